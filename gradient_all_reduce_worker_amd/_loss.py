"""Binding of the loss operators of libga.so (include/ga_loss.h), under the same
names: argument marshalling only, no fallback implementation. The calls go
through ctypes; _tensors.so looks the tensors over.

Every call takes one tensor per worker: matrices of rows x columns whose rows
may be strided (the same stride for all workers) and whose row counts may
differ, or be 0. Outputs that are not given are allocated, on the stream that
the call runs on; a workspace that is given (``ws``, uint8) may be used by one call at
a time, so two captured graphs that may run at once need one each.

The tensors' device need not be the current one. ``stream`` is a
torch.cuda.Stream of that device, its handle, or None for its current stream.
Tensors that another stream wrote have to be waited for by the caller.

Autograd does not record the calls: the losses and gradients they return have
no history. The gradients go on to what the logits were made from with
``torch.autograd.backward(logits, grads)``. Outputs that are given count as
changed in place, so with the gradients in the logits' own memory a backward
pass that needs those logits (a tanh's output, say) is refused.
"""
import ctypes as C
from contextlib import contextmanager
from typing import List, Optional, Sequence, Tuple, Union

import torch

from . import _native
from ._native import BF16, F32, _check

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
TOP_MAX = 1024
MAX_EXPERTS = 1024

LOSS_EXPORTS = (
    "ga_top_logits", "ga_distill_loss", "ga_distill_loss_ws_bytes", "ga_balance_loss",
    "ga_balance_loss_ws_bytes", "ga_balance_groups",
)

# type codes of _tensors.so beside F32 and BF16
I32, U8, BOOL = 2, 3, 4

Tensors = Sequence[torch.Tensor]
_bound = None
_looks = None


def _tensors():
    """_tensors.so (built by __graft_entry__.build()); raise if absent."""
    global _looks
    if _looks is None:
        try:
            from . import _tensors as looks
        except ImportError as e:
            raise ImportError("_tensors.so is not built; run __graft_entry__.build() first") from e
        _looks = looks
    return _looks


def _dtype(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"{what} are float32 or bfloat16, not {t.dtype}")


def load() -> C.CDLL:
    """libga.so with the loss operators' signatures."""
    global _bound
    if _bound is None:
        L = _native.load()
        vp, i64, i32, f32, sz = C.c_void_p, C.c_int64, C.c_int32, C.c_float, C.c_size_t
        L.ga_top_logits.argtypes = [vp, vp, i32, i64, i64, i32, i32, f32, vp, vp, vp, vp]
        L.ga_distill_loss.argtypes = [vp, vp, i32, i64, i64, i32, vp, vp, i32, vp, i32, vp, f32, f32, vp, i64, vp,
                                      vp, vp, sz, vp]
        L.ga_distill_loss_ws_bytes.argtypes = [i64]
        L.ga_distill_loss_ws_bytes.restype = sz
        L.ga_balance_loss.argtypes = [vp, vp, i32, i32, i64, i32, vp, i32, vp, i32, i64, f32, vp, i64, vp, vp, vp,
                                      sz, vp]
        L.ga_balance_loss_ws_bytes.argtypes = [vp, i32, i32, i64]
        L.ga_balance_loss_ws_bytes.restype = sz
        L.ga_balance_groups.argtypes = [vp, i32, i64]
        L.ga_balance_groups.restype = i64
        for name in ("ga_top_logits", "ga_distill_loss", "ga_balance_loss"):
            getattr(L, name).restype = C.c_int
        _bound = L
    return _bound


@contextmanager
def _elsewhere(index: int, stream):
    """For a call on another device than the current one, or on a given
    stream: its handle; what is allocated inside belongs to that stream."""
    dev = torch.device("cuda", index)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    if stream.device != dev:
        raise ValueError(f"the tensors are on {dev}, the stream on {stream.device}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield stream.cuda_stream


class _Logits:
    """The workers' logits, looked over (by _tensors.so, loaded from here on):
    pointers and row counts (bytes for the C ABI), rows together, columns, row
    stride, type and device."""
    __slots__ = ("ptrs", "tokens", "rows", "cols", "ld", "dt", "device", "P", "first")

    def __init__(self, ts: Tensors):
        self.ptrs, self.tokens, self.rows, self.cols, self.ld, self.dt, self.device = _tensors().logits(ts)
        self.P = len(ts)
        self.first = ts

    def dense(self, ts: Optional[Tensors], what: str, code: int, cols: int = -1):
        """Pointers of one dense tensor per worker, [rows] or [rows, cols]."""
        return None if ts is None else _looks.dense(ts, what, code, self.device, self.tokens, cols)

    def one(self, t: torch.Tensor, what: str, code: int, numel: int) -> int:
        return _looks.one(t, what, code, self.device, numel)

    def new(self, dtype: torch.dtype, cols: Optional[int] = None) -> List[torch.Tensor]:
        return [torch.empty((t.shape[0],) if cols is None else (t.shape[0], cols), dtype=dtype, device=t.device)
                for t in self.first]

    def empty(self, shape, dtype: torch.dtype) -> torch.Tensor:
        return torch.empty(shape, dtype=dtype, device=self.first[0].device)

    def grads(self, grads):
        """(gradients or None, their pointers, their row stride)."""
        if grads is None or grads is False:
            return None, None, 0
        if grads is True:
            grads = self.new(self.first[0].dtype, self.cols)
        return (grads, *_looks.matrices(grads, "gradients", self.dt, self.device, self.tokens, self.cols))

    def workspace(self, ws: Optional[torch.Tensor], need: int):
        """(workspace, address, bytes)."""
        if ws is None:
            ws = self.empty(max(need, 8), torch.uint8)
            return ws, ws.data_ptr(), max(need, 8)
        n = ws.numel()
        return ws, self.one(ws, "the workspace", U8, n), n

    def run(self, stream, call):
        """call(stream handle) with the logits' device current."""
        if stream is None and self.device == torch.cuda.current_device():
            return call(torch._C._cuda_getCurrentRawStream(self.device))
        with _elsewhere(self.device, stream) as handle:
            return call(handle)


def _slots(idx: Tensors) -> int:
    if not len(idx) or idx[0].dim() != 2:
        raise ValueError("idx must be one matrix per worker, rows x slots")
    return idx[0].shape[1]


def ga_top_logits(logits: Tensors, k: int, temp: float = 1.0, vals: Optional[Tensors] = None,
                  idx: Optional[Tensors] = None, lse: Union[bool, Tensors] = True,
                  stream=None) -> Tuple[Tensors, Tensors, Optional[Tensors]]:
    """Every row's k largest logits in descending order (vals, the logits'
    dtype), their columns (idx, int32; equal values by column) and the row's
    log-sum-exp at `temp` (lse, float32; False: none)."""
    lg = _Logits(logits)

    def call(s):
        v = lg.new(logits[0].dtype, k) if vals is None else vals
        i = lg.new(torch.int32, k) if idx is None else idx
        e = lg.new(torch.float32) if lse is True else None if lse is False else lse
        _check(load().ga_top_logits(lg.ptrs, lg.tokens, lg.P, lg.cols, lg.ld, lg.dt, k, temp,
                                    lg.dense(v, "vals", lg.dt, k), lg.dense(i, "idx", I32, k),
                                    lg.dense(e, "lse", F32), s))
        _looks.written(vals, idx, lse)
        return v, i, e

    return lg.run(stream, call)


def ga_distill_loss_ws_bytes(rows: int) -> int:
    return int(load().ga_distill_loss_ws_bytes(rows))


def ga_distill_loss(logits: Tensors, idx: Tensors, vals: Tensors, lse: Optional[Tensors] = None,
                    weight: Optional[Tensors] = None, temp: float = 1.0, scale: float = 1.0,
                    grads: Union[bool, Tensors, None] = True, row_loss: Optional[Tensors] = None,
                    out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, Optional[Tensors]]:
    """Distillation from a teacher's top logits (idx, vals, and its lse or
    None to renormalise over the slots): (loss, grads). loss holds sum w l,
    sum w and scale times their ratio; grads are the logits' gradients, in
    tensors given (the logits themselves: in place), new ones (True) or none
    (None); row_loss receives every row's l."""
    lg = _Logits(logits)
    k = _slots(idx)
    vdt = _dtype(vals[0], "vals") if len(vals) else F32
    L = load()

    def call(s):
        g, gp, ldg = lg.grads(grads)
        o = lg.empty(3, torch.float32) if out is None else out
        w, wp, wn = lg.workspace(ws, L.ga_distill_loss_ws_bytes(lg.rows))
        _check(L.ga_distill_loss(lg.ptrs, lg.tokens, lg.P, lg.cols, lg.ld, lg.dt, lg.dense(idx, "idx", I32, k),
                                 lg.dense(vals, "vals", vdt, k), vdt, lg.dense(lse, "lse", F32), k,
                                 lg.dense(weight, "weights", F32), temp, scale, gp, ldg,
                                 lg.dense(row_loss, "row losses", F32), lg.one(o, "out", F32, 3), wp, wn, s))
        _looks.written(grads, row_loss, out)
        return o, g

    return lg.run(stream, call)


def ga_balance_groups(tokens: Sequence[int], group_len: int = 0) -> int:
    """Groups (rows of the counts) of workers with these row counts."""
    return int(load().ga_balance_groups((C.c_int64 * len(tokens))(*tokens), len(tokens), group_len))


def ga_balance_loss_ws_bytes(tokens: Sequence[int], experts: int, group_len: int = 0) -> int:
    return int(load().ga_balance_loss_ws_bytes((C.c_int64 * len(tokens))(*tokens), len(tokens), experts, group_len))


def ga_balance_loss(logits: Tensors, idx: Tensors, mask: Optional[Tensors] = None, score: int = SCORE_SOFTMAX,
                    group_len: int = 0, scale: float = 1.0, grads: Union[bool, Tensors, None] = True,
                    counts: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[Tensors]]:
    """A router's balance loss from its logits and the experts it chose (idx):
    (loss, counts, grads). loss holds the sum of the groups' losses, the
    number of groups with a row that counts and scale times their ratio;
    counts is [groups, experts]; mask (uint8 or bool) drops rows; grads as in
    ga_distill_loss."""
    lg = _Logits(logits)
    k = _slots(idx)
    mdt = BOOL if mask is not None and len(mask) and mask[0].dtype == torch.bool else U8
    L = load()

    def call(s):
        g, gp, ldg = lg.grads(grads)
        groups = 1 if group_len == 0 else L.ga_balance_groups(lg.tokens, lg.P, group_len)
        o = lg.empty(3, torch.float32) if out is None else out
        c = lg.empty((groups, lg.cols), torch.int32) if counts is None else counts
        w, wp, wn = lg.workspace(ws, L.ga_balance_loss_ws_bytes(lg.tokens, lg.P, lg.cols, group_len))
        _check(L.ga_balance_loss(lg.ptrs, lg.tokens, lg.P, lg.cols, lg.ld, lg.dt, lg.dense(idx, "idx", I32, k), k,
                                 lg.dense(mask, "mask", mdt), score, group_len, scale, gp, ldg,
                                 lg.one(c, "counts", I32, groups * lg.cols) or None, lg.one(o, "out", F32, 3),
                                 wp, wn, s))
        _looks.written(grads, counts, out)
        return o, c, g

    return lg.run(stream, call)
