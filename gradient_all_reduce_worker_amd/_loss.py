"""ctypes binding of the loss operators of libga.so (include/ga_loss.h), under
the same names: argument marshalling only, no fallback implementation.

Every call takes one tensor per worker: matrices of rows x columns whose rows
may be strided (the same stride for all workers) and whose row counts may
differ, or be 0. Outputs that are not given are allocated, on the stream that
the call runs on; a workspace that is given (``ws``) may be used by one call at
a time, so two captured graphs that may run at once need one each.

The tensors' device need not be the current one. ``stream`` is a
torch.cuda.Stream of that device, its handle, or None for its current stream.
Tensors that another stream wrote have to be waited for by the caller.
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

Tensors = Sequence[torch.Tensor]
_bound = None


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
def _launch(dev: torch.device, stream):
    """The handle of the stream that a call on `dev` runs on; what is
    allocated inside belongs to that stream."""
    if stream is None:
        if dev.index == torch.cuda.current_device():
            yield torch.cuda.current_stream().cuda_stream
            return
        stream = torch.cuda.current_stream(dev)
    elif not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    if stream.device != dev:
        raise ValueError(f"the tensors are on {dev}, the stream on {stream.device}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield stream.cuda_stream


def _dtype(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"{what} are float32 or bfloat16, not {t.dtype}")


def _ptrs(ts: Tensors):
    return (C.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


class _Logits:
    """The workers' logits: pointers, row counts, columns and row stride."""

    def __init__(self, ts: Tensors):
        if not len(ts):
            raise ValueError("no workers")
        t0 = ts[0]
        self.device, self.dtype = t0.device, t0.dtype
        self.dt = _dtype(t0, "logits")
        if not t0.is_cuda:
            raise ValueError("logits must be GPU tensors")
        if t0.dim() != 2:
            raise ValueError("logits are matrices, rows x columns")
        self.cols = t0.shape[1]
        self.rows = [t.shape[0] for t in ts]
        self.ld = self.stride(ts, "logits")
        self.P = len(ts)
        self.tokens = (C.c_int64 * self.P)(*self.rows)
        self.ptrs = _ptrs(ts)

    def stride(self, ts: Tensors, what: str) -> int:
        """The row stride of matrices that match the logits."""
        if len(ts) != len(self.rows):
            raise ValueError(f"{len(ts)} {what} for {len(self.rows)} workers")
        ld = None
        for t, n in zip(ts, self.rows):
            if t.dtype != self.dtype or t.device != self.device:
                raise TypeError(f"{what} must all be {self.dtype} on {self.device}")
            if t.shape != (n, self.cols):
                raise ValueError(f"{what} of shape {tuple(t.shape)}, not {(n, self.cols)}")
            if n and self.cols > 1 and t.stride(1) != 1:
                raise ValueError(f"{what} must have consecutive columns")
            if n > 1:
                if ld is not None and t.stride(0) != ld:
                    raise ValueError(f"all workers' {what} need the same row stride")
                ld = t.stride(0)
        if ld is not None and ld < self.cols:
            raise ValueError(f"rows of {what} overlap")
        return self.cols if ld is None else ld

    def dense(self, ts: Optional[Tensors], what: str, dtype: torch.dtype, cols: Optional[int] = None):
        """Pointers of one dense tensor per worker, [rows] or [rows, cols]."""
        if ts is None:
            return None
        if len(ts) != self.P:
            raise ValueError(f"{len(ts)} {what} for {self.P} workers")
        for t, n in zip(ts, self.rows):
            if t.dtype != dtype or t.device != self.device:
                raise TypeError(f"{what} must be {dtype} on {self.device}, not {t.dtype} on {t.device}")
            if t.shape != ((n,) if cols is None else (n, cols)) or not t.is_contiguous():
                raise ValueError(f"{what} must be dense, of shape {(n,) if cols is None else (n, cols)}")
        return _ptrs(ts)

    def one(self, t: torch.Tensor, what: str, dtype: torch.dtype, numel: int) -> int:
        if t.dtype != dtype or t.device != self.device or t.numel() != numel or not t.is_contiguous():
            raise ValueError(f"{what} must be {numel} dense {dtype} values on {self.device}")
        return t.data_ptr()

    def new(self, dtype: torch.dtype, cols: Optional[int] = None) -> List[torch.Tensor]:
        return [torch.empty((n,) if cols is None else (n, cols), dtype=dtype, device=self.device)
                for n in self.rows]

    def workspace(self, ws: Optional[torch.Tensor], need: int) -> torch.Tensor:
        if ws is None:
            return torch.empty(max(need, 8), dtype=torch.uint8, device=self.device)
        if ws.device != self.device or not ws.is_contiguous():
            raise ValueError(f"the workspace must be dense, on {self.device}")
        return ws


def _grads(lg: _Logits, grads: Union[bool, Tensors, None]):
    """(gradients or None, their row stride)."""
    if grads is None or grads is False:
        return None, 0
    if grads is True:
        return lg.new(lg.dtype, lg.cols), lg.cols
    return grads, lg.stride(grads, "gradients")


def ga_top_logits(logits: Tensors, k: int, temp: float = 1.0, vals: Optional[Tensors] = None,
                  idx: Optional[Tensors] = None, lse: Union[bool, Tensors] = True,
                  stream=None) -> Tuple[Tensors, Tensors, Optional[Tensors]]:
    """Every row's k largest logits in descending order (vals, the logits'
    dtype), their columns (idx, int32; equal values by column) and the row's
    log-sum-exp at `temp` (lse, float32; False: none)."""
    lg = _Logits(logits)
    with _launch(lg.device, stream) as s:
        vals = lg.new(lg.dtype, k) if vals is None else vals
        idx = lg.new(torch.int32, k) if idx is None else idx
        lse = lg.new(torch.float32) if lse is True else None if lse is False else lse
        _check(load().ga_top_logits(lg.ptrs, lg.tokens, lg.P, lg.cols, lg.ld, lg.dt, k, temp,
                                    lg.dense(vals, "vals", lg.dtype, k), lg.dense(idx, "idx", torch.int32, k),
                                    lg.dense(lse, "lse", torch.float32), s))
    return vals, idx, lse


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
    if len(idx) != lg.P or idx[0].dim() != 2:
        raise ValueError("idx must be one matrix per worker, rows x slots")
    k = idx[0].shape[1]
    tdt = vals[0].dtype
    vdt = _dtype(vals[0], "vals")
    with _launch(lg.device, stream) as s:
        grads, ldg = _grads(lg, grads)
        if out is None:
            out = torch.empty(3, dtype=torch.float32, device=lg.device)
        L = load()
        ws = lg.workspace(ws, L.ga_distill_loss_ws_bytes(sum(lg.rows)))
        _check(L.ga_distill_loss(lg.ptrs, lg.tokens, lg.P, lg.cols, lg.ld, lg.dt,
                                 lg.dense(idx, "idx", torch.int32, k), lg.dense(vals, "vals", tdt, k), vdt,
                                 lg.dense(lse, "lse", torch.float32), k,
                                 lg.dense(weight, "weights", torch.float32), temp, scale,
                                 None if grads is None else _ptrs(grads), ldg,
                                 lg.dense(row_loss, "row losses", torch.float32),
                                 lg.one(out, "out", torch.float32, 3), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), s))
    return out, grads


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
    if len(idx) != lg.P or idx[0].dim() != 2:
        raise ValueError("idx must be one matrix per worker, rows x slots")
    k = idx[0].shape[1]
    with _launch(lg.device, stream) as s:
        grads, ldg = _grads(lg, grads)
        L = load()
        groups = L.ga_balance_groups(lg.tokens, lg.P, group_len)
        if out is None:
            out = torch.empty(3, dtype=torch.float32, device=lg.device)
        if counts is None:
            counts = torch.empty(groups, lg.cols, dtype=torch.int32, device=lg.device)
        need = L.ga_balance_loss_ws_bytes(lg.tokens, lg.P, lg.cols, group_len)
        ws = lg.workspace(ws, need)
        mdt = mask[0].dtype if mask and mask[0].dtype == torch.bool else torch.uint8
        _check(L.ga_balance_loss(lg.ptrs, lg.tokens, lg.P, lg.cols, lg.ld, lg.dt,
                                 lg.dense(idx, "idx", torch.int32, k), k, lg.dense(mask, "mask", mdt), score,
                                 group_len, scale, None if grads is None else _ptrs(grads), ldg,
                                 lg.one(counts, "counts", torch.int32, groups * lg.cols) or None,
                                 lg.one(out, "out", torch.float32, 3), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), s))
    return out, counts, grads
