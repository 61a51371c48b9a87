"""The loss operators on the GPU against the binary64 oracle: odd sizes,
strides, empty rows and workers, masks, both types, in place, other streams,
captured graphs, and the three run together with the ring.

Tolerances are derived, not chosen. u = 2^-24 is half a step of binary32; h of
the stored type (bf16: 2^-8, binary32: u) the rounding of a stored gradient.
For a term e = exp2((x - b) c), c = log2(e) / temp: x - b, the product and c
(two roundings) leave the exponent off by 4 u relative, so e is off by
(4 A + 2) u with A = |x - b| / temp (2 u: the hardware exp2, 1 ulp). A sum of n
terms per thread and a tree over the workgroup adds (n + 25) u, each change of
a running maximum another (2 + 1 + 1.5) u (a rescaling by exp(-A') loses 4 A' u
of a part exp(-A') <= 1/e A'), at most one per vector. A teacher's q = exp(lq)
is off by the error of its logits (6 |t| u), the sum over K slots and expf,
logf of 2 ulp: (6 t + K + 24) u. A gradient coef (p sum q - slot) adds these up
with ten roundings of its own; a row's loss the same per slot.
"""
import ctypes as C

import numpy as np
import pytest
import torch

import gradient_all_reduce_worker_amd as ga
from gradient_all_reduce_worker_amd import _loss
from oracle import loss as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def _f64(t):
    return t.detach().cpu().double().numpy()


def _logits(rng, rows, cols, tdt, pad=0, spread=3.0):
    """One strided matrix per worker; the padding between rows holds NaN."""
    out = []
    for n in rows:
        x = torch.full((n, cols + pad), float("nan"), dtype=tdt)
        x[:, :cols] = torch.from_numpy(rng.standard_normal((n, cols)) * spread).to(tdt)
        out.append(x.to(DEV)[:, :cols])
    return out


# ------------------------------------------------------------------ top logits
def _check_top(logits, k, temp, got):
    for x, v, i, l in zip(logits, *got):
        z = _f64(x)
        if not z.shape[0]:
            continue
        idx, vals, lse = ol.top_logits(z, k, temp)
        assert np.array_equal(i.cpu().numpy(), idx)
        assert np.array_equal(_f64(v), vals)
        n = z.shape[1]
        for r in range(z.shape[0]):
            if np.isneginf(z[r]).all():
                assert np.isneginf(float(l[r]))
                continue
            a = (z[r].max() - z[r]) / temp
            p = np.exp(z[r] / temp - lse[r])
            abar = float((p * np.where(p > 0, a, 0)).sum())
            per = -(-n // 64)                            # terms of a thread, at most
            tol = (4 * abar + 2 + 2.2 * per + 25 + 4 + 2 * abs(lse[r]) + 3 * abs(z[r].max() / temp)) * U
            assert abs(float(l[r]) - lse[r]) <= tol, (r, float(l[r]), lse[r], tol)


TOP = [([1], 1, 1, 0), ([3, 0, 2], 2, 2, 0), ([1], 7, 7, 0), ([2], 8, 3, 0), ([5], 9, 9, 3), ([4, 1], 63, 20, 0),
       ([3], 64, 64, 8), ([2, 2], 100, 100, 1), ([2], 513, 512, 0), ([3], 1000, 64, 0), ([2], 1024, 1024, 0),
       ([2], 2047, 1000, 0), ([2, 3], 4097, 16, 7), ([2], 8191, 128, 0), ([1] * 7, 16384, 33, 0), ([2], 32768, 256, 0),
       ([1, 2], 50003, 64, 0), ([2], 65537, 700, 0), ([2], 131072, 128, 0), ([1], 160001, 256, 5),
       ([1], 300007, 1024, 0), ([1], 1100001, 40, 0), ([600], 40, 5, 0)]


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("case", range(len(TOP)))
def test_top_logits(case, tdt):
    rows, V, k, pad = TOP[case]
    print(f"top rows={rows} V={V} k={k} pad={pad} {tdt}", flush=True)
    x = _logits(np.random.default_rng(case), rows, V, tdt, pad)
    temp = (1.0, 2.0, 0.7)[case % 3]
    _check_top(x, k, temp, ga.ga_top_logits(x, k, temp))


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("kind", ["equal", "up", "down", "few", "zeros", "inf", "all_inf", "lowest", "peaks", "half"])
@pytest.mark.parametrize("V,k", [(300, 50), (5003, 200), (70000, 64), (70000, 1024)])
def test_top_logits_in_order_and_tied(kind, V, k, tdt):
    print(f"top {kind} V={V} k={k} {tdt}", flush=True)
    rng = np.random.default_rng(9)
    if kind == "equal":
        z = np.full((2, V), -1.5)
    elif kind == "up":
        z = np.tile(np.arange(V) * 0.001, (2, 1))
    elif kind == "down":
        z = np.tile(-np.arange(V) * 0.001, (2, 1))
    elif kind == "few":
        z = rng.integers(-2, 3, (2, V)).astype(float)
    elif kind == "zeros":
        z = rng.choice([0.0, -0.0, -1.0], (2, V))
    elif kind == "inf":
        z = np.where(rng.random((2, V)) < 0.999, -INF, rng.standard_normal((2, V)))
    elif kind == "all_inf":
        z = np.full((2, V), -INF)
    elif kind == "lowest":
        z = np.full((2, V), float(torch.finfo(tdt).min))
        z[0, V // 2] = 1.0
    elif kind == "peaks":                                # all large ones next to each other
        z = rng.standard_normal((2, V))
        z[:, V // 3:V // 3 + k] += 50
    else:
        z = np.where(np.arange(V) < V // 2, rng.standard_normal((2, V)), -INF)
    x = [torch.from_numpy(z).to(tdt).to(DEV)]
    _check_top(x, k, 1.0, ga.ga_top_logits(x, k))


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_top_logits_with_nan_stays_in_bounds(tdt, sign):
    x = torch.randn(4, 5000, device=DEV).to(tdt)
    x[0, ::3] = float("nan")
    x[1] = float("nan")
    x[2, 7] = float("nan")
    x[3, 5] = INF
    if sign < 0:
        x = -x
    _, idx, lse = ga.ga_top_logits([x], 100)
    for r in range(4):
        i = idx[0][r].cpu()
        assert len(set(i.tolist())) == 100 and int(i.min()) >= 0 and int(i.max()) < 5000
    assert torch.isnan(lse[0][:3]).all()


def test_log_sum_exp_rounds_once():
    """Rows with one logit x in [64, 128), whose log-sum-exp is x: off by its
    one rounding (half a step, 2^-18), log2(e)'s in binary32 (0.23 u x) and
    those of exp2 and log2 next to 1 (4 u)."""
    x = torch.full((4096, 9), -INF, device=DEV)
    x[:, 4] = 64 + 64 * torch.rand(4096, generator=torch.Generator().manual_seed(1)).to(DEV)
    _, _, (lse,) = ga.ga_top_logits([x], 1)
    err = (lse.double() - x[:, 4].double()).abs()
    assert float(err.max()) <= 2.0 ** -18 + (0.23 * 128 + 4) * U


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("vectors", [128, 129, 512, 513, 1024, 1025, 2048, 2049, 8193])
def test_top_logits_at_every_kernels_ends(vectors, tdt):
    """Rows of so many 16-byte vectors, whole and with one element more or less."""
    E = 4 if tdt == F32 else 8
    for V in (vectors * E - 1, vectors * E, vectors * E + 1):
        for k in (40, 384, 385):
            print(f"top V={V} k={k} {tdt}", flush=True)
            x = _logits(np.random.default_rng(V), [2], V, tdt)
            _check_top(x, k, 1.0, ga.ga_top_logits(x, k))


def test_top_logits_leaves_the_rest_alone():
    """Without lse, into given buffers with guards behind them."""
    x = _logits(np.random.default_rng(1), [3, 2], 777, BF16, pad=5)
    big = [torch.full((n * 9 + 16,), 77, dtype=torch.int32, device=DEV) for n in (3, 2)]
    idx = [b[: n * 9].view(n, 9) for b, n in zip(big, (3, 2))]
    vals, _, lse = ga.ga_top_logits(x, 9, idx=idx, lse=False)
    assert lse is None
    for b, n, z in zip(big, (3, 2), x):
        assert (b[n * 9:] == 77).all()
        assert np.array_equal(b[: n * 9].view(n, 9).cpu().numpy(), ol.top_logits(_f64(z), 9, 1.0)[0])


# ------------------------------------------------------------------ distillation
def _teacher(rng, rows, V, K, vdt, z=None, empty=True, twice=True, spread=2.0):
    idx, vals = [], []
    for w, n in enumerate(rows):
        i = np.stack([rng.permutation(V)[:K] if K <= V else rng.integers(0, V, K) for _ in range(n)]) if n else \
            np.zeros((0, K), int)
        if n and empty and K > 2:
            i[0, K // 2] = -1
            i[-1, 0] = V                                 # out of range: empty as well
            i[-1, 1] = -2 ** 31
        if n and twice and K > 3:
            i[0, K - 1] = i[0, 0]
            i[n // 2, 1:4] = i[n // 2, 2]
        v = rng.standard_normal((n, K)) * spread + 2
        if z is not None:                                # near the student's own logits
            v = np.take_along_axis(_f64(z[w]), np.clip(i, 0, V - 1), 1) + 0.3 * rng.standard_normal((n, K))
        idx.append(torch.from_numpy(i.astype(np.int32)).to(DEV))
        vals.append(torch.from_numpy(v).to(vdt).to(DEV))
    return idx, vals


def _check_distill(logits, idx, vals, lse, weight, temp, scale, loss, grads, rows=None, tdt=None):
    """Everything against the oracle, to the bounds derived above."""
    tdt = tdt or logits[0].dtype
    z64, v64 = [_f64(x) for x in logits], [_f64(v) for v in vals]
    i64 = [i.cpu().numpy() for i in idx]
    l64 = None if lse is None else [_f64(l) for l in lse]
    w64 = None if weight is None else [_f64(w) for w in weight]
    o = ol.distill(z64, i64, v64, l64, w64, temp, scale)
    E, num_tol = (4 if tdt == F32 else 8), 0.0
    for w in range(len(z64)):
        z, n = z64[w], z64[w].shape[0]
        V, K = z.shape[1], i64[w].shape[1]
        per = -(-V // 64 // E + 1) * E if V > 64 * E else E     # terms of a thread, at most
        for r in range(n):
            wt = 1.0 if w64 is None else (w64[w][r] if w64[w][r] > 0 else 0.0)
            q, coef = o["q"][w][r], o["coef"][w][r]
            if wt == 0 or not q.any() or np.isneginf(z[r]).all():
                if grads is not None:
                    assert not _f64(grads[w][r]).any(), (w, r)
                if rows is not None:
                    assert float(rows[w][r]) == 0.0
                continue
            on = q > 0
            b = z[r].max()
            A = np.where(np.isneginf(z[r]), 0.0, (b - z[r]) / temp)
            p = ol.softmax(z[r:r + 1] / temp)[0]
            t = v64[w][r][on] / temp
            L = l64[w][r] if l64 is not None else ol.logsumexp(v64[w][r][(i64[w][r] >= 0) & (i64[w][r] < V)][None] / temp)[0]
            eS = (4 * float((p * A).sum()) + 2 + 2.2 * per + 25) * U
            eq = (6 * np.abs(t).max() + np.abs(t - L).max() + K + 24) * U
            if grads is not None:
                want, mass, slot = o["grads"][w][r], o["mass"][w][r], o["slot"][w][r]
                err = abs(coef) * (mass * ((4 * A + 2 + K + 10) * U + eS + eq) + slot * (eq + (K + 6) * U))
                err += 3 * U * np.abs(want) + abs(coef) * 1e-37 + 1e-40
                err += HALF[tdt] * (np.abs(want) + err)
                d = np.abs(_f64(grads[w][r]) - want)
                assert (d <= err).all(), (w, r, float((d / err).max()), int((d / err).argmax()))
            s, lnS = i64[w][r][on], ol.logsumexp((z[r:r + 1] - b) / temp)[0]
            lq, lp = t - L, (z[r, s] - b) / temp - lnS
            l_tol = INF
            if np.isfinite(lp).all():
                D = np.abs(lq - lp)
                l_tol = temp ** 2 * float((q[on] * (eq * D + eq + 2 * U * np.abs(lq) + 3 * U * A[s] + eS
                                                    + (2 + 3) * U * (np.abs(lnS) + np.abs(lq) + A[s])
                                                    + (K + 14) * U * D)).sum())
            num_tol += wt * l_tol
            if rows is not None:
                want = o["rows"][w][r]
                assert float(rows[w][r]) == want if np.isinf(want) else abs(float(rows[w][r]) - want) <= l_tol, (w, r)
    got = _f64(loss)
    assert abs(got[1] - o["den"]) <= U * o["den"]
    if np.isfinite(num_tol):
        num_tol += 2 * U * abs(o["num"])
        assert abs(got[0] - o["num"]) <= num_tol
        assert abs(got[2] - o["loss"]) <= (abs(scale) * num_tol / o["den"] if o["den"] > 0 else 0) + 2 * U * abs(o["loss"])
    else:
        assert np.isinf(got[0]) and np.isinf(got[2])


DISTILL = [([1], 1, 1, 0), ([2, 0, 1], 2, 2, 0), ([3], 7, 5, 0), ([2], 8, 8, 0), ([3, 1], 9, 4, 3), ([2], 63, 3, 0),
           ([4], 65, 70, 0), ([3, 2], 1000, 64, 8), ([2], 2048, 16, 0), ([2, 1], 4097, 100, 0), ([2], 8192, 65, 0),
           ([2], 8200, 1, 0), ([1, 2], 16385, 256, 1), ([2], 32768, 16, 0), ([1, 1, 1], 50003, 64, 0), ([2], 65536, 40, 64),
           ([1], 70001, 1024, 0), ([2], 131072, 64, 0), ([1], 140003, 32, 0), ([1], 163840, 16, 0), ([1], 262147, 50, 3),
           ([300, 0, 40], 33, 6, 0)]


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("case", range(len(DISTILL)))
def test_distill(case, tdt):
    rows, V, K, pad = DISTILL[case]
    print(f"distill rows={rows} V={V} K={K} pad={pad} {tdt}", flush=True)
    rng = np.random.default_rng(100 + case)
    x = _logits(rng, rows, V, tdt, pad)
    vdt = (F32, BF16)[case % 2]
    idx, vals = _teacher(rng, rows, V, K, vdt, x if case % 3 else None)
    temp, scale = (1.0, 2.0, 0.6)[case % 3], (1.0, -0.25)[case % 2]
    lse = weight = None
    if case % 4 >= 2:
        lse = [torch.logsumexp(v.float() / temp, 1) + 0.1 for v in vals]
    if case % 5 >= 2:
        weight = [torch.from_numpy(rng.random(n).astype(np.float32)).to(DEV) for n in rows]
        if rows[0] > 1:
            weight[0][-1] = 0
            x[0][-1] = float("nan")                      # not read
    row_loss = [torch.full((n,), 7.0, device=DEV) for n in rows]
    loss, grads = ga.ga_distill_loss(x, idx, vals, lse, weight, temp, scale, row_loss=row_loss)
    _check_distill(x, idx, vals, lse, weight, temp, scale, loss, grads, row_loss)
    alone, none = ga.ga_distill_loss(x, idx, vals, lse, weight, temp, scale, grads=None)
    assert none is None                                  # (the loss alone may be summed in another order)
    _check_distill(x, idx, vals, lse, weight, temp, scale, alone, None)
    again, same = ga.ga_distill_loss(x, idx, vals, lse, weight, temp, scale)
    assert torch.equal(again, loss) and all(torch.equal(a, b) for a, b in zip(same, grads))
    # strided gradients, with what lies between and behind the rows left alone
    big = [torch.full((n + 1, V + 5), 3.0, dtype=tdt, device=DEV) for n in rows]
    _, gr = ga.ga_distill_loss(x, idx, vals, lse, weight, temp, scale, grads=[b[:n, :V] for b, n in zip(big, rows)])
    for b, n, g in zip(big, rows, grads):
        assert torch.equal(b[:n, :V], g) and (b[:, V:] == 3).all() and (b[n:] == 3).all()
    # in place
    here = [t.clone(memory_format=torch.preserve_format) for t in x]
    here = [torch.empty_strided(t.shape, t.stride(), dtype=tdt, device=DEV).copy_(t) for t in x]
    l2, g2 = ga.ga_distill_loss(here, idx, vals, lse, weight, temp, scale, grads=here)
    assert torch.equal(l2, loss) and all(torch.equal(a, b) for a, b in zip(here, grads))


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("vectors", [127, 128, 255, 256, 511, 512, 639, 640, 767, 768, 1024, 1025, 2300, 4607, 4608, 6200,
                                     9215, 9216, 15000, 20480, 22527, 22528])
def test_distill_at_every_kernels_ends(vectors, tdt):
    """Rows of so many whole 16-byte vectors and some elements more, with the
    gradient, in place, and without."""
    rng, E = np.random.default_rng(vectors), 4 if tdt == F32 else 8
    V, rows, K = vectors * E + vectors % E, [2, 1], 20
    print(f"distill V={V} {tdt}", flush=True)
    x = _logits(rng, rows, V, tdt)
    idx, vals = _teacher(rng, rows, V, K, tdt, x)
    row_loss = [torch.full((n,), 7.0, device=DEV) for n in rows]
    loss, grads = ga.ga_distill_loss(x, idx, vals, row_loss=row_loss)
    _check_distill(x, idx, vals, None, None, 1.0, 1.0, loss, grads, row_loss)
    alone, _ = ga.ga_distill_loss(x, idx, vals, grads=False)
    _check_distill(x, idx, vals, None, None, 1.0, 1.0, alone, None)
    here, same = ga.ga_distill_loss(x, idx, vals, grads=x)
    assert torch.equal(here, loss) and all(torch.equal(a, b) for a, b in zip(same, grads))


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_distill_masked_entries(V, tdt):
    """-inf and the type's lowest value among the logits, whole rows of them,
    a teacher without slots, and all weights zero."""
    rng = np.random.default_rng(V)
    x = _logits(rng, [8], V, tdt)
    z = x[0]
    low = torch.finfo(tdt).min
    z[0, 1:] = -INF
    z[1] = -INF
    z[2, ::2] = low
    z[3] = low
    z[4, : V - 2] = -INF
    z[5] = torch.finfo(tdt).max
    idx, vals = _teacher(rng, [8], V, 6, F32, twice=False, empty=False)
    idx[0][0] = torch.tensor([0, -1, -1, -1, -1, -1])
    idx[0][4, 0] = V - 1
    idx[0][4, 1:] = V - 2
    idx[0][6] = -1
    vals[0][7, 2:] = -INF
    vals[0][5, 0] = low if tdt == F32 else -3e38
    row_loss = [torch.empty(8, device=DEV)]
    loss, grads = ga.ga_distill_loss(x, idx, vals, row_loss=row_loss)
    _check_distill(x, idx, vals, None, None, 1.0, 1.0, loss, grads, row_loss)
    assert torch.isfinite(loss).all()
    # a slot of weight on a column that the student rules out
    idx[0][0, 1] = 1
    loss, grads = ga.ga_distill_loss(x, idx, vals, row_loss=row_loss)
    assert float(row_loss[0][0]) == INF and float(loss[2]) == INF and torch.isfinite(grads[0].float()).all()
    zero = [torch.zeros(8, device=DEV)]
    x[0][:] = float("nan")
    loss, grads = ga.ga_distill_loss(x, idx, vals, weight=zero, row_loss=row_loss)
    assert not loss.any() and not grads[0].any() and not row_loss[0].any()


def _past_the_end(got, want):
    """`got` with the numbers that binary32 cannot hold put in, where it has
    them as infinities."""
    got, far = _f64(got), np.abs(want) > 3.41e38
    assert (got[far] == np.sign(want[far]) * INF).all()
    return torch.from_numpy(np.where(far, want, got))


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("temp", [1.0, 2.0, 0.7])
@pytest.mark.parametrize("V", [700, 5000, 40000, 180000])
def test_large_finite_masks(V, temp, tdt):
    """Entries masked out by a large finite number, whole threads' shares of a
    row at once, and rows of nothing but large numbers. A product with
    log2(e) / temp is then off by up to 2^104 in units of the exponent."""
    low = float(torch.finfo(tdt).min)
    rng = np.random.default_rng(V)
    fills = (-1e4, -1e9, -1e10, -1e11, -1e20, -1e30, low, 1e10, 3e37)
    x = _logits(rng, [3 * len(fills)], V, tdt)
    z = x[0]
    for k, m in enumerate(fills):
        z[3 * k, V // 7:] = m                            # one unmasked end
        z[3 * k + 1, : V - 5] = m                        # a few unmasked at the other
        z[3 * k + 2] = m                                 # none
        z[3 * k + 2, V // 2] = 0.75 * m
    print(f"masks V={V} temp={temp} {tdt}", flush=True)
    k = 8
    v, i, lse = ga.ga_top_logits(x, k, temp)
    _check_top(x, k, temp, (v, i, [_past_the_end(lse[0], ol.top_logits(_f64(z), k, temp)[2])]))
    idx, vals = _teacher(rng, [3 * len(fills)], V, k, F32, twice=False)
    for r in range(3 * len(fills)):                      # slots on masked and on unmasked columns
        idx[0][r, :4] = torch.tensor([0, V // 2, V - 1, V - 2])
    row_loss = [torch.empty(3 * len(fills), device=DEV)]
    for grads in (True, False):
        loss, g = ga.ga_distill_loss(x, idx, vals, temp=temp, grads=grads, row_loss=row_loss)
        # rows of the lowest value have losses near 3.4e38 temp
        o = ol.distill([_f64(z)], [idx[0].cpu().numpy()], [_f64(vals[0])], None, None, temp, 1.0)
        rows = [_past_the_end(row_loss[0], o["rows"][0])]
        if o["num"] > 3.41e38:
            assert torch.isposinf(loss[0])
            loss = torch.tensor([o["num"], o["den"], o["loss"]], dtype=torch.float64)
        _check_distill(x, idx, vals, None, None, temp, 1.0, loss, g, rows)


@pytest.mark.parametrize("tdt", [F32, BF16])
def test_distill_nan_stays_in_its_row(tdt):
    rng = np.random.default_rng(2)
    x = _logits(rng, [4], 3000, tdt)
    idx, vals = _teacher(rng, [4], 3000, 8, F32)
    x[0][1, 17] = float("nan")
    x[0][2, 5] = INF
    _, grads = ga.ga_distill_loss(x, idx, vals)
    assert torch.isnan(grads[0][1]).any() and torch.isnan(grads[0][2]).any()
    assert torch.isfinite(grads[0][0].float()).all() and torch.isfinite(grads[0][3].float()).all()


def test_distill_gradient_against_differences():
    """Along a direction d of entries in [-1, 1] the loss of a row is
    temp^2 (Q logsumexp((z + h d) / temp) - linear), whose third derivative is
    temp^-1 Q times a third cumulant of a variable in [-1, 1] (at most 1): the
    central difference is off by h^2 / 6 of it and by the loss's own error / h."""
    rng = np.random.default_rng(12)
    V, K, temp, h = 3001, 40, 1.5, 2.0 ** -6
    x = _logits(rng, [3, 2], V, F32)
    idx, vals = _teacher(rng, [3, 2], V, K, F32, x)
    weight = [torch.rand(n, device=DEV) + 0.5 for n in (3, 2)]
    loss, grads = ga.ga_distill_loss(x, idx, vals, weight=weight, temp=temp)
    for seed in range(4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        d = [(torch.randint(0, 3, t.shape, generator=g, device=DEV) - 1).float() for t in x]
        up = [(a + h * b) for a, b in zip(x, d)]
        dn = [(a - h * b) for a, b in zip(x, d)]
        lu, _ = ga.ga_distill_loss(up, idx, vals, weight=weight, temp=temp, grads=None)
        ld, _ = ga.ga_distill_loss(dn, idx, vals, weight=weight, temp=temp, grads=None)
        # the points' own rounding (x + h d in binary32) is in the denominators
        diff = (_f64(lu)[2] - _f64(ld)[2])
        step = [(_f64(a) - _f64(b)) for a, b in zip(up, dn)]
        want = sum(float((_f64(q) * s).sum()) for q, s in zip(grads, step))
        terms = V // 64 + 40
        own = 2 * temp ** 2 * (2.2 * terms + 8 * K + 200) * U      # of each loss, per row, averaged
        assert abs(diff - want) <= 2 * own + 2 * h ** 3 / 6 / temp + 40 * U, (diff, want)


# ------------------------------------------------------------------ balance
def _route(rng, x, K, drop=True, twice=True):
    out = []
    for z in x:
        n, E = z.shape
        i = rng.integers(0, E, (n, K))
        if n and drop:
            i[0, 0] = -1
            i[-1, K - 1] = E
            i[n // 2, 0] = 2 ** 31 - 1
        out.append(torch.from_numpy(i.astype(np.int32)).to(DEV))
    return out


def _check_balance(x, idx, mask, sigmoid, group_len, scale, got):
    loss, counts, grads = got
    tdt = x[0].dtype
    E, K = x[0].shape[1], idx[0].shape[1]
    z64 = [_f64(t) for t in x]
    o = ol.balance(z64, [i.cpu().numpy() for i in idx], None if mask is None else [m.cpu().numpy() for m in mask],
                   sigmoid, group_len, scale)
    assert np.array_equal(counts.cpu().numpy(), o["counts"])
    groups = ol.groups_of([z.shape[0] for z in z64], group_len)
    tol = 0.0
    for w, z in enumerate(z64):
        for r in range(z.shape[0]):
            g = groups[w][r]
            p, s = o["p"][w][r], o["s"][w][r]
            if not p.any():
                if grads is not None:
                    assert not _f64(grads[w][r]).any()
                continue
            f = E * o["counts"][g] / (K * o["n"][g])
            zr = np.where(np.isneginf(z[r]), 0.0, np.abs(z[r]) if sigmoid else z[r].max() - z[r])
            ep = (4 * zr + 6) * U                        # of one score
            es = 2 * (float((p * ep).sum()) + (E + 20) * U) + float((p * f * ep).sum()) / max(s, 1e-300)
            tol += s * es / o["n"][g]
            if grads is None:
                continue
            want = o["grads"][w][r]
            coef = abs(scale) / (o["den"] * o["n"][g])
            slope = p
            if sigmoid:
                with np.errstate(over="ignore"):
                    slope = p / (1 + np.exp(z[r]))
            err = coef * slope * (np.abs(f - s) * (ep * 2 + es + 10 * U) + 2 * U * f + es * s) + 1e-38
            err += 2 * U * np.abs(want)
            err += HALF[tdt] * (np.abs(want) + err)
            d = np.abs(_f64(grads[w][r]) - want)
            assert not (d > err).any(), (w, r, float((d / err).max()))
    got = _f64(loss)
    assert got[1] == o["den"]
    assert abs(got[0] - o["num"]) <= tol + 2 * U * o["num"]
    want = o["loss"]
    assert abs(got[2] - want) <= (abs(scale) * tol / o["den"] if o["den"] else 0) + 3 * U * abs(want)


BALANCE = [([1], 1, 1, 0, 0), ([3, 0, 2], 2, 2, 0, 0), ([5], 3, 2, 0, 2), ([64], 8, 2, 0, 0), ([70, 33], 8, 8, 4, 16),
           ([200, 0, 130], 16, 4, 0, 0), ([65, 64, 63], 60, 6, 0, 32), ([300], 64, 6, 0, 0), ([257, 500], 100, 3, 3, 100),
           ([600, 100], 128, 8, 0, 0), ([520], 160, 6, 0, 500), ([300, 200], 256, 8, 8, 0), ([130], 384, 8, 0, 64),
           ([90, 45], 512, 10, 0, 0), ([40], 513, 3, 0, 7), ([33], 1000, 33, 1, 0), ([50], 1024, 8, 0, 1),
           ([3000, 2500], 32, 2, 0, 0), ([1] * 20, 12, 2, 0, 1), ([1500, 0, 700], 20, 3, 0, 600)]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("case", range(len(BALANCE)))
def test_balance(case, tdt, sigmoid):
    rows, E, K, pad, group_len = BALANCE[case]
    print(f"balance rows={rows} E={E} K={K} pad={pad} group={group_len} {tdt} sigmoid={sigmoid}", flush=True)
    rng = np.random.default_rng(200 + case)
    x = _logits(rng, rows, E, tdt, pad)
    idx = _route(rng, x, K)
    score = ga.SCORE_SIGMOID if sigmoid else ga.SCORE_SOFTMAX
    scale = (1.0, 0.01, -3.0)[case % 3]
    mask = None
    if case % 2:
        mask = [torch.from_numpy((rng.random(n) < 0.8).astype(np.uint8) * 3).to(DEV) for n in rows]
        if group_len and rows[0] >= group_len:
            mask[0][:group_len] = 0                      # a group that is empty
        for t, m in zip(x, mask):
            t[m == 0] = float("nan")                     # not read
    got = ga.ga_balance_loss(x, idx, mask, score, group_len, scale)
    _check_balance(x, idx, mask, sigmoid, group_len, scale, got)
    loss, counts, grads = got
    alone, c2, none = ga.ga_balance_loss(x, idx, mask, score, group_len, scale, grads=None)
    assert none is None and torch.equal(alone, loss) and torch.equal(c2, counts)
    big = [torch.full((n + 1, E + 3), 3.0, dtype=tdt, device=DEV) for n in rows]
    ga.ga_balance_loss(x, idx, mask, score, group_len, scale, grads=[b[:n, :E] for b, n in zip(big, rows)])
    for b, n, g in zip(big, rows, grads):
        assert torch.equal(b[:n, :E], g) and (b[:, E:] == 3).all() and (b[n:] == 3).all()
    if mask is not None:
        l3, _, g3 = ga.ga_balance_loss(x, idx, [m != 0 for m in mask], score, group_len, scale)
        assert torch.equal(l3, loss)
    here = [torch.empty_strided(t.shape, t.stride(), dtype=tdt, device=DEV).copy_(t) for t in x]
    l2, _, _ = ga.ga_balance_loss(here, idx, mask, score, group_len, scale, grads=here)
    assert torch.equal(l2, loss) and all(torch.equal(a, b) for a, b in zip(here, grads))


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("E", [3, 4, 6, 8, 9, 12, 16, 20, 24, 30, 32, 40, 48, 56, 64, 72, 96, 100, 144, 176, 192, 200, 224,
                               256, 260, 320, 512, 516, 640, 768, 1020, 1024])
def test_balance_at_every_team(E, tdt):
    """Every way that rows of E experts are laid out over lanes; few rows (one
    workgroup does everything) and more than that."""
    rng = np.random.default_rng(E)
    for rows in ([20, 9], [700, 350]):
        print(f"balance rows={rows} E={E} {tdt}", flush=True)
        x = _logits(rng, rows, E, tdt)
        idx = _route(rng, x, min(E, 6))
        got = ga.ga_balance_loss(x, idx)
        _check_balance(x, idx, None, False, 0, 1.0, got)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("E", [5, 64, 300])
def test_balance_masked_entries(E, tdt, sigmoid):
    rng = np.random.default_rng(E)
    x = _logits(rng, [40, 30], E, tdt)
    low = torch.finfo(tdt).min
    x[0][0, 1:] = -INF
    x[0][1] = -INF
    x[0][2, ::2] = low
    x[0][4] = 80.0
    x[0][5, :2] = torch.tensor([60.0, -60.0])
    if not sigmoid:
        x[0][3] = low                                    # softmax: even; sigmoid: all 0
        x[1][0] = torch.finfo(tdt).max
    idx = _route(rng, x, 3)
    score = ga.SCORE_SIGMOID if sigmoid else ga.SCORE_SOFTMAX
    _check_balance(x, idx, None, sigmoid, 0, 1.0, ga.ga_balance_loss(x, idx, None, score))
    none = [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (40, 30)]
    for group_len in (0, 16):
        loss, counts, grads = ga.ga_balance_loss(x, idx, none, score, group_len)
        assert not loss.any() and not counts.any() and not grads[0].any() and not grads[1].any()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("E", [5, 8, 64, 160, 300, 1024])
@pytest.mark.parametrize("n", [20, 600])
def test_balance_infinity(n, E, tdt, sigmoid):
    """NaN in a row that counts, and +inf in a softmax: NaN in the loss and all
    over the row, and nowhere else. A sigmoid of +inf is 1 with slope 0, as one
    of 200 is in binary32. In a row that does not count, nothing."""
    rng = np.random.default_rng(E)
    x = _logits(rng, [n, 3], E, tdt)
    idx = _route(rng, x, 3)
    mask = [torch.ones(t.shape[0], dtype=torch.uint8, device=DEV) for t in x]
    score = ga.SCORE_SIGMOID if sigmoid else ga.SCORE_SOFTMAX
    mask[0][11], x[0][11, 1] = 0, INF
    _, _, clean = ga.ga_balance_loss(x, idx, mask, score)
    rest = torch.arange(n, device=DEV) != 7

    def put(v, at):
        y = [t.clone() for t in x]
        y[0][7, at] = v
        loss, _, grads = ga.ga_balance_loss(y, idx, mask, score)
        assert torch.equal(grads[0][rest], clean[0][rest]) and torch.equal(grads[1], clean[1])
        return loss, grads[0][7]

    for at in (0, E // 2, E - 1):
        for bad in (INF, float("nan")):
            loss, row = put(bad, at)
            if sigmoid and bad == INF:
                like, as_row = put(200.0, at)
                assert torch.equal(loss, like) and torch.equal(row, as_row) and torch.isfinite(row).all()
            else:
                assert torch.isnan(loss[0]) and torch.isnan(loss[2]) and torch.isnan(row).all()


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("E", [8, 300])
def test_balance_sigmoids_next_to_zero(E, tdt):
    """Logits just above the point where a sigmoid leaves the normal numbers
    still have their shares, those below it none."""
    rng = np.random.default_rng(E)
    x = _logits(rng, [40], E, tdt)
    x[0][:8] = torch.from_numpy(-86.0 + rng.random((8, E))).to(tdt)
    idx = _route(rng, x, 3)
    _check_balance(x, idx, None, True, 0, 1.0, ga.ga_balance_loss(x, idx, None, ga.SCORE_SIGMOID))
    x[0][8:16] = -88.0
    loss, _, grads = ga.ga_balance_loss(x, idx, None, ga.SCORE_SIGMOID)
    x[0][8:16] = -INF
    same, _, none = ga.ga_balance_loss(x, idx, None, ga.SCORE_SIGMOID)
    assert torch.equal(loss, same) and not grads[0][8:16].any() and torch.equal(grads[0], none[0])


def test_balance_gradient_against_differences():
    """The counts stay as they are, so along d in [-1, 1] each s_t is a mean of
    f (at most F) under a softmax: its third derivative is at most 8 F."""
    rng = np.random.default_rng(13)
    x = _logits(rng, [200, 100], 40, F32, spread=1.0)
    idx = _route(rng, x, 4)
    for score in (ga.SCORE_SOFTMAX, ga.SCORE_SIGMOID):
        loss, counts, grads = ga.ga_balance_loss(x, idx, None, score)
        F, h = 40 * int(counts.max()) / (4 * 300), 2.0 ** -6
        d = [(torch.randint(0, 3, t.shape, device=DEV) - 1).float() for t in x]
        up, dn = [a + h * b for a, b in zip(x, d)], [a - h * b for a, b in zip(x, d)]
        lu, _, _ = ga.ga_balance_loss(up, idx, None, score, grads=None)
        ld, _, _ = ga.ga_balance_loss(dn, idx, None, score, grads=None)
        step = [_f64(a) - _f64(b) for a, b in zip(up, dn)]
        want = sum(float((_f64(g) * s).sum()) for g, s in zip(grads, step))
        own = 2 * (40 + 60) * U * float(loss[2])
        assert abs(_f64(lu)[2] - _f64(ld)[2] - want) <= 2 * own + 8 * F * 2 * h ** 3 / 6 + 40 * U


# ------------------------------------------------------------------ no rows, other streams, graphs, far offsets
def test_no_rows_at_all():
    x = [torch.empty(0, 40, device=DEV), torch.empty(0, 40, device=DEV)]
    i = [torch.empty(0, 3, dtype=torch.int32, device=DEV)] * 2
    v = [torch.empty(0, 3, device=DEV)] * 2
    out = torch.full((3,), 5.0, device=DEV)
    ga.ga_distill_loss(x, i, v, out=out)
    assert out.tolist() == [0, 0, 0]
    for group_len in (0, 4):
        out.fill_(5)
        loss, counts, _ = ga.ga_balance_loss(x, i, None, group_len=group_len, out=out)
        assert out.tolist() == [0, 0, 0] and not counts.any() and counts.shape[0] == (1 if group_len == 0 else 0)
    ga.ga_top_logits(x, 3)


def test_no_rows_with_another_gradient_stride():
    """Without rows no gradient lies on its logits, whatever the strides."""
    L = _loss.load()
    out = torch.full((3,), 5.0, device=DEV)
    counts = torch.full((40,), 5, dtype=torch.int32, device=DEV)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    none, tokens, s = (C.c_void_p * 2)(), (C.c_int64 * 2)(0, 0), torch.cuda.current_stream().cuda_stream
    assert L.ga_distill_loss(none, tokens, 2, 40, 40, 0, none, none, 0, None, 3, None, 1.0, 1.0, none, 48, None,
                             out.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
    assert out.tolist() == [0, 0, 0]
    out.fill_(5)
    assert L.ga_balance_loss(none, tokens, 2, 40, 40, 0, none, 3, None, 0, 0, 1.0, none, 48, counts.data_ptr(),
                             out.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
    assert out.tolist() == [0, 0, 0] and not counts.any()


def test_more_rows_than_a_grid_is_wide():
    """1.1 million rows: two rows of the grid, sums of sums, partial weights.
    Checked against the same formulas in binary64, all rows at once: a row's
    log-probability is off by (4 A + 2 + 8 + 25) u, its loss by that, and the
    same of the teacher's two slots; gradients by a step of bf16 besides."""
    rows, V, K = [1_000_003, 0, 99_999], 8, 2
    g = torch.Generator(device=DEV).manual_seed(8)
    x = [torch.randn(n, V, generator=g, device=DEV).to(BF16) for n in rows]
    vals, idx, lse = ga.ga_top_logits(x, K)
    for z, v, i, l in zip(x, vals, idx, lse):
        d = z.double()
        assert torch.equal(i.long(), torch.sort(d + 0.0, dim=1, descending=True, stable=True)[1][:, :K])
        assert torch.equal(v.double(), torch.gather(d, 1, i.long()))
        assert ((l.double() - torch.logsumexp(d, 1)).abs() <= 120 * U).all()
    weight = [torch.rand(n, generator=g, device=DEV) for n in rows]
    y = [torch.randn(n, V, generator=g, device=DEV).to(BF16) for n in rows]
    row_loss = [torch.empty(n, device=DEV) for n in rows]
    loss, grads = ga.ga_distill_loss(y, idx, vals, weight=weight, row_loss=row_loss)
    alone, _ = ga.ga_distill_loss(y, idx, vals, weight=weight, grads=None)
    den = sum(w.double().sum() for w in weight)
    num = sum((w.double() * l.double()).sum() for w, l in zip(weight, row_loss))
    assert abs(float(loss[1]) - float(den)) <= U * float(den)
    assert abs(float(loss[0]) - float(num)) <= 1.01 * U * float(num)
    assert abs(float(alone[2]) - float(num / den)) <= 300 * U * float(num / den) + 300 * U
    for z, v, i, w, l, gr in zip(y, vals, idx, weight, row_loss, grads):
        p = torch.softmax(z.double(), 1)
        q = torch.softmax(v.double(), 1)
        want = (q * (q.log() - torch.gather(p, 1, i.long()).log())).sum(1)
        assert ((l.double() - want).abs() <= 400 * U).all()
        gw = (p.scatter_add(1, i.long(), -q)) * (w.double() / den)[:, None]
        err = 200 * U * (w.double() / den)[:, None]
        assert ((gr.double() - gw).abs() <= err + HALF[BF16] * (gw.abs() + err)).all()


def test_balance_of_many_rows():
    """70,000 rows in one group and in groups of 1000, against binary64 at once:
    scores off by (4 A + 6) u, the sums by (E + 20) u."""
    g = torch.Generator(device=DEV).manual_seed(9)
    rows, E, K = [50_000, 20_001], 16, 3
    x = [torch.randn(n, E, generator=g, device=DEV) for n in rows]
    idx = [torch.randint(-1, E, (n, K), generator=g, device=DEV, dtype=torch.int32) for n in rows]
    for group_len in (0, 1000):
        loss, counts, grads = ga.ga_balance_loss(x, idx, group_len=group_len)
        group = torch.from_numpy(np.concatenate(ol.groups_of(rows, group_len))).to(DEV)
        G = int(group.max()) + 1
        i = torch.cat(idx).long()
        flat = (group[:, None] * E + i)[i >= 0]
        want = torch.bincount(flat, minlength=G * E).view(G, E)
        assert torch.equal(counts.long(), want)
        n = torch.bincount(group, minlength=G).double()
        p = torch.softmax(torch.cat(x).double(), 1)
        f = (E * want.double() / (K * n[:, None]))[group]
        s = (f * p).sum(1)
        total = (s / n[group]).sum()
        tol = (4 * 12 + 2 * (E + 26)) * U
        assert abs(float(loss[0]) - float(total)) <= tol * float(total) and int(loss[1]) == G
        gw = p * (f - s[:, None]) / (G * n[group])[:, None]
        err = 3 * tol * (p * (f + s[:, None])) / (G * n[group])[:, None]
        assert ((torch.cat(grads).double() - gw).abs() <= err + 1e-38).all()


def test_workers_stacked_in_one_tensor():
    """A tensor is a sequence of its slices: [workers, rows, columns]."""
    x, r = torch.randn(3, 6, 40, device=DEV), torch.randn(3, 6, 8, device=DEV)
    mask = torch.rand(3, 6, device=DEV) < 0.7
    vals, idx, lse = (torch.stack(t) for t in ga.ga_top_logits(x, 4))
    experts = torch.stack(ga.ga_top_logits(r, 2, lse=False)[1])
    g, gr, was = torch.empty_like(x), torch.empty_like(r), torch.empty(1)._version
    loss, _ = ga.ga_distill_loss(x, idx, vals, lse, weight=mask.float(), grads=g)
    one, og = ga.ga_distill_loss(list(x), list(idx), list(vals), list(lse), weight=list(mask.float()))
    assert torch.equal(loss, one) and torch.equal(g, torch.stack(og)) and g._version > was
    for m in (mask, mask.to(torch.uint8)):
        loss, counts, _ = ga.ga_balance_loss(r, experts, m, grads=gr)
        one, oc, og = ga.ga_balance_loss(list(r), list(experts), list(m))
        assert torch.equal(loss, one) and torch.equal(counts, oc) and torch.equal(gr, torch.stack(og))


def test_binding_refusals():
    """Tensors that do not fit each other are refused before the library is
    called."""
    x = [torch.randn(4, 32, device=DEV), torch.randn(2, 32, device=DEV)]
    i = [torch.zeros(4, 3, dtype=torch.int32, device=DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV)]
    v = [torch.zeros(4, 3, device=DEV), torch.zeros(2, 3, device=DEV)]
    wide = torch.randn(4, 64, device=DEV)
    bad = [
        (TypeError, lambda: ga.ga_top_logits([x[0], x[1].to(BF16)], 3)),
        (TypeError, lambda: ga.ga_top_logits([x[0], x[1].cpu()], 3)),
        (TypeError, lambda: ga.ga_top_logits([x[0].half()], 3)),
        (TypeError, lambda: ga.ga_top_logits([x[0], 3], 3)),
        (TypeError, lambda: ga.ga_top_logits([torch._neg_view(x[0])], 3)),
        (ValueError, lambda: ga.ga_top_logits([x[0].T], 3)),
        (ValueError, lambda: ga.ga_top_logits([wide[:, ::2]], 3)),
        (ValueError, lambda: ga.ga_top_logits([x[0][0]], 3)),
        (ValueError, lambda: ga.ga_top_logits([x[0][:1].expand(4, 32)], 3)),
        (ValueError, lambda: ga.ga_top_logits([wide[:, :32], x[0]], 3)),          # two strides
        (ValueError, lambda: ga.ga_top_logits(x, 3, idx=i[:1])),
        (ValueError, lambda: ga.ga_top_logits(x, 4, idx=i)),
        (TypeError, lambda: ga.ga_top_logits(x, 3, idx=v)),
        (ga.GAError, lambda: ga.ga_top_logits(x, 33)),
        (ga.GAError, lambda: ga.ga_top_logits(x, 3, temp=0.0)),
        (TypeError, lambda: ga.ga_distill_loss(x, [t.long() for t in i], v)),
        (ValueError, lambda: ga.ga_distill_loss(x, i, v[::-1])),
        (TypeError, lambda: ga.ga_distill_loss(x, i, [t.half() for t in v])),
        (ValueError, lambda: ga.ga_distill_loss(x, i, v, weight=[torch.ones(4, device=DEV), torch.ones(3, device=DEV)])),
        (TypeError, lambda: ga.ga_distill_loss(x, i, v, grads=[t.to(BF16) for t in x])),
        (ValueError, lambda: ga.ga_distill_loss(x, i, v, out=torch.empty(2, device=DEV))),
        (ValueError, lambda: ga.ga_distill_loss(x, i, v, grads=[wide[:, :32], torch.empty(2, 32, device=DEV)])),
        (ga.GAError, lambda: ga.ga_distill_loss(x, i, v, ws=torch.empty(16, dtype=torch.uint8, device=DEV))),
        (ga.GAError, lambda: ga.ga_distill_loss(x, i, v, grads=[x[0], torch.empty(2, 32, device=DEV)])),
        (TypeError, lambda: ga.ga_balance_loss(x, i, [torch.ones(4, device=DEV), torch.ones(2, device=DEV)])),
        (ValueError, lambda: ga.ga_balance_loss(x, i, counts=torch.empty(2, 32, dtype=torch.int32, device=DEV))),
        (ga.GAError, lambda: ga.ga_balance_loss(x, i, group_len=-1)),
        (ga.GAError, lambda: ga.ga_balance_loss(x, i, score=7)),
    ]
    for k, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            print(f"refusal {k} was not refused")
    torch.cuda.synchronize()


def test_written_outputs_have_new_versions():
    """Autograd sees that a call wrote into a tensor: a backward pass that
    needs what stood there before is refused, as after torch's own calls."""
    x = [torch.randn(4, 32, device=DEV, requires_grad=True), torch.randn(2, 32, device=DEV, requires_grad=True)]
    i = [torch.zeros(4, 3, dtype=torch.int32, device=DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV)]
    v = [torch.zeros(4, 3, device=DEV), torch.zeros(2, 3, device=DEV)]

    def like(*shape, dtype=F32):
        return [torch.empty(n, *shape, dtype=dtype, device=DEV) for n in (4, 2)]

    capped = [torch.tanh(t) for t in x]
    loss, g = ga.ga_distill_loss(capped, i, v)
    torch.autograd.backward(capped, g)                   # how a gradient goes on
    assert all(torch.isfinite(t.grad).all() for t in x)
    capped = [torch.tanh(t) for t in x]
    ga.ga_distill_loss(capped, i, v, grads=capped)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.backward(capped, [torch.ones_like(t) for t in capped])

    vals, idx, lse, rows, grads = like(3), like(3, dtype=torch.int32), like(), like(), like(32)
    out, counts = torch.empty(3, device=DEV), torch.empty(1, 32, dtype=torch.int32, device=DEV)
    logits = [t.detach() for t in x]

    def versions(*ts):
        return [t._version for t in ts]

    for call, wrote in ((lambda: ga.ga_top_logits(logits, 3, vals=vals, idx=idx, lse=lse), [*vals, *idx, *lse]),
                        (lambda: ga.ga_distill_loss(logits, i, v, grads=grads, row_loss=rows, out=out),
                         [*grads, *rows, out]),
                        (lambda: ga.ga_balance_loss(logits, i, grads=grads, counts=counts, out=out),
                         [*grads, counts, out])):
        was, read = versions(*wrote), versions(*logits, *i, *v)
        call()
        assert all(a > b for a, b in zip(versions(*wrote), was))
        assert versions(*logits, *i, *v) == read
    was = versions(*grads, out)
    with pytest.raises(ga.GAError):
        ga.ga_distill_loss(logits, i, v, temp=0.0, grads=grads, out=out)
    assert versions(*grads, out) == was
    with torch.inference_mode():                         # tensors that have no versions
        o = torch.empty(3, device=DEV)
        ga.ga_distill_loss(logits, i, v, grads=False, out=o)
    ga.ga_distill_loss(logits, i, v, grads=False, out=o)
    torch.cuda.synchronize()


@pytest.mark.parametrize("temp", [1e-30, 1e-3, 1e30])
def test_far_temperatures(temp):
    """A softmax that is one-hot, and one that is even; teachers at the type's
    ends. Probabilities are then exact up to a few roundings."""
    x = torch.tensor([[1.0, 3.0, 2.0, -5.0], [3e38, -3e38, 0.0, 1.0]], device=DEV)
    i = torch.tensor([[1, 2], [0, 1]], dtype=torch.int32, device=DEV)
    v = torch.tensor([[4.0, 1.0], [3e38, -3e38]], device=DEV)
    loss, (g,) = ga.ga_distill_loss([x], [i], [v], temp=temp)
    p = torch.softmax(x.double() / temp, 1)
    q = torch.softmax(v.double() / temp, 1)
    want = (p.scatter_add(1, i.long(), -q)) * (temp / 2)
    assert torch.isfinite(g).all()
    assert ((g.double() - want).abs() <= 40 * U * temp).all()
    _, _, (l,) = ga.ga_top_logits([x], 2, temp=temp)
    exact = torch.logsumexp(x.double() / temp, 1)
    assert torch.equal(torch.isinf(l), exact.abs() > 3.4028235e38)
    ok = ~torch.isinf(l)
    assert ((l.double() - exact).abs()[ok] <= 40 * U * exact.abs()[ok] + 40 * U).all()


@pytest.mark.parametrize("temp", [5e-39, 1e-38, 1e-30, 1e-20, 1e-10])
def test_losses_at_low_temperatures(temp):
    """The teacher's softmax is one-hot, the student's too: a row's loss is
    temp times how far the teacher's column lies below the student's maximum,
    to ten roundings of the logits' sizes (the end's own, below 2^-126, half of
    its last place)."""
    x = torch.tensor([[1.0, 3.0, 2.0, -5.0], [1.0, 3.0, 2.0, -5.0], [3e38, -3e38, 0.0, 1.0], [-1e30, 7.0, 7.5, 0.0]],
                     device=DEV)
    i = torch.tensor([[1, 2], [1, 2], [0, 1], [0, 1]], dtype=torch.int32, device=DEV)
    v = torch.tensor([[4.0, 1.0], [1.0, 4.0], [-1.0, 5.0], [0.0, 1.0]], device=DEV)
    col = torch.tensor([1, 2, 1, 1])
    rows = [torch.empty(4, device=DEV)]
    loss, _ = ga.ga_distill_loss([x], [i], [v], temp=temp, row_loss=rows)
    z = _f64(x)
    t = float(np.float32(temp))
    at = z[np.arange(4), col]
    want = t * (z.max(1) - at)
    tol = 10 * U * t * (np.abs(z.max(1)) + np.abs(at)) + 2.0 ** -149
    print(want, _f64(rows[0]), flush=True)
    assert (np.abs(_f64(rows[0]) - want) <= tol).all()
    assert abs(_f64(loss)[0] - want.sum()) <= tol.sum() + U * want.sum()
    assert abs(_f64(loss)[2] - want.mean()) <= tol.mean() + U * want.mean()


@pytest.mark.parametrize("temp", [1e15, 1.9e19, 2.5e19, 1e30])
def test_losses_at_high_temperatures(temp):
    """Both softmaxes are even, over the teacher's slots and over all columns:
    temp^2 log(V / K), where temp^2 alone passes binary32's range."""
    V, K = 64, 60
    x = [torch.zeros(3, V, device=DEV)]
    i = [torch.arange(K, dtype=torch.int32, device=DEV).repeat(3, 1)]
    v = [torch.zeros(3, K, device=DEV)]
    rows = [torch.empty(3, device=DEV)]
    loss, grads = ga.ga_distill_loss(x, i, v, temp=temp, row_loss=rows)
    t = float(np.float32(temp))
    if t * t * np.log(V / K) > 3.5e38:
        assert torch.isposinf(rows[0]).all() and torch.isposinf(loss[[0, 2]]).all()
    else:
        _check_distill(x, i, v, None, None, t, 1.0, loss, grads, rows)


def test_the_lowest_temperatures_log_sum_exp():
    x = torch.full((2, 1003), -1.0, device=DEV)
    x[:, [5, 900]] = 0.0
    for temp in (4.5e-39, 1e-38):
        _, _, (lse,) = ga.ga_top_logits([x], 3, temp=temp)
        assert (np.abs(_f64(lse) - np.log(2)) <= 4 * U).all()


def _kernels(call):
    """How many kernels a call launches."""
    call()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    n = C.c_size_t()
    assert _loss.load().hipGraphGetNodes(C.c_void_p(g.raw_cuda_graph()), None, C.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("rows,launches", [([64], 1), ([8], 1), ([0], 1), ([192], 1), ([193], 3), ([1000], 3),
                                           ([1, 1, 1], 1), ([40, 70], 1), ([1] * 4, 3), ([3] * 16, 3), ([1] * 64, 3),
                                           ([4] * 64, 3), ([8] + [0] * 63, 1), ([0, 5, 0, 7, 0], 1),
                                           ([0] * 8, 1), ([0, 1000, 0, 5], 3)])
def test_one_launch_only_for_few_units(rows, launches):
    """One workgroup takes units one after another, at least one per worker:
    only a few of them."""
    x = [torch.randn(n, 8, device=DEV) for n in rows]
    idx = [torch.randint(0, 8, (n, 2), dtype=torch.int32, device=DEV) for n in rows]
    grads, out = [torch.empty_like(t) for t in x], torch.empty(3, device=DEV)
    counts, ws = torch.empty(1, 8, dtype=torch.int32, device=DEV), torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    assert _kernels(lambda: ga.ga_balance_loss(x, idx, grads=grads, counts=counts, out=out, ws=ws)) == launches
    _check_balance(x, idx, None, False, 0, 1.0, (out, counts, grads))


def _job(seed, tdt=BF16):
    rng = np.random.default_rng(seed)
    x = _logits(rng, [5, 3], 9001, tdt)
    idx, vals = _teacher(rng, [5, 3], 9001, 20, F32)
    weight = [torch.rand(n, device=DEV) for n in (5, 3)]
    r = _logits(rng, [300, 200], 64, tdt)
    return x, idx, vals, weight, r, _route(rng, r, 4)


def _all(j, stream=None):
    x, idx, vals, weight, r, e = j
    t = ga.ga_top_logits(x, 17, stream=stream)
    d = ga.ga_distill_loss(x, idx, vals, weight=weight, stream=stream)
    b = ga.ga_balance_loss(r, e, group_len=128, stream=stream)
    return [*t[0], *t[1], *t[2], d[0], *d[1], b[0], b[1], *b[2]]


def test_two_streams_at_once():
    jobs = [_job(1), _job(2)]
    want = [_all(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for k in (0, 1):
            got[k] = _all(jobs[k], streams[k] if k else streams[k].cuda_stream)
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(got[k], want[k]))


def test_captured_and_replayed():
    """Two graphs with allocations of their own, replayed in turn with eager
    work between and new inputs each time."""
    jobs = [_job(3), _job(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for j in jobs:
            _all(j)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_all(j))
        graphs.append(g)
    for rep in range(4):
        for j in jobs:
            j[0][0].copy_(torch.randn_like(j[0][0].float()).to(BF16) * 3)
            j[4][1].copy_(torch.randn_like(j[4][1].float()).to(BF16))
        for o in outs:
            for t in o:
                t.fill_(1)
        for g in graphs:
            g.replay()
        want = [_all(j) for j in jobs]
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w)), rep


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31 from the buffer's start, and workers'
    row counts that put them there."""
    V, ld, n = 1000, 1 << 20, 2200                       # 2.3e9 elements, 4.6 GB
    rng = np.random.default_rng(7)
    store = torch.zeros(n * ld, dtype=BF16, device=DEV)
    x = store.view(n, ld)[:, :V]
    last = _logits(rng, [4], V, BF16)[0]
    x[n - 4:] = last
    idx, vals = _teacher(rng, [4], V, 12, F32)
    full_i = torch.full((n, 12), -1, dtype=torch.int32, device=DEV)
    full_v = torch.zeros(n, 12, device=DEV)
    full_i[n - 4:], full_v[n - 4:] = idx[0], vals[0]
    w = torch.zeros(n, device=DEV)
    w[n - 4:] = 1
    _, ti, _ = ga.ga_top_logits([x], 9)
    assert np.array_equal(ti[0][n - 4:].cpu().numpy(), ol.top_logits(_f64(last), 9, 1.0)[0])
    loss, grads = ga.ga_distill_loss([x], [full_i], [full_v], weight=[w], grads=[x])
    _check_distill([last], idx, vals, None, None, 1.0, 1.0, loss, [x[n - 4:]], tdt=BF16)
    x[n - 4:] = last
    e = [torch.randint(0, 1000, (n, 2), dtype=torch.int32, device=DEV)]
    b, c, g = ga.ga_balance_loss([x], e, [w.to(torch.uint8)])
    _check_balance([last], [e[0][n - 4:]], None, False, 0, 1.0, (b, c, [g[0][n - 4:]]))


# ------------------------------------------------------------------ together, as a data-parallel step uses them
def test_the_longest_row():
    """2^31 - 1 columns: the last ones, and those past 2^30, have their numbers;
    masked ones count nothing."""
    V = 2 ** 31 - 1
    x = torch.empty(1, V, dtype=BF16, device=DEV)
    at = [V - 1, 5, 2 ** 30 + 3, V - 9]
    for rest in (-1.0, -INF):
        x.fill_(rest)
        for i, c in enumerate(at):
            x[0, c] = 8.0 - i
        print(f"longest row, the rest {rest}", flush=True)
        vals, idx, lse = ga.ga_top_logits([x], 6)
        assert idx[0][0].tolist() == at + [0, 1]         # equal values by column
        assert vals[0][0].tolist() == [8.0, 7.0, 6.0, 5.0, rest, rest]
        want = np.log(sum(np.exp(8.0 - i) for i in range(4)) + (V - 4) * np.exp(rest))
        # a thread's sum of 2^22 equal terms rounds each by half a step of it
        assert abs(float(lse[0]) - want) <= (2 ** 22 * U if rest == -1.0 else 30 * U) + 4 * U * want
    x.fill_(0.0)
    idx, vals = torch.tensor([[V - 1]], dtype=torch.int32, device=DEV), torch.zeros(1, 1, device=DEV)
    print("longest row, distilled", flush=True)
    loss, _ = ga.ga_distill_loss([x], [idx], [vals], grads=False)
    # 2^23 ones per thread are summed without rounding
    assert abs(float(loss[2]) - np.log(V)) <= 8 * U * np.log(V)


def test_a_long_rows_sum():
    """2^31 - 1 columns, all of them in the log-sum-exp: a part of 2^-11 of the
    row that was left out or taken twice would show. A thread's sum is rounded
    by the terms of a vector, of a run of rounds and by the runs: fewer than
    2^12 additions, each half a step."""
    V = 2 ** 31 - 1
    x = torch.full((1, V), -1.0, dtype=BF16, device=DEV)
    x[0, 77] = 0.0
    bound = 2.0 ** 12 * U
    want = np.log((V - 1) * np.exp(-1.0) + 1)
    for k in (4, 600):                                   # both kernels of long rows
        print(f"long row's sum, k={k}", flush=True)
        _, _, lse = ga.ga_top_logits([x], k)
        print(float(lse[0]) - want, bound, flush=True)
        assert abs(float(lse[0]) - want) <= bound + 4 * U * want
    idx, vals = torch.tensor([[77]], dtype=torch.int32, device=DEV), torch.zeros(1, 1, device=DEV)
    print("long row's sum, distilled", flush=True)
    for grads in (False, [x]):
        loss, _ = ga.ga_distill_loss([x], [idx], [vals], grads=grads)
        print(float(loss[2]) - want, bound, flush=True)
        assert abs(float(loss[2]) - want) <= bound + 8 * U * want


def test_workers_gradients_sum_to_the_batchs():
    """A teacher's top logits, the student's loss over four workers with
    different shares of the batch, each worker's parameter gradient, and the
    ring's sum of them: the gradient of the whole batch on one worker. The
    products are binary32 sums of n terms: off by (n + 2) u of their
    magnitudes' sum each, and the ring adds three roundings."""
    g = torch.Generator(device=DEV).manual_seed(5)
    rows, D, V, E, K = [37, 5, 64, 22], 48, 5000, 32, 4
    h = [torch.randn(n, D, generator=g, device=DEV) for n in rows]
    wt, ws = (torch.randn(D, V, generator=g, device=DEV) * 0.2 for _ in range(2))
    wr = torch.randn(D, E, generator=g, device=DEV) * 0.2
    weight = [torch.ones(n, device=DEV) for n in rows]
    weight[2][40:] = 0
    vals, idx, lse = ga.ga_top_logits([a @ wt for a in h], 50, temp=2.0)

    def step(hs, idx, vals, lse, weight):
        loss, gz = ga.ga_distill_loss([a @ ws for a in hs], idx, vals, lse, weight, temp=2.0)
        r = [a @ wr for a in hs]
        chosen = [t[:, :K].contiguous() for t in ga.ga_top_logits(r, K, lse=False)[1]]
        aux, counts, gr = ga.ga_balance_loss(r, chosen, [(w > 0) for w in weight], scale=0.1)
        flat = [torch.cat([(a.T @ z).reshape(-1), (a.T @ q).reshape(-1)]) for a, z, q in zip(hs, gz, gr)]
        mag = sum(torch.cat([(a.abs().T @ z.abs()).reshape(-1), (a.abs().T @ q.abs()).reshape(-1)])
                  for a, z, q in zip(hs, gz, gr))
        return loss, aux, counts, flat, mag

    loss, aux, counts, flat, mag = step(h, idx, vals, lse, weight)
    ga.ga_ring_allreduce_sim(flat, ga.SUM)
    one = step([torch.cat(h)], [torch.cat(idx)], [torch.cat(vals)], [torch.cat(lse)], [torch.cat(weight)])
    assert torch.equal(counts, one[2])
    assert int(counts.sum()) == K * (37 + 5 + 40 + 22)
    n = sum(rows)
    # the two runs' logits are the same products of the same rows, but a
    # library product may add in another order for another shape: 2 (D + 2) u
    # of each logit's magnitude, which moves a gradient's p by as much / temp
    zmag = max(float((a.abs() @ ws.abs()).max()) for a in h)
    rel = (2 * (D + 2) * zmag + 2 * n + 2000) * U
    assert abs(float(loss[2] - one[0][2])) <= 4 * rel * max(1.0, float(loss[2]))
    assert abs(float(aux[2] - one[1][2])) <= 4 * rel * max(1.0, float(aux[2]))
    for f in flat[1:]:
        assert torch.equal(f, flat[0])
    assert (_f64((flat[0] - one[3][0]).abs()) <= 4 * rel * _f64(one[4]) + 1e-30).all()
