"""The loss oracle against facts fixed outside it: torch's autograd in
binary64, closed forms and brute force."""
import numpy as np
import pytest
import torch

from oracle import loss as ol


def _distill_by_autograd(zs, idx, vals, lse, weight, temp, scale):
    zs = [torch.tensor(z, requires_grad=True) for z in zs]
    num, den = 0.0, 0.0
    for i, z in enumerate(zs):
        lp = torch.log_softmax(z / temp, 1)
        t = torch.tensor(vals[i]) / temp
        on = torch.tensor(idx[i]) >= 0
        t = t.masked_fill(~on, -np.inf)
        L = torch.logsumexp(t, 1) if lse is None else torch.tensor(lse[i])
        lq = t - L[:, None]
        q = lq.exp()
        at = lp.gather(1, torch.tensor(idx[i]).clamp(min=0))
        row = temp ** 2 * torch.where(on, q * (lq.masked_fill(~on, 0) - at), 0.0).sum(1)
        w = torch.ones(z.shape[0], dtype=torch.float64) if weight is None else torch.tensor(weight[i])
        num, den = num + (w * row).sum(), den + w.sum()
    loss = scale * num / den
    loss.backward()
    return float(loss), [z.grad.numpy() for z in zs]


@pytest.mark.parametrize("with_lse,with_w,temp", [(False, False, 1.0), (True, True, 2.0), (False, True, 0.5)])
def test_distill_equals_autograd(with_lse, with_w, temp):
    rng = np.random.default_rng(3)
    zs, idx, vals, lse, w = [], [], [], [], []
    for n in (3, 1, 4):
        zs.append(rng.standard_normal((n, 11)))
        i = rng.integers(0, 11, (n, 4))                       # repeats happen
        i[0, 1] = -1
        idx.append(i)
        vals.append(rng.standard_normal((n, 4)))
        lse.append(rng.standard_normal(n) + 3)
        w.append(rng.random(n))
    o = ol.distill(zs, idx, vals, lse if with_lse else None, w if with_w else None, temp, 0.7)
    loss, grads = _distill_by_autograd(zs, idx, vals, lse if with_lse else None, w if with_w else None, temp, 0.7)
    assert abs(o["loss"] - loss) <= 1e-12 * abs(loss)
    for a, b in zip(o["grads"], grads):
        assert np.abs(a - b).max() <= 1e-14


def test_distill_of_the_teacher_itself_is_zero():
    rng = np.random.default_rng(4)
    z = rng.standard_normal((5, 6))
    idx, vals, _ = ol.top_logits(z, 6, 1.0)
    o = ol.distill([z], [idx], [vals], None, None, 1.5, 1.0)
    assert abs(o["loss"]) <= 1e-15 and np.abs(o["grads"][0]).max() <= 1e-16


def test_distill_rows_that_hold_nothing():
    z = np.array([[-np.inf, -np.inf], [0.0, -np.inf], [1.0, 2.0]])
    idx = np.array([[0], [0], [-1]])
    o = ol.distill([z], [idx], [np.ones((3, 1))], None, None, 1.0, 1.0)
    assert o["num"] == 0.0 and o["den"] == 3.0 and not np.abs(o["grads"][0]).any()


def test_top_logits_by_brute_force():
    rng = np.random.default_rng(5)
    z = rng.integers(-2, 3, (20, 9)).astype(np.float64)       # many ties
    idx, vals, lse = ol.top_logits(z, 4, 1.0)
    for r in range(20):
        want = sorted(range(9), key=lambda v: (-z[r, v], v))[:4]
        assert idx[r].tolist() == want and vals[r].tolist() == [z[r, v] for v in want]
        assert abs(lse[r] - np.log(np.exp(z[r]).sum())) <= 1e-14 * 10


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("group_len", [0, 2, 3])
def test_balance_equals_autograd(sigmoid, group_len):
    rng = np.random.default_rng(6)
    E, K = 5, 2
    zs = [rng.standard_normal((n, E)) for n in (4, 1, 5)]
    idx = [rng.integers(-1, E, (z.shape[0], K)) for z in zs]
    mask = [rng.random(z.shape[0]) < 0.7 for z in zs]
    mask[1][:] = False
    o = ol.balance(zs, idx, mask, sigmoid, group_len, 0.3)
    ts = [torch.tensor(z, requires_grad=True) for z in zs]
    groups = ol.groups_of([z.shape[0] for z in zs], group_len)
    loss, live = 0.0, 0
    for g in range(o["counts"].shape[0]):
        rows = [(i, r) for i in range(3) for r in range(zs[i].shape[0]) if groups[i][r] == g and mask[i][r]]
        if not rows:
            assert not o["counts"][g].any()
            continue
        c = np.bincount([e for i, r in rows for e in idx[i][r] if e >= 0], minlength=E)
        assert (c == o["counts"][g]).all()
        x = torch.stack([ts[i][r] for i, r in rows])
        p = torch.sigmoid(x) if sigmoid else torch.softmax(x, 1)
        p = p / p.sum(1, keepdim=True)
        loss = loss + (torch.tensor(c) * E / (K * len(rows)) * p.mean(0)).sum()
        live += 1
    loss = 0.3 * loss / live
    loss.backward()
    assert abs(o["loss"] - float(loss)) <= 1e-14 and o["den"] == live
    for t, g in zip(ts, o["grads"]):
        assert np.abs((t.grad.numpy() if t.grad is not None else 0) - g).max() <= 1e-15


def test_balance_of_an_even_router_is_one():
    E, n = 4, 8
    idx = (np.arange(n) % E)[:, None]
    o = ol.balance([np.zeros((n, E))], [idx], None, False, 0, 1.0)
    assert abs(o["loss"] - 1.0) <= 1e-15 and np.abs(o["grads"][0]).max() <= 1e-16
