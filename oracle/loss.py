"""Oracle for the loss operators, in numpy binary64: a teacher's top logits,
distillation from them, and a router's balance loss with its counts.

Test infrastructure, like the rest of this folder. Rows come as one float64
matrix per worker. Written from the definitions, row by row:

* softmax with temperature tau: p = softmax(z / tau); an entry of -inf has
  probability 0, a row of -inf alone has no distribution (all 0);
* distillation (the forward divergence of the softened distributions, scaled
  by tau^2 so that its gradient keeps its size when tau changes):
  l = tau^2 sum_k q_k (log q_k - log p[idx_k]);
* balance: groups of rows, load f_e = E c_e / (K n), L = sum_e f_e mean_t p_te.
"""
from typing import List, Optional, Sequence

import numpy as np


def softmax(z: np.ndarray) -> np.ndarray:
    m = z.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.exp(z - np.where(np.isinf(m) & (m < 0), 0.0, m))
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s != 0)


def logsumexp(z: np.ndarray) -> np.ndarray:
    m = z.max(axis=1)
    base = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        return base + np.log(np.exp(z - base[:, None]).sum(axis=1))


def top_logits(z: np.ndarray, k: int, temp: float):
    """(columns of the k largest, their values, lse) of every row; equal
    values by column."""
    idx = np.argsort(-(z + 0.0), axis=1, kind="stable")[:, :k]
    return idx, np.take_along_axis(z, idx, axis=1), logsumexp(z / temp)


def distill(logits: Sequence[np.ndarray], idx: Sequence[np.ndarray], vals: Sequence[np.ndarray],
            lse: Optional[Sequence[np.ndarray]], weight: Optional[Sequence[np.ndarray]], temp: float,
            scale: float) -> dict:
    """num = sum w l, den = sum w, loss, per worker: rows (l), grads, and the
    parts of a gradient for error bounds: mass (p sum q) and slot (sum of q)
    with the factor coef of each row."""
    P = len(logits)
    if weight is None:
        weight = [np.ones(z.shape[0]) for z in logits]
    weight = [np.where(w > 0, w, 0.0).astype(np.float64) for w in weight]
    den = float(sum(w.sum() for w in weight))
    num = 0.0
    out = {"rows": [], "grads": [], "mass": [], "slot": [], "coef": [], "q": []}
    for i in range(P):
        z, n = logits[i], logits[i].shape[0]
        V, K = z.shape[1], idx[i].shape[1]
        rows, mass, slot = np.zeros(n), np.zeros((n, V)), np.zeros((n, V))
        coef, qs = np.zeros(n), np.zeros((n, K))
        for r in range(n):
            if weight[i][r] == 0:
                continue
            coef[r] = scale * temp * weight[i][r] / den
            if np.isneginf(z[r]).all():
                continue
            p = softmax(z[r:r + 1] / temp)[0]
            on = [k for k in range(K) if 0 <= idx[i][r, k] < V and not np.isneginf(vals[i][r, k])]
            if not on:
                continue
            t = vals[i][r, on] / temp
            L = lse[i][r] if lse is not None else logsumexp(t[None])[0]
            for j, k in enumerate(on):
                q = np.exp(t[j] - L)
                qs[r, k] = q
                v = idx[i][r, k]
                slot[r, v] += q
                # from the row's maximum: next to the type's lowest value a
                # log-sum-exp does not keep what it adds to it
                lp = (z[r, v] - z[r].max()) / temp - logsumexp((z[r:r + 1] - z[r].max()) / temp)[0]
                if q > 0:
                    rows[r] += temp ** 2 * q * ((t[j] - L) - lp)
            mass[r] = p * qs[r].sum()
        num += float((weight[i] * rows)[weight[i] > 0].sum())
        out["rows"].append(rows)
        out["mass"].append(mass)
        out["slot"].append(slot)
        out["coef"].append(coef)
        out["q"].append(qs)
        out["grads"].append((mass - slot) * coef[:, None])
    out.update(num=num, den=den, loss=scale * num / den if den > 0 else 0.0)
    return out


def groups_of(tokens: Sequence[int], group_len: int) -> List[np.ndarray]:
    """The group of every row, per worker."""
    out, first = [], 0
    for t in tokens:
        if group_len == 0:
            out.append(np.zeros(t, dtype=np.int64))
        else:
            out.append(first + np.arange(t) // group_len)
            first += -(-t // group_len)
    return out


def balance(logits: Sequence[np.ndarray], idx: Sequence[np.ndarray], mask: Optional[Sequence[np.ndarray]],
            sigmoid: bool, group_len: int, scale: float) -> dict:
    tokens = [z.shape[0] for z in logits]
    E, K = logits[0].shape[1], idx[0].shape[1]
    groups = groups_of(tokens, group_len)
    G = 1 if group_len == 0 else sum(-(-t // group_len) for t in tokens)
    counts, n = np.zeros((G, E), dtype=np.int64), np.zeros(G, dtype=np.int64)
    on = [np.ones(t, bool) if mask is None else np.asarray(mask[i]) != 0 for i, t in enumerate(tokens)]
    for i, t in enumerate(tokens):
        for r in range(t):
            if on[i][r]:
                n[groups[i][r]] += 1
                for e in idx[i][r]:
                    if 0 <= e < E:
                        counts[groups[i][r], e] += 1
    live = int((n > 0).sum())
    total, grads, scores, means = 0.0, [], [], []
    for i, t in enumerate(tokens):
        g = np.zeros((t, E))
        p = np.zeros((t, E))
        s = np.zeros(t)
        for r in range(t):
            if not on[i][r]:
                continue
            k = groups[i][r]
            f = E * counts[k] / (K * n[k])
            x = logits[i][r]
            if sigmoid:
                with np.errstate(over="ignore"):
                    a = 1 / (1 + np.exp(-x))
                    rest = 1 / (1 + np.exp(x))                 # 1 - a, which cancels for large x
                p[r] = a / a.sum() if a.sum() > 0 else 0.0
                slope = p[r] * rest
            else:
                p[r] = softmax(x[None])[0]
                slope = p[r]
            s[r] = f @ p[r]
            total += s[r] / n[k]
            g[r] = scale / (live * n[k]) * slope * (f - s[r])
        grads.append(g)
        scores.append(p)
        means.append(s)
    return {"num": total, "den": live, "loss": scale * total / live if live else 0.0, "counts": counts, "n": n,
            "grads": grads, "p": scores, "s": means}
