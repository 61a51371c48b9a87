"""The loss operators over P data-parallel workers and the cases they are
measured on: the teacher's top logits (ga_top_logits), the distillation loss
that reads them, with its gradient (ga_distill_loss), and the balance loss of
a router with the per-expert counts and its gradient (ga_balance_loss).

run() computes each either in plain torch operations (own = False) or with
the library's kernels (own = True), on the same inputs and into the same
outputs. exact() is the definition in binary64.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a teacher decoding one sequence: one row, latency is all there is
        dict(name="top 1x32768 bf16", op="top", P=1, T=1, V=32768, dt="bf16", K=16, pad=0, temp=1.0),
        # four workers' ragged batches, an odd vocabulary: rows start anywhere
        dict(name="top 4x~300x50003 bf16", op="top", P=4, T=300, V=50003, dt="bf16", K=64, pad=0, temp=2.0),
        # binary32 logits of a small vocabulary, padded rows
        dict(name="top 2x1024x32000 f32", op="top", P=2, T=1024, V=32000, dt="f32", K=32, pad=64, temp=1.0),
        # a teacher's pass over two workers' batches with a large vocabulary
        dict(name="top 2x1024x131072 bf16", op="top", P=2, T=1024, V=131072, dt="bf16", K=128, pad=0, temp=1.0),

        # a few positions of one sequence (a short fine-tuning sample)
        dict(name="distill 1x8x32768 bf16", op="distill", P=1, T=8, V=32768, dt="bf16", K=16, pad=0, temp=1.0,
             lse=False, weights=False, grad=True),
        # binary32 logits, ragged batches with padded positions, odd vocabulary
        dict(name="distill 4x~300x50003 f32", op="distill", P=4, T=300, V=50003, dt="f32", K=32, pad=0, temp=2.0,
             lse=False, weights=True, grad=True),
        # evaluation: the loss alone, of the whole batch and of every position
        dict(name="distill eval 2x1024x65536", op="distill", P=2, T=1024, V=65536, dt="bf16", K=64, pad=0,
             temp=1.0, lse=True, weights=True, grad=False),
        # a training step of eight workers with a large vocabulary
        dict(name="distill 8x512x131072 bf16", op="distill", P=8, T=512, V=131072, dt="bf16", K=64, pad=0,
             temp=1.0, lse=True, weights=True, grad=True),

        # one short sequence through a small router
        dict(name="balance 1x64x8 f32", op="balance", P=1, T=64, E=8, dt="f32", K=2, score="softmax", group=0,
             masked=False),
        # eight workers, 64 experts, padded positions, one global batch
        dict(name="balance 8x~4096x64 bf16", op="balance", P=8, T=4096, E=64, dt="bf16", K=6, score="softmax",
             group=0, masked=True),
        # sigmoid scores, the loss of every sequence for itself
        dict(name="balance 4x~16384x160 f32", op="balance", P=4, T=16384, E=160, dt="f32", K=6, score="sigmoid",
             group=4096, masked=True),
        # eight workers' full batches over 256 experts
        dict(name="balance 8x16384x256 bf16", op="balance", P=8, T=16384, E=256, dt="bf16", K=8, score="softmax",
             group=0, masked=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["top", "distill", "balance"])
    P = rng.choice([1, 1, 2, 3, 4, 8])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "balance":
        E = rng.choice([8, 16, 32, 60, 64, 128, 160, 256, 384, 512])
        T = _log_int(rng, 1, min(32768, (1 << 24) // (P * E)))
        return dict(op=op, P=P, T=T, E=E, dt=dt, K=rng.randint(1, min(8, E)),
                    score=rng.choice(["softmax", "sigmoid"]), group=rng.choice([0, 0, 512, 4096]),
                    masked=rng.random() < 0.5)
    V = _log_int(rng, 1000, 160000)
    if rng.random() < 0.5:
        V = V // 64 * 64
    T = _log_int(rng, 1, max(1, min(4096, (1 << 28) // (P * V))))
    case = dict(op=op, P=P, T=T, V=V, dt=dt, K=_log_int(rng, 1, 256), pad=rng.choice([0, 0, 8, 64]),
                temp=rng.choice([1.0, 1.0, 2.0, 0.7]))
    if op == "distill":
        case.update(lse=rng.random() < 0.5, weights=rng.random() < 0.5, grad=rng.random() < 0.8)
    return case


def _tokens(case):
    """Rows of each worker: the first holds T, the others up to 12% fewer
    where the name of the case says so (an odd T, or a masked batch)."""
    T, P = case["T"], case["P"]
    ragged = case.get("masked") or case.get("weights") or case.get("V", 0) % 2
    return [max(1, T - (T * (i % 4)) // 25) if ragged else T for i in range(P)]


def _padding(case, t):
    """Rows at a worker's end that are padding (weight 0, or masked)."""
    return t // 9 if case.get("weights") or case.get("masked") else 0


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    tdt = DTYPES[case["dt"]]
    tok = _tokens(case)
    if case["op"] == "balance":
        return _prepare_balance(case, gen, dev, tdt, tok)
    V, K, pad = case["V"], case["K"], case["pad"]
    s = {"case": case, "temp": case["temp"], "k": K}
    s["logits"] = [(torch.randn(t, V + pad, generator=gen, device=dev, dtype=tdt) * 2)[:, :V] for t in tok]
    if case["op"] == "top":
        # a peak at a few places, as a language model's logits have them
        for x in s["logits"]:
            at = torch.randint(V, (x.shape[0], 4), generator=gen, device=dev)
            x.scatter_add_(1, at, torch.rand(at.shape, generator=gen, device=dev).to(tdt) * 8)
        s["vals"] = [torch.empty(t, K, dtype=tdt, device=dev) for t in tok]
        s["idx"] = [torch.empty(t, K, dtype=torch.int32, device=dev) for t in tok]
        s["lse"] = [torch.empty(t, dtype=torch.float32, device=dev) for t in tok]
        return s
    s["idx"], s["vals"] = [], []
    for x in s["logits"]:
        t = x.shape[0]
        first = torch.randint(V, (t, 1), generator=gen, device=dev)
        step = torch.randint(1, V // K + 1, (t, 1), generator=gen, device=dev)
        at = (first + step * torch.arange(K, device=dev)) % V             # K places, none twice
        top = torch.sort(torch.randn(t, K, generator=gen, device=dev) * 2 + 7, dim=1, descending=True)[0]
        x.scatter_(1, at, (top + 0.7 * torch.randn(t, K, generator=gen, device=dev)).to(tdt))
        # every fifth row of the teacher holds fewer: its last slots are empty
        short = (torch.arange(t, device=dev) % 5 == 4)[:, None] & (torch.arange(K, device=dev) >= K - K // 4)
        s["idx"].append(torch.where(short, -1, at).to(torch.int32))
        s["vals"].append(top.to(tdt))
    s["teacher_lse"] = None
    if case["lse"]:
        # the teacher's own sum over its vocabulary: 5% of it outside its top
        s["teacher_lse"] = [torch.logsumexp(v.float() / case["temp"], 1) + 0.05 for v in s["vals"]]
    s["weight"] = None
    if case["weights"]:
        s["weight"] = [torch.rand(t, generator=gen, device=dev) + 0.5 for t in tok]
        for w in s["weight"]:
            w[w.numel() - _padding(case, w.numel()):] = 0
    s["grads"] = [torch.empty(t, V, dtype=tdt, device=dev) for t in tok] if case["grad"] else None
    s["row_loss"] = None if case["grad"] else [torch.empty(t, dtype=torch.float32, device=dev) for t in tok]
    s["loss"] = torch.empty(3, dtype=torch.float32, device=dev)
    return s


def _prepare_balance(case, gen, dev, tdt, tok):
    E, K = case["E"], case["K"]
    s = {"case": case}
    liked = torch.randn(E, generator=gen, device=dev) * 0.5               # some experts are liked more
    s["logits"] = [(torch.randn(t, E, generator=gen, device=dev) * 1.5 + liked).to(tdt) for t in tok]
    s["idx"] = []
    for x in s["logits"]:
        at = torch.topk(x.float() + 0.1 * torch.randn(x.shape, generator=gen, device=dev), K, dim=1)[1]
        full = torch.rand(at.shape, generator=gen, device=dev) < 0.02      # slots an expert had no room for
        s["idx"].append(torch.where(full, -1, at).to(torch.int32))
    s["mask"] = None
    if case["masked"]:
        s["mask"] = [torch.ones(t, dtype=torch.uint8, device=dev) for t in tok]
        for m in s["mask"]:
            m[m.numel() - _padding(case, m.numel()):] = 0
    s["grads"] = [torch.empty(t, E, dtype=tdt, device=dev) for t in tok]
    s["loss"] = torch.empty(3, dtype=torch.float32, device=dev)
    s["counts"] = torch.empty(_groups(case, tok)[0], E, dtype=torch.int32, device=dev)
    return s


def _groups(case, tok):
    """(number of groups, first group of each worker)."""
    g = case["group"]
    if not g:
        return 1, [0] * len(tok)
    n = [-(-t // g) for t in tok]
    return sum(n), [sum(n[:i]) for i in range(len(n))]


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if op == "top":
        return _run_top(state)
    if op == "distill":
        return _run_distill(state)
    return _run_balance(state)


def _run_top(s):
    if own:
        import gradient_all_reduce_worker_amd as ga
        vals, idx, lse = ga.ga_top_logits(s["logits"], s["k"], temp=s["temp"], vals=s["vals"], idx=s["idx"],
                                          lse=s["lse"])
        return {"vals": vals, "idx": idx, "lse": lse}
    rows = [_plain_top(x, s["k"], s["temp"]) for x in s["logits"]]
    return {"vals": [r[0] for r in rows], "idx": [r[1] for r in rows], "lse": [r[2] for r in rows]}


def _plain_top(x, k, temp):
    V = x.shape[1]
    f = x.float() + 0.0
    bits = f.view(torch.int32)
    order = bits ^ ((bits >> 31) & 0x7FFFFFFF)                  # as signed integers, in the values' order
    # the lower column is the larger key among equal values
    key = (order.to(torch.int64) << 32) + (V - 1 - torch.arange(V, device=x.device))
    idx = V - 1 - (torch.topk(key, k, dim=1)[0] & 0xFFFFFFFF)
    f = f / temp
    m = f.amax(1, keepdim=True)
    lse = m[:, 0] + (f - m).exp().sum(1).log()
    return x.gather(1, idx), idx.to(torch.int32), lse


def _run_distill(s):
    if own:
        import gradient_all_reduce_worker_amd as ga
        loss, grads = ga.ga_distill_loss(s["logits"], s["idx"], s["vals"], lse=s["teacher_lse"],
                                         weight=s["weight"], temp=s["temp"], grads=s["grads"],
                                         row_loss=s["row_loss"], out=s["loss"])
        return {"loss": loss, "grads": grads, "row_loss": s["row_loss"]}
    c = s["case"]
    none = [None] * len(s["logits"])
    weight = s["weight"] or [torch.ones(x.shape[0], device=x.device) for x in s["logits"]]
    den = sum(w.double().sum() for w in weight)
    rows = [_plain_distill(z, i, v, l, w, den, s["temp"], c["grad"])
            for z, i, v, l, w in zip(s["logits"], s["idx"], s["vals"], s["teacher_lse"] or none, weight)]
    num = sum(r[0] for r in rows)
    return {"loss": torch.stack([num, den, num / den]).float(), "grads": [r[1] for r in rows] if c["grad"] else None,
            "row_loss": None if c["grad"] else [r[1] for r in rows]}


def _plain_distill(z, idx, vals, lse, w, den, temp, grad):
    x = z.float() / temp
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(1, keepdim=True)
    kept = idx >= 0
    at = idx.clamp(min=0).long()
    t = torch.where(kept, vals.float() / temp, -math.inf)
    if lse is None:
        top = t.amax(1, keepdim=True)
        log_q = t - top - (t - top).exp().sum(1, keepdim=True).log()
    else:
        log_q = t - lse[:, None]
    q = torch.where(kept, log_q.exp(), 0.0)
    log_p = x.gather(1, at) - m - total.log()
    row = temp * temp * torch.where(kept, q * (log_q - log_p), 0.0).sum(1)
    row = torch.where(w > 0, row, 0.0)
    num = (w.double() * row.double()).sum()
    if not grad:
        return num, row
    g = e / total * q.sum(1, keepdim=True)
    g.scatter_add_(1, at, -q)
    return num, (g * (temp * w / den.float())[:, None]).to(z.dtype)


def _run_balance(s):
    c = s["case"]
    if own:
        import gradient_all_reduce_worker_amd as ga
        loss, counts, grads = ga.ga_balance_loss(
            s["logits"], s["idx"], mask=s["mask"],
            score=ga.SCORE_SIGMOID if c["score"] == "sigmoid" else ga.SCORE_SOFTMAX, group_len=c["group"],
            grads=s["grads"], counts=s["counts"], out=s["loss"])
        return {"loss": loss, "counts": counts, "grads": grads}
    E, K = c["E"], c["K"]
    dev = s["loss"].device
    tok = [x.shape[0] for x in s["logits"]]
    G, first = _groups(c, tok)
    group = torch.cat([b + (torch.arange(t, device=dev) // c["group"] if c["group"]
                            else torch.zeros(t, dtype=torch.int64, device=dev)) for b, t in zip(first, tok)])
    x = torch.cat(s["logits"]).float()
    idx = torch.cat(s["idx"]).long()
    valid = torch.cat(s["mask"]) != 0 if s["mask"] else torch.ones(x.shape[0], dtype=torch.bool, device=dev)
    n = torch.zeros(G, dtype=torch.int64, device=dev).index_add_(0, group, valid.long())
    kept = (idx >= 0) & valid[:, None]
    counts = torch.zeros(G * E, dtype=torch.int64, device=dev)
    counts = counts.index_add_(0, (group[:, None] * E + idx.clamp(min=0)).view(-1), kept.view(-1).long()).view(G, E)
    if c["score"] == "sigmoid":
        a = 1 / (1 + (-x).exp())
        p = a / a.sum(1, keepdim=True)
        slope = p * (1 - a)
    else:
        e = (x - x.amax(1, keepdim=True)).exp()
        p = slope = e / e.sum(1, keepdim=True)
    live = n.clamp(min=1)
    f = E * counts / (K * live[:, None]).float()                # load of each expert: 1 where it is even
    f = f[0] if G == 1 else f[group]
    mean = (p * f).sum(1, keepdim=True)
    per_row = torch.where(valid, 1.0 / live.double()[group], 0.0)
    num = (mean[:, 0].double() * per_row).sum()
    den = (n > 0).sum().double()
    grad = slope * (f - mean) * (per_row / den).float()[:, None]
    grad = grad.to(s["logits"][0].dtype)
    return {"loss": torch.stack([num, den, num / den]).float(), "counts": counts.to(torch.int32),
            "grads": list(torch.split(grad, tok))}


# ------------------------------------------------------------------ what a pass needs
def work(case):
    tok = _tokens(case)
    rows = sum(tok)
    live = sum(t - _padding(case, t) for t in tok)
    es = 4 if case["dt"] == "f32" else 2
    K = case["K"]
    if case["op"] == "balance":
        E = case["E"]
        moved = live * (E * es + 4 * K) + rows * E * es + (rows if case["masked"] else 0)
        return {"bytes": moved + _groups(case, tok)[0] * E * 4 + 12, "flops": 12.0 * live * E}
    V = case["V"]
    if case["op"] == "top":
        return {"bytes": rows * (V * es + K * (es + 4) + 4), "flops": 5.0 * rows * V}
    moved = live * (V * es + K * (es + 4) + (4 if case["lse"] else 0)) + (4 * rows if case["weights"] else 0) + 12
    moved += 0 if case["grad"] else 4 * rows
    return {"bytes": moved + (rows * V * es if case["grad"] else 0), "flops": (9.0 if case["grad"] else 5.0) * live * V}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "top":
        vals, lse = [], []
        for x in s["logits"]:
            v, l = [], []
            for part in torch.split(x, 64):
                d = part.double()
                v.append(torch.sort(d, dim=1, descending=True)[0][:, :case["K"]])
                l.append(torch.logsumexp(d / case["temp"], 1))
            vals.append(torch.cat(v))
            lse.append(torch.cat(l))
        return {"vals": vals, "idx": [None] * len(vals), "lse": lse}
    if case["op"] == "distill":
        return _exact_distill(case, s)
    return _exact_balance(case, s)


def _exact_distill(case, s):
    tau, total_w, num, grads, row_loss = case["temp"], 0.0, 0.0, [], []
    P = len(s["logits"])
    weight = [s["weight"][i].double() if s["weight"] else
              torch.ones(s["logits"][i].shape[0], dtype=torch.float64, device=s["loss"].device) for i in range(P)]
    total_w = float(torch.cat(weight).sum())
    for i in range(P):
        z, out, losses = s["logits"][i], [], []
        for lo in range(0, z.shape[0], 64):
            rows = slice(lo, lo + 64)
            log_p = torch.log_softmax(z[rows].double() / tau, 1)
            at, u = s["idx"][i][rows].long(), s["vals"][i][rows].double() / tau
            dense = torch.zeros_like(log_p)                      # the teacher's distribution, spread out
            ent = torch.zeros(at.shape[0], dtype=torch.float64, device=z.device)
            u = u.masked_fill(at < 0, -math.inf)
            log_q = u - (torch.logsumexp(u, 1) if s["teacher_lse"] is None
                         else s["teacher_lse"][i][rows].double())[:, None]
            for k in range(at.shape[1]):
                on = at[:, k] >= 0
                dense[on, at[on, k]] += log_q[on, k].exp()
                ent[on] += log_q[on, k].exp() * log_q[on, k]
            row = tau ** 2 * (ent - (dense * log_p).sum(1))
            row = torch.where(weight[i][rows] > 0, row, 0.0)
            num += float((weight[i][rows] * row).sum())
            losses.append(row)
            if case["grad"]:
                g = log_p.exp() * dense.sum(1, keepdim=True) - dense
                out.append(g * (tau * weight[i][rows] / total_w)[:, None])
        if case["grad"]:
            grads.append(torch.cat(out))
        else:
            row_loss.append(torch.cat(losses))
    return {"loss": torch.tensor([num, total_w, num / total_w], dtype=torch.float64),
            "grads": grads if case["grad"] else None, "row_loss": None if case["grad"] else row_loss}


def _exact_balance(case, s):
    """By the chain rule group after group: the loss of a group as a function
    of its probabilities, and theirs of the logits."""
    E, K = case["E"], case["K"]
    tok = [x.shape[0] for x in s["logits"]]
    grads = [torch.zeros(t, E, dtype=torch.float64, device=s["loss"].device) for t in tok]
    valid = [s["mask"][i] != 0 if s["mask"] else torch.ones(t, dtype=torch.bool, device=s["loss"].device)
             for i, t in enumerate(tok)]
    if case["group"]:
        parts = [[(i, lo, min(lo + case["group"], t))] for i, t in enumerate(tok) for lo in range(0, t, case["group"])]
    else:
        parts = [[(i, 0, t) for i, t in enumerate(tok)]]
    losses, todo = [], []
    for part in parts:
        x = torch.cat([s["logits"][i][a:b][valid[i][a:b]] for i, a, b in part]).double()
        at = torch.cat([s["idx"][i][a:b][valid[i][a:b]] for i, a, b in part]).long().view(-1)
        n = x.shape[0]
        if not n:
            continue
        load = torch.bincount(at[at >= 0], minlength=E).double() * E / (K * n)
        if case["score"] == "sigmoid":
            a = torch.sigmoid(x)
            p = a / a.sum(1, keepdim=True)
            back = load - p @ load[:, None]
            g = a * torch.sigmoid(-x) / a.sum(1, keepdim=True) * back
        else:
            p = torch.softmax(x, 1)
            g = p * load - p * (p @ load[:, None])
        losses.append(float(load @ p.mean(0)))
        todo.append((part, g / n))
    for part, g in todo:
        g = g / len(losses)
        for i, a, b in part:
            m = int(valid[i][a:b].sum())
            grads[i][a:b][valid[i][a:b]] = g[:m]
            g = g[m:]
    num = sum(losses)
    return {"loss": torch.tensor([num, len(losses), num / len(losses)], dtype=torch.float64), "counts": None,
            "grads": grads}
