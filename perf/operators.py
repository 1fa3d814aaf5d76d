"""Measurement cases of the decode-step operators of a streaming codec decoder: the attention
of one new token over a paged key-value cache, the eviction that bounds that cache, and the
sampling of the next code.

Three operators, by a case's ``op``:

attend   q [B, Hq, D] attends to the n_b = len_b + 1 rows that sequence b has in a paged cache
         once its new row (k_new, v_new) has been put at slot len_b:
             p[b, h, j] = softmax_j(q[b, h] . k[b, h // G, j] / sqrt(D)),  out = sum_j p v,
         G = Hq / Hkv, over the last ``window`` slots if there is a window; with ``weights``
         also  w_out[b, hk, j] = w_in[b, hk, j] + sum_{h of hk's group} p[b, h, j].
evict    of the len_b slots of every (sequence, head), keeps the first ``sinks``, the last
         ``recent`` and those with the largest accumulated weight, ``budget`` in all (ties: the
         lowest slot), and copies their K and V rows and weights, in order, to other pages.
sample   one token a row from logits: temperature, then top-k, top-p and min-p, each a prefix
         of the tokens by (logit descending, index ascending), then the race
         argmax_i exp((l_i - max) / T) / e_i of given Exp(1) numbers e.

Sizes are generic: codebooks of 2048 entries and heads of 64 for a codec's own decoder, heads
of 128 and vocabularies of 10^5 for a language model that writes its codes.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _attend(name, **kw):
    case = dict(op="attend", B=1, Hq=32, Hkv=8, D=128, page=64, lo=128, hi=128, dtype="bf16",
                layout="head", window=0, weights=False)
    case.update(kw, name=name)
    return case


def listed():
    return [
        # One stream of a codec's decoder: ten seconds of frames, every head its own K and V.
        # The smallest call, where only latency counts.
        _attend("attend one stream", Hq=16, Hkv=16, D=64, page=16, lo=125, hi=125),
        # A small serving batch at ordinary, ragged lengths.
        _attend("attend ragged batch", B=16, page=16, lo=37, hi=4099, dtype="f16"),
        # One long session: all the work lies along one sequence's length.
        _attend("attend long session", lo=131071, hi=131071),
        # A full serving batch, lengths from one token up: the largest call.
        _attend("attend full batch", B=128, lo=0, hi=8191),
        # fp32 caches, token-major pages, an odd page size, a sliding window of 250 frames
        # and a head size that is no power of two.
        _attend("attend f32 window", B=24, Hq=16, Hkv=8, D=80, page=20, lo=3, hi=1501,
                dtype="f32", layout="token", window=750),
        # A batch whose caches are kept bounded: attention that also accumulates its weights.
        _attend("attend with weights", B=8, page=32, lo=5000, hi=9001, weights=True),
        # The steady state of bounded caches: a few pages over the budget, some rows under it.
        dict(name="evict steady", op="evict", B=16, Hkv=8, D=128, page=16, lo=1500, hi=2304,
             budget=2048, sinks=4, recent=256, dtype="bf16", layout="head"),
        # After a long prompt: one row in thirty stays.
        dict(name="evict long prompt", op="evict", B=2, Hkv=8, D=64, page=64, lo=30011, hi=32767,
             budget=1000, sinks=8, recent=128, dtype="f16", layout="token"),
        # The eight codebooks of one frame.
        dict(name="sample codebooks", op="sample", rows=8, V=2048, dtype="f32", T=1.0, k=250,
             p=1.0, minp=0.0),
        # One row of a large vocabulary, all filters on.
        dict(name="sample one row", op="sample", rows=1, V=131072, dtype="f32", T=0.7, k=50,
             p=0.95, minp=0.02),
        # A serving batch: nucleus sampling.
        dict(name="sample batch", op="sample", rows=64, V=32768, dtype="bf16", T=0.8, k=0, p=0.9,
             minp=0.0),
        # A full batch with an odd vocabulary, whose rows start at odd addresses.
        dict(name="sample full batch", op="sample", rows=256, V=100003, dtype="f16", T=1.0, k=0,
             p=0.95, minp=0.05),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "evict", "sample"])
    if op == "attend":
        dtype = rng.choice(["bf16", "f16", "f32"])
        D = rng.choice([64, 80, 96, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        G = rng.choice([1, 2, 3, 4, 8])
        B = _log_uniform(rng, 1, 128)
        row = 2 * Hkv * D * (4 if dtype == "f32" else 2)
        hi = min(_log_uniform(rng, 1, 131072), int(1.0e9 / (B * row)))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, page=rng.choice([8, 16, 24, 64, 128]),
                    lo=rng.randint(0, hi), hi=hi, dtype=dtype,
                    layout=rng.choice(["head", "token"]),
                    window=rng.choice([0, 0, max(1, hi // 2)]), weights=rng.random() < 0.25)
    if op == "evict":
        B, Hkv, D = _log_uniform(rng, 1, 32), rng.choice([2, 4, 8]), rng.choice([64, 80, 128])
        hi = min(_log_uniform(rng, 256, 65536), int(5.0e8 / (B * Hkv * D * 4)))
        budget = _log_uniform(rng, 64, hi)
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=rng.choice([8, 16, 24, 64]),
                    lo=rng.randint(hi // 2, hi), hi=hi, budget=budget,
                    sinks=rng.randint(0, budget // 4), recent=rng.randint(0, budget // 2),
                    dtype=rng.choice(["bf16", "f16", "f32"]), layout=rng.choice(["head", "token"]))
    V = _log_uniform(rng, 1000, 200000)
    rows = min(_log_uniform(rng, 1, 256), 25000000 // V)
    return dict(op=op, rows=rows, V=V, dtype=rng.choice(["bf16", "f16", "f32"]),
                T=round(rng.uniform(0.5, 1.3), 2), k=rng.choice([0, _log_uniform(rng, 1, 999)]),
                p=rng.choice([1.0, round(rng.uniform(0.5, 0.99), 3)]),
                minp=rng.choice([0.0, round(rng.uniform(0.01, 0.2), 3)]))


def _lengths(case):
    """B lengths spread evenly over lo..hi, in an order that is not sorted."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    even = [lo + (hi - lo) * i // max(1, B - 1) for i in range(B)] if B > 1 else [hi]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, B) == 1)
    return [even[(i * step) % B] for i in range(B)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

    s = dict(case=dict(case))
    if case["op"] == "sample":
        rows, V = case["rows"], case["V"]
        s["logits"] = normal(rows, V, scale=3.0)
        s["noise"] = torch.empty(rows, V, device="cuda").exponential_(generator=g)
        # Every eighth request of a batch asks for the most likely token (temperature 0).
        T = [0.0 if i % 8 == 7 else case["T"] for i in range(rows)]
        s["T"] = torch.tensor(T, dtype=torch.float32, device="cuda")
        s["k"] = torch.full((rows,), case["k"], dtype=torch.int32, device="cuda")
        s["p"] = torch.full((rows,), case["p"], dtype=torch.float32, device="cuda")
        s["minp"] = torch.full((rows,), case["minp"], dtype=torch.float32, device="cuda")
        if own:   # the plan that a program keeps; the plain form has none
            import transposed_convolution_gb300 as ctr
            s["plan"] = ctr.Sampler(rows, V, dtype=dt)
        return s

    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    lens = _lengths(case)
    evict = case["op"] == "evict"
    # The cache: as many pages as the lengths need, dealt out in a random order.
    need = [max(1, -(-(n if evict else n + 1) // page)) for n in lens]
    most, used = max(need), sum(need)
    order = torch.randperm(used, generator=g, device="cuda").tolist()
    tables, at = np.zeros((B, most), np.int32), 0
    for b in range(B):
        tables[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["tables"] = torch.from_numpy(tables).cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    total = used
    if evict:
        most_to = -(-case["budget"] // page)
        s["to"] = torch.arange(used, used + B * most_to, dtype=torch.int32,
                               device="cuda").view(B, most_to)
        s["first"] = used
        total += B * most_to
    shape = (total, Hkv, page, D) if case["layout"] == "head" else (total, page, Hkv, D)
    s["k"], s["v"] = normal(*shape), normal(*shape)
    if evict:
        # Weights accumulated over a run are uneven: a few slots hold most of the mass.
        s["w"] = torch.empty(B, Hkv, most * page, device="cuda").exponential_(generator=g) ** 3
        s["w_out"] = torch.zeros(B, Hkv, case["budget"], device="cuda")
    else:
        # Projections of one buffer, as a fused QKV product leaves them: strided rows.
        Hq = case["Hq"]
        qkv = normal(B, Hq + 2 * Hkv, D)
        qkv[:, :Hq] *= 2.0
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if case["weights"]:
            s["w"] = torch.rand(B, Hkv, most * page, generator=g, device="cuda") * 0.01
            s["w_out"] = torch.zeros(B, Hkv, most * page, device="cuda")
    if own:       # the plan that a program keeps, on the cache it has
        import transposed_convolution_gb300 as ctr
        s["plan"] = ctr.PagedAttention(
            B, case.get("Hq", Hkv), Hkv, D, page, most, k_pages=s["k"], v_pages=s["v"],
            layout=case["layout"], window=case.get("window", 0),
            weights=case.get("weights", False))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "attend":
            out = s["plan"].forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"],
                                    weights=s.get("w"), weights_out=s.get("w_out"))
            got = dict(out=out, k=s["k"], v=s["v"])
            return dict(got, w=s["w_out"]) if "w" in s else got
        if op == "evict":
            c = s["case"]
            slots, lens, w = s["plan"].evict(s["tables"], s["lens"], s["w"], s["to"], c["budget"],
                                             sinks=c["sinks"], recent=c["recent"],
                                             weights_out=s["w_out"])
            return dict(slots=slots, lens=lens, w=w, k=s["k"][s["first"]:], v=s["v"][s["first"]:])
        return s["plan"].forward(s["logits"], s["noise"], s["T"], s["k"], s["p"], s["minp"])
    return {"attend": _plain_attend, "evict": _plain_evict, "sample": _plain_sample}[op](s)


def _plain_attend(s):
    c = s["case"]
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    G, k, v = c["Hq"] // Hkv, s["k"], s["v"]
    tables, lens = s["tables"].long(), s["lens"].long()
    at = tables.gather(1, (lens // page)[:, None])[:, 0]
    if c["layout"] == "head":
        k[at, :, lens % page], v[at, :, lens % page] = s["k_new"], s["v_new"]
        kd, vd = (x[tables].transpose(2, 3).reshape(B, -1, Hkv, D).float() for x in (k, v))
    else:
        k[at, lens % page], v[at, lens % page] = s["k_new"], s["v_new"]
        kd, vd = (x[tables].reshape(B, -1, Hkv, D).float() for x in (k, v))
    j = torch.arange(kd.shape[1], device="cuda")
    on = j <= lens[:, None]
    if c["window"]:
        on = on & (j > lens[:, None] - c["window"])
    q = s["q"].float().reshape(B, Hkv, G, D) * (1.0 / math.sqrt(D))
    x = torch.matmul(q, kd.permute(0, 2, 3, 1))
    x = torch.where(on[:, None, None], x, float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    vd = torch.where(on[:, :, None, None], vd, 0.0)
    out = torch.matmul(p, vd.transpose(1, 2)).reshape(B, c["Hq"], D).to(k.dtype)
    got = dict(out=out, k=k, v=v)
    if c["weights"]:
        old = torch.where((j < lens[:, None])[:, None], s["w"], 0.0)
        have = (j <= lens[:, None])[:, None]
        s["w_out"].copy_(torch.where(have, old + p.sum(2), s["w_out"]))
        got["w"] = s["w_out"]
    return got


def _plain_evict(s):
    c = s["case"]
    B, Hkv, page, budget, first = c["B"], c["Hkv"], c["page"], c["budget"], s["first"]
    tables, lens, w = s["tables"].long(), s["lens"].long(), s["w"]
    j = torch.arange(w.shape[2], device="cuda")
    n = lens[:, None]
    x = torch.where(((j < c["sinks"]) | (j >= n - c["recent"]))[:, None], float("inf"), w)
    x = torch.where((j < n)[:, None], x, float("-inf"))
    _, best = torch.sort(x, dim=-1, descending=True, stable=True)
    kept = torch.clamp(lens, max=budget)
    i = torch.arange(budget, device="cuda")
    best = best[..., :budget]
    best = torch.cat([best, best.new_zeros(B, Hkv, budget - best.shape[2])], -1)
    on = (i < kept[:, None])[:, None]
    best = torch.where(on, best, w.shape[2])
    best, _ = torch.sort(best, dim=-1)
    take = torch.where(on, best, 0)
    b, h, r = torch.nonzero(on.expand(B, Hkv, budget), as_tuple=True)
    slot = take[b, h, r]
    src, dst = tables[b, slot // page], s["to"].long()[b, r // page]
    for x in (s["k"], s["v"]):
        if c["layout"] == "head":
            x[dst, h, r % page] = x[src, h, slot % page]
        else:
            x[dst, r % page, h] = x[src, slot % page, h]
    s["w_out"].copy_(torch.where(on, w.gather(2, take), s["w_out"]))
    return dict(slots=torch.where(on, best, -1).int(), lens=kept.int(), w=s["w_out"],
                k=s["k"][first:], v=s["v"][first:])


def _plain_sample(s):
    l, T, k, p, minp = s["logits"].float(), *(s[a][:, None] for a in ("T", "k", "p", "minp"))
    V = l.shape[1]
    l = torch.where(torch.isnan(l), float("-inf"), l)
    l, index = torch.sort(l, dim=-1, descending=True, stable=True)
    top = l[:, :1]
    w = torch.where(l == top, 1.0, torch.exp((l - top) / torch.where(T > 0, T, 1.0)))
    rank = torch.arange(V, device="cuda")[None]
    keep = (rank < torch.where(k > 0, k, V)) & (T > 0)
    before = torch.cumsum(w, -1) - w
    mass = torch.where(keep, w, 0.0).sum(-1, keepdim=True)
    keep = keep & ((p >= 1) | (before < p * mass)) & (w >= minp)
    keep = (keep | (rank == 0)) & (l > float("-inf"))
    noise = s["noise"].gather(1, index).clamp_min(torch.finfo(torch.float32).tiny)
    score = torch.where(keep, w / noise, -1.0)
    best = score.amax(-1, keepdim=True)
    token = torch.where(score == best, index, V).amin(-1)
    return torch.where(best[:, 0] >= 0, token, -1)


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "sample":
        # Every logit decides; of the noise only the numbers of the tokens that may be kept.
        rows, V = case["rows"], case["V"]
        kept = min(case["k"], V) if case["k"] else V if case["p"] >= 1 and not case["minp"] else 1
        return dict(bytes=rows * (V * es + kept * 4 + 16 + 8), flops=rows * V * 4)
    lens, Hkv, D = _lengths(case), case["Hkv"], case["D"]
    if case["op"] == "evict":
        # Weights in; the kept rows of K and V in and out, with their weights and slots.
        kept = sum(min(n, case["budget"]) for n in lens)
        return dict(bytes=4 * Hkv * sum(lens) + Hkv * kept * (4 * D * es + 4)
                    + 4 * Hkv * case["B"] * case["budget"], flops=Hkv * sum(lens))
    seen = sum(min(n + 1, case["window"] or n + 1) for n in lens)
    B, Hq = case["B"], case["Hq"]
    # The window's K and V rows, with the new ones read from the arguments and written too.
    nbytes = es * (2 * Hkv * D * (seen + B) + 2 * B * Hq * D) + 4 * (seen // case["page"] + 2 * B)
    if case["weights"]:
        nbytes += 8 * Hkv * (sum(lens) + B)
    return dict(bytes=nbytes, flops=4 * Hq * D * seen)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "evict":
        return _exact_evict(s)
    c, G, page = case, case["Hq"] // case["Hkv"], case["page"]
    out = torch.zeros(c["B"], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    w = s["w_out"].double() if c["weights"] else None
    for b, n in enumerate(_lengths(c)):
        # The sequence's rows in slot order, [n + 1, Hkv, D], the new one last.
        slot = torch.arange(n, device="cuda")
        pg, off = s["tables"][b].long()[slot // page], slot % page
        rows = [(x[pg, :, off] if c["layout"] == "head" else x[pg, off]).double()
                for x in (s["k"], s["v"])]
        K, Vv = (torch.cat([x, y[b][None].double()]) for x, y in
                 zip(rows, (s["k_new"], s["v_new"])))
        first = max(0, n + 1 - c["window"]) if c["window"] else 0
        K, Vv = K[first:], Vv[first:]
        for h in range(c["Hkv"]):
            q = s["q"][b, h * G:(h + 1) * G].double()
            p = torch.softmax(q @ K[:, h].T / math.sqrt(c["D"]), -1)
            out[b, h * G:(h + 1) * G] = p @ Vv[:, h]
            if w is not None:
                w[b, h, :n] = s["w"][b, h, :n].double()
                w[b, h, n] = 0
                w[b, h, first:n + 1] += p.sum(0)
    got = dict(out=out, k=None, v=None)
    return dict(got, w=w) if w is not None else got


def _exact_evict(s):
    c = s["case"]
    w = s["w"].cpu().numpy().astype(np.float64)
    B, Hkv, budget = c["B"], c["Hkv"], c["budget"]
    slots = np.full((B, Hkv, budget), -1, np.int32)
    w_out = np.zeros((B, Hkv, budget))
    lens = _lengths(c)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            held = set(range(min(c["sinks"], n))) | set(range(max(0, n - c["recent"]), n))
            rest = sorted((i for i in range(n) if i not in held), key=lambda i: (-w[b, h, i], i))
            keep = sorted(list(held) + rest[:max(0, budget - len(held))])[:n]
            slots[b, h, :len(keep)] = keep
            w_out[b, h, :len(keep)] = w[b, h, keep]
    return dict(slots=slots, lens=np.minimum(lens, budget).astype(np.int32), w=w_out, k=None,
                v=None)


def _exact_sample(s):
    c, V = s["case"], s["case"]["V"]
    logits, noise = (s[a].float().cpu().numpy().astype(np.float64) for a in ("logits", "noise"))
    got = np.empty(c["rows"], np.int64)
    for i, T in enumerate(s["T"].cpu().numpy().astype(np.float64)):
        order = np.argsort(-logits[i], kind="stable")
        if T <= 0:
            got[i] = order[0]
            continue
        order = order[:c["k"] or V]
        w = np.exp((logits[i, order] - logits[i, order[0]]) / T)
        share = np.cumsum(w / w.sum())
        p, minp = (float(np.float32(c[a])) for a in ("p", "minp"))
        count = len(order) if p >= 1 else 1 + int(np.sum(share[:-1] < p))
        count = max(1, min(count, int(np.sum(w >= minp))))
        kept = order[:count]
        score = w[:count] / np.maximum(noise[i, kept], np.finfo(np.float32).tiny)
        got[i] = kept[score == score.max()].min()
    return got
