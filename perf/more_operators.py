"""Measurement cases of the operators that take a chunk of new tokens into a paged key-value cache:
the pages for them, their rotary positions, and their attention.

Three operators, by a case's ``op``:

chunk    the n_b new tokens of sequence b (rows starts[b] .. starts[b + 1] - 1 of q [T, Hq, D]), whose
         K and V rows are in the cache already, attend to the cache: token i, at slot len_b + i, to the
         slots up to its own (the last ``window`` of them if there is a window):
             out[t, h] = sum_j softmax_j(q[t, h] . K[j, h // G] / sqrt(D)) V[j, h // G],  G = Hq / Hkv.
rotary   pairs (x, y) of the first R of a head's D columns, columns (i, i + R/2) ("half") or
         (2i, 2i + 1) ("interleaved"), turned by the token's position times the pair's frequency,
             x' = m (x cos a - y sin a),  y' = m (x sin a + y cos a),  a = position * f_i,
             f_i = base^(-2i/R), divided by ``factor`` for pairs that turn less than ``low`` times
             over ``original`` positions, kept for those that turn more than ``high`` times, blended
             linearly in the number of turns between (factor 1: no scaling).
         With ``put`` K is turned on its way into its slots of the cache, and V copied beside it.
pages    each sequence's last count_b tokens are given back (their pages go to the free list) and as
         many reserved again: pages from the end of the free list into the sequence's table, and for
         each token the slot page * page_size + row and its position.

Sizes are generic: heads of 64 and 80 for a codec's own decoder, heads of 128 and 256 for a language
model that writes its codes.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _chunk(name, **kw):
    case = dict(op="chunk", B=1, Hq=32, Hkv=8, D=128, page=64, lo=0, hi=0, n_lo=1, n_hi=1,
                dtype="bf16", layout="head", window=0)
    case.update(kw, name=name)
    return case


def _rotary(name, **kw):
    case = dict(op="rotary", T=1, Hq=32, Hkv=8, D=128, R=128, style="half", base=10000.0, factor=1.0,
                original=4096, low=1.0, high=32.0, magnitude=1.0, first=0, put=False, page=16,
                layout="head", dtype="bf16")
    case.update(kw, name=name)
    return case


def listed():
    return [
        # Four drafted frames of one stream of a codec's decoder, checked at once: only latency counts.
        _chunk("chunk drafted frames", Hq=16, Hkv=16, D=64, page=16, lo=125, hi=125, n_lo=4, n_hi=4),
        # A serving step that mixes single tokens with pieces of prompts, at ragged lengths.
        _chunk("chunk mixed batch", B=16, page=16, lo=37, hi=4099, n_lo=1, n_hi=131, dtype="f16"),
        # A long session's next piece: few rows, most of the work along the cache.
        _chunk("chunk long session", lo=65531, hi=65531, n_lo=512, n_hi=512),
        # A whole prompt at once, the cache empty before it: the largest call.
        _chunk("chunk prompt", n_lo=8192, n_hi=8192),
        # fp32 caches, token-major pages, an odd page size, a sliding window, a head size that is no
        # power of two.
        _chunk("chunk f32 window", B=6, Hq=16, Hkv=8, D=80, page=20, lo=3, hi=1501, n_lo=100, n_hi=311,
               dtype="f32", layout="token", window=750),
        # Wide heads, three to a KV head, prompts of several users.
        _chunk("chunk wide heads", B=4, Hq=12, Hkv=4, D=256, page=24, lo=0, hi=2500, n_lo=601,
               n_hi=1400),
        # The new token of one stream: only latency counts.
        _rotary("rotary one token", first=5000),
        # A prompt past the trained length, frequencies scaled.
        _rotary("rotary prompt", T=8192, base=500000.0, factor=8.0, original=8192, high=4.0,
                magnitude=1.0 + 0.1 * math.log(8.0), first=1000000),
        # fp32, pairs side by side, part of the head, an odd number of tokens.
        _rotary("rotary f32 part", T=1001, Hq=16, Hkv=8, D=80, R=32, style="interleaved", dtype="f32"),
        # A mixed step's tokens, turned and put into the cache in one pass.
        _rotary("rotary and put", T=2011, R=64, put=True, layout="token", dtype="f16", first=300),
        # A batch of single tokens: every sixteenth needs a new page.
        dict(name="pages one token each", op="pages", B=64, page=16, lo=0, hi=8191, n_lo=1, n_hi=1),
        # A full batch of prompts' pieces.
        dict(name="pages prompts", op="pages", B=256, page=16, lo=0, hi=4000, n_lo=1, n_hi=2001),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rotary", "rotary", "pages"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    layout = rng.choice(["head", "token"])
    if op == "chunk":
        D = rng.choice([64, 80, 96, 128, 256])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        B = _log_uniform(rng, 1, 64)
        # Products of a query and a slot, padding included: at most a quarter of the largest case's
        # (an eighth in fp32, whose products take longer).
        most = (1 << 28) // Hq // (2 if dtype == "f32" else 1) * 128 // D
        n_hi = min(_log_uniform(rng, 1, 4096), max(1, most // B // 64))
        hi = min(_log_uniform(rng, 1, 65536), max(1, most // B // n_hi - n_hi))
        hi = max(1, min(hi, int(5.0e8 / (B * Hkv * D * (8 if dtype == "f32" else 4)))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([8, 16, 20, 24, 64, 128]),
                    lo=rng.randint(0, hi), hi=hi, n_lo=rng.randint(1, n_hi), n_hi=n_hi, dtype=dtype,
                    layout=layout, window=rng.choice([0, 0, 0, max(1, (hi + n_hi) // 3)]))
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 256])
        G = rng.choice([1, 2, 4, 8])
        most = int(4.0e7 / ((G + 2) * Hkv * D))
        return dict(op=op, T=_log_uniform(rng, 1, most), Hq=G * Hkv, Hkv=Hkv, D=D,
                    R=rng.choice([D, D, D // 2, 32]), style=rng.choice(["half", "interleaved"]),
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 32.0]),
                    original=8192, low=1.0, high=rng.choice([4.0, 32.0]),
                    magnitude=rng.choice([1.0, 1.25]), first=_log_uniform(rng, 1, 4000000),
                    put=rng.random() < 0.5, page=rng.choice([8, 16, 20, 64]), layout=layout,
                    dtype=dtype)
    B, page = _log_uniform(rng, 1, 256), rng.choice([8, 16, 20, 64, 128])
    n_hi = _log_uniform(rng, 1, 2000)
    hi = _log_uniform(rng, 1, 16000)
    return dict(op=op, B=B, page=page, lo=rng.randint(0, hi), hi=hi, n_lo=rng.randint(0, n_hi),
                n_hi=n_hi)


def _spread(B, lo, hi, strides):
    """B numbers spread evenly over lo..hi, in an order that is not sorted."""
    even = [lo + (hi - lo) * i // max(1, B - 1) for i in range(B)] if B > 1 else [hi]
    step = next(s for s in strides if math.gcd(s, B) == 1)
    return [even[(i * step) % B] for i in range(B)]


def _lengths(case):
    return _spread(case["B"], case["lo"], case["hi"], (7, 5, 3, 1))


def _counts(case):
    return _spread(case["B"], case["n_lo"], case["n_hi"], (11, 13, 3, 1))


def _frequencies(c):
    """The R/2 frequencies of a case, in 64 bits."""
    f = c["base"] ** (-2.0 * np.arange(c["R"] // 2) / c["R"])
    turns = c["original"] * f / (2 * np.pi)
    keep = np.clip((turns - c["low"]) / (c["high"] - c["low"]), 0.0, 1.0)
    return (1 - keep) * f / c["factor"] + keep * f


def _positions(c):
    return np.arange(c["first"], c["first"] + c["T"], dtype=np.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=dict(case))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["dtype"]])

    def shuffled(n):
        return torch.randperm(n, generator=g, device="cuda").to(torch.int32)

    if case["op"] == "rotary":
        T, Hq, Hkv, D, page = (case[a] for a in ("T", "Hq", "Hkv", "D", "page"))
        # Projections of one buffer, as a fused QKV product leaves them: strided rows.
        qkv = normal(T, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["positions"] = torch.from_numpy(_positions(case)).to(torch.int32).cuda()
        if case["put"]:
            # Slots of shuffled pages, a few of them more than there are tokens.
            pages = -(-T // page) + 3
            at = torch.arange(T, device="cuda")
            s["slots"] = shuffled(pages).long()[at // page] * page + at % page
            shape = (pages, Hkv, page, D) if case["layout"] == "head" else (pages, page, Hkv, D)
            s["k_pages"], s["v_pages"] = normal(*shape), normal(*shape)
        if own:       # the plans that a program keeps
            import transposed_convolution_gb300 as ctr
            s["rotary"] = ctr.Rotary(
                D, case["R"], layout=case["style"], base=case["base"], scaling="parts",
                factor=case["factor"], original=case["original"], low=case["low"], high=case["high"],
                magnitude=case["magnitude"], dtype=DTYPES[case["dtype"]])
            if case["put"]:
                s["plan"] = ctr.PagedAttention(1, Hq, Hkv, D, page, pages, k_pages=s["k_pages"],
                                               v_pages=s["v_pages"], layout=case["layout"])
        return s

    B, page = case["B"], case["page"]
    lens, counts = np.array(_lengths(case)), np.array(_counts(case))
    need = -(-(lens + counts) // page)
    most, used = max(1, int(need.max())), int(need.sum())
    total = used + (used // 4 + 1 if case["op"] == "pages" else 0)
    # The cache's pages, dealt out in a random order.
    order = shuffled(total)
    first = np.concatenate([[0], np.cumsum(need)[:-1]])
    held = np.arange(most)[None] < need[:, None]
    at = torch.from_numpy(np.where(held, first[:, None] + np.arange(most), 0)).cuda()
    tables = torch.where(torch.from_numpy(held).cuda(), order[at], -1).to(torch.int32)
    s["tables"] = tables.contiguous()
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    if case["op"] == "pages":
        s["full"] = torch.from_numpy((lens + counts).astype(np.int32)).cuda()
        s["counts"] = torch.from_numpy(counts.astype(np.int32)).cuda()
        s["rows"] = int(counts.sum()) + 5        # a buffer of a fixed size, not quite filled
        s["free"], s["count"] = order.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        s["free"][:total - used] = order[used:]
        s["count"].fill_(total - used)
        if own:       # the plan that a program keeps, with the free list it has
            import transposed_convolution_gb300 as ctr
            s["plan"] = ctr.PagePool(B, page, most, free=s["free"], count=s["count"])
        return s

    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    s["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    shape = (total, Hkv, page, D) if case["layout"] == "head" else (total, page, Hkv, D)
    s["k"], s["v"] = normal(*shape), normal(*shape)
    s["q"] = (normal(int(counts.sum()), Hq + 2 * Hkv, D) * 2)[:, :Hq]
    if own:           # the plan that a program keeps, on the cache it has
        import transposed_convolution_gb300 as ctr
        s["plan"] = ctr.PagedAttention(B, Hq, Hkv, D, page, most, k_pages=s["k"], v_pages=s["v"],
                                       layout=case["layout"], window=case["window"], chunks=True)
    return s


def run(s):
    c = s["case"]
    if own:
        if c["op"] == "chunk":
            return s["plan"].forward_chunk(s["q"], s["tables"], s["lens"], s["starts"])
        if c["op"] == "rotary":
            if c["put"]:
                q = s["plan"].put(s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"],
                                  rotary=s["rotary"])
                return dict(q=q, k=s["k_pages"], v=s["v_pages"])
            q, k = s["rotary"].forward(s["q"], s["k"], s["positions"])
            return dict(q=q, k=k)
        s["plan"].release(s["tables"], s["full"], s["lens"])
        granted, starts, slots, positions, lens = s["plan"].reserve(
            s["tables"], s["lens"], s["counts"], s["rows"])
        return dict(tables=s["tables"], granted=granted, starts=starts, slots=slots,
                    positions=positions, lens=lens, count=s["count"])
    return {"chunk": _plain_chunk, "rotary": _plain_rotary, "pages": _plain_pages}[c["op"]](s)


def _plain_chunk(s):
    c, dev = s["case"], s["q"].device
    B, Hq, Hkv, D, G = c["B"], c["Hq"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    most, T = max(_counts(c)), s["q"].shape[0]
    tables, lens, starts = s["tables"].long().clamp(min=0), s["lens"].long(), s["starts"].long()
    if c["layout"] == "head":
        k, v = (x[tables].transpose(2, 3).reshape(B, -1, Hkv, D).float() for x in (s["k"], s["v"]))
    else:
        k, v = (x[tables].reshape(B, -1, Hkv, D).float() for x in (s["k"], s["v"]))
    i = torch.arange(most, device=dev)
    rows = (starts[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float()[rows].view(B, most, Hkv, G, D).permute(0, 2, 3, 1, 4)
    scores = q.reshape(B, Hkv, G * most, D) @ k.permute(0, 2, 3, 1)
    scores = scores.mul_(1 / math.sqrt(D)).view(B, Hkv, G, most, -1)
    j, at = torch.arange(scores.shape[-1], device=dev), lens[:, None] + i
    hidden = j > at[:, :, None]
    if c["window"]:
        hidden |= j <= at[:, :, None] - c["window"]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()   # rows of padding may be empty
    total = scores.sum(-1, keepdim=True)
    v = v.masked_fill(j[:, None, None] >= (lens + starts.diff())[:, None, None, None], 0.0)
    out = scores.view(B, Hkv, G * most, -1) @ v.transpose(1, 2)
    out = out.view(B, Hkv, G, most, D) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(B, most, Hq, D)
    return out[i < starts.diff()[:, None]].to(s["q"].dtype)


def _plain_rotary(s):
    c, dev = s["case"], s["q"].device
    f = torch.from_numpy(_frequencies(c)).to(dev)
    angle = s["positions"].double()[:, None] * f
    cos, sin = ((x * c["magnitude"]).float()[:, None] for x in (angle.cos(), angle.sin()))

    def turned(x):
        head, rest = x[..., :c["R"]].float(), x[..., c["R"]:]
        if c["style"] == "half":
            a, b = head.chunk(2, -1)
            head = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = head[..., ::2], head[..., 1::2]
            head = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([head.to(x.dtype), rest], -1)

    q, k = turned(s["q"]), turned(s["k"])
    if not c["put"]:
        return dict(q=q, k=k)
    pg, row = s["slots"] // c["page"], s["slots"] % c["page"]
    if c["layout"] == "head":
        s["k_pages"][pg, :, row], s["v_pages"][pg, :, row] = k, s["v"]
    else:
        s["k_pages"][pg, row], s["v_pages"][pg, row] = k, s["v"]
    return dict(q=q, k=s["k_pages"], v=s["v_pages"])


def _plain_pages(s):
    c, page, dev = s["case"], s["case"]["page"], s["lens"].device
    tables, lens, full, counts = s["tables"], s["lens"].long(), s["full"].long(), s["counts"].long()
    most, free, count = tables.shape[1], s["free"], s["count"].long()
    j = torch.arange(most, device=dev)
    # Give back: the last sequence's last page first, so that the first one's comes out first.
    back = (j >= (-(-lens // page))[:, None]) & (j < (-(-full // page))[:, None])
    order = back.flatten().flip(0).cumsum(0).flip(0).view(back.shape) - 1
    free[(count + order)[back]] = tables[back]
    count = count + back.sum()
    tables.masked_fill_(back, -1)
    # Reserve: first come, first served.
    need = -(-(lens + counts) // page) - -(-lens // page)
    ends = counts.cumsum(0)
    ok = ((need.cumsum(0) <= count) | (need == 0)) & (ends <= s["rows"])
    granted = torch.where(ok, counts, 0)
    starts = torch.cat([ends.new_zeros(1), granted.cumsum(0)])
    take = (j >= (-(-lens // page))[:, None]) & (j < (-(-(lens + granted) // page))[:, None])
    order = take.flatten().cumsum(0).view(take.shape) - 1
    tables[take] = free[(count - 1 - order)[take]]
    s["count"].copy_(count - take.sum())
    t = torch.arange(s["rows"], device=dev)
    b = torch.searchsorted(starts[1:], t, right=True).clamp(max=c["B"] - 1)
    position = lens[b] + t - starts[b]
    on = t < starts[-1]
    held = tables[b, (position // page).clamp(max=most - 1)].long()
    slots = torch.where(on, held * page + position % page, -1)
    i32 = torch.int32
    return dict(tables=tables, granted=granted.to(i32), starts=starts.to(i32), slots=slots,
                positions=torch.where(on, position, 0).to(i32), lens=(lens + granted).to(i32),
                count=s["count"])


def work(case):
    if case["op"] == "pages":
        tokens, B, page = sum(_counts(case)), case["B"], case["page"]
        moved = sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(_lengths(case), _counts(case)))
        # Lengths and counts in; each page's number from the table to the list and back; a slot and
        # a position a token.
        return dict(bytes=24 * B + 16 * moved + 12 * tokens, flops=0)
    size = 4 if case["dtype"] == "f32" else 2
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        T = case["T"]
        heads = 2 * (Hq + Hkv) + (2 * Hkv if case["put"] else 0)
        return dict(bytes=T * (heads * D * size + 4 + (8 if case["put"] else 0)),
                    flops=3 * T * (Hq + Hkv) * case["R"])
    w = case["window"] or 1 << 40
    pairs = slots = 0
    for n, m in zip(_lengths(case), _counts(case)):
        slots += n + m - max(0, n + 1 - w)
        full = max(0, n + m - max(n, w))        # tokens whose window is full
        pairs += full * w + sum(range(n + 1, n + m - full + 1))
    bytes_ = (2 * slots * Hkv + 2 * sum(_counts(case)) * Hq) * D * size
    return dict(bytes=bytes_ + 4 * (slots // case["page"] + 2 * case["B"]), flops=4 * pairs * Hq * D)


def exact(case, seed):
    s = _bare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(s)
    return _exact_chunk(s) if case["op"] == "chunk" else _exact_rotary(s)


def _bare(case, seed):
    """The inputs without the plans."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_chunk(s):
    c = s["case"]
    G, page, w, dev = c["Hq"] // c["Hkv"], c["page"], c["window"], s["q"].device
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    t0 = 0
    for b, (n, m) in enumerate(zip(_lengths(c), _counts(c))):
        total = n + m
        j = torch.arange(total, device=dev)
        pg, row = s["tables"][b].long()[j // page], j % page
        for hk in range(c["Hkv"]):
            if c["layout"] == "head":
                K, V = s["k"][pg, hk, row].double(), s["v"][pg, hk, row].double()
            else:
                K, V = s["k"][pg, row, hk].double(), s["v"][pg, row, hk].double()
            for i0 in range(0, m, 2048):
                pos = torch.arange(n + i0, n + min(m, i0 + 2048), device=dev)
                seen = j[None] <= pos[:, None]
                if w:
                    seen &= j[None] > pos[:, None] - w
                for h in range(hk * G, hk * G + G):
                    q = s["q"][t0 + i0:t0 + i0 + len(pos), h].double()
                    x = torch.where(seen, q @ K.T / math.sqrt(c["D"]), -math.inf)
                    p = torch.exp(x - x.max(1, keepdim=True).values)
                    out[t0 + i0:t0 + i0 + len(pos), h] = (p @ V) / p.sum(1, keepdim=True)
        t0 += m
    return out


def _exact_rotary(s):
    c = s["case"]
    R, half = c["R"], c["R"] // 2
    got = {}
    pos = _positions(c).astype(np.float64)
    for name in ("q", "k"):
        x = s[name].double().cpu().numpy()
        y = x.copy()
        for i in range(half):
            f = c["base"] ** (-2.0 * i / R)
            turns = c["original"] * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - c["low"]) / (c["high"] - c["low"])))
            f = f * keep + f / c["factor"] * (1 - keep)
            a, b = (i, i + half) if c["style"] == "half" else (2 * i, 2 * i + 1)
            cos, sin = np.cos(pos * f)[:, None], np.sin(pos * f)[:, None]
            y[:, :, a] = c["magnitude"] * (x[:, :, a] * cos - x[:, :, b] * sin)
            y[:, :, b] = c["magnitude"] * (x[:, :, a] * sin + x[:, :, b] * cos)
        got[name] = y
    if not c["put"]:
        return got
    k, v = s["k_pages"].double().cpu().numpy(), s["v_pages"].double().cpu().numpy()
    new_v = s["v"].double().cpu().numpy()
    for t, slot in enumerate(s["slots"].tolist()):
        pg, row = divmod(slot, c["page"])
        at = (pg, slice(None), row) if c["layout"] == "head" else (pg, row)
        k[at], v[at] = got["k"][t], new_v[t]
    return dict(q=got["q"], k=k, v=v)


def _exact_pages(s):
    page, tables = s["case"]["page"], s["tables"].cpu().numpy()
    lens, full, counts = (s[a].tolist() for a in ("lens", "full", "counts"))
    free, rows = s["free"].tolist()[:int(s["count"])], s["rows"]
    for b in reversed(range(len(lens))):
        for j in reversed(range(-(-lens[b] // page), -(-full[b] // page))):
            free.append(int(tables[b, j]))
            tables[b, j] = -1
    left, room, granted, starts, slots, positions = len(free), rows, [], [0], [], []
    for b, (n, m) in enumerate(zip(lens, counts)):
        need = -(-(n + m) // page) - -(-n // page)
        left, room = left - need, room - m
        m = m if (left >= 0 or not need) and room >= 0 else 0
        for at in range(n, n + m):
            if at % page == 0:
                tables[b, at // page] = free.pop()
            slots.append(int(tables[b, at // page]) * page + at % page)
            positions.append(at)
        granted.append(m)
        starts.append(len(slots))
    empty = rows - len(slots)
    i32 = np.int32
    return dict(tables=tables, granted=np.array(granted, i32), starts=np.array(starts, i32),
                slots=np.array(slots + [-1] * empty, np.int64),
                positions=np.array(positions + [0] * empty, i32),
                lens=np.array(lens, i32) + np.array(granted, i32), count=np.array([len(free)], i32))
