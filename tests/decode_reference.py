"""64-bit numpy forms of the decode-step operators, written from their formulas, and the error
bounds that their fp32 sums allow."""
import numpy as np

UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # unit roundoff of one rounding


def slot_rows(pages, table, n, page, layout):
    """The first n slots of a sequence as [n, H_kv, D]."""
    j = np.arange(n)
    pg, off = table[j // page], j % page
    return pages[pg, :, off] if layout == "head" else pages[pg, off]


def attention(q, k_pages, v_pages, tables, lens, page, layout="head", k_new=None, v_new=None,
              window=0, scale=None, hidden=()):
    """out [B, Hq, D], p (a list of [Hq, n] probabilities) and, for the error bound, the largest
    score error and the sums of p |v|.  All arguments float64 (tables, lens int).  ``hidden``:
    (sequence, slot) pairs that a bad page number hides."""
    B, Hq, D = q.shape
    Hkv = k_pages.shape[1] if layout == "head" else k_pages.shape[2]
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, mass, ds, probs = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.zeros((B, Hq)), []
    for b in range(B):
        n = max(int(lens[b]), 0)
        K, V = (slot_rows(x, tables[b], n, page, layout) for x in (k_pages, v_pages))
        if k_new is not None and lens[b] >= 0:
            K, V = (np.concatenate([x, y[b][None]]) for x, y in ((K, k_new), (V, v_new)))
            n += 1
        on = np.arange(n) >= (max(0, n - window) if window else 0)
        for bb, j in hidden:
            if bb == b and j < n:
                on[j] = False
        P = np.zeros((Hq, n))
        for h in range(Hq):
            if not on.any():
                continue
            k, v = K[on, h // G], V[on, h // G]
            s = scale * (k @ q[b, h])
            e = np.exp(s - s.max())
            P[h, on] = e / e.sum()
            out[b, h] = P[h, on] @ v
            mass[b, h] = P[h, on] @ np.abs(v)
            # A dot product of D terms in fp32, its scaling and the conversion to powers of two.
            ds[b, h] = (D + 4) * 2.0 ** -24 * abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
        probs.append(P)
    return out, probs, ds, mass


def attention_bound(out, ds, mass, longest, dtype):
    """Largest error of each output: the exponent's error enters the numerator and the
    denominator; sums of up to ``longest`` terms run at least sixteen abreast; 16-bit types
    multiply V with a probability kept to at least 15 bits; one rounding at the end."""
    u = 2.0 ** -24
    c = (longest / 16 + 64) * u + (2.0 ** -15 if dtype != "f32" else 0.0)
    return (2 * ds[:, :, None] + c) * mass * 1.01 + UNIT[dtype] * 1.01 * np.abs(out) + 2.0 ** -24


def evict(w, n, budget, sinks, recent):
    """The kept slots of one head, ascending."""
    keep = min(n, budget)
    held = sorted(set(range(min(sinks, n))) | set(range(max(0, n - recent), n)))
    others = [j for j in range(n) if j not in set(held)]
    weight = {j: -np.inf if np.isnan(w[j]) else float(w[j]) for j in others}
    # NaN ranks below every number, -inf included.
    others.sort(key=lambda j: (bool(np.isnan(w[j])), -weight[j], j))
    return sorted((held + others)[:keep]) if len(held) <= keep else held[:keep]


def sample(logits, noise, T=1.0, k=0, p=1.0, min_p=0.0, slack=1e-5):
    """The set of tokens one row may give: the formula's, and those that fp32 rounding of the
    weights and of the mass (relative error far below ``slack``) could give instead."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    m = l.max()
    if m == -np.inf:
        return {-1}
    order = np.argsort(-l, kind="stable")
    if T <= 0:
        return {int(order[0])}
    if 0 < k < len(order):
        order = order[:k]
    with np.errstate(invalid="ignore"):
        w = np.where(l[order] == m, 1.0, np.exp((l[order] - m) / T))
    before = np.cumsum(w) - w
    tokens = set()
    tiny = float(np.finfo(np.float32).tiny)
    for f in (1 - slack, 1.0, 1 + slack):
        on = np.ones(len(order), bool)
        if p < 1:
            on &= before < p * f * w.sum()
        on &= w >= min_p * f
        on[0] = True
        on &= l[order] > -np.inf
        score = np.where(on, w / np.maximum(np.asarray(noise, np.float64)[order], tiny), -1.0)
        best = score.max()
        near = order[score >= best * (1 - slack)]
        exact = order[score == best]
        # Equal weights and equal noise tie exactly in fp32 too: then the lowest index only.
        tokens.add(int(exact.min()))
        tokens |= {int(i) for i in near if not (score[order == i] == best).any()}
    return tokens
