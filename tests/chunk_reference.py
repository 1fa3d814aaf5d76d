"""64-bit numpy forms of the operators of a chunk of new tokens (attention over the paged cache,
rotary positions, pages), written from their formulas, and the error bounds that their sums allow."""
import numpy as np

from decode_reference import UNIT, slot_rows


def attention(q, k_pages, v_pages, tables, lens, starts, page, layout="head", window=0, scale=None,
              cap=None, hidden=()):
    """out [T, Hq, D] (NaN in rows that no sequence has) and, for the error bound, the largest score
    error [T, Hq] and the sums of p |v|.  ``hidden``: (sequence, slot) pairs that a bad page hides."""
    T, Hq, D = q.shape
    Hkv = k_pages.shape[1] if layout == "head" else k_pages.shape[2]
    G = Hq // Hkv
    cap = tables.shape[1] * page if cap is None else cap
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, mass, ds = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        if n <= 0:
            continue
        rows = slice(int(starts[b]), int(starts[b + 1]))
        out[rows] = 0.0
        if lens[b] < 0:
            continue
        end = np.minimum(lens[b] + np.arange(n) + 1, cap)
        lo = np.maximum(0, end - window) if window else np.zeros(n, int)
        j0, j1 = int(lo[0]), int(end[-1])
        j = np.arange(j0, j1)
        pg, off = tables[b, j // page], j % page
        on = (j >= lo[:, None]) & (j < end[:, None])
        for bb, x in hidden:
            if bb == b and j0 <= x < j1:
                on[:, x - j0] = False
        seen = on.any(0)
        pg = np.where(seen, pg, 0)
        for hk in range(Hkv):
            K, V = ((x[pg, hk, off] if layout == "head" else x[pg, off, hk]) for x in (k_pages, v_pages))
            K, V = np.where(seen[:, None], K, 0.0), np.where(seen[:, None], V, 0.0)
            for h in range(hk * G, hk * G + G):
                qh = q[rows, h]
                s = np.where(on, scale * (qh @ K.T), -np.inf)
                top = s.max(1, keepdims=True)
                e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
                total = e.sum(1, keepdims=True)
                p = e / np.where(total > 0, total, 1.0)
                out[rows, h] = p @ V
                mass[rows, h] = p @ np.abs(V)
                # A dot product of D terms in fp32, its scaling and the conversion to powers of two.
                a = np.where(on, np.abs(qh) @ np.abs(K).T, 0.0).max(1)
                ds[rows, h] = (D + 4) * 2.0 ** -24 * abs(scale) * a
    return out, ds, mass


def attention_bound(out, ds, mass, longest, dtype):
    """Largest error of each output: the exponent's error enters the numerator and the denominator; sums
    of up to ``longest`` terms, one after the other in the worst case; 16-bit types round each probability
    once (fp16 to no less than 2^-38 of the largest); one rounding at the end."""
    u = 2.0 ** -24
    c = (longest + 64) * u + (UNIT[dtype] if dtype != "f32" else 0.0)
    if dtype == "f16":
        c += longest * 2.0 ** -38
    return (2 * ds[:, :, None] + c) * mass * 1.01 + UNIT[dtype] * 1.01 * np.abs(out) + 2.0 ** -24


def frequencies(R, base=10000.0, scaling=None, factor=1.0, original=0.0, low=1.0, high=32.0):
    f = base ** (-2.0 * np.arange(R // 2) / R)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        g = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = (1 - g) * f / factor + g * f
    return f


def rotary(x, positions, f, layout="half", magnitude=1.0):
    """x [T, H, D] turned, and the largest error of each output: an angle within 2^-31 turn, a sine and a
    cosine within 2^-22 (fp32 argument and function), two products and a sum in fp32.  The rounding to
    the type is the caller's to add."""
    R = 2 * len(f)
    a = np.asarray(positions, np.float64)[:, None] * f
    cos, sin = magnitude * np.cos(a)[:, None], magnitude * np.sin(a)[:, None]
    y = np.array(x, np.float64)
    i, j = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., i] * sin + x[..., j] * cos
    err = np.zeros_like(y)
    slack = (np.abs(x[..., i]) + np.abs(x[..., j])) * abs(magnitude) * (2.0 ** -22 + 4 * 2.0 ** -24)
    # The 53-bit rounding of the frequency, times the position, on either side.
    slack = slack * (1 + np.abs(a)[:, None] * 2.0 ** -52 / 2.0 ** -22)
    err[..., i] = err[..., j] = slack
    return y, err


class Pool:
    """The free list, tables and lengths as Python lists."""

    def __init__(self, B, page, max_pages, num_pages):
        self.page, self.cap = page, page * max_pages
        self.tables = [[-1] * max_pages for _ in range(B)]
        self.free = list(range(num_pages))[::-1]

    def pages(self, n):
        return -(-n // self.page)

    def reserve(self, lens, counts, rows):
        granted, starts, slots, positions, bad = [], [0], [], [], False
        left, room = len(self.free), rows
        for b, (n, m) in enumerate(zip(lens, counts)):
            if n >= 0 and (m < 0 or n > self.cap or m > self.cap - n):
                m, bad = 0, True
            m = 0 if n < 0 else m
            need = self.pages(n + m) - self.pages(n) if m else 0
            left, room = left - need, room - m
            m = m if (left >= 0 or not need) and room >= 0 else 0
            for at in range(n, n + m):
                if at % self.page == 0:
                    self.tables[b][at // self.page] = self.free.pop()
                slots.append(self.tables[b][at // self.page] * self.page + at % self.page)
                positions.append(at)
            granted.append(m)
            starts.append(len(slots))
        empty = rows - len(slots)
        return (granted, starts, slots + [-1] * empty, positions + [0] * empty,
                [n + m for n, m in zip(lens, granted)], bad)

    def release(self, lens, keep):
        for b in reversed(range(len(lens))):
            for j in reversed(range(self.pages(max(keep[b], 0)), self.pages(max(lens[b], 0)))):
                self.free.append(self.tables[b][j])
                self.tables[b][j] = -1
        return [n if n < 0 else -1 if m < 0 else min(n, m) for n, m in zip(lens, keep)]
