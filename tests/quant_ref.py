"""A plain float64 model of the 4-bit KV cache and of windowed decode attention,
for the tests (not a test module).  It shares no code with the library: values
are quantised by counting the borders below them, and found in the cache by the
place of each code."""
from __future__ import annotations

import math

import numpy as np

LIMIT = 16384.0
HALVES = np.arange(0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)  # finite, >= 0, ascending
GRID = np.concatenate([-HALVES[:0:-1], HALVES])


def quantise(x):
    """Codes [.., GR, 32] and s, b [.., GR] (float64; NaN for a group with a NaN) of fp16 x [.., d]."""
    y = np.clip(np.asarray(x).astype(np.float64), -LIMIT, LIMIT)
    y = y.reshape(*y.shape[:-1], y.shape[-1] // 32, 32)
    nan = np.isnan(y).any(-1)
    y = np.where(nan[..., None], 0.0, y)
    lo, hi = y.min(-1), y.max(-1)
    s = HALVES[np.searchsorted(15 * HALVES, hi - lo)]
    want = lo - 16 * s
    j = np.clip(np.searchsorted(GRID, want), 1, GRID.size - 1)
    under, over = GRID[j - 1], GRID[j]
    b = np.where(over - want < want - under, over, under)
    n = np.zeros(y.shape, np.int64)
    for k in range(15):
        n += y >= (b + (16.5 + k) * s)[..., None]
    n = np.where((s > 0)[..., None], n, 0)
    return np.where(nan[..., None], 0, n), np.where(nan, np.nan, s), np.where(nan, np.nan, b)


def values(x):
    """The fp16 values that x [.., d] is stored as, as float64."""
    n, s, b = quantise(x)
    with np.errstate(invalid="ignore"):
        return (s[..., None] * (16 + n) + b[..., None]).astype(np.float16).astype(np.float64).reshape(np.shape(x))


def places(P, d):
    """For token slot and dim: index of the 16-bit half and field of the code, and the halves of s and b, in
    one head's page; for K and for V: arrays [P, d]."""
    tb, gr = min(P, 64), d // 32
    slot, dim = np.arange(P)[:, None], np.arange(d)[None, :]
    base, r = slot // tb * (tb * d * 5 // 8), slot % tb
    j, f = dim // 32, dim // 8 % 4
    field = np.broadcast_to(f, (P, d))
    kp = base + tb * d // 4 + r * 2 * gr + j
    k = (base + r * (d // 4) + (dim // 2 % 4 * gr + j) * 2 + dim % 2, field, kp, kp + gr)
    v0 = base + tb * d * 5 // 16
    c, t, e = r // 8, r % 8 // 2, r % 2
    vp = v0 + tb * d // 4 + c * 16 * gr + (t * gr + j) * 4 + e
    v = (v0 + c * 2 * d + ((dim % 8 * 4 + t) * gr + j) * 2 + e, field, vp, vp + 2)
    return k, v


def page_values(page, P, d):
    """K and V [Hkv, P, d] (float64) of one page, uint8 [Hkv, P * d * 5 / 4]."""
    h = np.ascontiguousarray(page).view(np.uint16)
    out = []
    for at, f, sp, bp in places(P, d):
        w = h[:, at].astype(np.int64)
        turned = ((w << 8) | (w >> 8)) & 0xFFFF
        n = np.choose(np.broadcast_to(f, w.shape), [w >> 6, w >> 2, w >> 10, turned >> 6]) & 15
        s, b = (h[:, x].view(np.float16).astype(np.float64) for x in (sp, bp))
        with np.errstate(invalid="ignore"):
            out.append((s * (16 + n) + b).astype(np.float16).astype(np.float64))
    return out


def pack_token(page, slot, k, v, P, d):
    """Store K and V [Hkv, d] (fp16) of one token in a page, uint8 [Hkv, P * d * 5 / 4]."""
    h = page.view(np.uint16)
    for x, (at, f, sp, bp) in zip((k, v), places(P, d)):
        n, s, b = quantise(x)
        n = n.reshape(x.shape)
        word = np.choose(np.broadcast_to(f[slot], n.shape), [n << 6, n << 2, n << 10, (n & 3) << 14 | n >> 2])
        mask = np.choose(f[slot], [15 << 6, 15 << 2, 15 << 10, 0xC003])
        for dim in range(d):  # several dims share a half
            cell = h[:, at[slot, dim]]
            h[:, at[slot, dim]] = (cell & np.uint16(0xFFFF ^ int(mask[dim]))) | word[:, dim].astype(np.uint16)
        bits = lambda y: np.where(np.isnan(y), 0x7FFF, y.astype(np.float16).view(np.uint16)).astype(np.uint16)
        h[:, sp[slot, ::32]] = bits(s)
        h[:, bp[slot, ::32]] = bits(b)


def visible(n, window, sinks):
    t = np.arange(n)
    return t if window is None else t[(t < sinks) | (t >= n - window)]


def attention(q, ks, vs, scale, window=None, sinks=0):
    """o, lse of q [B, Hq, d] over rows ks[i], vs[i] [N, Hkv, d] (float64), with an element-wise bound on
    what a kernel with fp32 sums, one fp16 rounding of the softmax weights and one of o may be off:
      - half an fp16 step of o, 2^-11 |o|, or 2^-25 among the subnormals;
      - half a step of each weight: 2^-11 sum p |v| / l, and 2^-25 for each one among the subnormals,
        in units where the greatest weight is 1 or more: 2^-25 N max |v| / l;
      - scores: a product sum of d terms in fp32, d 2^-24 sum |q k|, and as much again for exp and log."""
    B, Hq, d = q.shape
    G = Hq // (ks[0].shape[1] if B else 1)
    o, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    to, tl = np.full((B, Hq, d), 2.0 ** -25), np.zeros((B, Hq))
    q = q.astype(np.float64)
    for i in range(B):
        t = visible(ks[i].shape[0], window, sinks)
        if not t.size:
            continue
        for h in range(Hq):
            k, v = ks[i][t, h // G], vs[i][t, h // G]
            x = k @ q[i, h] * scale
            m = x.max()
            p = np.exp(x - m)
            l = p.sum()
            o[i, h] = p @ v / l
            lse[i, h] = m + math.log(l)
            es = 2 * d * 2.0 ** -24 * (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale) + 2.0 ** -20
            a = p @ np.abs(v) / l
            to[i, h] += 2.0 ** -11 * np.abs(o[i, h]) + (2.0 ** -11 + 2 * es) * a + \
                2.0 ** -25 * t.size * np.abs(v).max() / l
            tl[i, h] = es + 2.0 ** -22 * abs(lse[i, h])
    return o, lse, to, tl
