"""A plain float64 model of the 8-bit KV cache, of decode attention over it and of
the page map, for the tests (not a test module).  It shares no code with the
library: codes are found by comparing with a table of all numbers that have one,
tokens join their blocks one call at a time, and bytes are found by their place."""
from __future__ import annotations

import math

import numpy as np

INT8, E4M3 = 0, 1
LEAST = {INT8: -24, E4M3: -15}
MOST = {INT8: 9, E4M3: 7}
TOP = {INT8: 127.0, E4M3: 448.0}


def _e4m3_numbers():
    """The 127 numbers >= 0 of codes 0 .. 126."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


NUMBERS = {INT8: np.arange(128, dtype=np.float64), E4M3: _e4m3_numbers()}


def nearest(y, fmt):
    """The numbers with a code nearest to y (|y| <= TOP), the even code's on a tie."""
    g, a = NUMBERS[fmt], np.abs(y)
    j = np.clip(np.searchsorted(g, a), 1, g.size - 1)
    under, over = a - g[j - 1], g[j] - a
    j = np.where((under < over) | ((under == over) & (j % 2 == 1)), j - 1, j)
    return np.copysign(g[j], y)


def codes(y, fmt):
    """Code bytes of numbers that have one; e4m3 has a zero of either sign."""
    if fmt == INT8:
        return y.astype(np.int64).astype(np.int8).view(np.uint8)
    j = np.searchsorted(NUMBERS[fmt], np.abs(y))
    return (j + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def numbers(c, fmt):
    if fmt == INT8:
        return c.view(np.int8).astype(np.float64)
    return np.where(c < 128, 1.0, -1.0) * np.append(NUMBERS[fmt], np.nan)[c & 127]


class Side:
    """K or V of one row: numbers y [n, Hkv, d] and exponents e [blocks, Hkv] (NaN: the block has joined a NaN)."""

    def __init__(self, fmt, P, Hkv, d):
        self.fmt, self.sb = fmt, min(P, 16)
        self.y = np.zeros((0, Hkv, d))
        self.e = np.zeros((0, Hkv))

    def append(self, x):
        fmt, n = self.fmt, len(self.y)
        x = np.asarray(x).astype(np.float64)
        bound = TOP[fmt] * 2.0 ** MOST[fmt]
        first = n // self.sb
        ys, es = [self.y[:first * self.sb]], [self.e[:first]]
        for b in range(first, -(-(n + len(x)) // self.sb) if len(x) else 0):
            old = self.y[b * self.sb:]
            new = x[max(0, b * self.sb - n):(b + 1) * self.sb - n]
            nan = np.isnan(new).any((0, 2))
            clipped = np.clip(np.where(np.isnan(new), 0, new), -bound, bound)
            top = np.abs(clipped).max((0, 2))
            e = np.full(top.shape, float(LEAST[fmt]))
            for k in range(LEAST[fmt], MOST[fmt]):
                e = np.where(top > TOP[fmt] * 2.0 ** k, k + 1, e)
            if len(old):
                was = self.e[b]
                nan |= np.isnan(was)
                e = np.maximum(e, np.where(np.isnan(was), e, was))
                old = nearest(old * 2.0 ** (np.where(np.isnan(was), e, was) - e)[:, None], fmt)
            ys += [old, nearest(clipped * 2.0 ** -e[:, None], fmt)]
            es.append(np.where(nan, np.nan, e)[None])
        if len(x):
            self.y, self.e = np.concatenate(ys), np.concatenate(es)

    def scales(self):
        """2^e of every token [n, Hkv]."""
        return 2.0 ** self.e.repeat(self.sb, 0)[:len(self.y)]

    def values(self):
        return self.y * self.scales()[:, :, None]


def head_bytes(P, d):
    tb = min(P, 64)
    return P // tb * (2 * tb * d + (32 if tb == 64 else 16))


def places(P, d):
    """Byte of token slot and dim in one head's page, K's and V's [P, d], and the bytes where the fp32 scales of a
    slot start, K's and V's [P]."""
    tb, sb = min(P, 64), min(P, 16)
    slot, dim = np.arange(P)[:, None], np.arange(d)[None, :]
    base, r = slot // tb * (2 * tb * d + (32 if tb == 64 else 16)), slot % tb
    x = np.where((r % 4 >= 2) & (d == 128), (dim + 64) % 128, dim)
    k = base + r * d + x
    u = r % sb
    v = base + tb * d + r // sb * sb * d + ((dim // 4 * (sb // 4) + u // 4) * 4 + dim % 4) * 4 + u % 4
    s = (base + 2 * tb * d + r // sb * 8)[:, 0]
    return k, v, s, s + 4


def pack(page, slot, y, e, side, P, d, fmt):
    """Store numbers y [Hkv, d] of one token and its block's exponents e [Hkv] in a page, uint8 [Hkv, bytes]."""
    at = places(P, d)
    page[:, at[side][slot]] = codes(y, fmt)
    s = at[2 + side][slot]
    page[:, s:s + 4] = np.where(np.isnan(e), np.float32(np.nan), 2.0 ** np.nan_to_num(e)).astype(np.float32)[:, None].view(np.uint8)


def unpack(page, P, d, fmt):
    """K and V values [Hkv, P, d] of one page."""
    page = np.ascontiguousarray(page)
    at = places(P, d)
    out = []
    for side in (0, 1):
        s = np.stack([np.ascontiguousarray(page[:, b:b + 4]).view(np.float32)[:, 0] for b in at[2 + side]], 1).astype(np.float64)
        out.append(numbers(page[:, at[side]], fmt) * s[:, :, None])
    return out


def visible(n, window, sinks):
    t = np.arange(n)
    return t if window is None else t[(t < sinks) | (t >= n - window)]


def attention(q, ks, vs, scale, window=None, sinks=0):
    """o, lse of q [B, Hq, d] over rows ks[i], vs[i] (Side), with an element-wise bound on what a kernel with fp32
    sums, one fp16 rounding of the softmax weights and one of o may be off:
      - half an fp16 step of o, 2^-11 |o|, or 2^-25 among the subnormals;
      - half a step of each weight times its V block's scale: 2^-11 sum p |v| / l, and for each one among the
        subnormals 2^-25 in units where the greatest is 1 or more: 2^-25 N max (p TOP 2^e) / l, p <= 1;
      - scores: a product sum of d terms in fp32, d 2^-24 sum |q k|, and as much again for exp and log."""
    B, Hq, d = q.shape
    G = Hq // ks[0].y.shape[1]
    o, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    to, tl = np.full((B, Hq, d), 2.0 ** -25), np.zeros((B, Hq))
    q = q.astype(np.float64)
    for i in range(B):
        t = visible(len(ks[i].y), window, sinks)
        if not t.size:
            continue
        kv, vv, vs_ = ks[i].values(), vs[i].values(), vs[i].scales()
        for h in range(Hq):
            k, v, unit = kv[t, h // G], vv[t, h // G], TOP[vs[i].fmt] * vs_[t, h // G].max()
            x = k @ q[i, h] * scale
            m = x.max()
            p = np.exp(x - m)
            l = p.sum()
            o[i, h] = p @ v / l
            lse[i, h] = m + math.log(l)
            es = 2 * d * 2.0 ** -24 * (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale) + 2.0 ** -20
            to[i, h] += 2.0 ** -11 * np.abs(o[i, h]) + (2.0 ** -11 + 2 * es) * (p @ np.abs(v) / l) + 2.0 ** -25 * t.size * unit / l
            tl[i, h] = es + 2.0 ** -22 * abs(lse[i, h])
    return o, lse, to, tl


def map_pages(lens, new, table, free, count, P, num_pages, T):
    """table, slots, positions, offsets, lengths and free count after pkv_map_pages; `free` is the free list."""
    table, cap = [list(r) for r in table], len(table[0]) * P
    count = min(max(count, 0), len(free))
    slots, positions, offsets, out = [-1] * T, [0] * T, [], []
    off = rank = taken = 0
    last = 0  # where a row begins, behind one whose tokens pass T the latter's place
    for i, (N, n) in enumerate(zip(lens, new)):
        last = off if off <= T else last
        offsets.append(last)
        valid = N >= 0 and n >= 0 and N + n <= cap
        have, need = -(-N // P), (-(-(N + n) // P) - -(-N // P)) if valid else 0
        served = valid and off + max(n, 0) <= T and (need == 0 or rank + need <= count)
        good = served
        for k in range(min(n, T - off) if valid else 0):
            x, pos = off + k, N + k
            j = pos // P - have
            if j >= 0 and pos % P == 0:
                page = free[count - 1 - rank - j] if served else -1
                table[i][pos // P] = page if 0 <= page < num_pages else -1
            if served:
                page = table[i][pos // P]
                if 0 <= page < num_pages:
                    slots[x], positions[x] = page * P + pos % P, pos
                else:
                    good = False
        if served and need:
            taken = rank + need
        rank += need
        off += max(n, 0)
        out.append(N + n if good else N)
    return table, slots, positions, offsets + [off if off <= T else last], out, count - taken
