"""The 8-bit cache where it could lose what it holds: decode of blocks of unequal
scales, element by element, and appends that are refused."""
import numpy as np
import pytest
import torch

import byte_ref as R
from paged_kv_gqa_09_gb300 import _lib, api
from test_gpu_byte import Batch, bits, dev, queries

pytestmark = pytest.mark.gpu
FORMATS = pytest.mark.parametrize("fmt", [R.INT8, R.E4M3], ids=["int8", "e4m3"])


def per_element(b, q, window=None, sinks=0):
    """o of the model, and what a kernel with fp32 sums may be off at each element, whatever the other dims of a
    value's block hold:
      - half an fp16 step of o, 2^-11 |o|, or 2^-25 among the subnormals;
      - weights held to 2^-11 of themselves or, the smallest, to 2^-25 where the greatest is 1 or more:
        (2^-11 sum p |v| + 2^-25 sum |v|) / l;
      - scores and exponentials in fp32, as in byte_ref.attention()."""
    ro, rl, to, tl = R.attention(q.cpu().numpy(), b.k, b.v, float(np.float32(b.shape.scale)), window, sinks)
    x = q.cpu().numpy().astype(np.float64)
    bound = np.zeros_like(to)
    for i in range(b.B):
        t = R.visible(len(b.k[i].y), window, sinks)
        for h in range(b.Hq if t.size else 0):
            k, v = b.k[i].values()[t, h // b.G], np.abs(b.v[i].values()[t, h // b.G])
            s = k @ x[i, h] * float(np.float32(b.shape.scale))
            p = np.exp(s - s.max())
            es = 2 * b.d * 2.0 ** -24 * (np.abs(k) @ np.abs(x[i, h])).max() * abs(b.shape.scale) + 2.0 ** -20
            bound[i, h] = 2.0 ** -11 * np.abs(ro[i, h]) + 2.0 ** -25 + ((2.0 ** -11 + 2 * es) * (p @ v) + 2.0 ** -25 * v.sum(0)) / p.sum()
    return ro, bound


# ------------------------------------------------------------------ decode

@FORMATS
@pytest.mark.parametrize("wide", [0, 4096])
@pytest.mark.parametrize("d,P", [(128, 16), (64, 8), (128, 8), (64, 64), (128, 128)])
def test_small_values_beside_a_block_of_a_large_scale(fmt, wide, d, P):
    """One value at the format's end, in one dim of one block; the other dims are left to blocks whose scale and
    softmax weight come to less than 2^-33 of that block's."""
    size, score = (2.0 ** -15, -4.0) if fmt == R.INT8 else (2.0 ** -9, -8.0)
    n = [64, 40, 17, 200]
    b = Batch(fmt, n, Hkv=2, G=4, d=d, P=P, seed=d + P, scale=1.0, wide=wide)
    ks, vs = [], []
    for i, m in enumerate(n):
        k, v = np.zeros((m, 2, d), np.float16), (np.clip(b.normal(m), -3, 3) * size).astype(np.float16)
        first = 8 * (i % 2)  # also a block that is not the row's first
        k[:, :, 0] = score
        k[first:first + 8, :, 0] = 0
        v[first:16 if P > 8 else first + 8] = 0
        v[first, :, 0] = R.TOP[fmt] * 2.0 ** R.MOST[fmt]
        ks.append(k)
        vs.append(v)
    b.append(ks, vs)
    q = np.zeros((4, 8, d), np.float16)
    q[:, :, 0] = 1.0
    q = dev(q)
    for window, sinks in ((None, 0), (9, 16)):
        ro, bound = per_element(b, q, window, sinks)
        o, lse = b.decode(q, window, sinks)
        x = o.cpu().numpy().astype(np.float64)
        bad = ~(np.abs(x - ro) <= bound)
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], x[bad][:4], ro[bad][:4], bound[bad][:4])
        assert (np.abs(ro[:, :, 1:]).max((1, 2)) > 2.0 ** -23).all()  # to lose them is beyond the bound, some 2^-25 there
        b.compare(o, lse, q, window, sinks)
    b.ok()


@FORMATS
@pytest.mark.parametrize("wide", [0, 4096])
def test_every_element_of_blocks_of_unequal_scales(fmt, wide):
    lens = [700, 33, 400]
    b = Batch(fmt, lens, Hkv=2, G=4, d=128, P=16, seed=15, wide=wide)
    ks, vs = [], []
    for n in lens:
        size = (2.0 ** b.rng.integers(-20, 14, (n + 15) // 16)).repeat(16)[:n, None, None]
        ks.append(b.normal(n))
        vs.append((np.clip(b.normal(n), -3, 3) * size * (b.rng.random((n, 2, 128)) < 0.2)).astype(np.float16))
    b.append(ks, vs)
    for scale in (0.0, 0.3, 1.0, 3.0):
        q = queries(b, scale=scale)
        for window, sinks in ((None, 0), (100, 20)):
            ro, bound = per_element(b, q, window, sinks)
            o, _ = b.decode(q, window, sinks)
            assert (np.abs(o.cpu().numpy().astype(np.float64) - ro) <= bound).all()
    b.ok()


@FORMATS
@pytest.mark.parametrize("wide", [0, 4096])
@pytest.mark.parametrize("d,P,G", [(128, 16, 1), (128, 8, 3), (64, 16, 4), (64, 8, 4), (128, 64, 4), (128, 16, 5), (64, 32, 7), (128, 8, 8),
                                   (64, 8, 6), (128, 256, 8)])
def test_weights_are_not_rounded_to_a_half(fmt, wide, d, P, G):
    """Scores that are exact, one dim of K alone, so that nothing but weights, sums and o's rounding is off:
      - o's rounding, 2^-11 |o| or 2^-25;
      - a weight's exponent and exponential, 2^-20 of it, and no more than that again where it is held in two fp16
        numbers: 2^-22, or 2^-25 of the least where the greatest is 1 or more;
      - sums in fp32: no term passes more than 64 roundings of 2^-23 (16 in a product, some 20 blocks of a warp's, the
        merges): 2^-17 sum p |v| / l."""
    lens = [33, 700, 64, 5, 300]
    b = Batch(fmt, lens, Hkv=2, G=G, d=d, P=P, seed=d + P + G, scale=1.0, wide=wide)
    ks = []
    for n in lens:
        k = np.zeros((n, 2, d), np.float16)
        k[:, :, 0] = b.rng.uniform(-4, 4, (n, 2))
        ks.append(k)
    b.append(ks, [b.normal(n) for n in lens])
    q = np.zeros((5, 2 * G, d), np.float16)
    q[:, :, 0] = np.linspace(0.3, 1.5, 2 * G)
    q = dev(q)
    for window, sinks in ((None, 0), (40, 9)):
        o, lse = b.decode(q, window, sinks)
        b.compare(o, lse, q, window, sinks)
        x, qn = o.cpu().numpy().astype(np.float64), q.cpu().numpy().astype(np.float64)
        for i, n in enumerate(lens):
            t = R.visible(n, window, sinks)
            for h in range(2 * G):
                v = b.v[i].values()[t, h // G]
                s = b.k[i].values()[t, h // G, 0] * qn[i, h, 0]
                p = np.exp(s - s.max())
                want = p @ v / p.sum()
                bound = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + ((2.0 ** -17 + 2.0 ** -19) * (p @ np.abs(v)) + 2.0 ** -25 * np.abs(v).sum(0)) / p.sum()
                assert (np.abs(x[i, h] - want) <= bound).all(), (i, h, np.abs(x[i, h] - want).max(), bound.max())
    b.ok()


@FORMATS
@pytest.mark.parametrize("d,P", [(128, 16), (64, 8), (128, 256)])
def test_bytes_behind_the_rows_beside_the_greatest_scale(fmt, d, P):
    """Masked tokens of a block whose scale is the format's greatest: any code there, -128 and NaNs among them, counts
    as nothing."""
    for fill in (0x80, 0x7F, 0xFF, 0x81):
        b = Batch(fmt, [5, 21, 100, 3], d=d, P=P, seed=31, fill=fill)
        top = R.TOP[fmt] * 2.0 ** R.MOST[fmt]
        with np.errstate(over="ignore"):  # to infinity, and back to the greatest
            vs = [np.clip(b.normal(n, top / 2), -top, top) for n in (5, 21, 100, 3)]
        for v in vs:
            v[-1] = top
        b.append([b.normal(n) for n in (5, 21, 100, 3)], [v.astype(np.float16) for v in vs])
        b.check(queries(b))
        b.check(queries(b), 3, 2)


@pytest.mark.parametrize("P", [8, 16, 32, 64, 128])
def test_a_wait_that_runs_out_with_more_heads_than_ctas(P):
    rng = np.random.default_rng(P)
    lens = rng.integers(100, 400, 90).tolist()
    for fmt in (R.INT8, R.E4M3):
        b = Batch(fmt, lens, Hkv=4, G=3, d=128, P=P, seed=P)
        b.grow(lens)
        q = queries(b)
        b.check(q)
        assert _lib.load().pkv_test_starve_next_decodes(1) == 0
        b.decode(q)
        assert api.pkv_get_error(b.ws)[0] == _lib.PKV_ETIMEOUT
        b.ws.zero_()  # the counters of a launch that gave up
        b.check(q)


# ------------------------------------------------------------------ refused appends

@FORMATS
@pytest.mark.parametrize("d,P,Hkv,rows", [(128, 16, 2, 3), (64, 8, 3, 3), (128, 64, 8, 3), (64, 16, 1, 70), (128, 256, 1, 130)])
@pytest.mark.parametrize("value", [3000.0, np.inf, np.nan])
def test_a_refused_row_keeps_its_earlier_tokens(fmt, d, P, Hkv, rows, value):
    """A row whose last page is partly filled and whose new tokens need a page that is not there: neither the length
    nor a value of the earlier tokens changes, whatever the new ones are; the other rows are served."""
    held = [P + 3 + i % 4 for i in range(rows)]
    new = [2 * P + i % 5 for i in range(rows)]
    new[1] = 40 * P  # the missing page is far off
    b = Batch(fmt, [x + y for x, y in zip(held, new)], Hkv=Hkv, G=1, d=d, P=P, seed=rows + P)
    b.grow(held)
    before = [(x.y.copy(), x.e.copy()) for side in (b.k, b.v) for x in side]
    refused = {0: 3, 1: 41, rows - 1: 2}
    keep = b.bt.clone()
    for i, page in refused.items():
        b.bt[i, page] = -1 if i else b.num_pages
    x = [b.normal(n) for n in new]
    for y in x:
        y[:, :, 5] = value
        y[0, :, 7] = 1.0
    b.append(x, [y[::-1].copy() for y in x])
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    assert b.lens.tolist() == [held[i] if i in refused else held[i] + new[i] for i in range(rows)]
    for j, side in enumerate((b.k, b.v)):
        for i in refused:
            side[i].y, side[i].e = before[j * rows + i]
    b.bt.copy_(keep)
    b.same()
    b.ok()


@FORMATS
@pytest.mark.parametrize("rows", [4, 64, 65, 300])
@pytest.mark.parametrize("value", [3000.0, np.nan])
def test_a_call_with_bad_offsets_keeps_every_row(fmt, rows, value):
    """Offsets that descend, pass the packed tokens or begin before them, in any row: no row's value changes."""
    held, new = [5 + i % 9 for i in range(rows)], [1 + i % 4 for i in range(rows)]
    b = Batch(fmt, [x + y for x, y in zip(held, new)], Hkv=2, G=1, d=128, P=16, seed=rows)
    b.grow(held)
    want = b.read()
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(off[-1])
    x = torch.full((T, 2, 128), value, dtype=torch.float16, device="cuda")
    down, past, ahead, middle = off.copy(), off.copy(), off.copy(), off.copy()
    down[rows // 2] = off[rows // 2 + 1] + 1
    past[rows] = T + 1
    ahead[0] = -1
    middle[rows - 1] = -4
    for bad in (down, past, ahead, middle):
        api.pkv_byte_append(b.shape, b.ws, fmt, x, x, b.bt, b.lens, b.cache, new_offsets=dev(bad))
        assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
        assert b.lens.tolist() == held
        for got, was in zip(b.read(), want):
            assert np.array_equal(bits(got), bits(was))
    b.ok()
