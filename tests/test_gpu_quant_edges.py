"""Calls of the 4-bit cache and windowed decode at their edges: rows without
new tokens, very many KV heads, a decoder on another stream,
scores of -inf and very large ones, weights far below the greatest,
groups of a few steps of fp16."""
import numpy as np
import pytest
import torch

import quant_ref as R
from paged_kv_gqa_09_gb300 import _lib, api
from test_gpu_quant import Batch, Pages, bits, clean, compare, dev, queries, widen

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows without new tokens

@pytest.mark.parametrize("d,P", [(128, 16), (64, 8)])
@pytest.mark.parametrize("new", [[0, 0, 4], [0, 0, 0, 9, 0], [0, 17, 0], [0, 1]])
def test_rows_without_new_tokens_among_the_others(d, P, new):
    """Empty rows first, last and between, at lengths that end inside eight positions; their own last page's entry
    is not looked at."""
    lens = [(3, 5, 9, 7, 1)[i] for i in range(len(new))]
    b = Batch([n + m + 8 for n, m in zip(lens, new)], d=d, P=P, seed=81, fill=0)
    b.grow(lens)
    for i, n in enumerate(new):
        if n == 0:
            b.bt[i] = -1
    b.grow(new)
    assert api.pkv_get_error(b.ws)[0] == 0
    assert b.lens.cpu().tolist() == [a + n for a, n in zip(lens, new)]
    b.bt.copy_(dev(b.table))
    k, v = b.read()
    assert np.array_equal(bits(k), bits(np.concatenate([R.values(x) for x in b.k])))
    assert np.array_equal(bits(v), bits(np.concatenate([R.values(x) for x in b.v])))
    b.ok()


def test_an_append_of_nothing_hands_the_lengths_on():
    b = Batch([20, 20, 20], seed=82, fill=0)
    b.grow([5, 9, 0])
    keep = b.cache.clone()
    none = torch.empty((0, 2, 128), dtype=torch.float16, device="cuda")
    out = torch.full_like(b.lens, -1)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    api.pkv_quant_append(b.shape, b.ws, none, none, b.bt, b.lens, b.cache, new_offsets=off, seq_lens_out=out)
    api.pkv_quant_append(b.shape, b.ws, none, none, b.bt, b.lens, b.cache, new_offsets=off)
    assert out.cpu().tolist() == [5, 9, 0] and b.lens.cpu().tolist() == [5, 9, 0]
    assert torch.equal(b.cache, keep)
    b.ok()
    b.lens[1] = -4
    api.pkv_quant_append(b.shape, b.ws, none, none, b.bt, b.lens, b.cache, new_offsets=off)
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE and int(b.lens[1]) == -4


# ------------------------------------------------------------------ very many KV heads

@pytest.mark.parametrize("Hkv", [1824, 2048])
def test_few_tokens_of_very_many_heads(Hkv):
    b = Batch([16], Hkv=Hkv, G=1, d=64, P=8, seed=83, fill=0)
    b.grow([3])
    b.grow([2])
    assert b.lens.cpu().tolist() == [5]
    k, v = b.read()
    assert np.array_equal(bits(k), bits(R.values(b.k[0])))
    assert np.array_equal(bits(v), bits(R.values(b.v[0])))
    b.check(queries(b))


# ------------------------------------------------------------------ a decoder on another stream

@pytest.mark.parametrize("handle", [False, True])
def test_a_decoders_first_call_on_another_stream(handle):
    """The current stream is busy while a new decoder appends and decodes on another one, its workspace taken from
    memory that held other values."""
    b = Batch([60, 33], Hkv=2, G=4, d=64, P=8, seed=84)
    k, v = [b.normal(50), b.normal(20)], [b.normal(50), b.normal(20)]
    kn, vn, off, q = dev(np.concatenate(k)), dev(np.concatenate(v)), dev(np.array([0, 50, 70], np.int32)), queries(b)
    f = Pages([700, 5], Hkv=2, G=4, d=64, P=8, seed=85)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    for where in (torch.cuda.current_stream(), side):  # whichever pool the workspace comes from
        with torch.cuda.stream(where):
            stale = [torch.full((api.pkv_attn_workspace_size(s),), 1, dtype=torch.uint8, device="cuda") for s in (b.shape, f.shape)]
        torch.cuda.synchronize()
        del stale
    dec = api.PagedDecoder()
    torch.cuda._sleep(100_000_000)
    dec.append_quant(kn, vn, b.cache, b.bt, b.lens, off, stream=stream)
    got = dec.step_quant(q, b.cache, b.bt, b.lens, stream=stream)
    win = dec.step_window(f.q, f.kc, f.vc, f.bt, f.lens, 600, 3, stream=stream)
    side.synchronize()
    torch.cuda.synchronize()
    compare(*got, q, [R.values(x) for x in k], [R.values(x) for x in v], b.shape.scale, None, 0)
    compare(*win, f.q, f.k, f.v, f.shape.scale, 600, 3)
    assert b.lens.cpu().tolist() == [50, 20]


# ------------------------------------------------------------------ scores of -inf

@pytest.mark.parametrize("d,lens", [(64, [700, 40, 0, 3000]), (128, [900, 1]), (128, [30] * 90)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("every", [None, 1, 301])
def test_keys_of_minus_infinity(d, lens, wide, every):
    """Every `every`-th token's score is finite (None: no token's), the others' are -inf, in clusters and in runs: o
    and lse are those of the finite ones alone, 0 and -inf where there is none."""
    b = Pages(lens, Hkv=2, G=4, d=d, P=16, seed=86)
    if wide:
        b = widen(b)
    b.q[..., 3] = 1.0
    keep = [np.zeros(n, bool) for n in lens]
    for i, n in enumerate(lens):
        if every:
            keep[i][n // 3::every] = True
        gone = torch.from_numpy(np.flatnonzero(~keep[i])).cuda()
        b.kc[b.bt[i, gone // 16].long(), gone % 16, :, 3] = -float("inf")
    o, lse = b.decode(10 ** 6, 0)
    compare(o, lse, b.q, [k[m] for k, m in zip(b.k, keep)], [v[m] for v, m in zip(b.v, keep)], b.shape.scale, None, 0)
    assert api.pkv_get_error(b.ws)[0] == 0
    clean(b.ws)
    # a weight of 0 and an infinite value make NaN, as in the definition
    i, t = len(lens) - 1, lens[-1] - 1
    if keep[i][t]:
        return
    b.vc[int(b.bt[i, t // 16]), t % 16, 1, 5] = float("inf")
    o, lse2 = b.decode(10 ** 6, 0)
    nan = torch.zeros_like(o, dtype=torch.bool)
    nan[i, 4:, 5] = True
    assert torch.equal(torch.isnan(o), nan) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("finite", [0, 3])
def test_scores_beyond_the_type_over_the_4_bit_cache(d, wide, finite):
    """Scores of -1e40, which are -inf in fp32; of the last row's tokens the first, one in the middle and the last
    have scores of 0."""
    lens = [500, 1, 1200]
    b = Batch(lens, Hkv=2, G=3, d=d, P=32, seed=87, scale=1e38)
    ks = [np.zeros((n, 2, d), np.float16) for n in lens]
    for k in ks:
        k[:, :, 0] = -100
    if finite:
        ks[2][[0, 611, 1199]] = 0
    b.append(ks, [b.normal(n) for n in lens])
    if wide:
        b = widen(b)
    q = torch.zeros((3, 6, d), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    o, lse = b.decode(q)
    mean = [R.values(v[[0, 611, 1199]]) if i == 2 and finite else R.values(v[:0]) for i, v in enumerate(b.v)]
    compare(o, lse, q, [np.zeros_like(v) for v in mean], mean, b.shape.scale, None, 0)
    b.ok()


# ------------------------------------------------------------------ very large scores

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("top,rest", [(16000, (8000, 15992)), (-8000, (-16000, -8008))])
@pytest.mark.parametrize("quant", [False, True])
def test_equal_greatest_scores_far_from_zero(d, wide, top, rest, quant):
    """Scores of 10^5 .. 10^10, of which three tokens' are the greatest, in tiles, warps and pieces of their own: o is
    the mean of their values, however the scale's product is rounded."""
    lens, Hkv, G, dims = [1500, 3, 700], 2, 4, 8
    rng = np.random.default_rng(88)
    ks = []
    for n in lens:
        c = rng.integers(rest[0] // 8, rest[1] // 8 + 1, (n, Hkv)) * 8.0
        c[[0, n // 2, n - 1]] = top
        k = np.zeros((n, Hkv, d), np.float16)
        k[:, :, :32] = c[:, :, None]  # a group of one value is kept as it is
        ks.append(k)
    if quant:
        b = Batch(lens, Hkv=Hkv, G=G, d=d, P=16, seed=89)
        b.append(ks, [b.normal(n) for n in lens])
        vs = [R.values(v) for v in b.v]
    else:
        b = Pages(lens, Hkv=Hkv, G=G, d=d, P=16, seed=89)
        for i, n in enumerate(lens):
            t = torch.arange(n, device="cuda")
            b.kc[b.bt[i, t // 16].long(), t % 16] = dev(ks[i])
        vs = b.v
    if wide:
        b = widen(b)
    q = torch.zeros((3, Hkv * G, d), dtype=torch.float16, device="cuda")
    q[..., :dims] = dev(np.array([60000, 31008, 7000, 1000, 301, 100, 20000, 50016], np.float16))[None, :, None]
    if quant:
        o, lse = b.decode(q)
    else:
        b.q = q
        o, lse = b.decode(10 ** 6, 0)
    o, lse = (x.cpu().numpy().astype(np.float64) for x in (o, lse))
    score = q[0, :, 0].double().cpu().numpy() * dims * top * float(np.float32(b.shape.scale))
    for i, n in enumerate(lens):
        for h in range(Hkv * G):
            v = vs[i][[0, n // 2, n - 1], h // G].astype(np.float64)
            # o's rounding to fp16, and that of the weights, which are equal
            assert (np.abs(o[i, h] - v.mean(0)) <= 2.0 ** -11 * (np.abs(v.mean(0)) + np.abs(v).mean(0)) + 2.0 ** -22).all()
            # a score's product with the scale, that with log2 e, and the way back from log2 units: fp32
            assert abs(lse[i, h] - score[h] - np.log(3)) <= 4 * 2.0 ** -24 * abs(score[h]) + 2.0 ** -20
    assert api.pkv_get_error(b.ws)[0] == 0
    clean(b.ws)


# ------------------------------------------------------------------ weights far below the greatest

@pytest.mark.parametrize("lead", [20.0, 24.6, 25.4, 28.0])
@pytest.mark.parametrize("B", [1, 80])  # many pieces of a row, and rows of a piece or two
@pytest.mark.parametrize("quant", [False, True])
def test_a_long_rows_tokens_far_behind_its_first(lead, B, quant):
    """10^6 tokens with a weight of 2^-lead of the first one's, whose value is 0 where theirs is 1."""
    P, d, Hkv, pages, times = 16, 64, 8, 64, 1040
    k, v = np.zeros((P * pages, Hkv, d), np.float16), np.ones((P * pages, Hkv, d), np.float16)
    k[0, :, 0] = 1
    v[0] = 0
    if quant:
        b = Batch([P * pages], Hkv=Hkv, G=2, d=d, P=P, seed=90)
        b.append([k], [v])
        first = float(R.values(k[0])[0, 0])
    else:
        b = Pages([P * pages], Hkv=Hkv, G=2, d=d, P=P, seed=90)
        t = torch.arange(P * pages, device="cuda")
        b.kc[b.bt[0, t // P].long(), t % P] = dev(k)
        b.vc[b.bt[0, t // P].long(), t % P] = dev(v)
        first = 1.0
    b.shape.scale = lead * float(np.log(2)) / first
    # the row's first page, then the others again and again; B such rows
    b.bt = torch.cat([b.bt[:, :1], b.bt[:, 1:].repeat(1, times)], 1).repeat(B, 1).contiguous()
    b.shape.bt_stride, b.shape.B, b.B = b.bt.shape[1], B, B
    n = P * (1 + (pages - 1) * times)
    b.lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.zeros((B, 2 * Hkv, d), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    if quant:
        o, lse = b.decode(q)
    else:
        b.q = q
        o, lse = b.decode(1 << 30, 0)
    o, lse = (x.cpu().numpy().astype(np.float64) for x in (o, lse))
    score = first * float(np.float32(b.shape.scale))
    rest = (n - 1) * np.exp(-score)
    # roundings of o and of the weights; 2^-32 of each small weight; a warp's sums of up to n / 4 tokens, 16 a step,
    # in fp32: 2^-24 of half their end for each step
    tol = 2.0 ** -11 * 2 + n * 2.0 ** -32 / rest + n / 64 * 2.0 ** -25
    # and the sum, in which a lane holds the first token's weight: what it adds to that, two tokens of sixteen of a
    # quarter of the row, may be lost
    assert np.abs(o * (rest + 1) / rest - 1).max() <= tol + rest / 32, (o.min(), o.max(), rest / (rest + 1))
    # six roundings of 2^-24 between the score, up to 20, and lse, and those sums
    assert np.abs(lse - score - np.log1p(rest)).max() <= 2.0 ** -16 + rest / 32 + n / 64 * 2.0 ** -25
    assert api.pkv_get_error(b.ws)[0] == 0
    clean(b.ws)


# ------------------------------------------------------------------ groups of a few steps of fp16

@pytest.mark.parametrize("d", [64, 128])
def test_groups_that_span_a_few_steps(d):
    """The values furthest from 0 in units of their range: one to three steps of fp16 at the limit, at either side of
    a power of two and among the subnormals, with 15 times the range on and off the grid."""
    rng = np.random.default_rng(91)
    at = np.array([16384.0, 16360.0, 8192.0, 8184.0, 4095.0, 1.0, 2.0 - 2.0 ** -10, 2.0 ** -14, 3 * 2.0 ** -24])
    rows = []
    for base in at:
        for steps in range(4):
            x = np.abs(np.float16(base)).view(np.uint16) - rng.integers(0, steps + 1, (4, 2, d // 32, 32))
            x[..., 0], x[..., 1] = x[..., 0].max(), x[..., 0].max() - steps
            x = np.maximum(x, 0).astype(np.uint16).view(np.float16).reshape(4, 2, d)
            rows += [x, -x]
    x = np.concatenate(rows)
    b = Batch([len(x) + 20], Hkv=2, G=1, d=d, P=16, seed=92, fill=0)
    b.append([x], [-x])
    k, v = b.read()
    assert np.array_equal(bits(k), bits(R.values(x)))
    assert np.array_equal(bits(v), bits(R.values(-x)))
    b.ok()
