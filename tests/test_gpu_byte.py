"""The 8-bit KV cache on the GPU: writing, reading back, and decode over it,
against the plain float64 model."""
import numpy as np
import pytest
import torch

import byte_ref as R
from paged_kv_gqa_09_gb300 import _lib, api

pytestmark = pytest.mark.gpu
FORMATS = pytest.mark.parametrize("fmt", [R.INT8, R.E4M3], ids=["int8", "e4m3"])


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bits(x):
    """fp16 bits with one NaN and one zero."""
    x = np.asarray(x).astype(np.float16)
    return np.where(np.isnan(x), 0x7FFF, np.where(x == 0, 0, x.view(np.uint16)))


class Batch:
    """A batch over the 8-bit cache: shuffled pages, a workspace, device tensors, and the model's rows.  What no
    token was written to is filled with `fill`: 0xFF is a NaN in either format's codes, int8's -1 and a NaN scale."""

    def __init__(self, fmt, cap, Hkv=2, G=4, d=128, P=16, seed=0, spare=3, fill=0xFF, scale=None, wide=0):
        rng = np.random.default_rng(seed)
        self.rng, self.fmt, self.B, self.Hkv, self.G, self.Hq, self.d, self.P = rng, fmt, len(cap), Hkv, G, Hkv * G, d, P
        pages = [-(-c // P) for c in cap]
        self.num_pages = max(1, sum(pages)) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((self.B, max(1, max(pages, default=1), wide)), order[-1], np.int32)
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.cache = torch.full((self.num_pages, Hkv, R.head_bytes(P, d)), fill, dtype=torch.uint8, device="cuda")
        self.bt = dev(self.table)
        self.lens = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        self.shape = api.make_byte_shape(self.Hq, d, self.cache, self.bt, scale)
        self.ws = torch.zeros(api.pkv_attn_workspace_size(self.shape), dtype=torch.uint8, device="cuda")
        self.k = [R.Side(fmt, P, Hkv, d) for _ in cap]
        self.v = [R.Side(fmt, P, Hkv, d) for _ in cap]

    def normal(self, n, scale=1.0):
        return (self.rng.standard_normal((n, self.Hkv, self.d)) * scale).astype(np.float16)

    def append(self, ks, vs, one=False, pad=0, **kw):
        """Append ks[i], vs[i] [n, Hkv, d] to each row, through one packed buffer."""
        off = np.concatenate([[0], np.cumsum([len(x) for x in ks])]).astype(np.int32)
        w = self.Hkv * self.d
        buf = torch.full((int(off[-1]), 2 * w + pad), float("nan"), dtype=torch.float16, device="cuda")
        if off[-1]:
            buf[:, :w] = dev(np.concatenate(ks).reshape(-1, w))
            buf[:, w:2 * w] = dev(np.concatenate(vs).reshape(-1, w))
        api.pkv_byte_append(self.shape, self.ws, self.fmt, buf[:, :w].unflatten(1, (self.Hkv, self.d)),
                            buf[:, w:2 * w].unflatten(1, (self.Hkv, self.d)), self.bt, self.lens, self.cache,
                            new_offsets=None if one else dev(off), **kw)
        for i in range(self.B):
            self.k[i].append(ks[i])
            self.v[i].append(vs[i])

    def grow(self, counts, scale=1.0, **kw):
        self.append([self.normal(n, scale) for n in counts], [self.normal(n, scale) for n in counts], **kw)

    def read(self, first=None, counts=None):
        f = [0] * self.B if first is None else first
        n = [len(x.y) - a for x, a in zip(self.k, f)] if counts is None else counts
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        ko = torch.full((int(off[-1]) + 2, self.Hkv, self.d), 7.0, dtype=torch.float16, device="cuda")
        vo = torch.full_like(ko, 7.0)
        api.pkv_byte_read(self.shape, self.ws, self.fmt, self.cache, self.bt, self.lens, dev(off), ko, vo,
                          first=None if first is None else dev(np.asarray(first, np.int32)))
        assert (ko[off[-1]:] == 7.0).all() and (vo[off[-1]:] == 7.0).all()  # rows behind the last span
        return ko[:off[-1]].cpu().numpy(), vo[:off[-1]].cpu().numpy()

    def same(self, first=None):
        """What is read back is what the model holds, bit for bit."""
        f = [0] * self.B if first is None else first
        for got, side in zip(self.read(first), (self.k, self.v)):
            assert np.array_equal(bits(got), bits(np.concatenate([x.values()[a:] for x, a in zip(side, f)])))

    def decode(self, q, window=None, sinks=0, **kw):
        o = torch.full((self.B, self.Hq, self.d), float("nan"), dtype=torch.float16, device="cuda")
        lse = torch.full((self.B, self.Hq), float("nan"), dtype=torch.float32, device="cuda")
        api.pkv_byte_decode(self.shape, self.ws, self.fmt, q, self.cache, self.bt, self.lens, o, lse, window=window,
                            sinks=sinks, **kw)
        return o, lse

    def ok(self):
        st, msg = api.pkv_get_error(self.ws)
        assert st == 0, msg
        assert int(self.ws[64:64 + 4 * 1920].view(torch.int32).abs().sum()) == 0  # the counters are back at zero
        assert int(self.ws[16:64].view(torch.int32).abs().sum()) == 0

    def check(self, q, window=None, sinks=0):
        o, lse = self.decode(q, window, sinks)
        self.compare(o, lse, q, window, sinks)
        self.ok()

    def compare(self, o, lse, q, window=None, sinks=0):
        ro, rl, to, tl = R.attention(q.cpu().numpy(), self.k, self.v, float(np.float32(self.shape.scale)), window, sinks)
        x, y = o.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        bad = ~(np.abs(x - ro) <= to)
        assert not bad.any(), (np.argwhere(bad)[:4], x[bad][:4], ro[bad][:4], to[bad][:4])
        none = ~np.isfinite(rl)
        assert np.array_equal(y[none], rl[none])
        assert (np.abs(y[~none] - rl[~none]) <= tl[~none]).all(), (y[~none] - rl[~none], tl[~none])


def queries(b, seed=5, scale=1.0):
    return dev((np.random.default_rng(seed).standard_normal((b.B, b.Hq, b.d)) * scale).astype(np.float16))


# ------------------------------------------------------------------ write and read

SHAPES = [(128, 16, 2, [5, 0, 33, 1]), (64, 8, 3, [9, 1, 0, 17]), (128, 64, 1, [130, 7]), (64, 256, 8, [300]),
          (128, 8, 1, [64]), (64, 128, 2, [1, 2, 3, 4, 5, 6, 7, 129]), (64, 32, 5, [40, 31]), (128, 8, 3, [7, 8, 9, 1])]


@FORMATS
@pytest.mark.parametrize("d,P,Hkv,counts", SHAPES)
def test_append_writes_the_format_and_read_returns_it(fmt, d, P, Hkv, counts):
    b = Batch(fmt, [c + 40 for c in counts], Hkv=Hkv, G=1, d=d, P=P, seed=d + P)
    first = [3 * i % 11 for i in range(b.B)]
    b.grow(first)
    b.grow(counts, scale=3.0, pad=24)
    assert b.lens.cpu().tolist() == [a + c for a, c in zip(first, counts)]
    cache, touched = b.cache.cpu().numpy(), set()
    for i in range(b.B):
        for t in range(len(b.k[i].y)):
            page = int(b.table[i, t // P])
            touched.add(page)
            for u, side in enumerate((b.k[i], b.v[i])):
                want = np.zeros_like(cache[page])
                R.pack(want, t % P, side.y[t], side.e[t // side.sb], u, P, d, fmt)
                at = R.places(P, d)
                where = np.concatenate([at[u][t % P], at[2 + u][t % P] + np.arange(4)])
                assert np.array_equal(cache[page][:, where], want[:, where]), (i, t, u)
    rest = [p for p in range(b.num_pages) if p not in touched]
    assert (cache[rest] == 0xFF).all()  # no other page is written
    b.same()
    b.same(first)
    b.ok()


@FORMATS
@pytest.mark.parametrize("d,P", [(128, 16), (64, 8), (128, 256), (64, 32)])
def test_tokens_join_their_blocks_call_by_call(fmt, d, P):
    """Calls of one token and of a few, with magnitudes that rise and fall: blocks whose scale grows once, often or
    never."""
    b = Batch(fmt, [120, 80, 50], Hkv=3, G=1, d=d, P=P, seed=P + d)
    for step in range(40):
        size = 2.0 ** b.rng.integers(-6, 7, 3)
        if step % 5 < 3:
            b.append([b.normal(1, x) for x in size], [b.normal(1, x) for x in size[::-1]], one=True)
        else:
            n = b.rng.integers(0, 4, 3)
            b.append([b.normal(k, x) for k, x in zip(n, size)], [b.normal(k, x) for k, x in zip(n, size)])
        if step % 8 == 7:
            b.same()
    b.same()
    assert any(np.diff(np.nan_to_num(x.e), axis=0).any() for x in b.k)
    b.ok()


@FORMATS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("one", [False, True])
def test_hard_values_round_as_defined(fmt, d, one):
    """Every magnitude of fp16 as a block's greatest; ties, the greatest code's borders, subnormals, values beyond
    the limit, infinities."""
    top = R.TOP[fmt]
    b = Batch(fmt, [64 * 16], Hkv=2, G=1, d=d, P=16, seed=3)
    rows = []
    for j in range(64):
        size = np.array(2.0 ** min(j % 41 - 24, 15)).astype(np.float16)
        if j % 41 == 40:
            size = np.float16(np.inf)
        x = b.normal(1 if one else 16, 1.0) * 0
        y = b.rng.integers(-4 * int(top), 4 * int(top) + 1, x.shape) / (4 * top)  # quarters of a step: ties among them
        with np.errstate(invalid="ignore"):
            x = (y * float(size)).astype(np.float16)
        x[0, 0, 0] = size * np.float16([1.0, top / 2 ** 8, top / 2 ** 8 + 2 ** -8, 1.9][j % 4])
        if j % 16 == 13:
            x[0, 1, 5] = [np.inf, -np.inf, 65504, -65504][j // 16]
        rows.append(x)
    for x in rows:
        if one:
            b.append([x], [-x[:, ::-1]], one=True)
            while len(b.k[0].y) % 16:  # to the next block
                z = np.zeros_like(x)
                b.append([z], [z], one=True)
        else:
            b.append([x], [-x[:, ::-1]])
    b.same()
    assert not np.isinf(b.read()[0]).any()  # a size beyond the type makes NaNs of its zeros
    b.ok()


@FORMATS
def test_random_bit_patterns_round_as_defined(fmt):
    b = Batch(fmt, [1500], Hkv=4, G=1, d=128, P=64, seed=4)
    x = b.rng.integers(0, 1 << 16, (2, 1500, 4, 128)).astype(np.uint16)
    x = np.where((x & 0x7C00) == 0x7C00, x & 0x83FF, x).astype(np.uint16)  # finite
    shift = np.broadcast_to(b.rng.integers(0, 31, (2, 94, 1, 1)).repeat(16, 1)[:, :1500], x.shape)
    x = np.where((x >> 10 & 31) > shift, (x & 0x83FF) | shift << 10, x).astype(np.uint16).view(np.float16)
    b.append([x[0]], [x[1]])
    b.same()
    b.ok()


@FORMATS
@pytest.mark.parametrize("one", [False, True])
def test_a_nan_is_its_blocks_until_the_block_starts_anew(fmt, one):
    b = Batch(fmt, [64, 64], Hkv=2, G=1, d=128, P=16, seed=6)
    b.grow([20, 5])
    k, v = [b.normal(1), b.normal(1)], [b.normal(1), b.normal(1)]
    k[0][0, 1, 77] = np.nan
    b.append(k, v, one=one)
    b.same()
    assert np.isnan(b.read()[0][16:21, 1]).all() and not np.isnan(b.read()[1]).any()
    b.grow([1, 1], one=True)  # a block that has joined a NaN keeps it
    b.same()
    q = queries(b)
    o, lse = b.decode(q)
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, 1]) and not torch.isnan(o[0, 0]).any() and not torch.isnan(o[1]).any()
    o, lse = b.decode(q, window=3, sinks=16)  # its block is seen in part
    assert torch.isnan(o[0, 1]).all() and not torch.isnan(o[1]).any()
    o, lse = b.decode(q, window=0, sinks=16)  # not at all
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    b.lens[0] = 16  # the row is cut back to before the block, which then starts anew
    for side in (b.k[0], b.v[0]):
        side.y, side.e = side.y[:16], side.e[:1]
    b.grow([1, 0], one=False)
    b.same()
    b.check(q)


@FORMATS
def test_append_to_other_lengths_leaves_the_old_ones(fmt):
    b = Batch(fmt, [60, 60], seed=8)
    b.grow([20, 3])
    out = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    b.grow([7, 30], seq_lens_out=out)
    assert b.lens.cpu().tolist() == [20, 3] and out.cpu().tolist() == [27, 33]
    b.lens = out
    b.same()


@FORMATS
@pytest.mark.parametrize("new", [[0, 0, 4], [0, 0, 0, 9, 0], [0, 17, 0], [0, 1], [0, 0]])
def test_rows_without_new_tokens_among_the_others(fmt, new):
    b = Batch(fmt, [50] * len(new), d=64, P=8, seed=9)
    b.grow([5 + i for i in range(len(new))])
    b.table[0, 0] = 10 ** 6  # such a row's page is not looked at
    keep = b.bt.clone()
    b.bt.copy_(dev(b.table))
    b.grow(new)
    b.bt.copy_(keep)
    b.same()
    b.ok()


@FORMATS
def test_rows_that_cannot_take_their_tokens_keep_their_length(fmt):
    b = Batch(fmt, [64, 64, 64, 64], seed=10)
    b.grow([10, 20, 30, 16])
    bt = b.bt.clone()
    b.bt[1, 1] = b.num_pages  # its last block's page; row 3: the next page
    b.bt[3, 1] = -1
    before = b.cache.clone()
    k = [b.normal(n) for n in (60, 5, 5, 2)]
    off = dev(np.array([0, 60, 65, 70, 72], np.int32))
    x = dev(np.concatenate(k))
    for one in (False, True):
        b.lens.copy_(dev(np.array([10, 20, 30, 16], np.int32)))
        if one:
            b.lens[0] = 64
            api.pkv_byte_append(b.shape, b.ws, fmt, x[:4], x[:4], b.bt, b.lens, b.cache)
            assert b.lens.cpu().tolist() == [64, 20, 31, 16]
        else:
            api.pkv_byte_append(b.shape, b.ws, fmt, x, x, b.bt, b.lens, b.cache, new_offsets=off)
            assert b.lens.cpu().tolist() == [10, 20, 35, 16]
        assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
        assert torch.equal(b.cache[bt[1, :2].long()], before[bt[1, :2].long()])
    for bad in ([0, 60, 50, 70, 72], [0, 60, 65, 70, 73], [-1, 60, 65, 70, 72], [5, 4, 3, 2, 1]):
        b.lens.copy_(dev(np.array([10, 20, 30, 16], np.int32)))
        api.pkv_byte_append(b.shape, b.ws, fmt, x, x, bt, b.lens, b.cache, new_offsets=dev(np.array(bad, np.int32)))
        assert b.lens.cpu().tolist() == [10, 20, 30, 16]
        assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    b.lens[2] = -4
    b.grow([0, 0, 3, 0])
    assert b.lens[2] == -4 and "negative" in api.pkv_get_error(b.ws)[1]
    b.ok()


@FORMATS
def test_read_outside_a_row_is_zeros_and_an_error(fmt):
    b = Batch(fmt, [40, 40], seed=11)
    b.grow([33, 20])
    want = [np.concatenate([x.values(), np.zeros((7, 2, 128))]) for x in b.k]
    k, v = b.read(first=[30, 16], counts=[10, 8])
    assert np.array_equal(bits(k), bits(np.concatenate([want[0][30:40], want[1][16:24]])))
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    k, v = b.read(first=[-3, 0], counts=[5, 1])
    assert (k[:3] == 0).all() and (v[:3] == 0).all() and np.array_equal(bits(k[3:5]), bits(want[0][:2]))
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    b.bt[0, 1] = -7
    k, v = b.read()
    assert (k[16:32] == 0).all() and (v[16:32] == 0).all() and np.array_equal(bits(k[33:]), bits(want[1][:20]))
    assert "row 0" in api.pkv_get_error(b.ws)[1]
    b.read(first=[0, 2 ** 31 - 1], counts=[0, 5])
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    b.ok()


@FORMATS
def test_read_into_strided_outputs(fmt):
    b = Batch(fmt, [70, 9], Hkv=3, d=64, P=32, seed=12)
    b.grow([70, 9])
    buf = torch.full((80, 2 * 192 + 40), 5.0, dtype=torch.float16, device="cuda")
    ko, vo = buf[:, 8:200].unflatten(1, (3, 64)), buf[:, 208:400].unflatten(1, (3, 64))
    api.pkv_byte_read(b.shape, b.ws, fmt, b.cache, b.bt, b.lens, dev(np.array([1, 71, 80], np.int32)), ko, vo)
    for got, side in ((ko, b.k), (vo, b.v)):
        assert np.array_equal(bits(got[1:].cpu().numpy()), bits(np.concatenate([x.values() for x in side])))
    assert (buf[:, :8] == 5).all() and (buf[:, 200:208] == 5).all() and (buf[:, 400:] == 5).all() and (buf[0] == 5).all()
    b.ok()


def test_a_zero_filled_cache_holds_zeros():
    for fmt in (R.INT8, R.E4M3):
        b = Batch(fmt, [100, 30], d=64, P=64, fill=0, seed=13)
        b.lens.copy_(dev(np.array([100, 30], np.int32)))
        k, v = b.read(counts=[100, 30])
        assert (k == 0).all() and (v == 0).all()
        o, lse = b.decode(queries(b))
        assert (o == 0).all() and torch.allclose(lse, torch.log(b.lens.float()).unsqueeze(1).expand_as(lse), atol=1e-5)
        b.ok()


@FORMATS
@pytest.mark.parametrize("B", [33, 64, 65, 130, 1100])
def test_many_rows(fmt, B):
    """Rows found in one look and by a search, with and without new tokens, written, read and decoded."""
    rng = np.random.default_rng(B)
    first, new = rng.integers(0, 20, B).tolist(), (rng.integers(0, 40, B) * rng.integers(0, 2, B)).tolist()
    b = Batch(fmt, [x + y for x, y in zip(first, new)], Hkv=1, G=2, d=64, P=16, seed=B)
    b.grow(first)
    b.grow(new)
    b.same()
    b.same([x // 2 for x in first])
    b.check(queries(b))


@FORMATS
@pytest.mark.parametrize("d,P,Hkv,new", [(128, 16, 4, [5000, 0, 3, 4300, 1]), (64, 8, 8, [8200]), (128, 64, 11, [8000, 17, 700]),
                                         (64, 16, 19, [3, 9000]), (128, 8, 8, [1] * 100 + [8300]), (64, 256, 3, [8192, 64])])
def test_many_tokens(fmt, d, P, Hkv, new):
    """Prompts of many tokens behind rows of any length: blocks that hold earlier tokens, chunks of heads that are
    not whole, tokens with a stride, a page out of range in the middle."""
    first = [(7 * i) % 37 for i in range(len(new))]
    b = Batch(fmt, [x + y for x, y in zip(first, new)], Hkv=Hkv, G=1, d=d, P=P, seed=len(new) + d)
    b.grow(first, scale=0.1)
    b.grow(new, pad=40)
    b.same()
    b.ok()
    long = int(np.argmax(new))
    b.lens[long] = first[long]
    keep = b.bt.clone()
    bad = (first[long] + 100) // P + 1
    b.bt[long, bad] = b.num_pages + 3
    before = [len(x.y) for x in b.k]
    x = torch.zeros((8192 + sum(new), Hkv, d), dtype=torch.float16, device="cuda")  # tokens behind the last offset
    off = np.array([0] * (long + 1) + [new[long]] * (b.B - long), np.int32)
    api.pkv_byte_append(b.shape, b.ws, fmt, x, x, b.bt, b.lens, b.cache, new_offsets=dev(off))
    assert b.lens.tolist() == [first[long] if i == long else n for i, n in enumerate(before)]  # the row keeps its length
    st, msg = api.pkv_get_error(b.ws)
    assert st == _lib.PKV_EDEVICE and f"row {long}, logical page {bad}" in msg
    b.bt.copy_(keep)
    b.ok()


@pytest.mark.parametrize("Hkv", [1824, 2048])
def test_few_tokens_of_very_many_heads(Hkv):
    b = Batch(R.E4M3, [16], Hkv=Hkv, G=1, d=64, P=8, seed=14)
    b.grow([1])
    b.grow([2])
    b.grow([1], one=True)
    b.same()
    b.ok()


# ------------------------------------------------------------------ decode

HEADS = [(128, 16, 2, 4), (64, 8, 3, 5), (128, 64, 1, 8), (64, 256, 2, 1), (128, 8, 8, 2), (64, 32, 1, 7), (128, 128, 2, 3),
         (64, 16, 2, 6)]


@FORMATS
@pytest.mark.parametrize("wide", [0, 4096])
@pytest.mark.parametrize("d,P,Hkv,G", HEADS)
def test_decode_rows_of_every_length(fmt, wide, d, P, Hkv, G):
    """Around every border of a block, tile and page, on clusters (narrow tables) and on cut runs (wide ones)."""
    lens = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300, 511, 513]
    b = Batch(fmt, lens, Hkv=Hkv, G=G, d=d, P=P, seed=d + P + G, wide=wide)
    b.grow(lens)
    b.check(queries(b))
    b.check(queries(b, seed=6, scale=4.0))


@FORMATS
@pytest.mark.parametrize("wide", [0, 4096])
@pytest.mark.parametrize("lens,d", [([4097], 128), ([8000, 1, 0, 129], 128), ([1500] * 9, 64), ([64] * 40 + [3000], 128),
                                    ([0, 0, 5000], 64), ([0] * 70 + [300], 64), ([20000], 128)])
def test_decode_long_rows(fmt, wide, lens, d):
    b = Batch(fmt, lens, Hkv=2, G=4, d=d, P=16, seed=len(lens), wide=wide)
    b.grow(lens)
    b.check(queries(b))


@FORMATS
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (5, 0), (16, 4), (64, 1), (63, 17), (100, 64), (130, 70), (1000, 5)])
@pytest.mark.parametrize("d,P", [(128, 16), (64, 64), (64, 8), (128, 8)])
def test_decode_in_a_window(fmt, window, sinks, d, P):
    lens = [0, 1, 4, 16, 17, 63, 64, 130, 250, 400]
    b = Batch(fmt, lens, Hkv=2, G=3, d=d, P=P, seed=window + sinks)
    b.grow(lens)
    b.check(queries(b), window, sinks)


@FORMATS
@pytest.mark.parametrize("P", [8, 16, 32, 64, 128])
def test_more_heads_than_the_gpu_holds_ctas(fmt, P):
    """Batches of many rows, whose (row, head)s come to more than two CTAs per SM."""
    rng = np.random.default_rng(P)
    lens = rng.integers(0, 400, 90).tolist()
    lens[3] = lens[40] = 0
    b = Batch(fmt, lens, Hkv=4, G=3, d=128, P=P, seed=P)
    b.grow(lens)
    b.check(queries(b))
    b.check(queries(b, seed=6), 100, 5)
    first = b.decode(queries(b))
    again = b.decode(queries(b))
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    b.bt[7, 0] = -1
    for side in (b.k[7], b.v[7]):
        side.y[:P] = 0
    o, lse = b.decode(queries(b))
    assert lens[7] > 0 and api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    b.compare(o, lse, queries(b))
    assert _lib.load().pkv_test_starve_next_decodes(1) == 0
    b.decode(queries(b))
    assert api.pkv_get_error(b.ws)[0] in (_lib.PKV_ETIMEOUT, _lib.PKV_EDEVICE)
    b.ws.zero_()


@FORMATS
@pytest.mark.parametrize("wide", [0, 4096])
def test_blocks_of_very_unequal_scales(fmt, wide):
    """V blocks from 2^-20 to 2^14, K blocks alike with queries to match: the weights carry V's scales."""
    lens = [700, 33, 400]
    b = Batch(fmt, lens, Hkv=2, G=4, d=128, P=16, seed=15, wide=wide)
    ks, vs = [], []
    for n in lens:
        size = (2.0 ** b.rng.integers(-20, 14, (n + 15) // 16)).repeat(16)[:n, None, None]
        ks.append((b.normal(n) * np.minimum(size[::-1], 16.0)).astype(np.float16))
        vs.append((np.clip(b.normal(n), -3, 3) * size).astype(np.float16))
    b.append(ks, vs)
    for scale in (0.0, 0.3, 1.0):
        b.check(queries(b, scale=scale))
        b.check(queries(b, scale=scale), 100, 20)


@FORMATS
def test_decode_of_large_and_tiny_values(fmt):
    b = Batch(fmt, [200, 90], Hkv=2, G=2, d=64, P=16, seed=16)
    b.append([b.normal(200, 6000.0), b.normal(90, 1e-6)], [b.normal(200, 9000.0), b.normal(90, 2e-7)])
    b.check(queries(b, scale=1e-3))
    b.check(queries(b, scale=1e-6))


@FORMATS
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_any_scale_of_the_scores(fmt, scale):
    b = Batch(fmt, [300, 17], Hkv=2, G=3, d=128, P=32, seed=21, scale=scale)
    b.grow([300, 17])
    b.check(queries(b))
    b.check(queries(b), 40, 3)


@FORMATS
@pytest.mark.parametrize("wide", [0, 4096])
def test_scores_that_rise_and_fall_along_the_row(fmt, wide):
    b = Batch(fmt, [600, 600], Hkv=1, G=4, d=64, P=16, seed=17, scale=1.0, wide=wide)
    ramp = np.linspace(0, 1, 600)[:, None, None]
    ks = [(np.ones((600, 1, 64)) * r).astype(np.float16) for r in (ramp, ramp[::-1])]
    b.append(ks, [b.normal(600), b.normal(600)])
    for scale in (0.05, 1.0, 50.0):
        q = dev(np.full((2, 4, 64), scale, np.float16))
        b.check(q)


@FORMATS
def test_scores_beyond_the_type_have_a_greatest(fmt):
    """Scores far from zero, equal and unequal: o stays a mean of values."""
    b = Batch(fmt, [300], Hkv=1, G=2, d=64, P=16, seed=18, scale=1.0)
    k = np.zeros((300, 1, 64), np.float16)
    k[:, 0, 0] = np.where(np.arange(300) % 3 == 0, 1.0, 0.5)
    v = b.normal(300)
    b.append([k], [v])
    for size in (3e4, -3e4, 6e4):
        q = np.zeros((1, 2, 64), np.float16)
        q[0, :, 0] = size
        o, lse = b.decode(dev(q))
        pick = np.arange(300) % 3 == 0 if size > 0 else np.arange(300) % 3 != 0
        want = b.v[0].values()[pick, 0].mean(0)
        # half steps of weights and o: 2^-11 (mean |v| + |o|) with equal weights
        bound = 2.0 ** -11 * (np.abs(b.v[0].values()[pick, 0]).mean(0) + np.abs(want)) + 2.0 ** -16
        assert (np.abs(o[0].cpu().numpy().astype(np.float64) - want) <= bound).all()
        assert torch.isfinite(lse).all()
    b.ok()


@pytest.mark.parametrize("rows", [1, 300])
def test_a_mean_of_the_greatest_values_stays_finite(rows):
    for fmt, top in ((R.INT8, 65024.0), (R.E4M3, 57344.0)):
        b = Batch(fmt, [50] * rows, Hkv=1, G=4, d=64, P=16, seed=19)
        x = np.full((50, 1, 64), 65504, np.float16)
        x[:, 0, 1::2] *= -1
        b.append([np.zeros_like(x)] * rows, [x] * rows)
        o, lse = b.decode(queries(b))
        assert (o.abs() == top).all() or (o.float().abs() - top).abs().max() <= 32  # a step of fp16 there
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        b.ok()


@FORMATS
@pytest.mark.parametrize("fill", [0x00, 0x7F, 0x80, 0xFF, 0x7E])
def test_what_no_token_was_written_to_holds_anything(fmt, fill):
    """The places behind a row's end in its last page and block, whatever bytes they hold."""
    lens = [1, 5, 17, 40, 100, 130]
    b = Batch(fmt, lens, Hkv=2, G=4, d=128, P=64, seed=20, fill=fill)
    b.grow(lens)
    b.check(queries(b))
    b.check(queries(b), 9, 2)


@FORMATS
def test_decode_reports_bad_pages_and_lengths(fmt):
    b = Batch(fmt, [40, 40, 40], seed=26)
    b.grow([40, 40, 40])
    q = queries(b)
    b.bt[1, 1] = 9999
    o, lse = b.decode(q)
    st, msg = api.pkv_get_error(b.ws)
    assert st == _lib.PKV_EDEVICE and "row 1" in msg
    # the bad page counts as zeros
    for side in (b.k[1], b.v[1]):
        side.y[16:32] = 0
    b.compare(o, lse, q)
    o, lse = b.decode(q, 4, 4)  # the bad page lies between the sinks and the window
    b.compare(o, lse, q, 4, 4)
    b.ok()
    b.lens[0] = -1
    o, lse = b.decode(q, 4, 4)
    assert (o[0] == 0).all() and (lse[0] == -float("inf")).all()
    assert "negative" in api.pkv_get_error(b.ws)[1]
    b.lens[0] = 10 ** 6
    b.decode(q, 0, 4)
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    b.ok()


@FORMATS
@pytest.mark.parametrize("wide", [0, 4096])
@pytest.mark.parametrize("d,P", [(128, 8), (64, 16), (128, 64), (64, 128)])
def test_a_bad_page_counts_as_zeros(fmt, wide, d, P):
    """Whatever the memory it would have gone to held: a batch whose bytes behind the rows are NaNs' goes first."""
    b = Batch(fmt, [3 * P] * 6, d=d, P=P, seed=P, wide=wide)
    b.grow([3 * P] * 6)
    q = queries(b)
    dirty = Batch(fmt, [1] * 300, d=d, P=P, seed=1, fill=0x7F, wide=wide)
    dirty.grow([1] * 300)
    b.bt[:, 1] = -5
    for side in b.k + b.v:
        side.y[P:2 * P] = 0
    for _ in range(3):
        dirty.decode(queries(dirty))
        o, lse = b.decode(q)
        b.compare(o, lse, q)
        assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE


@FORMATS
def test_pages_beyond_32_bit_offsets(fmt):
    Hkv, d, P = 8, 128, 256
    pages = (1 << 32) // (Hkv * R.head_bytes(P, d)) + 40
    b = Batch(fmt, [600], Hkv=Hkv, G=1, d=d, P=P, seed=27)
    b.cache = torch.empty((pages, Hkv, R.head_bytes(P, d)), dtype=torch.uint8, device="cuda")
    b.bt.copy_(dev(np.array([[pages - 1, pages - 7, pages - 2]], np.int32)))
    b.shape.num_pages = pages
    b.grow([599])
    b.grow([1], one=True)
    b.check(queries(b))
    b.same()


@FORMATS
def test_append_decode_loop_captured_as_a_graph(fmt):
    """The serving step -- append a token, decode -- captured once and replayed, on a stream of its own, after an
    eager step on the same buffers."""
    b = Batch(fmt, [90, 60, 75], Hkv=2, G=4, d=128, P=16, seed=28)
    b.grow([40, 0, 25])
    kn, vn = (torch.zeros((3, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros((3, 8, 128), dtype=torch.float16, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros((3, 8), dtype=torch.float32, device="cuda")

    def step():
        api.pkv_byte_append(b.shape, b.ws, fmt, kn, vn, b.bt, b.lens, b.cache)
        api.pkv_byte_decode(b.shape, b.ws, fmt, q, b.cache, b.bt, b.lens, o, lse, window=30, sinks=2)

    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    for t in range(6):
        k, v = b.normal(3, 1.0 + t), b.normal(3)
        kn.copy_(dev(k))
        vn.copy_(dev(v))
        q.copy_(queries(b, seed=100 + t))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            if t == 1:
                with torch.cuda.graph(g, stream=st):
                    step()
            if t == 0:
                step()
            else:
                g.replay()
        torch.cuda.synchronize()
        for i in range(3):
            b.k[i].append(k[i:i + 1])
            b.v[i].append(v[i:i + 1])
        b.compare(o, lse, q, 30, 2)
    assert b.lens.cpu().tolist() == [46, 6, 31]
    b.same()
    b.ok()


@FORMATS
def test_the_same_call_gives_the_same_bits(fmt):
    b = Batch(fmt, [3000, 10, 700], Hkv=4, G=8, d=128, P=16, seed=29, wide=4096)
    b.grow([3000, 10, 700])
    q = queries(b)
    first = b.decode(q)
    for _ in range(5):
        again = b.decode(q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@FORMATS
def test_decode_of_runs_that_are_split(fmt):
    """Runs long enough that their ends are claimed by whichever CTA is free: every row repeats its pages 64 times,
    so o is that of one repetition and lse larger by ln 64."""
    times, P = 64, 64
    b = Batch(fmt, [16 * P] * 8, Hkv=8, G=8, d=128, P=P, seed=41)
    b.grow([16 * P] * 8)
    b.bt = b.bt.repeat(1, times).contiguous()
    b.shape.bt_stride = 16 * times
    b.lens = b.lens * times
    b.lens[3] = 0
    b.lens[5] = b.lens[5] // times
    q = queries(b)
    first = b.decode(q)
    for _ in range(4):
        again = b.decode(q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    for side in (b.k[3], b.v[3]):
        side.y, side.e = side.y[:0], side.e[:0]
    ro, rl, to, tl = R.attention(q.cpu().numpy(), b.k, b.v, float(np.float32(b.shape.scale)))
    rl[[0, 1, 2, 4, 6, 7]] += np.log(times)
    x, y = first[0].cpu().numpy().astype(np.float64), first[1].cpu().numpy().astype(np.float64)
    # a repetition adds to the weights' roundings below 2^-14 only: 64 times the term for those
    extra = 2.0 ** -25 * 1024 * times * max(R.TOP[fmt] * v.scales().max() for v in b.v if len(v.y))
    assert (np.abs(x - ro) <= to + extra).all()
    assert (y[3] == -np.inf).all()
    rows = [i for i in range(8) if i != 3]
    # fp32 sums of 65536 weights: 2^-24 times the depth of the sums (tiles per warp and merges, some 2^12)
    assert (np.abs(y[rows] - rl[rows]) <= tl[rows] + 2.0 ** -12).all()
    b.ok()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("wide", [0, 4096])
def test_a_wait_that_runs_out_is_reported(d, wide):
    b = Batch(R.INT8, [400, 30], d=d, seed=42, wide=wide)
    b.grow([400, 30])
    q = queries(b)
    b.check(q)
    assert _lib.load().pkv_test_starve_next_decodes(1) == 0
    b.decode(q)
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_ETIMEOUT
    b.ws.zero_()  # the counters of a launch that gave up
    b.check(q)


def test_calls_on_two_streams_with_a_workspace_each():
    bs = [Batch(f, [900, 30, 500], seed=60 + f, wide=4096) for f in (R.INT8, R.E4M3)]
    for b in bs:
        b.grow([900, 30, 500])
    qs = [queries(b) for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    outs = []
    for _ in range(5):
        outs = [b.decode(q, stream=s) for b, q, s in zip(bs, qs, streams)]
    torch.cuda.synchronize()
    for b, q, (o, lse) in zip(bs, qs, outs):
        b.compare(o, lse, q)
        b.ok()


def test_lse_may_be_left_out():
    b = Batch(R.E4M3, [300, 0], seed=61)
    b.grow([300, 0])
    q = queries(b)
    want, _ = b.decode(q)
    o = torch.empty_like(q)
    api.pkv_byte_decode(b.shape, b.ws, R.E4M3, q, b.cache, b.bt, b.lens, o)
    assert torch.equal(o, want)


def test_binding_refuses_wrong_tensors():
    b = Batch(R.INT8, [40, 40], seed=44)
    b.grow([20, 20])
    q = queries(b)
    o = torch.empty_like(q)
    good = dict(shape=b.shape, ws=b.ws, fmt=0, q=q, byte_cache=b.cache, block_table=b.bt, seq_lens=b.lens, o=o)
    for bad, kind in ((dict(q=q.float()), ValueError), (dict(q=q[:1]), ValueError), (dict(q=q.transpose(0, 1)), ValueError),
                      (dict(q=None), TypeError), (dict(ws=b.ws[:100]), ValueError), (dict(byte_cache=b.cache[1:]), ValueError),
                      (dict(byte_cache=b.cache.char()), ValueError), (dict(block_table=b.bt[:1]), ValueError),
                      (dict(seq_lens=b.lens[:1]), ValueError), (dict(o=o.float()), ValueError), (dict(window=2 ** 31), ValueError),
                      (dict(shape=3), TypeError), (dict(window=-1), _lib.PkvError), (dict(sinks=1), ValueError),
                      (dict(fmt=2), _lib.PkvError), (dict(fmt="e4m3"), TypeError)):
        with pytest.raises(kind):
            api.pkv_byte_decode(**{**good, **bad})
    x = torch.zeros(2, 2, 128, dtype=torch.float16, device="cuda")
    wide = torch.zeros(2, 2, 256, dtype=torch.float16, device="cuda")
    for k, v in ((x.float(), x), (x, x[:1]), (x[:, :1], x[:, :1]), (x, wide[:, :, :128]), (wide[:, :, ::2], wide[:, :, ::2]), (x[0], x[0])):
        with pytest.raises(ValueError):
            api.pkv_byte_append(b.shape, b.ws, 0, k, v, b.bt, b.lens, b.cache)
    with pytest.raises(_lib.PkvError):  # three tokens for two rows
        y = torch.zeros(3, 2, 128, dtype=torch.float16, device="cuda")
        api.pkv_byte_append(b.shape, b.ws, 0, y, y, b.bt, b.lens, b.cache)
    b.ok()


@FORMATS
def test_decoder_object_runs_the_byte_steps(fmt):
    dec = api.PagedDecoder()
    b = Batch(fmt, [60, 33], Hkv=2, G=4, d=64, P=8, seed=45)
    k, v = [b.normal(50), b.normal(20)], [b.normal(50), b.normal(20)]
    dec.append_byte(fmt, dev(np.concatenate(k)), dev(np.concatenate(v)), b.cache, b.bt, b.lens, dev(np.array([0, 50, 70], np.int32)))
    for i in range(2):
        b.k[i].append(k[i])
        b.v[i].append(v[i])
    b.same()
    q = queries(b)
    o, lse = dec.step_byte(fmt, q, b.cache, b.bt, b.lens)
    b.compare(o, lse, q)
    o, lse = dec.step_byte(fmt, q, b.cache, b.bt, b.lens, window=20, sinks=3)
    b.compare(o, lse, q, 20, 3)
    ko, vo = torch.empty(70, 2, 64, dtype=torch.float16, device="cuda"), torch.empty(70, 2, 64, dtype=torch.float16, device="cuda")
    dec.read_byte(fmt, b.cache, b.bt, b.lens, dev(np.array([0, 50, 70], np.int32)), ko, vo)
    assert np.array_equal(bits(vo.cpu().numpy()), bits(np.concatenate([x.values() for x in b.v])))
