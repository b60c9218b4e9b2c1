"""The 4-bit KV cache on the GPU: writing, reading back, and decode over it,
against the plain float64 model; and decode with a sliding window over the fp16
pages."""
import numpy as np
import pytest
import torch

import quant_ref as R
from paged_kv_gqa_09_gb300 import _lib, api

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def clean(ws):
    """The workspace's counters are back at zero."""
    assert int(ws[64:64 + 4 * 1920].view(torch.int32).abs().sum()) == 0
    assert int(ws[16:64].view(torch.int32).abs().sum()) == 0


class Batch:
    """A batch over the 4-bit cache: shuffled pages, a workspace, device tensors."""

    def __init__(self, cap, Hkv=2, G=4, d=128, P=16, seed=0, spare=3, fill=0xFF, scale=None):
        rng = np.random.default_rng(seed)
        self.rng, self.B, self.Hkv, self.G, self.Hq, self.d, self.P = rng, len(cap), Hkv, G, Hkv * G, d, P
        pages = [-(-c // P) for c in cap]
        self.num_pages = max(1, sum(pages)) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((self.B, max(1, max(pages, default=1))), order[-1], np.int32)
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = order[at:at + n]
            at += n
        # what no token was written to holds NaN params and code bits
        self.cache = torch.full((self.num_pages, Hkv, P * d * 5 // 4), fill, dtype=torch.uint8, device="cuda")
        self.bt = dev(self.table)
        self.lens = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        self.shape = api.make_quant_shape(self.Hq, d, self.cache, self.bt, scale)
        self.ws = torch.zeros(api.pkv_attn_workspace_size(self.shape), dtype=torch.uint8, device="cuda")
        self.k = [np.zeros((0, Hkv, d), np.float16) for _ in cap]
        self.v = [np.zeros((0, Hkv, d), np.float16) for _ in cap]

    def normal(self, n, scale=1.0):
        return (self.rng.standard_normal((n, self.Hkv, self.d)) * scale).astype(np.float16)

    def append(self, ks, vs, one=False, pad=0):
        """Append ks[i], vs[i] [n, Hkv, d] to each row, through one packed buffer."""
        off = np.concatenate([[0], np.cumsum([len(x) for x in ks])]).astype(np.int32)
        w = self.Hkv * self.d
        buf = torch.full((int(off[-1]), 2 * w + pad), float("nan"), dtype=torch.float16, device="cuda")
        if off[-1]:
            buf[:, :w] = dev(np.concatenate(ks).reshape(-1, w))
            buf[:, w:2 * w] = dev(np.concatenate(vs).reshape(-1, w))
        api.pkv_quant_append(self.shape, self.ws, buf[:, :w].unflatten(1, (self.Hkv, self.d)),
                             buf[:, w:2 * w].unflatten(1, (self.Hkv, self.d)), self.bt, self.lens, self.cache,
                             new_offsets=None if one else dev(off))
        for i in range(self.B):
            self.k[i] = np.concatenate([self.k[i], ks[i]])
            self.v[i] = np.concatenate([self.v[i], vs[i]])

    def grow(self, counts, scale=1.0, **kw):
        self.append([self.normal(n, scale) for n in counts], [self.normal(n, scale) for n in counts], **kw)

    def read(self, first=None, counts=None, lens=None):
        f = [0] * self.B if first is None else first
        n = [len(x) - a for x, a in zip(self.k, f)] if counts is None else counts
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        ko = torch.full((int(off[-1]) + 2, self.Hkv, self.d), 7.0, dtype=torch.float16, device="cuda")
        vo = torch.full_like(ko, 7.0)
        api.pkv_quant_read(self.shape, self.ws, self.cache, self.bt, self.lens, dev(off), ko, vo,
                           first=None if first is None else dev(np.asarray(first, np.int32)))
        assert (ko[off[-1]:] == 7.0).all() and (vo[off[-1]:] == 7.0).all()  # rows behind the last span
        return ko[:off[-1]].cpu().numpy(), vo[:off[-1]].cpu().numpy()

    def decode(self, q, window=None, sinks=0, **kw):
        o = torch.full((self.B, self.Hq, self.d), float("nan"), dtype=torch.float16, device="cuda")
        lse = torch.full((self.B, self.Hq), float("nan"), dtype=torch.float32, device="cuda")
        api.pkv_quant_decode(self.shape, self.ws, q, self.cache, self.bt, self.lens, o, lse, window=window, sinks=sinks, **kw)
        return o, lse

    def ok(self):
        st, msg = api.pkv_get_error(self.ws)
        assert st == 0, msg
        clean(self.ws)

    def check(self, q, window=None, sinks=0):
        o, lse = self.decode(q, window, sinks)
        compare(o, lse, q, [R.values(x) for x in self.k], [R.values(x) for x in self.v], self.shape.scale, window, sinks)
        self.ok()


def compare(o, lse, q, ks, vs, scale, window, sinks):
    ro, rl, to, tl = R.attention(q.cpu().numpy(), ks, vs, float(np.float32(scale)), window, sinks)
    x = o.cpu().numpy().astype(np.float64)
    bad = ~(np.abs(x - ro) <= to)
    assert not bad.any(), (np.argwhere(bad)[:4], x[bad][:4], ro[bad][:4], to[bad][:4])
    y = lse.cpu().numpy().astype(np.float64)
    none = ~np.isfinite(rl)
    assert np.array_equal(y[none], rl[none])
    assert (np.abs(y[~none] - rl[~none]) <= tl[~none]).all(), (y[~none] - rl[~none], tl[~none])


def queries(b, seed=5, scale=1.0):
    return dev((np.random.default_rng(seed).standard_normal((b.B, b.Hq, b.d)) * scale).astype(np.float16))


def bits(x):
    """fp16 bits with one NaN and one zero."""
    x = np.asarray(x).astype(np.float16)
    return np.where(np.isnan(x), 0x7FFF, np.where(x == 0, 0, x.view(np.uint16)))


# ------------------------------------------------------------------ write and read

SHAPES = [(128, 16, 2, [5, 0, 33, 1]), (64, 8, 3, [9, 1, 0, 17]), (128, 64, 1, [130, 7]), (64, 256, 8, [300]),
          (128, 8, 1, [64]), (64, 128, 2, [1, 2, 3, 4, 5, 6, 7, 129])]


@pytest.mark.parametrize("d,P,Hkv,counts", SHAPES)
def test_append_writes_the_format_and_read_returns_it(d, P, Hkv, counts):
    b = Batch([c + 40 for c in counts], Hkv=Hkv, G=1, d=d, P=P, seed=d + P, fill=0)
    first = [3 * i % 11 for i in range(b.B)]
    b.grow(first)
    b.grow(counts, pad=24)
    assert b.lens.cpu().tolist() == [a + c for a, c in zip(first, counts)]
    want = np.zeros((b.num_pages, Hkv, P * d * 5 // 4), np.uint8)
    for i in range(b.B):
        for t in range(len(b.k[i])):
            R.pack_token(want[b.table[i, t // P]], t % P, b.k[i][t], b.v[i][t], P, d)
    assert np.array_equal(b.cache.cpu().numpy(), want)
    k, v = b.read()
    assert np.array_equal(bits(k), bits(np.concatenate([R.values(x) for x in b.k])))
    assert np.array_equal(bits(v), bits(np.concatenate([R.values(x) for x in b.v])))
    k, v = b.read(first=first)
    assert np.array_equal(bits(v), bits(np.concatenate([R.values(x[a:]) for x, a in zip(b.v, first)])))
    b.ok()


def hard_groups(rng, n, d):
    """Groups where rounding decides: ties, tiny and huge values, one value, far offsets, infinities, NaN."""
    g = []
    for i in range(n * d // 32):
        kind = i % 12
        x = rng.standard_normal(32)
        if kind == 1:
            x = x * 2.0 ** -20
        elif kind == 2:
            x = x * 30000
        elif kind == 3:
            x = np.full(32, x[0])
        elif kind == 4:
            x = 1000 + x
        elif kind == 5:
            x[rng.integers(32)] = np.inf
        elif kind == 6:
            x[rng.integers(32)] = -np.inf
        elif kind == 7:
            x[rng.integers(32)] = np.nan
        elif kind == 8:
            x = rng.integers(0, 31, 32) / 2.0  # halves of a step where the range is 15
            x[:2] = 0.0, 15.0
        elif kind == 9:
            x = rng.integers(0, 3, 32) * 2.0 ** -24
        elif kind == 10:
            x = -16000 + rng.integers(0, 200, 32) * 8.0
        elif kind == 11:
            x = np.where(rng.integers(0, 2, 32) == 0, 0.0, -0.0)
        g.append(x)
    with np.errstate(over="ignore"):
        return np.concatenate(g).astype(np.float16).reshape(n, 1, d)


@pytest.mark.parametrize("d", [64, 128])
def test_hard_values_round_as_defined(d):
    b = Batch([200], Hkv=1, G=1, d=d, P=32, seed=3)
    rng = np.random.default_rng(7)
    b.append([hard_groups(rng, 180, d)], [hard_groups(rng, 180, d)])
    k, v = b.read()
    assert np.array_equal(bits(k), bits(R.values(b.k[0])))
    assert np.array_equal(bits(v), bits(R.values(b.v[0])))
    b.ok()


def test_random_bit_patterns_round_as_defined():
    """fp16 numbers drawn over all finite bit patterns: groups that span the whole range of exponents."""
    b = Batch([512], Hkv=2, G=1, d=128, P=64, seed=4)
    rng = np.random.default_rng(8)
    x = rng.integers(0, 0x7C00, (2, 512, 2, 128)).astype(np.uint16) | (rng.integers(0, 2, (2, 512, 2, 128)) << 15).astype(np.uint16)
    x = x.view(np.float16)
    x[:, :, 1] *= np.float16(2.0 ** -6)
    b.append([x[0]], [x[1]])
    k, v = b.read()
    assert np.array_equal(bits(k), bits(R.values(x[0])))
    assert np.array_equal(bits(v), bits(R.values(x[1])))


@pytest.mark.parametrize("d,P", [(128, 16), (64, 8), (128, 256)])
def test_tokens_one_at_a_time_equal_one_prompt(d, P):
    a = Batch([70, 41, 55], d=d, P=P, seed=9, fill=0)
    b = Batch([70, 41, 55], d=d, P=P, seed=9, fill=0)
    a.grow([67, 38, 52])
    for t in range(38):
        b.append([x[t:t + 1] for x in a.k], [x[t:t + 1] for x in a.v], one=True)
    b.append([x[38:] for x in a.k], [x[38:] for x in a.v])
    assert torch.equal(a.cache, b.cache) and torch.equal(a.lens, b.lens)
    a.ok()
    b.ok()


def test_append_to_other_lengths_leaves_the_old_ones():
    b = Batch([64, 64], seed=10, fill=0)
    b.grow([5, 9])
    out = torch.zeros_like(b.lens)
    x = dev(b.normal(2))
    before = None
    for _ in range(2):  # twice the same call: the same cache
        api.pkv_quant_append(b.shape, b.ws, x, x, b.bt, b.lens, b.cache, seq_lens_out=out)
        assert b.lens.cpu().tolist() == [5, 9] and out.cpu().tolist() == [6, 10]
        assert before is None or torch.equal(before, b.cache)
        before = b.cache.clone()


def test_rows_that_cannot_take_their_tokens_keep_their_length():
    b = Batch([32, 32, 32, 32], seed=11, fill=0)
    b.grow([30, 4, 6, 8])
    b.table[1, 0] = b.num_pages + 5
    b.bt.copy_(dev(b.table))
    bad = [len(b.table[0]) * 16 - 30 + 1, 2, 3, 0]  # no room; a bad page
    k = [b.normal(n) for n in bad]
    keep = b.cache.clone()
    off = dev(np.concatenate([[0], np.cumsum(bad)]).astype(np.int32))
    x = dev(np.concatenate(k))
    api.pkv_quant_append(b.shape, b.ws, x, x, b.bt, b.lens, b.cache, new_offsets=off)
    assert b.lens.cpu().tolist() == [30, 4, 9, 8]
    st, msg = api.pkv_get_error(b.ws)
    assert st == _lib.PKV_EDEVICE and ("row 0" in msg or "row 1" in msg), msg
    b.ok()
    page = int(b.table[2, 0])
    same = torch.ones(b.num_pages, dtype=torch.bool)
    same[page] = False
    assert torch.equal(b.cache[same.cuda()], keep[same.cuda()])
    # offsets that run backwards or out of the buffer, a negative length
    lens = b.lens.clone()
    api.pkv_quant_append(b.shape, b.ws, x, x, b.bt, lens, b.cache,
                         new_offsets=dev(np.array([0, 2, 1, 1, x.shape[0] + 9], np.int32)))
    assert lens.cpu().tolist() == [30, 4, 9, 8]
    assert "packed" in api.pkv_get_error(b.ws)[1]
    lens[2] = -3
    api.pkv_quant_append(b.shape, b.ws, x[:4], x[:4], b.bt, lens, b.cache)
    assert int(lens[2]) == -3
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    b.ok()


def test_read_outside_a_row_is_zeros_and_an_error():
    b = Batch([32, 32], seed=12)
    b.grow([10, 20])
    b.table[1, 1] = -1
    b.bt.copy_(dev(b.table))
    k, v = b.read(first=[8, 14], counts=[4, 4])
    assert (k[2:4] == 0).all() and (v[2:4] == 0).all() and (k[6:8] == 0).all() and (v[6:8] == 0).all()
    assert np.array_equal(bits(k[:2]), bits(R.values(b.k[0][8:10])))
    assert np.array_equal(bits(v[4:6]), bits(R.values(b.v[1][14:16])))
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    b.ok()


def test_read_into_strided_outputs():
    b = Batch([50], Hkv=2, d=64, P=16, seed=13)
    b.grow([50])
    buf = torch.full((50, 2 * 2 * 64 + 8), 3.0, dtype=torch.float16, device="cuda")
    ko, vo = (buf[:, a:a + 128].unflatten(1, (2, 64)) for a in (0, 128))
    api.pkv_quant_read(b.shape, b.ws, b.cache, b.bt, b.lens, dev(np.array([0, 50], np.int32)), ko, vo)
    assert np.array_equal(bits(ko.cpu().numpy()), bits(R.values(b.k[0])))
    assert np.array_equal(bits(vo.cpu().numpy()), bits(R.values(b.v[0])))
    assert (buf[:, 256:] == 3.0).all()


# ------------------------------------------------------------------ decode over the 4-bit cache

LENS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 200, 513]


@pytest.mark.parametrize("d,P,Hkv,G", [(128, 16, 2, 4), (64, 8, 3, 5), (128, 64, 1, 8), (64, 256, 2, 1), (128, 8, 8, 2),
                                       (64, 16, 1, 7), (128, 128, 2, 3), (64, 32, 4, 6)])
def test_quant_decode_rows_of_every_length(d, P, Hkv, G):
    b = Batch(LENS, Hkv=Hkv, G=G, d=d, P=P, seed=P + G)
    b.grow(LENS)
    b.check(queries(b))


def widen(b, columns=4096):
    """A wide block table, whose further entries are no pages: rows could be long, so the work is cut into runs
    instead of going to clusters."""
    more = torch.full((b.B, columns), -7, dtype=torch.int32, device="cuda")
    b.bt = torch.cat([b.bt, more], 1).contiguous()
    b.shape.bt_stride += columns
    return b


@pytest.mark.parametrize("d,P,Hkv,G", [(128, 16, 2, 4), (64, 8, 3, 5), (128, 64, 1, 8), (64, 256, 2, 1), (128, 8, 8, 2),
                                       (64, 16, 1, 7), (128, 128, 2, 3), (64, 32, 4, 6)])
def test_quant_decode_over_a_wide_table(d, P, Hkv, G):
    b = widen(Batch(LENS, Hkv=Hkv, G=G, d=d, P=P, seed=P + G))
    b.grow(LENS)
    q = queries(b)
    b.check(q)
    b.check(q, 10 ** 6, 0)
    b.check(q, 2 ** 31 - 1, 2 ** 31 - 1)


@pytest.mark.parametrize("lens", [[4097], [8000, 1, 0, 129], [1500] * 9, [64] * 40 + [3000], [0, 0, 5000], [0] * 70 + [300]])
def test_quant_decode_long_rows_over_a_wide_table(lens):
    b = widen(Batch(lens, Hkv=2, G=8, d=128, P=32, seed=22))
    b.grow(lens)
    b.check(queries(b))


@pytest.mark.parametrize("d,P,G", [(128, 16, 1), (64, 64, 3)])
def test_many_rows(d, P, G):
    """More (row, head) pairs than CTAs: runs of whole rows, and rows that see nothing among them."""
    lens = LENS * 4
    b = Batch(lens, Hkv=8, G=G, d=d, P=P, seed=51)
    b.grow(lens)
    f = Pages(lens, Hkv=8, G=G, d=d, P=P, seed=52)
    q = queries(b)
    b.check(q)
    for window, sinks in ((0, 0), (0, 3), (16, 4), (100, 64), (1000, 0)):
        b.check(q, window, sinks)
        f.check(window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (5, 0), (16, 4), (64, 1), (63, 17), (100, 64), (130, 70),
                                          (10 ** 6, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)])
@pytest.mark.parametrize("d,P", [(128, 16), (64, 64), (64, 8)])
def test_quant_decode_in_a_window(window, sinks, d, P):
    b = Batch(LENS, Hkv=2, G=4, d=d, P=P, seed=21)
    b.grow(LENS)
    b.check(queries(b), window, sinks)


@pytest.mark.parametrize("lens", [[4097], [8000, 1, 0, 129], [1500] * 9, [64] * 40 + [3000]])
def test_quant_decode_long_rows(lens):
    b = Batch(lens, Hkv=2, G=8, d=128, P=32, seed=22)
    b.grow(lens)
    b.check(queries(b))
    b.check(queries(b), 777, 5)


def test_quant_decode_of_large_and_tiny_values():
    """Score ranges that move the running maximum a long way, and V far from 1."""
    for ks, vs, qs in ((8.0, 1e-4, 4.0), (0.01, 3000.0, 0.01), (30.0, 1.0, 30.0)):
        b = Batch([300, 40], Hkv=1, G=4, d=128, P=16, seed=23)
        b.append([b.normal(n, ks) for n in (300, 40)], [b.normal(n, vs) for n in (300, 40)])
        b.check(queries(b, scale=qs))


def test_quant_decode_scores_that_rise_along_the_row():
    b = Batch([640], Hkv=1, G=2, d=64, P=16, seed=24)
    k = b.normal(640)
    q = queries(b)
    k[:, 0] += (np.arange(640)[:, None] / 200.0 * q[0, 0].cpu().numpy()).astype(np.float16)
    b.append([k], [b.normal(640)])
    b.check(q)


def test_a_nan_in_the_row_reaches_only_its_own_row_and_head():
    b = Batch([100, 100], Hkv=2, G=2, d=64, P=16, seed=25)
    k, v = [b.normal(100), b.normal(100)], [b.normal(100), b.normal(100)]
    v[0][3, 1, 5] = np.nan
    b.append(k, v)
    o, _ = b.decode(queries(b))
    x = torch.isnan(o).cpu().numpy()
    assert x[0, 2:, :32].all() and not x[0, :2].any() and not x[0, 2:, 32:].any() and not x[1].any()
    o, _ = b.decode(queries(b), 96, 3)  # token 3 is masked out
    assert not torch.isnan(o).any()
    b.ok()


def test_quant_decode_reports_bad_pages_and_lengths():
    b = Batch([40, 40, 40], seed=26)
    b.grow([40, 40, 40])
    q = queries(b)
    b.table[1, 1] = 9999
    b.bt.copy_(dev(b.table))
    b.decode(q)
    st, msg = api.pkv_get_error(b.ws)
    assert st == _lib.PKV_EDEVICE and "row 1" in msg
    o, lse = b.decode(q, 4, 4)  # the bad page lies between the sinks and the window
    ks, vs = ([R.values(x) for x in y] for y in (b.k, b.v))
    compare(o, lse, q, ks, vs, b.shape.scale, 4, 4)
    b.ok()
    b.lens[0] = -1
    o, lse = b.decode(q, 4, 4)
    assert (o[0] == 0).all() and (lse[0] == -float("inf")).all()
    assert "negative" in api.pkv_get_error(b.ws)[1]
    b.lens[0] = 10 ** 6
    b.decode(q)
    assert api.pkv_get_error(b.ws)[0] == _lib.PKV_EDEVICE
    b.ok()


def test_pages_beyond_32_bit_offsets():
    """Pages past 4 GiB of the 4-bit cache and past 8 GiB of the fp16 pages."""
    Hkv, d, P = 8, 128, 256
    pages = (1 << 32) // (Hkv * P * d * 5 // 4) + 40
    b = Batch([600], Hkv=Hkv, G=1, d=d, P=P, seed=27)
    b.cache = torch.empty((pages, Hkv, P * d * 5 // 4), dtype=torch.uint8, device="cuda")
    b.table[0, :3] = [pages - 1, pages - 7, pages - 2]
    b.bt.copy_(dev(b.table))
    b.shape.num_pages = pages
    b.grow([600])
    b.check(queries(b))
    k, v = b.read()
    assert np.array_equal(bits(k), bits(R.values(b.k[0])))
    assert np.array_equal(bits(v), bits(R.values(b.v[0])))


def test_append_decode_loop_captured_as_a_graph():
    """The serving step -- append a token, decode -- captured once and replayed, on a stream of its own,
    beside eager steps on the same buffers."""
    b = Batch([90, 60, 75], Hkv=2, G=4, d=128, P=16, seed=28)
    b.grow([40, 0, 25])
    kn, vn = (torch.zeros((3, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros((3, 8, 128), dtype=torch.float16, device="cuda")
    o = torch.zeros_like(q)
    lse = torch.zeros((3, 8), dtype=torch.float32, device="cuda")

    def step():
        api.pkv_quant_append(b.shape, b.ws, kn, vn, b.bt, b.lens, b.cache)
        api.pkv_quant_decode(b.shape, b.ws, q, b.cache, b.bt, b.lens, o, lse, window=30, sinks=2)

    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    for t in range(6):
        k, v = b.normal(3), b.normal(3)
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
            b.k[i] = np.concatenate([b.k[i], k[i:i + 1]])
            b.v[i] = np.concatenate([b.v[i], v[i:i + 1]])
        compare(o, lse, q, [R.values(x) for x in b.k], [R.values(x) for x in b.v], b.shape.scale, 30, 2)
    assert b.lens.cpu().tolist() == [46, 6, 31]
    b.ok()


def test_the_same_call_gives_the_same_bits():
    b = Batch([3000, 10, 700], Hkv=4, G=8, d=128, P=16, seed=29)
    b.grow([3000, 10, 700])
    q = queries(b)
    first = b.decode(q)
    for _ in range(5):
        again = b.decode(q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def repeated(B, Hkv, G, d, P, distinct, times, seed):
    """A batch whose rows repeat `distinct` pages `times` times over: long rows over a small cache."""
    b = Batch([distinct * P] * B, Hkv=Hkv, G=G, d=d, P=P, seed=seed)
    b.grow([distinct * P] * B)
    b.bt = b.bt.repeat(1, times).contiguous()
    b.shape.bt_stride = distinct * times
    b.lens = b.lens * times
    return b


def test_quant_decode_of_runs_that_are_split():
    """Runs long enough that their ends are claimed by whichever CTA is free (more than 48 tiles a CTA): every
    row repeats its pages 64 times, so o is that of one repetition and lse larger by ln 64."""
    times = 64
    b = repeated(8, 8, 8, 128, 64, 16, times, seed=41)
    b.lens[3] = 0
    b.lens[5] = b.lens[5] // times
    q = queries(b)
    first = b.decode(q)
    for _ in range(4):
        again = b.decode(q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ks, vs = ([R.values(x) for x in y] for y in (b.k, b.v))
    ks[3], vs[3] = ks[3][:0], vs[3][:0]
    ro, rl, to, tl = R.attention(q.cpu().numpy(), ks, vs, float(np.float32(b.shape.scale)))
    rl[[0, 1, 2, 4, 6, 7]] += np.log(times)
    x, y = first[0].cpu().numpy().astype(np.float64), first[1].cpu().numpy().astype(np.float64)
    # a repetition adds to the weights' roundings below 2^-14 only: 64 times the term for those
    extra = 2.0 ** -25 * 1024 * times * max(np.abs(v).max() for v in vs if v.size)
    assert (np.abs(x - ro) <= to + extra).all()
    assert (y[3] == -np.inf).all()
    rows = [i for i in range(8) if i != 3]
    # fp32 sums of 65536 weights: 2^-24 times the depth of the sums (tiles per warp and merges, some 2^12)
    assert (np.abs(y[rows] - rl[rows]) <= tl[rows] + 2.0 ** -12).all()
    b.ok()


def test_a_wait_that_runs_out_is_reported():
    """The bounded wait: CTA 0's first stage is left unfilled, the consumers give up after a second, the error
    is reported and the next launch is right."""
    for make in (lambda: Batch([400, 30], seed=42), lambda: Batch([400], d=64, seed=43)):
        b = make()
        b.grow([len_ for len_ in ([400, 30] if b.B == 2 else [400])])
        q = queries(b)
        b.check(q)
        assert _lib.load().pkv_test_starve_next_decodes(1) == 0
        b.decode(q)
        assert api.pkv_get_error(b.ws)[0] == _lib.PKV_ETIMEOUT
        b.ws.zero_()  # the counters of a launch that gave up
        b.check(q)


def test_binding_refuses_wrong_tensors():
    b = Batch([40, 40], seed=44)
    b.grow([20, 20])
    q = queries(b)
    o = torch.empty_like(q)
    good = dict(shape=b.shape, ws=b.ws, q=q, quant_cache=b.cache, block_table=b.bt, seq_lens=b.lens, o=o)
    for bad, kind in ((dict(q=q.float()), ValueError), (dict(q=q[:1]), ValueError), (dict(q=q.transpose(0, 1)), ValueError),
                      (dict(q=q.cpu()), ValueError), (dict(q=None), TypeError), (dict(ws=b.ws[:100]), ValueError),
                      (dict(ws=None), TypeError), (dict(quant_cache=b.cache[1:]), ValueError),
                      (dict(block_table=b.bt.long()), ValueError), (dict(block_table=b.bt[:1]), ValueError),
                      (dict(seq_lens=b.lens[:1]), ValueError), (dict(o=o.float()), ValueError),
                      (dict(lse=torch.empty(2, 8, dtype=torch.float16, device="cuda")), ValueError),
                      (dict(window=2 ** 31), ValueError), (dict(window="4"), TypeError), (dict(shape=3), TypeError),
                      (dict(window=-1), _lib.PkvError), (dict(sinks=1), ValueError)):
        with pytest.raises(kind):
            api.pkv_quant_decode(**{**good, **bad})
    x = torch.zeros(2, 2, 128, dtype=torch.float16, device="cuda")
    wide = torch.zeros(2, 2, 256, dtype=torch.float16, device="cuda")
    for k, v in ((x.float(), x), (x, x[:1]), (x[:, :1], x[:, :1]), (x, wide[:, :, :128]), (wide[:, :, ::2], wide[:, :, ::2]),
                 (x.cpu(), x.cpu()), (x[0], x[0])):
        with pytest.raises(ValueError):
            api.pkv_quant_append(b.shape, b.ws, k, v, b.bt, b.lens, b.cache)
    with pytest.raises(_lib.PkvError):  # three tokens for two rows
        y = torch.zeros(3, 2, 128, dtype=torch.float16, device="cuda")
        api.pkv_quant_append(b.shape, b.ws, y, y, b.bt, b.lens, b.cache)
    b.ok()


def test_decoder_object_runs_the_new_steps():
    """PagedDecoder: append, then decode over the 4-bit cache and over fp16 pages in a window, with its own
    workspaces."""
    dec = api.PagedDecoder()
    b = Batch([60, 33], Hkv=2, G=4, d=64, P=8, seed=45)
    k, v = [b.normal(50), b.normal(20)], [b.normal(50), b.normal(20)]
    off = dev(np.array([0, 50, 70], np.int32))
    dec.append_quant(dev(np.concatenate(k)), dev(np.concatenate(v)), b.cache, b.bt, b.lens, off)
    k1, v1 = b.normal(2), b.normal(2)
    dec.append_quant(dev(k1), dev(v1), b.cache, b.bt, b.lens)
    ks = [R.values(np.concatenate([k[i], k1[i:i + 1]])) for i in range(2)]
    vs = [R.values(np.concatenate([v[i], v1[i:i + 1]])) for i in range(2)]
    q = queries(b)
    o, lse = dec.step_quant(q, b.cache, b.bt, b.lens)
    compare(o, lse, q, ks, vs, b.shape.scale, None, 0)
    o, lse = dec.step_quant(q, b.cache, b.bt, b.lens, window=9, sinks=2)
    compare(o, lse, q, ks, vs, b.shape.scale, 9, 2)
    f = Pages([70, 5], Hkv=2, G=4, d=64, P=8, seed=46)
    o, lse = dec.step_window(f.q, f.kc, f.vc, f.bt, f.lens, 30, 3)
    compare(o, lse, f.q, f.k, f.v, f.shape.scale, 30, 3)
    o, lse = dec.step_window(f.q, f.kc, f.vc, f.bt, f.lens, 30, 3, want_lse=False)
    assert lse is None


# ------------------------------------------------------------------ the window over fp16 pages

class Pages:
    """fp16 pages: what no token was written to holds NaN."""

    def __init__(self, lens, Hkv=2, G=4, d=128, P=16, seed=0, spare=3, scale=None):
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.Hq, self.d = len(lens), Hkv, Hkv * G, d
        pages = [-(-n // P) for n in lens]
        num = max(1, sum(pages)) + spare
        order = rng.permutation(num)
        self.table = np.full((self.B, max(1, max(pages))), order[-1], np.int32)
        kc = np.full((num, P, Hkv, d), np.nan, np.float16)
        vc = np.full((num, P, Hkv, d), np.nan, np.float16)
        self.k, self.v, at = [], [], 0
        for i, n in enumerate(lens):
            self.table[i, :pages[i]] = order[at:at + pages[i]]
            at += pages[i]
            for store, cache in ((self.k, kc), (self.v, vc)):
                x = rng.standard_normal((n, Hkv, d)).astype(np.float16)
                t = np.arange(n)
                cache[self.table[i, t // P], t % P] = x
                store.append(x.astype(np.float64))
        self.kc, self.vc, self.bt = dev(kc), dev(vc), dev(self.table)
        self.lens = dev(np.asarray(lens, np.int32))
        self.q = dev(rng.standard_normal((self.B, self.Hq, d)).astype(np.float16))
        self.shape = api.make_shape(self.q, self.kc, self.bt, scale)
        self.ws = torch.zeros(api.pkv_attn_workspace_size(self.shape), dtype=torch.uint8, device="cuda")

    def decode(self, window, sinks):
        o = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
        api.pkv_window_decode(self.shape, self.ws, self.q, self.kc, self.vc, self.bt, self.lens, window, sinks, o, lse)
        return o, lse

    def check(self, window, sinks):
        o, lse = self.decode(window, sinks)
        compare(o, lse, self.q, self.k, self.v, self.shape.scale, window, sinks)
        assert api.pkv_get_error(self.ws)[0] == 0
        clean(self.ws)


@pytest.mark.parametrize("d,P,Hkv,G", [(128, 16, 2, 4), (64, 8, 3, 5), (128, 64, 1, 8), (64, 256, 2, 1), (128, 128, 8, 2),
                                       (64, 32, 1, 7)])
def test_window_decode_rows_of_every_length(d, P, Hkv, G):
    b = Pages(LENS, Hkv=Hkv, G=G, d=d, P=P, seed=P + G)
    for window, sinks in ((0, 0), (0, 3), (1, 0), (16, 4), (63, 17), (100, 64), (130, 70), (10 ** 6, 0),
                          (2 ** 31 - 1, 2 ** 31 - 1)):
        b.check(window, sinks)


@pytest.mark.parametrize("lens", [[4097], [8000, 1, 0, 129], [64] * 40 + [3000]])
def test_window_decode_long_rows(lens):
    b = Pages(lens, Hkv=2, G=8, d=128, P=16, seed=31)
    for window, sinks in ((4096, 4), (2000, 100), (1, 1), (65, 0)):
        b.check(window, sinks)


def test_window_that_holds_the_row_equals_the_full_decode():
    b = Pages([700, 3, 90], seed=32)
    o, lse = b.decode(1000, 0)
    full = api.PagedDecoder().step(b.q, b.kc, b.vc, b.bt, b.lens, 700)
    # both round o once and each weight once: at most a step of o and 2^-10 of the weighted |v| apart
    assert (o.float() - full[0].float()).abs().max() <= 2.0 ** -10 * 8
    assert (lse - full[1]).abs().max() <= 1e-5


def test_masked_tokens_hold_anything():
    """NaN and infinities in tokens outside the window, on pages that are read and on pages that are not."""
    b = Pages([500, 90], P=32, seed=33)
    want = b.decode(100, 10)
    for i, n in enumerate((500, 90)):
        for t in range(n):
            if 10 <= t < n - 100:
                page, slot = int(b.table[i, t // 32]), t % 32
                b.kc[page, slot] = float("nan") if t % 2 else float("inf")
                b.vc[page, slot] = float("inf") if t % 3 else float("nan")
    got = b.decode(100, 10)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_bad_pages_outside_the_window_are_not_read():
    b = Pages([300], P=16, seed=34)
    want = b.decode(40, 20)
    b.bt[0, 3:16] = 10 ** 8  # between the sinks and the window
    got = b.decode(40, 20)
    assert torch.equal(want[0], got[0])
    assert api.pkv_get_error(b.ws)[0] == 0
    b.bt[0, 17] = -4
    b.decode(40, 20)
    st, msg = api.pkv_get_error(b.ws)
    assert st == _lib.PKV_EDEVICE and "row 0" in msg


def test_lse_may_be_left_out():
    b = Pages([70], seed=35)
    o, _ = b.decode(30, 4)
    o2 = torch.zeros_like(o)
    api.pkv_window_decode(b.shape, b.ws, b.q, b.kc, b.vc, b.bt, b.lens, 30, 4, o2)
    assert torch.equal(o, o2)


def test_calls_on_two_streams_with_a_workspace_each():
    b = Pages([2000, 50], G=8, seed=36)
    want = b.decode(1500, 4)
    torch.cuda.synchronize()
    ws = [torch.zeros_like(b.ws) for _ in range(2)]
    out = [torch.zeros_like(want[0]) for _ in range(2)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for w, o, s in zip(ws, out, st):
            api.pkv_window_decode(b.shape, w, b.q, b.kc, b.vc, b.bt, b.lens, 1500, 4, o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[0])


def test_window_decode_of_runs_that_are_split():
    """As for the 4-bit cache: rows that repeat their pages, all of them inside the window."""
    times = 64
    b = Pages([1024] * 8, Hkv=8, G=4, d=64, P=64, seed=47)
    b.bt = b.bt.repeat(1, times).contiguous()
    b.shape.bt_stride *= times
    b.lens = b.lens * times
    o, lse = b.decode(1 << 30, 0)
    again = b.decode(1 << 30, 0)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    ro, rl, to, tl = R.attention(b.q.cpu().numpy(), b.k, b.v, float(np.float32(b.shape.scale)))
    extra = 2.0 ** -25 * 1024 * times * max(np.abs(v).max() for v in b.v)
    assert (np.abs(o.cpu().numpy().astype(np.float64) - ro) <= to + extra).all()
    assert (np.abs(lse.cpu().numpy().astype(np.float64) - np.log(times) - rl) <= tl + 2.0 ** -12).all()
    assert api.pkv_get_error(b.ws)[0] == 0
    clean(b.ws)


@pytest.mark.parametrize("d,P,Hkv,G", [(128, 16, 2, 4), (64, 8, 3, 5), (128, 64, 1, 8), (64, 256, 2, 1), (128, 128, 8, 2)])
def test_window_decode_over_a_wide_table(d, P, Hkv, G):
    b = widen(Pages(LENS, Hkv=Hkv, G=G, d=d, P=P, seed=P + G))
    for window, sinks in ((10 ** 6, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 10 ** 6)):
        b.check(window, sinks)


@pytest.mark.parametrize("lens", [[4097], [8000, 1, 0, 129], [64] * 40 + [3000]])
def test_window_decode_long_rows_over_a_wide_table(lens):
    b = widen(Pages(lens, Hkv=2, G=8, d=128, P=16, seed=31))
    for window, sinks in ((10 ** 6, 4), (20000, 100)):
        b.check(window, sinks)


@pytest.mark.parametrize("P", [8, 32, 128])
def test_windows_over_a_wide_table(P):
    """Windows and sinks that end inside a tile and at its ends, over rows around a tile's length (256, d = 64)."""
    lens = [255, 256, 257, 384, 511, 512, 513, 700, 0, 1]
    b = widen(Batch(lens, Hkv=2, G=4, d=64, P=P, seed=73))
    b.grow(lens)
    for window, sinks in ((None, 0), (255, 1), (256, 0), (257, 129), (64, 64), (1, 300), (0, 256)):
        b.check(queries(b), window, sinks)


@pytest.mark.parametrize("lens,Hkv,G,d", [([20000], 1, 8, 128), ([9000, 5], 1, 4, 64), ([16500, 0, 3000], 1, 5, 128)])
def test_rows_of_so_many_pieces_that_groups_are_merged_first(lens, Hkv, G, d):
    for b, window, sinks in ((widen(Batch(lens, Hkv=Hkv, G=G, d=d, P=64, seed=71)), None, 0),
                             (widen(Pages(lens, Hkv=Hkv, G=G, d=d, P=64, seed=72)), 10 ** 6, 3)):
        if isinstance(b, Batch):
            b.grow(lens)
            b.q = queries(b)
            b.check(b.q, window, sinks)
            first, again = b.decode(b.q), b.decode(b.q)
        else:
            b.check(window, sinks)
            first, again = b.decode(window, sinks), b.decode(window, sinks)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------ calls at the edges

def test_one_workspace_serves_batches_of_any_size():
    """Long rows whose states are split, then many rows, then an append that meets a bad page, over one workspace."""
    few = widen(Batch([5000, 700], Hkv=2, G=4, d=64, P=16, seed=61))
    many = Batch([300], Hkv=2, G=4, d=64, P=16, seed=62)
    B = 2000
    few.grow([5000, 700])
    many.grow([300])
    many.bt = many.bt.repeat(B, 1).contiguous()  # rows may share pages that are only read
    many.lens = many.lens.repeat(B)
    many.shape.B = B
    ws = few.ws  # made for the small batch
    q = dev(np.random.default_rng(63).standard_normal((1, many.Hq, 64)).astype(np.float16)).repeat(B, 1, 1)
    ref = few.decode(queries(few))

    def decode_many():
        o = torch.full_like(q, float("nan"))
        api.pkv_quant_decode(many.shape, ws, q, many.cache, many.bt, many.lens, o)
        return o

    for _ in range(2):
        got = few.decode(queries(few))
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
        o = decode_many()
        ro, _, to, _ = R.attention(q[:1].cpu().numpy(), [R.values(many.k[0])], [R.values(many.v[0])],
                                   float(np.float32(many.shape.scale)))
        assert (np.abs(o.cpu().numpy().astype(np.float64) - ro) <= to).all()
    # 2000 rows of one new token each, of which one names a bad page
    lone = Batch([3] * B, Hkv=2, G=4, d=64, P=8, seed=64)
    lone.bt[77, 0] = -1
    off = dev(np.arange(B + 1, dtype=np.int32))
    x = dev(np.random.default_rng(65).standard_normal((B, 2, 64)).astype(np.float16))
    api.pkv_quant_append(lone.shape, ws, x, x, lone.bt, lone.lens, lone.cache, new_offsets=off)
    assert lone.lens.cpu().tolist() == [0 if i == 77 else 1 for i in range(B)]
    st, msg = api.pkv_get_error(ws)
    assert st == _lib.PKV_EDEVICE and "row 77" in msg
    clean(ws)


@pytest.mark.parametrize("rows", [1, 300])  # a cluster's merge and a CTA's own rounding
def test_a_mean_of_the_greatest_values_stays_finite(rows):
    """Weights 1 and 128 (1 + 9/16 2^-10), of which fp16 holds the second as 128 (1 + 2^-10): over their sum
    before rounding, values at the type's end come out 2^-11.2 beyond it."""
    n = 600
    b = Pages([n], Hkv=1, G=1, d=64, P=16, seed=66)
    b.shape.scale = float(np.log(128 * (1 + 0.5625 / 1024)))
    b.kc.fill_(0)
    b.vc.fill_(65504.0)
    b.kc[..., 0] = -100.0
    b.q = torch.zeros_like(b.q)
    b.q[..., 0] = 1.0
    for t, x in ((0, 0.0), (256, 1.0)):  # the same warp's: tiles of 128 tokens
        b.kc[int(b.bt[0, t // 16]), t % 16, 0, 0] = x
    b.bt, b.lens, b.q = b.bt.repeat(rows, 1).contiguous(), b.lens.repeat(rows), b.q.repeat(rows, 1, 1).contiguous()
    b.shape.B = rows
    o, _ = b.decode(10 ** 6, 0)
    assert (o == 65504.0).all()
    b.vc.fill_(-65504.0)
    o, _ = b.decode(10 ** 6, 0)
    assert (o == -65504.0).all()
    b.vc.fill_(float("inf"))  # an infinite value stays one
    o, _ = b.decode(10 ** 6, 0)
    assert not torch.isfinite(o).any()


@pytest.mark.parametrize("wide", [False, True])
def test_scores_of_any_size_have_a_greatest(wide):
    """Equal scores of -1e32: their mean, not a row without a maximum."""
    b = Pages([200, 1], Hkv=1, G=2, d=64, P=16, seed=67)
    if wide:
        b = widen(b)
    b.shape.scale = -1e32
    b.kc.fill_(0)
    b.kc[..., 3] = 1.0
    b.q = torch.zeros_like(b.q)
    b.q[..., 3] = 1.0
    o, lse = b.decode(10 ** 6, 0)
    for i in range(2):
        # one rounding of the mean and fp32 sums of 200 terms of at most 8
        assert np.abs(o[i].cpu().numpy().astype(np.float64) - b.v[i].mean(0)).max() <= 2.0 ** -11 * 8 + 200 * 8 * 2.0 ** -24
        assert (lse[i] / -1e32 - 1).abs().max() <= 1e-6


def test_a_decoder_makes_its_workspace_before_a_capture():
    b = Batch([60, 33], Hkv=2, G=4, d=64, P=8, seed=68)
    b.grow([50, 20])
    dec, q = api.PagedDecoder(), queries(b)
    o = torch.zeros_like(q)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="before capturing"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            dec.step_quant(q, b.cache, b.bt, b.lens, o=o, want_lse=False)
    want, _ = dec.step_quant(q, b.cache, b.bt, b.lens, want_lse=False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.step_quant(q, b.cache, b.bt, b.lens, o=o, want_lse=False)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
