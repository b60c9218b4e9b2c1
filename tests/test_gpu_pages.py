"""The page map and the slot append on the GPU against plain models, and runs of
them with the fp16 and 8-bit caches as a serving loop has them."""
import numpy as np
import pytest
import torch

import byte_ref as R
import oracle
from gpu_util import close, close_lse, dev
from paged_kv_gqa_09_gb300 import _lib, api

pytestmark = pytest.mark.gpu


class Map:
    """Rows with pages of their own, a free list of what is left, and the map's outputs."""

    def __init__(self, lens, P, stride, free, seed=0, num_pages=None, count=None):
        self.rng = np.random.default_rng(seed)
        self.P, self.B, self.lens = P, len(lens), list(lens)
        have = [max(0, -(-n // P)) if n <= stride * P else stride for n in lens]
        self.num_pages = sum(have) + max(free, 1) if num_pages is None else num_pages
        order = self.rng.permutation(self.num_pages)
        self.table = np.full((self.B, stride), -99, np.int32)
        at = 0
        for i, n in enumerate(have):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.free = order[at:at + free].astype(np.int32)
        self.count = len(self.free) if count is None else count
        self.shape = _lib.Shape(self.B, 1, 1, 128, P, self.num_pages, stride, 1.0)
        self.ws = torch.zeros(api.pkv_attn_workspace_size(self.shape), dtype=torch.uint8, device="cuda")
        self.bt, self.sl = dev(self.table), dev(np.asarray(lens, np.int32))
        self.fp, self.fc = dev(self.free), dev(np.array([self.count], np.int32))

    def run(self, new, T, in_place=False, positions=True, stream=None):
        self.slots = torch.full((T,), -77, dtype=torch.int64, device="cuda")
        self.pos = torch.full((T,), -77, dtype=torch.int32, device="cuda") if positions else None
        self.off = torch.full((self.B + 1,), -77, dtype=torch.int32, device="cuda")
        out = None if in_place else torch.full_like(self.sl, -77)
        fout = None if in_place else torch.full_like(self.fc, -77)
        api.pkv_map_pages(self.shape, self.ws, self.sl, dev(np.asarray(new, np.int32)), self.bt, self.fp, self.fc, self.slots,
                          self.off, seq_lens_out=out, free_count_out=fout, positions=self.pos, stream=stream)
        return (self.sl, self.fc) if in_place else (out, fout)

    def check(self, new, T=None, error=False, **kw):
        T = int(sum(max(0, n) for n in new)) if T is None else T
        want = R.map_pages(self.lens, new, self.table.tolist(), self.free.tolist(), self.count, self.P, self.num_pages, T)
        out, fout = self.run(new, T, **kw)
        assert self.off.tolist() == want[3]
        assert self.slots.tolist() == want[1]
        assert self.pos is None or self.pos.tolist() == want[2]
        assert out.tolist() == want[4] and fout.tolist() == [want[5]]
        assert self.bt.cpu().numpy().tolist() == want[0]
        st, msg = api.pkv_get_error(self.ws)
        assert (st == _lib.PKV_EDEVICE) == error, msg
        assert int(self.ws[16:64].view(torch.int32).abs().sum()) == 0
        return msg


@pytest.mark.parametrize("P", [8, 16, 256])
@pytest.mark.parametrize("B,most", [(1, 1), (1, 5000), (7, 60), (64, 1), (300, 40), (1023, 1), (1024, 9), (1025, 3), (2500, 1), (3000, 30)])
def test_tokens_get_their_slots(P, B, most):
    rng = np.random.default_rng(B + P)
    lens = rng.integers(0, 3 * P, B)
    new = rng.integers(0 if most > 1 else 1, most + 1, B)
    need = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(lens.tolist(), new.tolist()))
    m = Map(lens.tolist(), P, int(-(-(lens + new).max() // P)) + 2, need + 3, seed=B)
    m.check(new.tolist())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pad", [0, 1, 2, 3, 5, 4000])
def test_a_padded_map(in_place, pad):
    m = Map([5, 0, 16, 31], 16, 8, 20)
    new = [3, 17, 0, 40]
    m.check(new, sum(new) + pad, in_place=in_place, positions=pad != 3)


@pytest.mark.parametrize("new", [[0], [0, 0, 0], [0, 1, 0], [0, 0, 7], [9, 0, 0]])
def test_rows_without_new_tokens(new):
    Map([5, 16, 0][:len(new)], 8, 9, 30).check(new)
    Map([5, 16, 0][:len(new)], 8, 9, 30).check(new, sum(new) + 9, in_place=True)


@pytest.mark.parametrize("B", [6, 1500])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.9, 0.99])
def test_rows_that_find_no_page(B, share):
    """Rows are served in order while pages last; those behind that need none are served too."""
    rng = np.random.default_rng(B)
    lens, new = rng.integers(0, 40, B).tolist(), rng.integers(0, 30, B).tolist()
    need = sum(-(-(a + b) // 16) - -(-a // 16) for a, b in zip(lens, new))
    m = Map(lens, 16, 6, int(need * share), seed=1)
    assert "no free page" in m.check(new, error=True)


def test_rows_that_are_refused():
    """Negative lengths, no room in the table, tokens beyond the packed buffer, counts outside the free list."""
    for lens, new, T, what in (([5, -1, 9], [3, 4, 5], 12, "negative"), ([5, 7, 9], [3, -4, 5], 8, "negative"),
                               ([5, 60, 9], [3, 4, 5], 12, ""), ([5, 61, 9], [3, 4, 5], 12, "beyond"),
                               ([5, 2 ** 31 - 1, 9], [3, 2 ** 31 - 1, 5], 30, "row"),  # of two rows that are refused, either
                               ([5, 7, 9], [3, 40, 5], 20, "outside"), ([5, 7, 9], [3, 4, 5], 0, "outside"),
                               ([5, 7, 9], [3, 4, 5], 10, "outside")):
        for in_place in (False, True):
            m = Map(lens, 16, 4, 12)
            assert what in m.check(new, T, error=what != "", in_place=in_place)  # 60 and 4 just fit
    m = Map([0, 0], 16, 4, 3, count=9)  # a count beyond the list is the list's end
    m.check([16, 30], error=False)
    m = Map([0, 0], 16, 4, 3, count=-2)
    m.check([16, 30], error=True)
    m = Map([0, 8], 16, 4, 0)
    m.check([0, 8])


@pytest.mark.parametrize("B", [4, 1100])
def test_page_ids_out_of_range(B):
    lens = [10, 16, 0, 33] + [1] * (B - 4)
    new = [9, 20, 40, 4000] + [1] * (B - 4)
    for where in ("table", "free"):
        m = Map(lens, 16, 300, 300, seed=2)
        if where == "table":
            m.table[0, 0] = m.num_pages
            m.bt.copy_(dev(m.table))
        else:
            m.free[-3] = -5
            m.free[-40] = m.num_pages
            m.fp.copy_(dev(m.free))
        assert "out of range" in m.check(new, error=True)


@pytest.mark.parametrize("T", [1 << 20])
def test_a_million_tokens(T):
    """Many CTAs: rows that begin and end anywhere within a CTA's share."""
    rng = np.random.default_rng(3)
    cuts = np.sort(rng.choice(T, 299, replace=False))
    new = np.diff(np.concatenate([[0], cuts, [T - 100]])).clip(0)
    lens = rng.integers(0, 200, 300)
    need = int((-(-(lens + new) // 64) - -(-lens // 64)).sum())
    m = Map(lens.tolist(), 64, int(-(-(lens + new).max() // 64)), need, seed=4)
    out, fout = m.run(new.tolist(), T)
    n = int(new.sum())
    row = np.repeat(np.arange(300), new)
    off = np.concatenate([[0], np.cumsum(new)])
    pos = lens[row] + np.arange(n) - off[row]
    table = m.bt.cpu().numpy()
    assert np.array_equal(m.slots.cpu().numpy()[:n], table[row, pos // 64].astype(np.int64) * 64 + pos % 64)
    assert np.array_equal(m.pos.cpu().numpy()[:n], pos) and (m.slots[n:] == -1).all() and (m.pos[n:] == 0).all()
    have = -(-lens // 64)
    pages = np.concatenate([table[i, have[i]:-(-(lens[i] + new[i]) // 64)] for i in range(300)])
    assert np.array_equal(pages, m.free[::-1][:need]) and fout.tolist() == [len(m.free) - need]
    for i in range(300):
        assert np.array_equal(table[i, :have[i]], m.table[i, :have[i]])
    assert np.array_equal(out.cpu().numpy(), lens + new) and np.array_equal(m.off.cpu().numpy(), off)
    assert api.pkv_get_error(m.ws)[0] == 0


# ------------------------------------------------------------------ slots

@pytest.mark.parametrize("Hkv,d,P,T,pad", [(8, 128, 16, 700, 0), (1, 64, 8, 1, 8), (3, 64, 32, 333, 296), (2, 128, 256, 5000, 0),
                                           (5, 128, 64, 77, 1024), (1, 64, 16, 9, 0)])
def test_tokens_go_to_their_slots(Hkv, d, P, T, pad):
    rng = np.random.default_rng(T)
    pages = T // P + 5
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    buf = torch.randn((T, 2 * Hkv * d + pad), device="cuda").half()
    k, v = buf[:, :Hkv * d].unflatten(1, (Hkv, d)), buf[:, Hkv * d:2 * Hkv * d].unflatten(1, (Hkv, d))
    kc, vc = (torch.randn((pages, P, Hkv, d), device="cuda").half() for _ in range(2))
    wk, wv = kc.clone(), vc.clone()
    live = dev(slots) >= 0
    wk.view(-1, Hkv, d)[dev(slots)[live]] = k[live]
    wv.view(-1, Hkv, d)[dev(slots)[live]] = v[live]
    shape = _lib.Shape(1, Hkv, Hkv, d, P, pages, 1, 1.0)
    ws = torch.zeros(api.pkv_attn_workspace_size(shape), dtype=torch.uint8, device="cuda")
    api.pkv_append_slots(shape, ws, k, v, dev(slots), kc, vc)
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    assert api.pkv_get_error(ws)[0] == 0
    bad = slots.copy()
    bad[T // 2] = pages * P
    bad[-1] = 2 ** 40
    api.pkv_append_slots(shape, ws, k, v, dev(bad), kc, vc)  # the same tokens again, but for those
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    st, msg = api.pkv_get_error(ws)
    assert st == _lib.PKV_EDEVICE and "slot" in msg


def test_slots_beyond_32_bit_offsets():
    pages = (1 << 32) // (256 * 8 * 128 * 2) + 9  # past 4 GiB, and past 2^31 elements
    kc, vc = (torch.zeros((pages, 256, 8, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    k, v = (torch.randn((3, 8, 128), device="cuda").half() for _ in range(2))
    slots = torch.tensor([pages * 256 - 1, pages * 256 - 700, 5], device="cuda")
    api.PagedDecoder().append_slots(k, v, slots, kc, vc)
    for got, want in ((kc, k), (vc, v)):
        assert torch.equal(got.view(-1, 8, 128)[slots], want)
        assert int(got.count_nonzero()) == int(want.count_nonzero())


def test_binding_refuses_wrong_tensors():
    m = Map([5, 7], 16, 4, 9)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    good = dict(shape=m.shape, ws=m.ws, seq_lens=m.sl, new_lens=i32(2), block_table=m.bt, free_pages=m.fp, free_count=m.fc,
                slot_map=torch.zeros(4, dtype=torch.int64, device="cuda"), new_offsets=i32(3))
    api.pkv_map_pages(**good)
    for bad in (dict(seq_lens=i32(1)), dict(new_lens=i32(2).long()), dict(new_lens=i32(2).cpu()), dict(block_table=m.bt[:1]),
                dict(free_pages=m.fp.long()), dict(free_count=i32(0)), dict(slot_map=i32(4)), dict(new_offsets=i32(2)),
                dict(seq_lens_out=i32(1)), dict(free_count_out=i32(0)), dict(positions=i32(3)), dict(ws=m.ws[:64]),
                dict(slot_map=torch.zeros(8, dtype=torch.int64, device="cuda")[::2])):
        with pytest.raises(ValueError):
            api.pkv_map_pages(**{**good, **bad})
    x = torch.zeros((4, 1, 128), dtype=torch.float16, device="cuda")
    pool = torch.zeros((m.num_pages, 16, 1, 128), dtype=torch.float16, device="cuda")
    good = dict(shape=m.shape, ws=m.ws, k_new=x, v_new=x, slot_map=torch.full((4,), -1, device="cuda"), k_cache=pool, v_cache=pool)
    api.pkv_append_slots(**good)
    for bad in (dict(k_new=x.float()), dict(v_new=x[:3]), dict(slot_map=good["slot_map"][:3]), dict(slot_map=i32(4)),
                dict(k_cache=pool[1:]), dict(v_cache=pool.float()), dict(k_new=x[:, :, ::2])):
        with pytest.raises(ValueError):
            api.pkv_append_slots(**{**good, **bad})


def test_calls_of_nothing():
    """Empty batches, calls without tokens, an empty free list."""
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    half = lambda *n: torch.zeros(n, dtype=torch.float16, device="cuda")
    i64 = torch.zeros(0, dtype=torch.int64, device="cuda")
    cache, pool, table = api.byte_cache_zeros(4, 16, 2, 64), half(4, 16, 2, 64), i32(0).view(0, 3)
    shape = api.make_byte_shape(8, 64, cache, table)
    assert shape.B == 0
    ws = torch.zeros(api.pkv_attn_workspace_size(shape), dtype=torch.uint8, device="cuda")
    api.pkv_map_pages(shape, ws, i32(0), i32(0), table, i32(0), i32(1), i64, i32(1))
    api.pkv_append_slots(shape, ws, half(0, 2, 64), half(0, 2, 64), i64, pool, pool)
    for fmt in (R.INT8, R.E4M3):
        api.pkv_byte_append(shape, ws, fmt, half(0, 2, 64), half(0, 2, 64), table, i32(0), cache)
        api.pkv_byte_read(shape, ws, fmt, cache, table, i32(0), i32(1), half(0, 2, 64), half(0, 2, 64))
        api.pkv_byte_decode(shape, ws, fmt, half(0, 8, 64), cache, table, i32(0), half(0, 8, 64))
    m = Map([5, 16, 0], 16, 2, 0)  # rows, but no pages and no tokens
    m.free, m.fp = m.free[:0], i32(0)
    m.count, m.fc = 0, i32(1)
    m.check([0, 0, 0])
    m.check([11, 0, 0], 16)  # what fits without a page
    table = dev(np.array([[0, 1, 2], [3, 2, 1]], np.int32))
    shape = api.make_byte_shape(8, 64, cache, table)
    lens = dev(np.array([20, 0], np.int32))
    out = i32(2)
    for fmt in (R.INT8, R.E4M3):
        api.pkv_byte_append(shape, ws, fmt, half(0, 2, 64), half(0, 2, 64), table, lens, cache, new_offsets=i32(3), seq_lens_out=out)
        assert out.tolist() == [20, 0]
    assert int(cache.count_nonzero()) == 0
    assert api.pkv_get_error(ws)[0] == 0


# ------------------------------------------------------------------ as they are used

def serve(kind, steps, captured):
    """Prompts enter an empty cache, then steps of one token per row, each step a map, an append and a decode, the
    last row's pages running out on the way; K and V of every step against the oracle."""
    rng = np.random.default_rng(7)
    P, Hkv, G, d, B = 16, 2, 4, 128, 4
    pages, stride = 24, 12
    prompts = [37, 0, 16, 150]
    dec = api.PagedDecoder()
    fmt = {"int8": R.INT8, "e4m3": R.E4M3}.get(kind)
    if kind == "fp16":
        kc, vc = (torch.full((pages, P, Hkv, d), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    else:
        cache = torch.full((pages, Hkv, R.head_bytes(P, d)), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.full((B, stride), -1, dtype=torch.int32, device="cuda")
    q = torch.zeros((B, Hkv * G, d), dtype=torch.float16, device="cuda")
    shape = api.make_shape(q, torch.empty((pages, P, Hkv, d), dtype=torch.float16, device="cuda"), table)
    free = dev(rng.permutation(pages).astype(np.int32))
    i32 = lambda x: dev(np.asarray(x, np.int32))
    lens, count, off = i32([0] * B), i32([pages]), i32([0] * (B + 1))
    o, lse = torch.zeros_like(q), torch.zeros((B, Hkv * G), dtype=torch.float32, device="cuda")
    held = [[np.zeros((0, Hkv, d), np.float16)] * B for _ in range(2)]
    sides = [[R.Side(fmt, P, Hkv, d) for _ in range(B)] for _ in range(2)] if fmt is not None else None

    def put(new, T, kn, vn, slots, pos, old):
        old.copy_(lens)
        dec.map_pages(shape, lens, new, table, free, count, slots, off, positions=pos)
        if kind == "fp16":
            dec.append_slots(kn, vn, slots, kc, vc)
            dec.step(q, kc, vc, table, lens, stride * P, path=_lib.PKV_PATH_WORKQUEUE, split_tokens=64, o=o, lse=lse)
        else:
            dec.append_byte(fmt, kn, vn, cache, table, old, off, seq_lens_out=old)
            dec.step_byte(fmt, q, cache, table, lens, o=o, lse=lse)

    want = list(prompts)
    have = [0] * B
    graph = torch.cuda.CUDAGraph()
    bufs = None
    for step in range(steps + 1):
        T = sum(prompts) + 5 if step == 0 else B + 3  # padded
        if step <= 1:  # the steps' buffers are made once
            bufs = (i32([0] * B), T, *(torch.zeros((T, Hkv, d), dtype=torch.float16, device="cuda") for _ in range(2)),
                    torch.zeros(T, dtype=torch.int64, device="cuda"), i32([0] * T), i32([0] * B))
        new = prompts if step == 0 else [1] * B
        kn, vn = (rng.standard_normal((T, Hkv, d)).astype(np.float16) for _ in range(2))
        bufs[0].copy_(i32(new))
        bufs[2].copy_(dev(kn))
        bufs[3].copy_(dev(vn))
        q.copy_(dev(rng.standard_normal(q.shape).astype(np.float16)))
        torch.cuda.synchronize()
        if captured and step >= 2:
            if step == 2:
                st = torch.cuda.Stream()
                with torch.cuda.graph(graph, stream=st):
                    put(*bufs)
            graph.replay()
        else:
            put(*bufs)
        torch.cuda.synchronize()
        at, left = 0, pages - sum(-(-n // P) for n in have)
        rank = 0
        for i in range(B):
            need = -(-(have[i] + new[i]) // P) - -(-have[i] // P)
            ok = have[i] + new[i] <= stride * P and (need == 0 or rank + need <= left)
            rank += need
            if ok:
                for u, x in enumerate((kn, vn)):
                    held[u][i] = np.concatenate([held[u][i], x[at:at + new[i]]])
                    if sides:
                        sides[u][i].append(x[at:at + new[i]])
                have[i] += new[i]
            at += new[i]
        assert lens.tolist() == have
        assert bufs[6].tolist() == (have if kind != "fp16" else bufs[6].tolist())
        if kind == "fp16":
            bt = table.cpu().numpy().clip(0)
            pool = [np.zeros((pages, P, Hkv, d), np.float16) for _ in range(2)]
            for u in range(2):
                for i in range(B):
                    for t in range(have[i]):
                        pool[u][bt[i, t // P], t % P] = held[u][i][t]
            ro, rl = oracle.attention(q.cpu().numpy(), pool[0], pool[1], bt, np.asarray(have, np.int32), float(shape.scale))
            close(o, ro)
            close_lse(lse, rl)
        else:
            ro, rl, to, tl = R.attention(q.cpu().numpy(), sides[0], sides[1], float(np.float32(shape.scale)))
            assert (np.abs(o.cpu().numpy().astype(np.float64) - ro) <= to).all()
            fin = np.isfinite(rl)
            got = lse.cpu().numpy().astype(np.float64)
            assert (np.abs(got[fin] - rl[fin]) <= tl[fin]).all() and (got[~fin] == rl[~fin]).all()
    return have, pages - sum(-(-n // P) for n in have)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind", ["fp16", "int8", "e4m3"])
def test_prompts_and_steps_of_a_serving_loop(kind, captured):
    """60 steps: rows reach the end of their pages' row in the table or the free list's end, and stay as they are
    while the others go on."""
    have, left = serve(kind, 60, captured)
    assert max(have) == 192 and sum(have) < sum([37, 0, 16, 150]) + 4 * 60
