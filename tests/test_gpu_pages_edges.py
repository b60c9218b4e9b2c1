"""The page map and the appends after it: rows that the map refuses take no
tokens in either cache."""
import numpy as np
import pytest
import torch

import byte_ref as R
from gpu_util import dev
from paged_kv_gqa_09_gb300 import _lib, api
from test_gpu_pages import Map

pytestmark = pytest.mark.gpu


def append(kind, m, cache, x, lens, off):
    """Packed tokens x into the 4-bit or 8-bit cache by the map's table and offsets; the lengths after it."""
    out = torch.full_like(lens, -7)
    if kind == "4-bit":
        shape = _lib.Shape(m.B, 1, 1, 128, m.P, m.num_pages, m.table.shape[1], 1.0)
        api.pkv_quant_append(shape, m.ws, x, x, m.bt, lens, cache, new_offsets=off, seq_lens_out=out)
    else:
        api.pkv_byte_append(m.shape, m.ws, {"int8": R.INT8, "e4m3": R.E4M3}[kind], x, x, m.bt, lens, cache, new_offsets=off,
                            seq_lens_out=out)
    return out


@pytest.mark.parametrize("kind", ["int8", "e4m3", "4-bit"])
@pytest.mark.parametrize("lens,new,T", [
    ([5, 7, 3, 40], [3, 4, 8, 2], 11),      # row 2's first four tokens would fit behind its three
    ([5, 7, 3, 40], [3, 4, 40, 2], 11),     # and where it would need pages for the rest
    ([5, 60, 9], [3, 9, 4], 5),             # a row too long for its table, whose first two would fit
    ([5, 7, 9], [3, 4, 5], 10), ([3], [8], 4), ([3, 20], [8, 0], 0), ([1, 2, 3], [5, 0, 0], 4),
    ([4] * 700, [3] * 700, 3 * 650 + 2), ([4] * 1300, [1, 2] * 650, 1502)])
def test_rows_that_pass_the_packed_tokens_are_not_appended(kind, lens, new, T):
    stride = 4
    m = Map(lens, 16, stride, 12 + sum(new) // 8)
    out, _ = m.run(new, T)
    want = [a + b if sum(new[:i + 1]) <= T and a + b <= 64 else a for i, (a, b) in enumerate(zip(lens, new))]
    assert out.tolist() == want and api.pkv_get_error(m.ws)[0] == _lib.PKV_EDEVICE
    off = m.off.tolist()
    assert off[0] == 0 and all(0 <= b - a <= n for a, b, n in zip(off, off[1:], new)) and off[-1] <= T
    if kind == "4-bit":
        cache = torch.full((m.num_pages, 1, m.P * 128 * 5 // 4), 0x5A, dtype=torch.uint8, device="cuda")
    else:
        cache = torch.full((m.num_pages, 1, R.head_bytes(16, 128)), 0x5A, dtype=torch.uint8, device="cuda")
    before = cache.clone()
    x = torch.randn((T, 1, 128), device="cuda").half()
    assert append(kind, m, cache, x, m.sl, m.off).tolist() == want
    served = {int(p) for i, n in enumerate(want) if n > lens[i] for p in m.bt[i, :-(-n // 16)].tolist()}
    rest = [p for p in range(m.num_pages) if p not in served]
    assert torch.equal(cache[rest], before[rest])


@pytest.mark.parametrize("kind", ["int8", "e4m3", "4-bit"])
def test_rows_that_find_no_page_are_not_appended(kind):
    """A row whose partly filled page has room for the first of its tokens, and no page for the others."""
    m = Map([3, 20, 5], 16, 4, 2)
    new = [9, 30, 4]  # row 1 needs two pages, after row 0, which needs none
    m.free, m.count = m.free[:1], 1
    m.fp, m.fc = dev(m.free), dev(np.array([1], np.int32))
    out, _ = m.run(new, 43)
    assert out.tolist() == [12, 20, 9]
    assert "no free page" in api.pkv_get_error(m.ws)[1]
    if kind == "4-bit":
        cache = torch.zeros((m.num_pages, 1, m.P * 128 * 5 // 4), dtype=torch.uint8, device="cuda")
    else:
        cache = torch.zeros((m.num_pages, 1, R.head_bytes(16, 128)), dtype=torch.uint8, device="cuda")
    x = torch.randn((43, 1, 128), device="cuda").half()
    assert append(kind, m, cache, x, m.sl, m.off).tolist() == [12, 20, 9]
    if kind != "4-bit":  # whose scales are each token's own: what lies behind a row's end is nobody's
        assert int(cache[m.table[1, :2].tolist()].count_nonzero()) == 0


@pytest.mark.parametrize("T", [0, 5, 4099, 700000])
@pytest.mark.parametrize("positions", [False, True])
def test_a_map_of_no_rows_writes_what_needs_none(T, positions):
    """A padded batch without a request: no slot of an earlier call is left, and no page is taken."""
    i32 = lambda n, x=-77: torch.full((n,), x, dtype=torch.int32, device="cuda")
    table = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    shape = _lib.Shape(0, 1, 1, 128, 16, 9, 3, 1.0)
    ws = torch.zeros(api.pkv_attn_workspace_size(shape), dtype=torch.uint8, device="cuda")
    slots, pos = torch.full((T,), 3, dtype=torch.int64, device="cuda"), i32(T) if positions else None
    off, count, left = i32(1), i32(1, 4), i32(1)
    for out in (left, None):
        api.pkv_map_pages(shape, ws, i32(0), i32(0), table, i32(9, 1), count, slots, off, free_count_out=out, positions=pos)
        assert (slots == -1).all() and (pos is None or (pos == 0).all()) and off.tolist() == [0] and count.tolist() == [4]
    assert left.tolist() == [4] and api.pkv_get_error(ws)[0] == 0
    assert int(ws.view(torch.int32).abs().sum()) == 0


@pytest.mark.parametrize("pages,Hkv", [(2 ** 31 - 1, 2 ** 18), (2 ** 30, 2 ** 17), (2 ** 31 - 1, 2 ** 17)])
def test_caches_whose_size_passes_64_bits_are_refused(pages, Hkv):
    """A shape that names more pages and heads than can be counted is no small cache's."""
    half = lambda *n: torch.zeros(n, dtype=torch.float16, device="cuda")
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    shape = _lib.Shape(1, Hkv, Hkv, 128, 256, pages, 1, 1.0)
    ws = torch.zeros(api.pkv_attn_workspace_size(shape), dtype=torch.uint8, device="cuda")
    q, small, codes, bt, lens = half(1, Hkv, 128), half(1, 256, 1, 128), torch.zeros(70000, dtype=torch.uint8, device="cuda"), i32(1, 1), i32(1)
    slots = torch.full((1,), -1, dtype=torch.int64, device="cuda")
    for call in (lambda: api.pkv_byte_decode(shape, ws, R.INT8, q, codes, bt, lens, torch.empty_like(q)),
                 lambda: api.pkv_byte_append(shape, ws, R.E4M3, q, q, bt, lens, codes),
                 lambda: api.pkv_byte_read(shape, ws, R.E4M3, codes, bt, lens, i32(2), q, q),
                 lambda: api.pkv_quant_decode(shape, ws, q, codes, bt, lens, torch.empty_like(q)),
                 lambda: api.pkv_quant_append(shape, ws, q, q, bt, lens, codes),
                 lambda: api.pkv_window_decode(shape, ws, q, small, small, bt, lens, 4, 0, torch.empty_like(q)),
                 lambda: api.pkv_append_slots(shape, ws, q, q, slots, small, small)):
        with pytest.raises(ValueError, match="elements, needs"):
            call()
