"""Calls of the 4-bit cache and windowed decode at their edges: rows without
new tokens, very many KV heads, a decoder on another stream."""
import numpy as np
import pytest
import torch

import quant_ref as R
from paged_kv_gqa_09_gb300 import _lib, api
from test_gpu_quant import Batch, Pages, bits, compare, dev, queries

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
