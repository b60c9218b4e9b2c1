"""CPU tests of the page map, the slot append and the 8-bit cache: sizes and
refusals (no call here launches a kernel), and the plain model they are tested
against."""
import ctypes

import numpy as np
import pytest
import torch

import byte_ref as R
from paged_kv_gqa_09_gb300 import _lib, api
from paged_kv_gqa_09_gb300 import build as build_mod

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return _lib.load()


def shape(**kw):
    base = dict(B=2, Hq=8, Hkv=2, d=128, page_size=16, num_pages=64, bt_stride=16, scale=0.088)
    base.update(kw)
    return _lib.Shape(*[base[k] for k, _ in _lib.Shape._fields_])


POINTERS = {"map": ("ws", "sl", "nl", "out", "bt", "fp", "fc", "fout", "off", "slots"),
            "slots": ("ws", "k_new", "v_new", "slots", "k", "v"),
            "append": ("ws", "k_new", "v_new", "bt", "sl", "out", "cache"),
            "read": ("ws", "cache", "bt", "sl", "ooff", "k_new", "v_new"),
            "decode": ("ws", "q", "cache", "bt", "sl", "o")}


def calls(L, s, **bad):
    """One call of each entry point; `bad` replaces arguments by name."""
    a = dict(ws=FAKE, k_new=FAKE, v_new=FAKE, stride=256, T=s.B, off=FAKE, aoff=None, bt=FAKE, sl=FAKE, nl=FAKE, out=FAKE,
             cache=FAKE, q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=None, first=None, ooff=FAKE, fp=FAKE, cap=9, fc=FAKE, fout=FAKE,
             slots=FAKE, pos=None, fmt=0, win=ctypes.byref(_lib.Window(4, 1)))
    a.update(bad)
    r = ctypes.byref(s)
    return {
        "map": lambda: L.pkv_map_pages(r, a["ws"], a["sl"], a["nl"], a["out"], a["bt"], a["fp"], a["cap"], a["fc"], a["fout"],
                                       a["off"], a["slots"], a["pos"], a["T"], None),
        "slots": lambda: L.pkv_append_slots(r, a["ws"], a["k_new"], a["v_new"], a["stride"], a["T"], a["slots"], a["k"],
                                            a["v"], None),
        "append": lambda: L.pkv_byte_append(r, a["ws"], a["fmt"], a["k_new"], a["v_new"], a["stride"], a["T"], a["aoff"],
                                            a["bt"], a["sl"], a["out"], a["cache"], None),
        "read": lambda: L.pkv_byte_read(r, a["ws"], a["fmt"], a["cache"], a["bt"], a["sl"], a["first"], a["ooff"], a["T"],
                                        a["k_new"], a["v_new"], a["stride"], None),
        "decode": lambda: L.pkv_byte_decode(r, a["win"], a["ws"], a["fmt"], a["q"], a["cache"], a["bt"], a["sl"], a["o"],
                                            a["lse"], None),
    }


@pytest.mark.parametrize("name", list(POINTERS))
@pytest.mark.parametrize("kw,status", [(dict(d=96), _lib.PKV_EUNSUPPORTED), (dict(Hq=6, Hkv=4), _lib.PKV_EINVAL),
                                       (dict(page_size=24), _lib.PKV_EUNSUPPORTED), (dict(num_pages=0), _lib.PKV_EINVAL),
                                       (dict(Hq=18), _lib.PKV_EUNSUPPORTED), (dict(B=-1), _lib.PKV_EINVAL)])
def test_bad_shapes_are_rejected(L, name, kw, status):
    s = shape(**kw)
    assert calls(L, s)[name]() == status
    assert L.pkv_byte_page_bytes(ctypes.byref(s)) == 0


@pytest.mark.parametrize("name,bad", [(n, {a: x}) for n, args in POINTERS.items() for a in args for x in (None, FAKE + 4)] + [
    ("append", dict(aoff=FAKE + 2)), ("read", dict(first=FAKE + 8)), ("decode", dict(lse=FAKE + 4)), ("map", dict(pos=FAKE + 4)),
    ("map", dict(T=-1)), ("map", dict(cap=-1)), ("append", dict(fmt=2)), ("read", dict(fmt=-1)), ("decode", dict(fmt=7)),
    ("append", dict(stride=255)), ("append", dict(stride=248)), ("append", dict(stride=260)), ("append", dict(T=-1)),
    ("append", dict(T=3)), ("slots", dict(stride=248)), ("slots", dict(T=-1)), ("read", dict(stride=8)), ("read", dict(T=-1)),
    ("decode", dict(win=ctypes.byref(_lib.Window(-1, 0)))), ("decode", dict(win=ctypes.byref(_lib.Window(4, -2))))])
def test_bad_arguments_are_rejected(L, name, bad):
    assert calls(L, shape(), **bad)[name]() == _lib.PKV_EINVAL
    assert _lib.last_error()


def test_calls_that_pass_an_index_are_rejected(L):
    big = dict(T=1 << 30, stride=1024, aoff=FAKE)
    for name in ("append", "read", "slots"):
        assert calls(L, shape(Hkv=8), **big)[name]() == _lib.PKV_EUNSUPPORTED
    for B in ((1 << 30) + 1, (1 << 31) - 1):
        for name in ("append", "read", "map", "slots"):
            assert calls(L, shape(B=B), T=7, aoff=FAKE)[name]() == _lib.PKV_EUNSUPPORTED
    assert calls(L, shape(), T=(1 << 31) - 4)["map"]() == _lib.PKV_EUNSUPPORTED
    s = shape(page_size=8, bt_stride=(1 << 28) - 1)  # rows whose last block ends beyond an int32
    for name in ("append", "read", "decode"):
        assert calls(L, s)[name]() == _lib.PKV_EUNSUPPORTED
    assert calls(L, shape(B=(1 << 25) + 1, Hq=1, Hkv=1, bt_stride=1, page_size=8))["decode"]() == _lib.PKV_EUNSUPPORTED
    many = shape(Hq=(1 << 20) + 1, Hkv=(1 << 20) + 1)
    assert calls(L, many, stride=128 * ((1 << 20) + 1))["slots"]() == _lib.PKV_EUNSUPPORTED


def test_empty_batches_are_no_ops(L):
    none = dict.fromkeys(("ws", "k_new", "v_new", "bt", "sl", "nl", "out", "cache", "q", "k", "v", "o", "ooff", "off", "fp", "fc",
                          "fout", "slots", "win"))
    for call in calls(L, shape(B=0), T=0, **none).values():
        assert call() == 0
    assert calls(L, shape(), T=0, k_new=None, v_new=None, slots=None)["slots"]() == 0
    assert calls(L, shape(), T=0, k_new=None, v_new=None)["read"]() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
def test_sizes(L, d, P):
    s = shape(d=d, page_size=P, Hkv=2)
    assert api.pkv_byte_page_bytes(s) == 2 * R.head_bytes(P, d)
    cache = api.byte_cache_zeros(5, P, 2, d, "cpu")
    assert cache.numel() == 5 * api.pkv_byte_page_bytes(s)
    got = api.make_byte_shape(8, d, cache, torch.zeros(2, 16, dtype=torch.int32))
    assert (got.page_size, got.d, got.Hkv, got.num_pages, got.B) == (P, d, 2, 5, 2)


def test_binding_refuses_what_the_library_cannot_see(L):
    s = shape()
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    t = torch.zeros(4, 2, 128, dtype=torch.float16)
    i32, i64 = torch.zeros(64, dtype=torch.int32), torch.zeros(64, dtype=torch.int64)
    for call in (lambda: api.pkv_byte_append(s, ws, 0, t, t, i32, i32, ws), lambda: api.pkv_byte_decode(s, ws, 0, t, ws, i32, i32, t),
                 lambda: api.pkv_byte_read(s, ws, 0, ws, i32, i32, i32, t, t), lambda: api.pkv_append_slots(s, ws, t, t, i64, t, t),
                 lambda: api.pkv_map_pages(s, ws, i32, i32, i32, i32, i32, i64, i32),
                 lambda: api.pkv_byte_decode(s, None, 0, t, t, t, t, t, sinks=4)):
        with pytest.raises(ValueError):  # host tensors
            call()
    with pytest.raises(TypeError):
        api.pkv_byte_append(s, ws, "int8", t, t, i32, i32, ws)
    with pytest.raises(ValueError):
        api.make_byte_shape(8, 128, torch.zeros(4, 2, 1001, dtype=torch.uint8), i32.view(2, 32))
    with pytest.raises(_lib.PkvError):
        api.pkv_byte_page_bytes(shape(page_size=5))


def test_a_decoders_byte_steps_go_to_the_stream_of_the_call(L, monkeypatch):
    """On a stream that is not the current one the workspace is made, and waited for, there, once; a stream that is
    being captured makes none."""
    log, now, capturing = [], ["current"], []

    class On:
        def __init__(self, stream):
            self.name = stream

        def __enter__(self):
            now.append(self.name)

        def __exit__(self, *_):
            now.pop()

    class Stream(str):
        pass

    class Zeros(torch.Tensor):
        is_cuda = True

    class Current:
        def synchronize(self):
            log.append(("wait", now[-1]))

    def zeros(*a, make=torch.zeros, **k):
        log.append(("workspace", now[-1]))
        return make(*a, **k).as_subclass(Zeros)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: Current())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[-1] in capturing)
    monkeypatch.setattr(torch, "zeros", zeros)
    for name in ("pkv_byte_decode", "pkv_byte_append", "pkv_byte_read", "pkv_append_slots", "pkv_map_pages"):
        monkeypatch.setattr(api, name, lambda *_: log.append(("launch", now[-1])))
    q, bt, lens = torch.ones(2, 8, 128, dtype=torch.float16), torch.ones(2, 16, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    cache = torch.ones(64, 2, R.head_bytes(16, 128), dtype=torch.uint8)
    pages = torch.ones(64, 16, 2, 128, dtype=torch.float16)
    new = torch.ones(2, 2, 128, dtype=torch.float16)
    side = Stream("side")
    for step in (lambda d, s: d.step_byte(0, q, cache, bt, lens, stream=s), lambda d, s: d.append_byte(1, new, new, cache, bt, lens, stream=s),
                 lambda d, s: d.read_byte(0, cache, bt, lens, lens, new, new, stream=s),
                 lambda d, s: d.append_slots(new, new, lens, pages, pages, stream=s),
                 lambda d, s: d.map_pages(shape(), lens, lens, bt, lens, lens, lens, lens, stream=s)):
        for stream, where in ((side, "side"), (None, "current")):
            log.clear()
            dec = api.PagedDecoder()
            step(dec, stream)
            assert log == [("workspace", where), ("wait", where), ("launch", "current")]
            log.clear()
            step(dec, stream)
            assert [what for what, _ in log] == ["launch"]
        capturing.append("side")
        with pytest.raises(RuntimeError, match="before capturing"):
            step(api.PagedDecoder(), side)
        capturing.clear()


# ------------------------------------------------------------------ the plain model

@pytest.mark.parametrize("P,d", [(8, 64), (16, 128), (32, 64), (64, 64), (128, 128)])
def test_places_use_every_byte_of_a_page_once(P, d):
    used = np.zeros(R.head_bytes(P, d), np.int64)
    k, v, sk, sv = R.places(P, d)
    np.add.at(used, k, 1)
    np.add.at(used, v, 1)
    for s in (sk, sv):
        for at in np.unique(s):
            used[at:at + 4] += 1
    tb, sb = min(P, 64), min(P, 16)
    unused = R.head_bytes(P, d) - P // tb * (2 * tb * d + tb // sb * 8)
    assert used.max() == 1 and (used == 0).sum() == unused


def test_numbers_of_e4m3_are_the_types():
    c = np.arange(256, dtype=np.uint8)
    got = R.numbers(c, R.E4M3)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    y = np.concatenate([np.linspace(-448, 448, 100001), np.float64(2.0) ** np.arange(-12, 9), R._e4m3_numbers()])
    y = np.concatenate([y, (R._e4m3_numbers()[1:] + R._e4m3_numbers()[:-1]) / 2])  # ties
    y = y.astype(np.float32).astype(np.float64)
    assert np.array_equal(R.nearest(y, R.E4M3), torch.from_numpy(y).float().to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_values_stay_within_the_stated_error(fmt):
    rng = np.random.default_rng(2)
    for scale in (1e-7, 1e-3, 1.0, 300.0, 9000.0):
        x = np.clip(rng.standard_normal((48, 2, 64)) * scale, -57344, 57344).astype(np.float16)
        s = R.Side(fmt, 16, 2, 64)
        s.append(x)
        y, unit = s.values(), s.scales()[:, :, None]
        bound = unit / 2 if fmt == R.INT8 else np.maximum(2.0 ** -4 * np.abs(x.astype(np.float64)), unit * 2.0 ** -10)
        assert (np.abs(y - x) <= bound).all()
        assert np.array_equal(y.astype(np.float16).astype(np.float64), y)  # fp16 numbers
        t = R.Side(fmt, 16, 2, 64)
        for n in (1, 4, 16, 3, 24):  # one more step for each growth of e
            t.append(x[len(t.y):len(t.y) + n])
        assert np.array_equal(t.e, s.e) and (np.abs(t.values() - x) <= 6 * bound).all()


def test_a_packed_token_reads_back():
    rng = np.random.default_rng(1)
    for fmt, P, d in ((0, 16, 128), (1, 64, 64), (0, 8, 64)):
        page = np.zeros((2, R.head_bytes(P, d)), np.uint8)
        sides = [R.Side(fmt, P, 2, d) for _ in range(2)]
        for side in sides:
            side.append(rng.standard_normal((P, 2, d)).astype(np.float16))
        for t in rng.permutation(P):
            for u, side in enumerate(sides):
                R.pack(page, t, side.y[t], side.e[t // side.sb], u, P, d, fmt)
        for got, side in zip(R.unpack(page, P, d, fmt), sides):
            assert np.array_equal(got, side.values().transpose(1, 0, 2))
