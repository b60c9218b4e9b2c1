"""CPU tests of the 4-bit cache and windowed decode entry points: sizes and
refusals (no call here launches a kernel), and the plain model they are tested
against."""
import ctypes

import numpy as np
import pytest
import torch

import quant_ref as R
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


def calls(L, s, **bad):
    """One call of each entry point; `bad` replaces arguments by name."""
    a = dict(ws=FAKE, k_new=FAKE, v_new=FAKE, stride=256, T=s.B, off=None, bt=FAKE, sl=FAKE, out=FAKE, cache=FAKE, q=FAKE,
             k=FAKE, v=FAKE, o=FAKE, lse=None, first=None, ooff=FAKE, win=ctypes.byref(_lib.Window(4, 1)))
    a.update(bad)
    r = ctypes.byref(s)
    return {
        "append": lambda: L.pkv_quant_append(r, a["ws"], a["k_new"], a["v_new"], a["stride"], a["T"], a["off"], a["bt"],
                                             a["sl"], a["out"], a["cache"], None),
        "read": lambda: L.pkv_quant_read(r, a["ws"], a["cache"], a["bt"], a["sl"], a["first"], a["ooff"], a["T"], a["k_new"],
                                         a["v_new"], a["stride"], None),
        "quant": lambda: L.pkv_quant_decode(r, a["win"], a["ws"], a["q"], a["cache"], a["bt"], a["sl"], a["o"], a["lse"],
                                            None),
        "window": lambda: L.pkv_window_decode(r, a["win"], a["ws"], a["q"], a["k"], a["v"], a["bt"], a["sl"], a["o"],
                                              a["lse"], None),
    }


@pytest.mark.parametrize("name", ["append", "read", "quant", "window"])
@pytest.mark.parametrize("kw,status", [(dict(d=96), _lib.PKV_EUNSUPPORTED), (dict(Hq=6, Hkv=4), _lib.PKV_EINVAL),
                                       (dict(page_size=24), _lib.PKV_EUNSUPPORTED), (dict(num_pages=0), _lib.PKV_EINVAL),
                                       (dict(Hq=18), _lib.PKV_EUNSUPPORTED)])
def test_bad_shapes_are_rejected(L, name, kw, status):
    s = shape(**kw)
    assert calls(L, s)[name]() == status
    assert L.pkv_attn_workspace_size(ctypes.byref(s)) == 0 and L.pkv_quant_page_bytes(ctypes.byref(s)) == 0


@pytest.mark.parametrize("name,bad", [(n, {a: x}) for n, args in {
    "append": ("ws", "k_new", "v_new", "bt", "sl", "out", "cache"), "read": ("ws", "cache", "bt", "sl", "ooff", "k_new", "v_new"),
    "quant": ("ws", "q", "cache", "bt", "sl", "o"), "window": ("ws", "q", "k", "v", "bt", "sl", "o")}.items()
    for a in args for x in (None, FAKE + 4)] + [("append", dict(off=FAKE + 2)), ("read", dict(first=FAKE + 8)),
                                                ("quant", dict(lse=FAKE + 4)), ("window", dict(win=None)),
                                                ("append", dict(stride=255)), ("append", dict(stride=248)),
                                                ("append", dict(stride=260)), ("append", dict(T=-1)), ("append", dict(T=3)),
                                                ("read", dict(stride=8)), ("read", dict(T=-1)),
                                                ("quant", dict(win=ctypes.byref(_lib.Window(-1, 0)))),
                                                ("window", dict(win=ctypes.byref(_lib.Window(4, -2))))])
def test_bad_arguments_are_rejected(L, name, bad):
    assert calls(L, shape(), **bad)[name]() == _lib.PKV_EINVAL
    assert _lib.last_error()


def test_too_many_tokens_are_rejected(L):
    s = shape(Hkv=8)
    big = dict(T=1 << 30, stride=1024, off=FAKE)
    assert calls(L, s, **big)["append"]() == _lib.PKV_EUNSUPPORTED
    assert calls(L, s, **big)["read"]() == _lib.PKV_EUNSUPPORTED


def test_too_many_rows_are_rejected(L):
    """The search for a token's row adds two rows' indices, and the lengths' loop one and a CTA's threads."""
    for B in ((1 << 30) + 1, (1 << 31) - 1):
        s = shape(B=B)
        assert calls(L, s, T=7, off=FAKE)["append"]() == _lib.PKV_EUNSUPPORTED
        assert calls(L, s, T=7)["read"]() == _lib.PKV_EUNSUPPORTED
        assert "rows" in _lib.last_error()


def test_rows_that_a_bounded_wait_does_not_cover_are_rejected(L):
    """A decode's CTAs look through all rows' lengths first, while a wait of one second runs."""
    s = shape(B=(1 << 25) + 1, Hq=1, Hkv=1, bt_stride=1, page_size=8)
    for name in ("quant", "window"):
        assert calls(L, s)[name]() == _lib.PKV_EUNSUPPORTED
        assert "rows" in _lib.last_error()


def test_rows_at_the_end_of_int32_are_rejected(L):
    s = shape(page_size=8, bt_stride=(1 << 28) - 1)
    assert calls(L, s)["quant"]() == _lib.PKV_EUNSUPPORTED
    assert calls(L, s)["window"]() == _lib.PKV_EUNSUPPORTED
    s = shape(B=1 << 20, page_size=64, bt_stride=1 << 14)  # more tiles than an int32 counts
    assert calls(L, s, win=None)["quant"]() == _lib.PKV_EUNSUPPORTED
    s = shape(B=(1 << 31) - 1)
    assert calls(L, s)["window"]() == _lib.PKV_EUNSUPPORTED


def test_empty_batches_are_no_ops(L):
    none = dict.fromkeys(("ws", "k_new", "v_new", "bt", "sl", "out", "cache", "q", "k", "v", "o", "ooff", "win"))
    for call in calls(L, shape(B=0), T=0, **none).values():
        assert call() == 0
    assert calls(L, shape(), T=0, k_new=None, v_new=None)["read"]() == 0


def test_sizes(L):
    s = shape(d=128, page_size=16, Hkv=2)
    assert api.pkv_quant_page_bytes(s) == 2 * 16 * 128 * 5 // 4
    assert api.pkv_attn_workspace_size(s) == api.pkv_attn_workspace_size(shape(num_pages=9999, bt_stride=3, page_size=64))
    with pytest.raises(_lib.PkvError):
        api.pkv_attn_workspace_size(shape(d=80))
    with pytest.raises(_lib.PkvError):
        api.pkv_quant_page_bytes(shape(page_size=5))


def test_binding_refuses_what_the_library_cannot_see(L):
    s = shape()
    t = torch.zeros(4, 2, 128, dtype=torch.float16)
    with pytest.raises(ValueError):  # host tensors
        api.pkv_quant_append(s, torch.zeros(1 << 20, dtype=torch.uint8), t, t, t, t, t)
    with pytest.raises(ValueError):
        api.pkv_quant_decode(s, torch.zeros(1 << 20, dtype=torch.uint8), t, t, t, t, t)
    with pytest.raises(ValueError):
        api.pkv_quant_decode(s, None, t, t, t, t, t, sinks=4)
    bt = torch.zeros(2, 16, dtype=torch.int32)
    assert api.make_quant_shape(8, 128, api.quant_cache_zeros(64, 16, 2, 128, "cpu"), bt).page_size == 16
    with pytest.raises(ValueError):
        api.make_quant_shape(8, 128, torch.zeros(4, 2, 1001, dtype=torch.uint8), bt)


def test_a_binding_built_for_another_pytorch_is_not_used(L, monkeypatch, tmp_path):
    """The compiled argument checks read tensors by the headers of the PyTorch that they were compiled against."""
    monkeypatch.setattr(_lib, "_call", None)
    assert build_mod.up_to_date()
    _lib.load_call()
    monkeypatch.setattr(_lib, "_call", None)
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    assert not build_mod.up_to_date()
    with pytest.raises(_lib.PkvLibraryError, match="1.2.3"):
        _lib.load_call()
    monkeypatch.undo()
    monkeypatch.setattr(build_mod, "CALL_FOR", str(tmp_path / "none"))  # one that does not say
    assert not build_mod.up_to_date()


def test_a_decoders_buffers_belong_to_the_stream_of_the_call(L, monkeypatch):
    """A decoder's first call on a stream that is not the current one: its workspace is zero before the launch, and
    the outputs it makes are memory of that stream; a stream that is being captured makes no workspace."""
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

    def made(what, make, wrap=lambda t: t):
        def f(*a, **k):
            log.append((what, now[-1]))
            return wrap(make(*a, **k))
        return f

    class Current:
        def synchronize(self):
            log.append(("wait", now[-1]))

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: Current())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[-1] in capturing)
    monkeypatch.setattr(torch, "zeros", made("workspace", torch.zeros, lambda t: t.as_subclass(Zeros)))
    monkeypatch.setattr(torch, "empty_like", made("o", torch.empty_like))
    monkeypatch.setattr(torch, "empty", made("lse", torch.empty))
    for name in ("pkv_quant_decode", "pkv_window_decode", "pkv_quant_append"):
        monkeypatch.setattr(api, name, lambda *_: log.append(("launch", now[-1])))
    q, bt = torch.ones(2, 8, 128, dtype=torch.float16), torch.ones(2, 16, dtype=torch.int32)
    cache = torch.ones(64, 2, 16 * 128 * 5 // 4, dtype=torch.uint8)
    pages = torch.ones(64, 16, 2, 128, dtype=torch.float16)
    new = torch.ones(2, 2, 128, dtype=torch.float16)
    side = Stream("side")
    for step in (lambda d, s: d.step_quant(q, cache, bt, None, stream=s), lambda d, s: d.step_window(q, pages, pages, bt, None, 9, stream=s),
                 lambda d, s: d.append_quant(new, new, cache, bt, None, stream=s)):
        for stream, where in ((side, "side"), (None, "current")):
            log.clear()
            dec = api.PagedDecoder()
            step(dec, stream)
            assert {at for what, at in log if what != "launch"} == {where}, log
            names = [what for what, _ in log]
            assert names.index("workspace") < names.index("wait") < names.index("launch"), log
            log.clear()
            step(dec, stream)
            assert "workspace" not in [what for what, _ in log] and "wait" not in [what for what, _ in log]
        capturing.append("side")
        with pytest.raises(RuntimeError, match="before capturing"):
            step(api.PagedDecoder(), side)
        capturing.clear()


def test_the_fp16_step_makes_its_buffers_on_its_stream(L, monkeypatch):
    """PagedDecoder.step on a stream that is not the current one: its workspace is zeroed in that stream, when it is
    made and when the configuration changes, and its other buffers are memory of it."""
    log, now = [], ["current"]

    class On:
        def __init__(self, stream):
            self.name = stream

        def __enter__(self):
            now.append(self.name)

        def __exit__(self, *_):
            now.pop()

    class Stream(str):
        pass

    class Workspace(torch.Tensor):
        def zero_(self):
            log.append(("zero", now[-1]))
            return self

    def made(what, make, kind=torch.Tensor):
        def f(*a, **k):
            log.append((what, now[-1]))
            return make(*a, **k).as_subclass(kind)
        return f

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "zeros", made("workspace", torch.zeros, Workspace))
    monkeypatch.setattr(torch, "empty_like", made("o", torch.empty_like))
    monkeypatch.setattr(torch, "empty", made("partials or lse", torch.empty))
    monkeypatch.setattr(api, "pkv_decode_step", lambda *_: log.append(("launch", now[-1])))
    q, bt = torch.ones(2, 8, 128, dtype=torch.float16), torch.ones(2, 64, dtype=torch.int32)
    pages = torch.ones(64, 16, 2, 128, dtype=torch.float16)
    dec = api.PagedDecoder()
    for chunk, first in ((256, "workspace"), (512, "zero")):
        log.clear()
        dec.step(q, pages, pages, bt, None, 1000, path=_lib.PKV_PATH_WORKQUEUE, split_tokens=chunk, stream=Stream("side"))
        assert log[0][0] == first and {at for what, at in log if what != "launch"} == {"side"}, log


# ------------------------------------------------------------------ the plain model

@pytest.mark.parametrize("P,d", [(8, 64), (16, 128), (64, 64), (128, 128)])
def test_places_use_every_bit_of_a_page_once(P, d):
    used = np.zeros((P * d * 5 // 8, 16), np.int64)
    cells = [[6, 7, 8, 9], [2, 3, 4, 5], [10, 11, 12, 13], [14, 15, 0, 1]]
    for at, f, sp, bp in R.places(P, d):
        for slot in range(P):
            for dim in range(d):
                used[at[slot, dim], cells[f[slot, dim]]] += 1
            used[sp[slot, ::32]] += 1
            used[bp[slot, ::32]] += 1
    assert (used == 1).all()


def test_a_packed_token_reads_back():
    rng = np.random.default_rng(1)
    page = np.zeros((2, 16 * 64 * 5 // 4), np.uint8)
    k, v = (rng.standard_normal((16, 2, 64)).astype(np.float16) for _ in range(2))
    for t in rng.permutation(16):
        R.pack_token(page, t, k[t], v[t], 16, 64)
    got = R.page_values(page, 16, 64)
    assert np.array_equal(got[0], R.values(k).transpose(1, 0, 2)) and np.array_equal(got[1], R.values(v).transpose(1, 0, 2))


def test_values_stay_within_the_stated_error():
    """|value - x| <= s / 2 + one fp16 step of b, for values within the limit."""
    rng = np.random.default_rng(2)
    for scale in (1e-6, 1e-3, 1.0, 300.0, 4000.0):
        x = np.clip(rng.standard_normal((200, 64)) * scale + rng.choice([0, scale * 5]), -R.LIMIT, R.LIMIT).astype(np.float16)
        _, s, b = R.quantise(x)
        step = np.spacing(np.abs(b).astype(np.float16)).astype(np.float64)
        err = np.abs(R.values(x) - x.astype(np.float64)).reshape(200, 2, 32)
        assert (err <= (s / 2 + step)[..., None]).all()
