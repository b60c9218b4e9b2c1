"""The launches of the 8-bit append and read on the CPU: every side of every scale
block has one warp, and calls beyond one launch are refused."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from paged_kv_gqa_09_gb300 import _lib
from test_byte_host import L, calls, shape  # noqa: F401 (L is a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 2 ** 31 - 1  # CTAs of a launch


@pytest.fixture(scope="module")
def grid(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = tmp_path_factory.mktemp("byte_grid") / "libbyte_grid.so"
    subprocess.run([nvcc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I",
                    os.path.join(ROOT, "paged_kv_gqa_09_gb300", "csrc"), "-o", str(out),
                    os.path.join(ROOT, "tests", "byte_grid_host.cu")], check=True)
    lib = ctypes.CDLL(str(out))
    for f in (lib.byte_append_units, lib.byte_read_units):
        f.argtypes = [ctypes.c_int] * 5 + [ctypes.c_void_p] * 2
    return lib


@pytest.mark.parametrize("lg", [3, 4])
@pytest.mark.parametrize("name", ["byte_append_units", "byte_read_units"])
def test_every_side_has_one_warp(grid, name, lg):
    rng = np.random.default_rng(lg)
    for k in range(1500):
        T, B = int(rng.choice([0, 1, 7, 100, 2000])), int(rng.integers(1, 40))
        Hkv, ctas = int(rng.choice([1, 2, 3, 5, 8, 19, 150])), int(rng.choice([1, 2, 9, 456]))
        T = T if Hkv < 100 else T // 10
        groups = (T >> lg) + 2 * B if T else 0
        units, out = np.zeros(groups * 2 * Hkv + 1, np.int32), np.zeros(4, np.int64)
        getattr(grid, name)(T, B, Hkv, lg, ctas, units.ctypes.data, out.ctypes.data)
        assert out[0] == groups and (units[:-1] == 1).all() and units[-1] == 0
        assert out[1] * out[2] >= 2 * Hkv
        assert name == "byte_read_units" or out[3] <= ctas


def test_the_sizes_of_large_launches(grid):
    out = np.zeros(4, np.int64)
    for T, B, Hkv, lg in ((1 << 30, 1, 1, 4), (1, 1 << 30, 8, 4), (5, 1 << 28, 64, 4), (1 << 20, 1 << 30, 128, 3), (2 ** 31 - 1, 3, 64, 3)):
        grid.byte_read_units(T, B, Hkv, lg, 608, None, out.ctypes.data)
        groups = (T >> lg) + 2 * B
        assert out[0] == groups and out[3] == -(-groups * Hkv // 8)  # two sides a warp, eight warps a CTA
        grid.byte_append_units(T, B, Hkv, lg, 456, None, out.ctypes.data)
        assert out[0] == groups and out[3] == 456


def test_reads_beyond_one_launch_are_refused(L):
    for B, Hkv, P in ((1 << 30, 8, 16), (1 << 28, 64, 16), (1 << 28, 32, 256), (1 << 30, 128, 8)):
        s = shape(B=B, Hq=Hkv, Hkv=Hkv, page_size=P, bt_stride=1)
        assert -(-2 * B * Hkv // 8) > MOST
        assert calls(L, s, T=5, stride=Hkv * 128)["read"]() == _lib.PKV_EUNSUPPORTED
        assert "one launch" in _lib.last_error()
