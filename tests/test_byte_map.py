"""The 8-bit append's and read's map from scale blocks to packed tokens, on the
CPU: every token is in one block's group, at its row's next position."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_gqa_09_gb300", "csrc")


@pytest.fixture(scope="module")
def bmap(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = tmp_path_factory.mktemp("byte_map") / "libbyte_map.so"
    subprocess.run([nvcc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC, "-o", str(out),
                    os.path.join(ROOT, "tests", "byte_map_host.cu")], check=True)
    L = ctypes.CDLL(str(out))
    L.byte_map_all.argtypes = [ctypes.c_int] * 3 + [ctypes.c_void_p] * 5
    return L


def check(L, lens, new, lg):
    lens, new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(off[-1])
    seen, places, out = np.zeros(T + 1, np.int32), np.zeros(T + 1, np.int64), np.zeros(2, np.int64)
    L.byte_map_all(lens.size, T, lg, *(x.ctypes.data for x in (off, lens, seen, places, out)))
    assert (seen[:T] == 1).all() and out[1] == 0
    row = np.repeat(np.arange(lens.size), new)
    assert np.array_equal(places[:T], (row.astype(np.int64) << 32) + lens[row] + np.arange(T) - off[row])
    size = 1 << lg
    assert out[0] == sum((a + n + size - 1) // size - a // size for a, n in zip(lens.tolist(), new.tolist()) if n)


@pytest.mark.parametrize("lg", [3, 4])
def test_random_batches(bmap, lg):
    rng = np.random.default_rng(lg)
    for _ in range(2000):
        B = int(rng.integers(1, 12))
        most = int(rng.choice([2, 17, 80]))
        check(bmap, rng.integers(0, 100, B), rng.integers(0, most, B) * rng.integers(0, 2, B), lg)


@pytest.mark.parametrize("lg", [3, 4])
def test_rows_at_the_end_of_their_range(bmap, lg):
    end = 2 ** 31 - 256
    check(bmap, [end - 20, 3, end - 1], [20, 0, 1], lg)
    check(bmap, [end - 40, -3], [40, 9], lg)  # a read may ask for tokens before a row's first
