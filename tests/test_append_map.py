"""The 4-bit append's map from groups of cache positions to packed tokens, on
the CPU.

The kernel reads and stores the tokens that append_map.cuh, a header of
host-and-device functions, names.  Here the header is compiled for the host and
every group of a batch is followed: each new token is stored once, at its row's
next position, and no token of another row or outside the packed buffer is
read -- rows without new tokens among the others, first and last, included.
"""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_gqa_09_gb300", "csrc")


@pytest.fixture(scope="module")
def amap(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = tmp_path_factory.mktemp("append_map") / "libappend_map.so"
    subprocess.run([nvcc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC, "-o", str(out),
                    os.path.join(ROOT, "tests", "append_map_host.cu")], check=True)
    L = ctypes.CDLL(str(out))
    L.append_map_all.argtypes = [ctypes.c_int, ctypes.c_int] + [ctypes.c_void_p] * 6
    L.append_units_all.argtypes = [ctypes.c_int] * 5 + [ctypes.c_void_p]
    L.append_units_all.restype = ctypes.c_longlong
    return L


def check(L, lens, new):
    lens, new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(off[-1])
    reads, stores, place = np.zeros(T + 1, np.int32), np.zeros(T + 1, np.int32), np.zeros(T + 1, np.int64)
    out = np.zeros(2, np.int64)
    L.append_map_all(lens.size, T, *(x.ctypes.data for x in (off, lens, reads, stores, place, out)))
    assert out[0] == 0, (lens.tolist(), new.tolist())
    assert (stores[:T] == 1).all() and (reads[:T] >= 1).all()
    row = np.repeat(np.arange(lens.size), new)
    assert np.array_equal(place[:T], (row.astype(np.int64) << 32) + lens[row] + np.arange(T) - off[row])
    # the groups that hold a new token, and no others
    assert out[1] == sum((a + n + 7) // 8 - a // 8 for a, n in zip(lens.tolist(), new.tolist()) if n)


@pytest.mark.parametrize("n", range(1, 10))
def test_an_empty_first_row_reads_nothing(amap, n):
    check(amap, [n, 3], [0, 4])
    check(amap, [n, n, n], [0, 0, 9])


@pytest.mark.parametrize("lens", [[5], [0], [5, 9], [8, 1, 7, 15]])
def test_an_append_of_nothing_reads_nothing(amap, lens):
    check(amap, lens, [0] * len(lens))


def test_random_batches(amap):
    rng = np.random.default_rng(11)
    for _ in range(2000):
        B = int(rng.integers(1, 12))
        most = int(rng.choice([2, 9, 40]))
        check(amap, rng.integers(0, 70, B), rng.integers(0, most, B) * rng.integers(0, 2, B))


def test_rows_at_the_end_of_int32(amap):
    end = 2 ** 31 - 1
    check(amap, [end - 20, 3, end - 1], [20, 0, 1])


@pytest.mark.parametrize("ctas", [456, 3])
@pytest.mark.parametrize("T,B,Hkv", [(1, 1, 2048), (1, 1, 1824), (1, 1, 1825), (5, 2, 5000), (1, 1, 1), (1, 1, 8), (400, 9, 3), (9, 3, 8),
                                     (40000, 8, 8), (3000, 1, 100), (0, 4, 8)])
def test_every_side_of_every_group_has_a_warp(amap, T, B, Hkv, ctas):
    """Very many KV heads and few tokens among the calls: as many parts as a group has sides would be more than
    there are warps."""
    units = np.zeros((max(1, T // 8 + 2 * B), 2 * Hkv), np.int32)
    groups = amap.append_units_all(T, B, Hkv, ctas, 8, units.ctypes.data)
    assert groups == (T // 8 + 2 * B if T else 0)
    assert (units[:groups] == 1).all()
