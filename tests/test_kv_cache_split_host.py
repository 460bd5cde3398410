"""The attention kernels' own split of their line of tiles over blocks (csrc/ar_split.h), compiled for the host: every tile
has one block, lines past 32 bits included, and the parts of an item lie where the join looks for them."""
import ctypes
import os
import random
import subprocess

import pytest

from tensor_allreduce_residual_gb300 import _build

SOURCE = """
#include "ar_split.h"
extern "C" void run_of(long long total, int blocks, int c, long long* lo, long long* n)
{
    const ar::Run r = ar::run_of(total, blocks, c);
    *lo = r.lo;
    *n = r.total == total ? r.n : -1;
}
extern "C" int block_of(long long total, int blocks, long long x) { return ar::block_of(total, blocks, x); }
extern "C" unsigned long long slot_of(int block, int begins) { return ar::slot_of(block, begins != 0); }
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{_build.CSRC}", str(d / "split.cpp"), "-o", str(d / "split.so")], check=True)
    lib = ctypes.CDLL(os.path.join(d, "split.so"))
    ll = ctypes.c_longlong
    lib.run_of.argtypes, lib.run_of.restype = [ll, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ll), ctypes.POINTER(ll)], None
    lib.block_of.argtypes, lib.slot_of.restype = [ll, ctypes.c_int, ll], ctypes.c_ulonglong
    return lib


def _run(split, total, blocks, c):
    lo, n = ctypes.c_longlong(), ctypes.c_longlong()
    split.run_of(total, blocks, c, lo, n)
    return lo.value, n.value


@pytest.mark.parametrize("total", [1, 7, 303, 304, 305, 456, 12345, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, (1 << 32) + 1, (1 << 45) + 77])
@pytest.mark.parametrize("blocks", [1, 7, 304, 456])
def test_runs_cover_the_line_and_blocks_find_their_tiles(split, total, blocks):
    at, sizes, r = 0, set(), random.Random(total)
    for c in range(blocks):
        lo, n = _run(split, total, blocks, c)
        assert lo == at and n >= 0
        for x in {lo, lo + n - 1, lo + n // 2, lo + r.randrange(max(n, 1))} if n else ():
            assert split.block_of(total, blocks, x) == c
        at += n
        sizes.add(n)
    assert at == total and max(sizes) - min(sizes) <= 1


@pytest.mark.parametrize("items,blocks", [([1, 5, 1, 9] * 3, 4), ([1] * 100, 7), ([40], 13), ([3, 1, 7] * 72, 304), ([1 << 34, 2, (1 << 33) + 5], 456)])
def test_parts_lie_where_the_join_reads_them(split, items, blocks):
    """Each block walks its run as the kernels do; the join takes an item's first block, its last, and a part of each."""
    total, starts = sum(items), [sum(items[:i]) for i in range(len(items))]
    written = {}
    for c in range(blocks):
        lo, n = _run(split, total, blocks, c)
        for item, (s, m) in enumerate(zip(starts, items)):
            a, b = max(lo, s), min(lo + n, s + m)
            if a < b and (a, b) != (s, s + m):
                slot = split.slot_of(c, a == s)
                assert slot not in written and 0 <= slot < 2 * blocks
                written[slot] = item
    for item, (s, m) in enumerate(zip(starts, items)):
        first, last = split.block_of(total, blocks, s), split.block_of(total, blocks, s + m - 1)
        read = [split.slot_of(first + p, p == 0) for p in range(last - first + 1)] if first != last else []
        assert [written.pop(slot) for slot in read] == [item] * len(read)
    assert not written
