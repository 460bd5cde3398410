"""The buffers that one call of ar_kv_compact or ar_kv_copy_pages moves in (csrc/ar_layers.h, compiled for the host): each once, however
many layers name it, as two owners of the same bytes would move what has moved already."""
import ctypes
import os
import random
import subprocess

import pytest

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build

SOURCE = """
#include "ar_layers.h"
extern "C" int distinct(void* const* k, void* const* v, int layers, void** out)
{
    ar::Layers to;
    const int n = ar::distinct_buffers(&to, k, v, layers);
    for (int i = 0; i < n; ++i)
        out[i] = (i & 1 ? to.odd : to.even)[i >> 1];
    return n;
}
"""


@pytest.fixture(scope="module")
def distinct(tmp_path_factory):
    d = tmp_path_factory.mktemp("layers")
    (d / "layers.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{_build.CSRC}", str(d / "layers.cpp"), "-o", str(d / "layers.so")], check=True)
    lib = ctypes.CDLL(os.path.join(d, "layers.so"))

    def call(k, v):
        out = (ctypes.c_void_p * (2 * len(k)))()
        n = lib.distinct((ctypes.c_void_p * len(k))(*k), (ctypes.c_void_p * len(v))(*v), len(k), out)
        return list(out[:n])

    return call


def _in_turn(k, v):
    return list(dict.fromkeys(x for pair in zip(k, v) for x in pair))


def test_layers_of_their_own_keep_their_order(distinct):
    for layers in (1, 2, 37, 128):
        k, v = [0x7f0000000000 + (i << 21) for i in range(layers)], [0x7f8000000000 + (i << 21) for i in range(layers)]
        assert distinct(k, v) == _in_turn(k, v) and len(distinct(k, v)) == 2 * layers


def test_a_buffer_that_several_layers_name_is_listed_once(distinct):
    assert distinct([0x1000, 0x1000], [0x2000, 0x2000]) == [0x1000, 0x2000]
    assert distinct([0x1000, 0x3000, 0x1000], [0x2000, 0x1000, 0x4000]) == [0x1000, 0x2000, 0x3000, 0x4000]
    assert distinct([0x1000], [0x1000]) == [0x1000]
    assert distinct([0x1000] * 128, [0x1000] * 128) == [0x1000]
    r = random.Random(4)
    for _ in range(300):
        layers, pool = r.randint(1, 128), [r.randrange(1, 1 << 47) for _ in range(r.randint(1, 200))]
        k, v = [r.choice(pool) for _ in range(layers)], [r.choice(pool) for _ in range(layers)]
        assert distinct(k, v) == _in_turn(k, v)
    for step in (1, 2, 16, 256, 1 << 10, 1 << 20, 1 << 30, 1 << 40):   # distances at which a hash may crowd
        k, v = [(1 << 46) + 2 * i * step for i in range(128)], [(1 << 46) + (2 * i + 1) * step for i in range(128)]
        assert distinct(k, v) == _in_turn(k, v)


def test_two_owners_of_one_buffer_would_move_tokens_twice(distinct):
    """The moves of one sequence by each owner of a buffer, whole or in part before the other's: only one owner gives the result."""
    kept = [1, 2, 4]
    want = [11, 12, 14, 13, 14]
    r = random.Random(1)

    def moved(owners):
        tokens, at = [10, 11, 12, 13, 14], [0] * owners
        while any(x < len(kept) for x in at):
            o = r.choice([o for o in range(owners) if at[o] < len(kept)])
            tokens[at[o]] = tokens[kept[at[o]]]
            at[o] += 1
        return tokens

    k, v = [0x1000, 0x1000], [0x2000, 0x2000]
    assert any(moved(k.count(0x1000)) != want for _ in range(100))
    assert all(moved(distinct(k, v).count(x)) == want for x in (0x1000, 0x2000) for _ in range(100))


FAKE = 0x10000   # never dereferenced: the calls are refused before a launch


def _cache(**kw):
    d = dict(k=None, v=None, dtype=ar.AR_FP8_E4M3, pages=8, page_size=1, kv_heads=1024, head_dim=1023, page_stride=1 << 40, token_stride=0,
             head_stride=1023, k_scale=1.0, v_scale=1.0, page_table=FAKE, batch=3, max_pages=4, table_stride=4, lengths=FAKE)
    d.update(kw)
    return ar.ArKVCache(**d)


def _pointers(layers, at):
    return (ctypes.c_void_p * layers)(*[at + (i << 30) for i in range(layers)])


def test_more_blocks_than_a_launch_has_are_refused_as_unsupported():
    """A token of 128 layers of 1024 heads of 1023 bytes: 268 million units of one byte; 2^31 - 1 pairs of pages of 5115 units."""
    _build.build()
    L = ar.lib()
    k, v = _pointers(128, 1 << 40), _pointers(128, 1 << 41)
    assert L.ar_kv_compact(_cache(), k, v, 128, FAKE, 5, 5, None, 5, 0x90000, None) == ar.AR_ERR_UNSUPPORTED
    small = _cache(kv_heads=1, page_size=5, token_stride=1023)
    assert L.ar_kv_copy_pages(small, k, v, 128, FAKE, FAKE, 2 ** 31 - 1, None) == ar.AR_ERR_UNSUPPORTED
    wide = _cache(kv_heads=1024, head_dim=1023, page_size=2 ** 20, token_stride=1 << 21, page_stride=1 << 50)
    assert L.ar_kv_copy_pages(wide, k, v, 128, FAKE, FAKE, 1, None) == ar.AR_ERR_UNSUPPORTED
