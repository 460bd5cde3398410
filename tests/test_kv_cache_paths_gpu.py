"""The paged key-value cache calls on paths that need many rows: joins whose rows do not end with their blocks, into each of
their partials too, and appends of several rows a block."""
import math

import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build
from tests.kv_cache_model import TORCH, check, half_step
from tests.test_kv_cache_gpu import _append_and_check, _gen, _join_room, _normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    _build.build()
    ar.lib()


def _partials(R, rows, dim, dtype, offset=0):
    """R partials, `offset` elements off the alignment, and their lse; some ranks have no key of some rows."""
    g = _gen(R * dim + rows)
    o = [_normal(g, rows * dim + offset).to(TORCH[dtype])[offset:].view(rows, dim) for _ in range(R)]
    lse = [_normal(g, rows, std=4.0) + 3 for _ in range(R)]
    for x, y in zip(o, lse):
        off = torch.rand(rows, generator=g, device="cuda") < 0.2
        y[off], x[off] = -math.inf, math.nan
    return o, lse


# rows of whole vectors; vectors over two rows, with and without elements after the last; rows of fewer elements than a
# vector, and rows off the alignment, by elements
@pytest.mark.parametrize("rows,dim,offset", [(3001, 64, 0), (2003, 33, 0), (2000, 100, 0), (1999, 9, 0), (4001, 3, 0), (701, 40, 1)])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("R", [1, 3, 12])
def test_join_over_many_blocks_and_into_each_partial(R, dtype, rows, dim, offset):
    o, lse = _partials(R, rows, dim, dtype, offset)
    ref, ref_lse, room, room_lse = _join_room(o, lse)
    out, got = ar.ar_attention_join(o, lse, return_lse=True)
    check(out, ref, room + half_step(ref, out.dtype), "out")
    check(got, ref_lse, room_lse, "lse")
    for r in range(R):
        kept = o[r].clone()
        into, again = ar.ar_attention_join(o, lse, out=o[r], return_lse=True)
        assert into is o[r] and torch.equal(into, out) and torch.equal(again, got)
        o[r].copy_(kept)


# The 16-bit vector path at several rows a block, whose table of cosines and sines is in another order: three and eight rows,
# one vector a half and several; the 8-byte vectors of an 8-bit cache; two rows in fp32.
@pytest.mark.parametrize("rows", [7301, 19998])
@pytest.mark.parametrize("dtype,cache,dim,rotary", [("bf16", "bf16", 16, 16), ("fp16", "e4m3", 64, 32), ("bf16", "bf16", 64, 64), ("fp32", "fp32", 16, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_of_several_rows_a_block(rows, dtype, cache, dim, rotary, interleaved):
    new = [2, 0, 0, rows // 3, 1, 0, rows // 2, 4]
    new.append(rows - sum(new))
    _append_and_check([n + 5 for n in new], new, 2, 1, dim, rotary, 64, dtype, cache, "NHD", interleaved=interleaved, padding=3, in_place=True)
