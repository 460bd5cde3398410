"""The paged key-value cache calls where a result shows the bits of what it is made of: weights against values that
cancel, factors at the ends of fp32, sines of small angles."""
import math

import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build
from tests import kv_cache_model as model
from tests.kv_cache_model import TORCH, check, half_step

pytestmark = pytest.mark.gpu

PAIRS = [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")]


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    _build.build()
    ar.lib()


def _ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("heads", [4, 16])
@pytest.mark.parametrize("pairs", [1, 50])
@pytest.mark.parametrize("dim", [16, 128])
def test_weights_keep_their_bits_against_values_that_cancel(dtype, cache, heads, pairs, dim):
    """Tokens in pairs of values -1 and n, the latter weighing about 1 / n: where n is the head's, the result is what is left
    of them, far below each.  The model's bound for fp32 queries has weights of 17 bits; one element of the query is not 0,
    so that no scaling of it loses any."""
    n = torch.tensor([3.0, 5.0, 7.0, 9.0, 11.0, 13.0, 15.0, 10.0], device="cuda")
    k, v = torch.zeros(pairs, 2, dim, device="cuda"), torch.full((pairs, 2, dim), -1.0, device="cuda")
    k[:, 1, 0] = -1.0
    v[:, 1] = n.repeat(dim // 8)
    tokens = 2 * pairs
    pages = torch.zeros(2, -(-tokens // 16) * 16, dim, device="cuda")
    pages[0, :tokens], pages[1, :tokens] = k.view(-1, dim), v.view(-1, dim)
    k, v = (x.reshape(-1, 16, 1, dim).to(TORCH[cache]) for x in pages)
    q = torch.zeros(1, heads, dim, device="cuda")
    q[0, :, 0] = n.log().repeat(2)[:heads]
    q = q.to(TORCH[dtype])
    table = torch.arange(k.shape[0], dtype=torch.int32, device="cuda")[None]
    out, lse = ar.ar_paged_attention(q, k, v, table, _ints(tokens), scale=1.0, return_lse=True)
    ref, ref_lse, room, room_lse = model.attention(q.float(), k, v, table, [tokens], scale=1.0)
    check(out, ref, room + half_step(ref, out.dtype), f"{dtype} {cache} out")
    check(lse, ref_lse, room_lse, f"{dtype} {cache} lse")


@pytest.mark.parametrize("dtype,cache", [p for p in PAIRS if p[0] != "fp16"])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_large_queries_and_scales_of_keys_that_are_zero(dtype, cache, softcap):
    """The query's size times the scale is over fp32's range, the scores are 0: every token weighs the same."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    k = torch.zeros(3, 16, 1, 64, device="cuda").to(TORCH[cache])
    v = torch.randn(3, 16, 1, 64, generator=g, device="cuda").to(TORCH[cache])
    q = torch.full((1, 4, 64), 2.0 ** 120, device="cuda").to(TORCH[dtype])
    q[0, 2] = -q[0, 2]
    table = _ints(0, 1, 2)[None]
    out, lse = ar.ar_paged_attention(q, k, v, table, _ints(37), scale=2.0 ** 40, softcap=softcap, return_lse=True)
    ref, ref_lse, room, room_lse = model.attention(q, k, v, table, [37], scale=2.0 ** 40, softcap=softcap)
    check(out, ref, room + half_step(ref, out.dtype), f"{dtype} {cache} out")
    check(lse, ref_lse, room_lse, f"{dtype} {cache} lse")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [2, 64])   # elements, and vectors
def test_rotation_of_small_angles_keeps_their_bits(interleaved, dim):
    """(0, 1) turns to (-sin a, cos a), each of the fp32 result's own size whatever the angle, near whole quarters of a turn
    too.  The angle of a position is off by less than 2^-64 turns for the fraction's 64 bits and its own size times 2^-62 for
    1 / 2 pi's, 2^-60 together up to pi; and relative to itself after whole quarters by u = 2^-24; sine and cosine by two
    steps, 4 u; the scale, the product and the sum by u each: 8 u of the result."""
    half = dim // 2
    freq = torch.tensor([1.0, 0.1, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 3e-8], device="cuda")
    freq = torch.cat([freq, math.pi / 2 ** torch.arange(8, device="cuda").float()]).repeat(2)
    positions = [0, 1, -1, 2, 3, 7, 100, 1000, 4097, -5000, 100003, (1 << 20) + 1]
    for f in freq[:16].split(half) if half < 16 else [freq]:
        rows = len(positions)
        x = torch.zeros(rows, 1, dim, device="cuda")
        x[..., 1::2] = 1.0
        if not interleaved:
            x = torch.cat([x[..., 0::2], x[..., 1::2]], -1).contiguous()
        k = torch.zeros(1, rows, 1, dim, device="cuda")
        v = torch.zeros_like(k)
        got = ar.ar_kv_append(k, v, _ints(0)[None], _ints(rows), x, x, q=x, seq_start=_ints(0, rows), positions=_ints(*positions),
                              inv_freq=f, interleaved=interleaved, rotary_scale=0.75)
        pos = _ints(*positions)
        ref = model.rotate(x.double(), pos, f, interleaved, 0.75)
        room = 8 * model.U32 * ref.abs() + ((pos.double().abs() + 1) * 2.0 ** -60)[:, None, None]
        check(got, ref, room, "q")
        check(k[0], ref, room, "k")
