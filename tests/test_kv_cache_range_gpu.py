"""Attention over the paged cache where numbers lie far apart: weights far below the largest, queries with elements far
below the largest, softcaps far above the scores."""
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


def _pages(keys, dtype):
    """keys or values [tokens, dim] as pages of 16 tokens of one head."""
    return keys.reshape(-1, 16, 1, keys.shape[1]).to(TORCH[dtype])


def _check(q, k, v, what, rows=1, **kw):
    """Attention of q [heads, dim], repeated over `rows` sequences that share all pages, against the formula."""
    tokens = k.shape[0] * 16
    table = torch.arange(k.shape[0], dtype=torch.int32, device="cuda").expand(rows, -1).contiguous()
    n = torch.full((rows,), tokens, dtype=torch.int32, device="cuda")
    out, lse = ar.ar_paged_attention(q.expand(rows, *q.shape).contiguous(), k, v, table, n, return_lse=True, **kw)
    ref, ref_lse, room, room_lse = model.attention(q[None], k, v, table[:1], [tokens], **kw)
    check(out, ref.expand_as(out), (room + half_step(ref, out.dtype)).expand_as(out), f"{what} out")
    check(lse, ref_lse.expand_as(lse), room_lse.expand_as(lse), f"{what} lse")


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("rows", [1, 600])   # split over many blocks, or a row in one
def test_many_weights_far_below_the_largest(dtype, cache, rows):
    """A few tokens whose weights are e^18 times the others' and whose values are 0: the result is all others'."""
    k, v = torch.zeros(4000, 64, device="cuda"), torch.full((4000, 64), 96.0, device="cuda")
    for j in (0, 16, 32, 48, 64, 96):
        k[j], v[j] = 18 / 256, 0.0
    q = torch.full((4, 64), 4.0, device="cuda").to(TORCH[dtype])
    _check(q, _pages(k, cache), _pages(v, cache), f"{dtype} {cache}", rows, scale=1.0)


@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_query_elements_far_below_the_largest(dtype, cache):
    """One element is 2^26 times the rest, where every key is 0: the scores are the rest's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    k, v = (torch.randn(496, 64, generator=g, device="cuda") for _ in range(2))
    k[:, 0] = 0.0
    q = torch.randn(4, 64, generator=g, device="cuda").to(TORCH["bf16"]).float() * 2.0 ** -12
    q[:, 0] = 2.0 ** 14
    _check(q.to(TORCH[dtype]), _pages(k, cache), _pages(v, cache), f"{dtype} {cache}", scale=2.0 ** 10)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("softcap", [0.5, 30.0, 1e4, 1e7])
def test_softcaps_near_to_and_far_above_the_scores(dtype, cache, softcap):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    k, v = (torch.randn(496, 64, generator=g, device="cuda") for _ in range(2))
    q = (torch.randn(4, 64, generator=g, device="cuda") * 2).to(TORCH[dtype])
    _check(q, _pages(k, cache), _pages(v, cache), f"{dtype} {cache}", scale=0.25, softcap=softcap)


@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_nan_passes_a_softcap(dtype, cache):
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    k, v = (_pages(torch.randn(96, 64, generator=g, device="cuda"), cache) for _ in range(2))
    k.view(torch.uint8 if cache == "e4m3" else k.dtype)[2, 3] = 0x7F if cache == "e4m3" else math.nan
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    q = torch.ones(1, 4, 64, device="cuda", dtype=TORCH[dtype])
    for n, nan in ((96, True), (35, False)):   # token 35 is the NaN
        out, lse = ar.ar_paged_attention(q, k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"), softcap=20.0, return_lse=True)
        assert bool((out.isnan() == nan).all()) and bool((lse.isnan() == nan).all())
