"""ar_tree_attention where a result shows the bits of what it is made of: weights against values that cancel, weights and elements of
queries far below the largest, softcaps far above the scores, tiles told apart by their values, and batches of more sequences than a
block has threads.

The bounds are relative to sum p |v| / sum p and follow the kernels' sums, u = 2^-24 being half a step of fp32:
  - a score: its dot product of `terms` numbers that are not 0, each product and sum off by 2 u at the most, the factor of base 2 and
    the exponential 8 u max(1, |s|), a softcap 16 u |s| more (derived in kv_cache_model.attention); a factor e^(+-delta) of a weight
    that each of sum p v and sum p takes: 4 delta, as there with the reference's own.
  - a weight is held in fp32 for fp32 caches, and else in two 16-bit numbers, a rounding and the rounding of what it leaves: bf16 2^-16
    of it, fp16 2^-22; where fp16's second number ends, 2^-25, of weights whose reference's is 2^11: 2^-36 of a weight that the sum holds.
  - sums: fp32 goes token after token through its block's tiles, a rounding each, and one for a moved reference; a product of the tensor
    core takes 16 tokens at once, and is taken to be off by eight; parts are joined by eight warps, then eight in a row."""
import math

import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build
from tests import drafts_model as model
from tests.drafts_model import Cache
from tests.kv_cache_model import TORCH, U32, check, half_step

pytestmark = pytest.mark.gpu

TYPES = [("fp32", "fp32"), ("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "e4m3"), ("bf16", "e4m3")]
BLOCKS = 152


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    _build.build()
    ar.lib()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(x, dtype, page=16):
    """[tokens, dim] as pages of one head, zeros behind."""
    wide = torch.zeros(-(-x.shape[0] // page) * page, x.shape[1], device="cuda")
    wide[: x.shape[0]] = x
    return wide.view(-1, page, 1, x.shape[1]).to(TORCH[dtype])


def _sums(cache_dtype, dim, tokens):
    """Roundings of a sum over a sequence's tokens, of one item that all blocks share."""
    tile = 32 if cache_dtype == "fp32" else 128 if dim <= 128 else 64
    tiles = -(-tokens // tile)
    mine = -(-tiles // BLOCKS)   # of a block
    parts = min(tiles, 2 * BLOCKS)
    a_tile = min(tokens, tile) + 1 if cache_dtype == "fp32" else 2 * -(-min(tokens, tile) // 16) * 8 + 1
    return mine * a_tile + (parts // 8 + 16 if parts > 1 else 0) + 4


def _attend(q, k, v, tokens, *, scale, softcap=0.0, terms=None, what="", page=16):
    """q [rows, heads, dim] are the last tokens of one sequence of `tokens`, and all see all of it; checks against 64 bits."""
    dtype, cache_dtype = ({t: n for n, t in TORCH.items()}[x.dtype] for x in (q, k))
    rows, heads, dim = q.shape
    table = torch.arange(k.shape[0], dtype=torch.int32, device="cuda")[None]
    mask = torch.full((rows, -(-rows // 64)), -1, dtype=torch.int64, device="cuda")
    out, lse = ar.ar_tree_attention(q, k, v, table, _ints([tokens]), mask=mask, scale=scale, softcap=softcap, return_lse=True)
    kd, vd, qd = (x.double() for x in (k.view(-1, dim)[:tokens], v.view(-1, dim)[:tokens], q))
    s = torch.einsum("rhd,jd->rhj", qd, kd) * scale
    mass = torch.einsum("rhd,jd->rhj", qd.abs(), kd.abs()) * abs(scale)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    delta = 2 * ((dim if terms is None else terms) + 2) * U32 * mass + (8 * s.abs().clamp(min=1) + (16 * s.abs() if softcap else 0)) * U32
    if dtype == "bf16" and cache_dtype == "e4m3":   # queries scaled to fp16: elements are off by 2^-39 of the largest
        delta = delta + 2.0 ** -39 * abs(scale) * qd.abs().amax(2)[..., None] * kd.abs().sum(1)
    delta = delta.amax(2, keepdim=True)
    p = torch.softmax(s, 2)
    ref, ref_lse = p @ vd, torch.logsumexp(s, 2)
    half16 = {"fp32": 0.0, "bf16": 2.0 ** -16}.get(cache_dtype, 2.0 ** -22)
    sums = 2 * _sums(cache_dtype, dim, tokens) * U32
    room = (p @ vd.abs()) * (4 * delta + half16 + 2 * sums) + 6 * U32 * ref.abs()
    if cache_dtype in ("fp16", "e4m3"):
        room = room + 2.0 ** -36 * vd.abs().sum(0)
    check(out, ref, room + half_step(ref, out.dtype), f"{what} out")
    check(lse, ref_lse, 2 * delta[..., 0] + 2 * sums + 4 * U32 * (1 + ref_lse.abs()), f"{what} lse")


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim,rows,heads", [(16, 1, 8), (128, 3, 8), (64, 20, 16), (256, 2, 4)])
def test_two_tokens_of_nearly_one_weight(dtype, cache, dim, rows, heads):
    """Values 1 and -1 leave tanh(s / 2) of two weights' bits: what the result rounds to is far finer than what a weight is held in."""
    k, v = torch.zeros(2, dim, device="cuda"), torch.ones(2, dim, device="cuda")
    k[1, 0], v[1] = 1.0, -1.0
    q = torch.zeros(rows, heads, dim, device="cuda")
    q[..., 0] = (torch.linspace(-1, 1, rows * heads, device="cuda") * 2.0 ** -8 + 2.0 ** -17).view(rows, heads)
    q = q.to(TORCH[dtype])
    tokens = rows   # the rows' own tokens are the last: two that weigh, and no more
    if rows <= 2:
        _attend(q, _pages(k, cache), _pages(v, cache), 2, scale=1.0, terms=1, what=f"{dtype} {cache}")
    else:   # the others alike in pairs, which cancel exactly
        wide_k, wide_v = k.repeat(-(-rows // 2), 1), v.repeat(-(-rows // 2), 1)
        tokens = wide_k.shape[0]
        _attend(q, _pages(wide_k, cache), _pages(wide_v, cache), tokens, scale=1.0, terms=1, what=f"{dtype} {cache}")


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("rows,heads", [(1, 4), (5, 16), (20, 8)])
@pytest.mark.parametrize("pairs", [1, 50])
@pytest.mark.parametrize("dim", [16, 128])
def test_weights_keep_their_bits_against_values_that_cancel(dtype, cache, rows, heads, pairs, dim):
    """Tokens in pairs of values -1 and n, the latter weighing about 1 / n: where n is the head's, the result is what is left of them."""
    pairs = max(pairs, -(-rows // 2))
    n = torch.tensor([3.0, 5.0, 7.0, 9.0, 11.0, 13.0, 15.0, 10.0], device="cuda")
    k, v = torch.zeros(pairs, 2, dim, device="cuda"), torch.full((pairs, 2, dim), -1.0, device="cuda")
    k[:, 1, 0] = -1.0
    v[:, 1] = n.repeat(dim // 8)
    q = torch.zeros(rows, heads, dim, device="cuda")
    q[..., 0] = n.log().repeat(2)[:heads]
    _attend(q.to(TORCH[dtype]), _pages(k.view(-1, dim), cache), _pages(v.view(-1, dim), cache), 2 * pairs, scale=1.0, terms=1, what=f"{dtype} {cache}")


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("rows", [1, 16, 40])
def test_many_weights_far_below_the_largest(dtype, cache, rows):
    """A few tokens whose weights are e^18 times the others' and whose values are 0: the result is all others'."""
    k, v = torch.zeros(4000, 64, device="cuda"), torch.full((4000, 64), 96.0, device="cuda")
    for j in (0, 16, 32, 48, 64, 96):
        k[j], v[j] = 18 / 256, 0.0
    q = torch.full((rows, 4, 64), 4.0, device="cuda").to(TORCH[dtype])
    _attend(q, _pages(k, cache), _pages(v, cache), 4000, scale=1.0, what=f"{dtype} {cache}")


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_query_elements_far_below_the_largest(dtype, cache):
    """One element is 2^26 times the rest, where every key is 0: the scores are the rest's."""
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(496, 64, generator=g, device="cuda") for _ in range(2))
    k[:, 0] = 0.0
    q = torch.randn(5, 4, 64, generator=g, device="cuda").to(TORCH["bf16"]).float() * 2.0 ** -12
    q[..., 0] = 2.0 ** 14
    _attend(q.to(TORCH[dtype]), _pages(k, cache), _pages(v, cache), 496, scale=2.0 ** 10, what=f"{dtype} {cache}")


@pytest.mark.parametrize("dtype,cache", [p for p in TYPES if p[0] != "fp16"])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_large_queries_and_scales_of_keys_that_are_zero(dtype, cache, softcap):
    """The query's size times the scale is over fp32's range, the scores are 0: every token weighs the same."""
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = torch.zeros(37, 64, device="cuda"), torch.randn(37, 64, generator=g, device="cuda")
    q = torch.full((3, 4, 64), 2.0 ** 120, device="cuda").to(TORCH[dtype])
    q[1, 2] = -q[1, 2]
    _attend(q, _pages(k, cache), _pages(v, cache), 37, scale=2.0 ** 40, softcap=softcap, what=f"{dtype} {cache}")


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("softcap", [0.5, 30.0, 1e4, 1e7, 1e20, 1e30])
def test_softcaps_near_to_and_far_above_the_scores(dtype, cache, softcap):
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(496, 64, generator=g, device="cuda") for _ in range(2))
    q = (torch.randn(7, 4, 64, generator=g, device="cuda") * 2).to(TORCH[dtype])
    _attend(q, _pages(k, cache), _pages(v, cache), 496, scale=0.25, softcap=softcap, what=f"{dtype} {cache}")


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_nan_passes_a_softcap(dtype, cache):
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = (_pages(torch.randn(96, 64, generator=g, device="cuda"), cache) for _ in range(2))
    k.view(torch.uint8 if cache == "e4m3" else k.dtype)[2, 3] = 0x7F if cache == "e4m3" else math.nan   # token 35
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    q = torch.ones(2, 4, 64, device="cuda", dtype=TORCH[dtype])
    for n, nan in ((96, True), (35, False)):
        out, lse = ar.ar_tree_attention(q, k, v, table, _ints([n]), softcap=20.0, return_lse=True)
        assert bool((out.isnan() == nan).all()) and bool((lse.isnan() == nan).all())


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim,tokens,rows,heads", [(128, 20011, 13, 8), (64, 40007, 2, 8), (128, 50001, 40, 4), (256, 30011, 6, 8)])
def test_long_contexts_miss_no_tile_and_take_none_twice(dtype, cache, dim, tokens, rows, heads):
    """Each 32 tokens have a value of 1 in one column, in turn: a column of the result is the weight of its tokens, some hundred of them,
    and a tile more or less shows in it whole."""
    g = torch.Generator(device="cuda").manual_seed(8)
    at = torch.arange(tokens, device="cuda")
    v = torch.zeros(tokens, dim, device="cuda")
    v[at, at // 32 % dim] = 1.0
    k = torch.randn(tokens, dim, generator=g, device="cuda")
    q = (torch.randn(rows, heads, dim, generator=g, device="cuda") / 2).to(TORCH[dtype])
    _attend(q, _pages(k, cache), _pages(v, cache), tokens, scale=dim ** -0.5, what=f"{dtype} {cache}")


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim,batch,page", [(64, 1100, 16), (128, 700, 17), (192, 800, 8)])
def test_more_sequences_than_a_block_has_threads(dtype, cache, dim, batch, page):
    """Each thread of the line's scan has several sequences, some without new tokens, some without any."""
    g = torch.Generator().manual_seed(9)
    news = torch.randint(0, 3, (batch,), generator=g).tolist()
    context = torch.randint(0, 40, (batch,), generator=g).tolist()
    news[0] = news[-1] = news[batch // 2] = 0
    context[5] = 300
    scales = (0.05, 0.02) if cache == "e4m3" else (1.0, 1.0)
    c = Cache([a + b for a, b in zip(context, news)], 2, dim, page, cache, "NHD", 3, scales)
    starts = [sum(news[:b]) for b in range(batch + 1)]
    q = torch.randn(starts[-1] + 2, 4, dim, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(TORCH[dtype])
    masks = [m for b, n in enumerate(news) for m in model.tree_masks(n, b)] + [0, 0]
    for use in (masks, None):
        out, lse = torch.full_like(q, 7.0), torch.full((q.shape[0], 4), 7.0, device="cuda")
        ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, mask=None if use is None else model.words_of(use, 1), seq_start=_ints(starts), out=out, lse=lse, **c.kw)
        ref, ref_lse, e_out, e_lse = model.attention(q, c, starts, use, scale=dim ** -0.5)
        mine = ~ref_lse.isnan()
        check(lse[mine], ref_lse[mine], e_lse[mine], "lse")
        check(out[mine], ref[mine], e_out[mine] + half_step(ref[mine], TORCH[dtype]), "out")
        assert bool((out[~mine] == 7).all()) and bool((lse[~mine] == 7).all()) and int((~mine).sum()) == 8


def test_fp32_weights_stay_in_32_bits():
    """Two tokens, values 1 and -1, scores up to a third: weights cut to two 16-bit numbers would be 2^-19 off.  In units of u: the factor
    of base 2 and its product with the score, 2 |s|; the exponential, 2 steps or 4; of a weight that is half of the sum or less.  The
    difference, the sum, the division and the product round the result by 4 of itself."""
    q = torch.zeros(2, 64, 64, device="cuda")
    q[..., 0] = (torch.linspace(-1, 1, 128, device="cuda") / 3).view(2, 64)
    k, v = torch.zeros(2, 64, device="cuda"), torch.ones(2, 64, device="cuda")
    k[1, 0], v[1] = 1.0, -1.0
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    mask = torch.full((2, 1), -1, dtype=torch.int64, device="cuda")
    out = ar.ar_tree_attention(q, _pages(k, "fp32"), _pages(v, "fp32"), table, _ints([2]), mask=mask, scale=1.0)
    s = q[..., :1].double()
    ref = -torch.tanh(s / 2).expand(-1, -1, 64)
    check(out, ref, U32 * ((2 * s.abs() + 4) / 2 * (1 + ref.abs()) + 5 * ref.abs()), "out")
