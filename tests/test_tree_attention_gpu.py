"""ar_tree_attention on the GPU against its formula in 64 bits: types, head sizes, layouts, pages, trees, chains, masks of no order,
windows, padding, idle sequences, values that a row must not see, and its place in a decoding step."""
import math

import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build
from tests import drafts_model as model
from tests.drafts_model import Cache
from tests.kv_cache_model import TORCH, by_token, check, half_step

pytestmark = pytest.mark.gpu
F = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    _build.build()
    ar.lib()


def _queries(rows, heads, dim, dtype, seed=1, std=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(rows, heads, dim, generator=g, device="cuda") * std).to(F[dtype])


def _starts(news):
    return [sum(news[:b]) for b in range(len(news) + 1)]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _compare(out, lse, want, dtype):
    ref, ref_lse, e_out, e_lse = want
    mine = ~ref_lse.isnan()
    assert bool(mine.any())
    check(lse[mine], ref_lse[mine], e_lse[mine], "lse")
    check(out[mine], ref[mine], e_out[mine] + half_step(ref[mine], F[dtype]), "out")
    return mine


def _case(dtype, cache_dtype, dim, heads, kv_heads, page, layout, context, news, kind="tree", window=0, softcap=0.0, seed=3, scale=None, std=1.5,
          joint=False, lead=0, tail=0):
    scales = (0.05, 0.02) if cache_dtype == "e4m3" else (1.0, 1.0)
    cache = Cache([c + n for c, n in zip(context, news)], kv_heads, dim, page, cache_dtype, layout, seed, scales, joint=joint)
    starts = [lead + x for x in _starts(news)]
    rows = starts[-1] + tail
    q = _queries(rows, heads, dim, dtype, seed + 1, std)
    masks = None
    if kind != "chain":
        masks = [0] * lead + [m for b, n in enumerate(news) for m in model.tree_masks(n, 10 * seed + b, kind)] + [0] * tail
    words = max(1, -(-max(news) // 64))
    out = torch.full_like(q, 7.0)
    lse = torch.full((rows, heads), 7.0, device="cuda")
    scale = dim ** -0.5 if scale is None else scale
    ar.ar_tree_attention(q, cache.k, cache.v, cache.table, cache.n, mask=None if masks is None else model.words_of(masks, words),
                         seq_start=_ints(starts), scale=scale, window=window, softcap=softcap, out=out, lse=lse, **cache.kw)
    mine = _compare(out, lse, model.attention(q, cache, starts, masks, scale=scale, window=window, softcap=softcap), dtype)
    assert bool((out[~mine] == 7).all()) and bool((lse[~mine] == 7).all())   # padding is left as it was
    return cache, q, starts, masks, out, lse


TYPES = [("fp32", "fp32"), ("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "e4m3"), ("bf16", "e4m3")]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,kv_heads,page,layout", [(8, 1, 16, "NHD"), (12, 3, 17, "HND"), (40, 2, 64, "NHD")])
def test_types_and_head_sizes(dtype, cache, dim, heads, kv_heads, page, layout):
    _case(dtype, cache, dim, heads, kv_heads, page, layout, [0, 1, 130, 300], [5, 1, 9, 3])


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
@pytest.mark.parametrize("window,softcap", [(0, 0.0), (1, 0.0), (3, 5.0), (100, 0.0), (1000, 20.0)])
def test_masks_windows_and_caps(dtype, cache, kind, window, softcap):
    _case(dtype, cache, 64, 6, 2, 24, "HND", [0, 2, 63, 190, 129], [7, 3, 70, 20, 64], kind, window, softcap)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim,group,new", [(128, 8, 1), (128, 8, 16), (128, 8, 17), (64, 16, 40), (128, 1, 129), (192, 4, 70), (256, 12, 30), (128, 5, 130)])
def test_numbers_of_rows(dtype, cache, dim, group, new):
    """Blocks of rows full, one over, and several, on one key-value head and on two."""
    _case(dtype, cache, dim, group, 1, 16, "NHD", [200], [new])
    _case(dtype, cache, dim, 2 * group, 2, 32, "HND", [150, 10], [new, 1], "any")


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("context,new", [(5000, 4), (20011, 13), (3000, 64)])
def test_long_contexts_are_split_and_joined(dtype, cache, context, new):
    _case(dtype, cache, 128, 8, 1, 64, "NHD", [context], [new])


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_ragged_batches(dtype, cache):
    r = torch.Generator().manual_seed(5)
    context = torch.randint(0, 700, (40,), generator=r).tolist()
    news = torch.randint(0, 24, (40,), generator=r).tolist()   # some sequences have no new token
    news[3] = news[20] = 0
    for kind in ("tree", "chain"):
        _case(dtype, cache, 128, 16, 4, 16, "NHD", context, news, kind, lead=2, tail=3)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("page,layout,joint", [(1, "NHD", False), (3, "HND", True), (128, "HND", False), (200, "NHD", True)])
def test_pages_of_any_size_and_halves_of_one_buffer(dtype, cache, page, layout, joint):
    _case(dtype, cache, 96, 4, 2, page, layout, [0, 99, 257], [6, 2, 11], joint=joint)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("n", [1, 200, 700])
def test_chunks_of_a_prompt(dtype, cache, n):
    """Without a mask a row sees the new tokens up to its own, whatever their number; with a window only the last."""
    _case(dtype, cache, 64, 4, 1, 16, "NHD", [33], [n], "chain")
    _case(dtype, cache, 64, 4, 2, 16, "NHD", [90], [n], "chain", window=50)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_the_same_number_of_rows_without_seq_start(dtype, cache):
    news, context = [6] * 5, [3, 0, 77, 140, 20]
    _, q, starts, masks, out, lse = _case(dtype, cache, 128, 8, 2, 16, "NHD", context, news)
    c = Cache([a + b for a, b in zip(context, news)], 2, 128, 16, cache, "NHD", 3, (0.05, 0.02) if cache == "e4m3" else (1.0, 1.0))
    got, got_lse = ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, mask=model.words_of(masks, 1), return_lse=True, **c.kw)
    assert torch.equal(got, out) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_one_new_token_is_ar_paged_attention(dtype, cache):
    lengths = [1, 40, 300, 0, 77]
    c = Cache(lengths, 2, 128, 16, cache, "NHD", 8, (0.05, 0.02) if cache == "e4m3" else (1.0, 1.0))
    q = _queries(5, 16, 128, dtype)
    one, one_lse = ar.ar_paged_attention(q, c.k, c.v, c.table, c.n, return_lse=True, **c.kw)
    out, lse = ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, return_lse=True, **c.kw)
    want = model.attention(q, c, list(range(6)), None, scale=128 ** -0.5)
    # an idle sequence (length 0) has no token, the row's own among them
    for o, s in ((one, one_lse), (out, lse)):
        _compare(o, s, want, dtype)
    assert bool((lse[3] == -math.inf).all()) and bool((out[3] == 0).all())


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_values_that_a_row_does_not_see_may_be_anything(dtype, cache):
    """NaN keys and values in drafted tokens and in front of the window reach the rows that see them, and no other."""
    context, n, dim, window = 200, 8, 64, 150
    c = Cache([context + n], 2, dim, 16, cache, "NHD", 4)
    q = _queries(n, 8, dim, dtype)
    masks = [0b1, 0b11, 0b101, 0b1101, 0b10001, 0b110001, 0b1000001, 0b11000001]
    bad = {context + 2: (True, False), context + 4: (False, True), 30: (True, True), 57: (False, True)}   # (key, value) NaN
    clean = Cache([context + n], 2, dim, 16, cache, "NHD", 4)
    for j, (key, value) in bad.items():
        p, s = int(c.table[0, j // 16]), j % 16
        nan = 0x7f if cache == "e4m3" else math.nan
        if key:
            model.bits(c.k)[p, s] = nan
        if value:
            model.bits(c.v)[p, s, :, 5] = nan
    out, lse = ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, mask=model.words_of(masks, 1), window=window, return_lse=True)
    ref, ref_lse, e_out, e_lse = model.attention(q, clean, [0, n], masks, scale=dim ** -0.5, window=window)
    for i in range(n):
        sees = set(model.seen(i, n, context + n, window, masks[i]))
        keys = any(key for j, (key, _) in bad.items() if j in sees)
        values = any(value for j, (_, value) in bad.items() if j in sees)
        if keys:
            assert bool(lse[i].isnan().all()) and bool(out[i].isnan().all()), i
            continue
        check(lse[i], ref_lse[i], e_lse[i], f"lse {i}")
        cols = [d for d in range(dim) if not (values and d == 5)]
        check(out[i][:, cols], ref[i][:, cols], (e_out[i] + half_step(ref[i], F[dtype]))[:, cols], f"out {i}")
        assert bool(out[i][:, 5].isnan().all()) == values, i
    infinite = Cache([context + n], 2, dim, 16, cache, "NHD", 4)
    if cache != "e4m3":   # which has no infinity
        for j in (context + 4, 57):
            infinite.v[int(c.table[0, j // 16]), j % 16, :, 5] = -math.inf
        out = ar.ar_tree_attention(q, infinite.k, infinite.v, c.table, c.n, mask=model.words_of(masks, 1), window=window)
        for i in range(n):
            sees = set(model.seen(i, n, context + n, window, masks[i]))
            if context + 4 in sees or 57 in sees:
                assert not bool(out[i][:, 5].isfinite().any())
            else:
                check(out[i], ref[i], e_out[i] + half_step(ref[i], F[dtype]), f"out {i}")


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_idle_sequences_bad_pages_and_lengths(dtype, cache):
    """Lengths below the number of rows, above the table and below 0; entries that are no page."""
    lengths, news = [3, 0, 64, 50, 40], [5, 4, 6, 3, 2]
    c = Cache(lengths, 1, 64, 16, cache, "NHD", 6)
    c.table[3, 1] = -1
    c.table[4, 0] = c.k.shape[0]
    starts = _starts(news)
    q = _queries(starts[-1], 4, 64, dtype)
    masks = [m for b, n in enumerate(news) for m in model.tree_masks(n, b)]
    for given in ([3, 0, 64, 50, 40], [3, -5, 70, 50, 40], [3, -2 ** 31, 67, 50, 40]):
        c.lengths = given
        for use in (masks, None):
            for window in (0, 9):
                out, lse = ar.ar_tree_attention(q, c.k, c.v, c.table, _ints(given), mask=None if use is None else model.words_of(use, 1),
                                                seq_start=_ints(starts), window=window, return_lse=True)
                _compare(out, lse, model.attention(q, c, starts, use, scale=1 / 8, window=window), dtype)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("std,scale", [(30.0, 1.0), (1e-3, 1.0), (2.0, -0.3), (1.0, 0.0)])
def test_scores_far_apart_small_and_negative(dtype, cache, std, scale):
    _case(dtype, cache, 64, 4, 1, 16, "NHD", [500, 20], [9, 4], scale=scale, std=std)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_scores_that_rise_along_the_sequence(dtype, cache):
    """The running reference has to follow scores that grow tile after tile."""
    c = Cache([1500], 1, 64, 16, cache, "NHD", 9)
    at = torch.arange(1500, device="cuda")
    x = torch.zeros(1500, 1, 64, device="cuda")
    x[:, 0, 0] = at / 8.0
    stored = x.to(TORCH[cache])
    model.bits(c.k)[c.table[0].long()[at // 16], at % 16] = model.bits(stored)
    q = torch.zeros(6, 8, 64, device="cuda")
    q[..., 0] = torch.linspace(-2, 2, 48, device="cuda").view(6, 8)
    q = q.to(F[dtype])
    out, lse = ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, scale=1.0, return_lse=True)
    _compare(out, lse, model.attention(q, c, [0, 6], None, scale=1.0), dtype)


def test_trees_over_many_words():
    """More drafted tokens than a word has bits, with masks wider and narrower than they need."""
    n, context = 200, 70
    c = Cache([context + n], 1, 64, 16, "bf16", "NHD", 2)
    q = _queries(n, 2, 64, "bf16")
    masks = model.tree_masks(n, 1, "any")
    for words in (1, 3, 4, 9):
        out, lse = ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, mask=model.words_of(masks, words), return_lse=True)
        cut = [m & (1 << 64 * words) - 1 for m in masks]
        _compare(out, lse, model.attention(q, c, [0, n], cut, scale=1 / 8), "bf16")


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "e4m3")])
def test_queries_out_of_a_projection_and_given_results(dtype, cache):
    c = Cache([90, 30], 2, 64, 16, cache, "NHD", 2)
    wide = _queries(6, 24, 64, dtype)
    q = wide[:, 4:12]
    dense = q.contiguous()
    out, lse = torch.empty_like(dense), torch.empty(6, 8, device="cuda")
    work = torch.empty(ar.ar_tree_attention_workspace_size(c.k, c.v, c.table, c.n, 8, 6), dtype=torch.uint8, device="cuda")
    got = ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, out=out, lse=lse, workspace=work)
    assert got[0] is out or got[0].data_ptr() == out.data_ptr()
    want = ar.ar_tree_attention(dense, c.k, c.v, c.table, c.n)
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "e4m3")])
def test_captured_steps_follow_lengths_masks_and_tables(dtype, cache):
    lengths, news = [40, 300, 9], [4, 7, 2]
    c = Cache(lengths, 2, 128, 16, cache, "NHD", 5, room=2)
    starts = _starts(news)
    q = _queries(starts[-1], 8, 128, dtype)
    masks = [m for b, n in enumerate(news) for m in model.tree_masks(n, b)]
    mask, first = model.words_of(masks, 1), _ints(starts)
    out, lse = torch.empty_like(q), torch.empty(starts[-1], 8, device="cuda")
    work = torch.empty(ar.ar_tree_attention_workspace_size(c.k, c.v, c.table, c.n, 8, starts[-1]), dtype=torch.uint8, device="cuda")
    call = lambda: ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, mask=mask, seq_start=first, out=out, lse=lse, workspace=work)  # noqa: E731
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for change in range(3):
        if change == 1:
            c.lengths = [33, 211, 8]
            c.n.copy_(_ints(c.lengths))
        if change == 2:
            starts = [0, 1, 5, 13]
            first.copy_(_ints(starts))
            masks = [m for b in range(3) for m in model.tree_masks(starts[b + 1] - starts[b], 40 + b, "any")]
            mask.copy_(model.words_of(masks, 1))
        graph.replay()
        torch.cuda.synchronize()
        _compare(out, lse, model.attention(q, c, starts, masks, scale=128 ** -0.5), dtype)
        again = out.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)


def test_two_streams_at_once_and_another_stream_than_the_current():
    c = Cache([700, 300], 2, 128, 16, "bf16", "NHD", 5)
    q = [_queries(8, 16, 128, "bf16", s) for s in range(4)]
    want = [ar.ar_tree_attention(x, c.k, c.v, c.table, c.n) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    got = []
    for x, s in zip(q, streams):
        s.wait_stream(torch.cuda.current_stream())
        got.append([ar.ar_tree_attention(x, c.k, c.v, c.table, c.n, stream=s) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for g, w in zip(got, want) for y in g)


def test_parts_of_ranks_join():
    """Each rank has half of the context; the drafted tokens lie with the second."""
    context, n = 300, 5
    c = Cache([context + n], 1, 64, 16, "fp16", "NHD", 5)
    q = _queries(n, 4, 64, "fp16")
    whole, whole_lse = ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, return_lse=True)
    half = 160   # whole pages
    every = model.words_of([0] * n, 1)   # no drafted token: the first rank has context only
    a = ar.ar_tree_attention(q, c.k, c.v, c.table, _ints([half + n]), mask=every, return_lse=True)
    b = ar.ar_tree_attention(q, c.k, c.v, c.table[:, half // 16:].contiguous(), _ints([context - half + n]), return_lse=True)
    out, lse = ar.ar_attention_join([a[0], b[0]], [a[1], b[1]], return_lse=True)
    want = model.attention(q, c, [0, n], None, scale=1 / 8)
    check(lse, want[1], 4 * want[3] + 1e-6, "lse")
    # each part is rounded to fp16 once, the whole once more
    part = half_step(a[0].double(), torch.float16) + half_step(b[0].double(), torch.float16)
    check(out, want[0], 4 * want[2] + part + half_step(want[0], torch.float16), "out")
    _compare(whole, whole_lse, want, "fp16")


@pytest.mark.parametrize("dtype,cache,page", [("bf16", "bf16", 16), ("bf16", "bf16", 17), ("fp32", "fp32", 16), ("fp16", "e4m3", 16), ("fp16", "e4m3", 17)])
def test_pages_gigabytes_apart(dtype, cache, page):
    """Offsets in the cache that pass 32 bits: pages 1 GB apart, for the attention, compacting and copying."""
    c = Cache([3 * page - 2, page + 1], 2, 64, page, cache, "NHD", 6, scales=(0.05, 0.02) if cache == "e4m3" else (1.0, 1.0))
    q = _queries(4, 8, 64, dtype)
    want = ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, **c.kw)
    pages = c.k.shape[0]
    assert 5 <= pages <= 8
    apart = (1 << 30) // c.k.element_size()
    far = []
    for x in (c.k, c.v):
        y = torch.empty((pages - 1) * apart + x[0].numel(), dtype=x.dtype, device="cuda").as_strided(x.shape, (apart, *x.stride()[1:]))
        y.view(torch.uint8)[:] = x.view(torch.uint8)
        far.append(y)
    assert torch.equal(ar.ar_tree_attention(q, *far, c.table, c.n, **c.kw), want)
    kept = _ints([[1], [0]])
    layout = c.kw["layout"]
    news = ar.ar_kv_compact(c.k, c.v, c.table, c.n, kept, drafted=2, layout=layout)
    assert torch.equal(ar.ar_kv_compact(*far, c.table, c.n, kept, drafted=2, layout=layout), news)
    src, dst = _ints([int(c.table[0, 2])]), _ints([int(c.table[0, 0])])
    ar.ar_kv_copy_pages(c.k, c.v, src, dst)
    ar.ar_kv_copy_pages(*far, src, dst)
    for x, y in zip((c.k, c.v), far):
        assert torch.equal(x.view(torch.uint8), y.contiguous().view(torch.uint8))
