"""Positions on several axes, compacting accepted drafts and copying pages on the GPU against plain loops, and a decoding step with
drafted tokens that uses all of them."""
import math
import random

import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build
from tests import drafts_model as model
from tests import kv_cache_model
from tests.drafts_model import Cache, bits
from tests.kv_cache_model import TORCH, U32, by_token, check, half_step

pytestmark = pytest.mark.gpu
F = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
TYPES = [("fp32", "fp32"), ("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "e4m3"), ("bf16", "e4m3")]


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    _build.build()
    ar.lib()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


# ------------------------------------------------------------------ positions on several axes

def _turned(x, positions, pair_axis, freq, interleaved, scale):
    """x [rows, heads, dim] in 64 bits; positions [axes, rows]."""
    half = freq.numel()
    angle = (positions.double()[torch.tensor(pair_axis, device="cuda", dtype=torch.long)].T * freq.double())[:, None]
    c, s = torch.cos(angle) * scale, torch.sin(angle) * scale
    out = x.clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return out


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim,rotary,axes,order,interleaved", [
    (128, 128, 3, "blocks", False), (128, 128, 3, "turns", True), (64, 32, 2, "turns", False), (80, 40, 4, "blocks", True), (24, 6, 3, "turns", False),
    (128, 64, 1, "blocks", False), (256, 256, 4, "any", True)])
def test_positions_on_several_axes(dtype, cache, dim, rotary, axes, order, interleaved):
    news, lengths = [3, 0, 20, 1], [9, 4, 20, 33]
    scales = (0.05, 0.02) if cache == "e4m3" else (1.0, 1.0)
    c = Cache(lengths, 2, dim, 16, cache, "NHD", 3, scales)
    start = [1, 4, 4, 24, 25]   # a row of padding before, two behind
    rows = 27
    qkv = _randn(5, rows, 6 + 4, dim).to(F[dtype])
    q, k, v = qkv.split([6, 2, 2], 1)
    half = rotary // 2
    r = random.Random(7)
    pair_axis = {"blocks": [j * axes // half for j in range(half)], "turns": [j % axes for j in range(half)],
                 "any": [r.randrange(axes) for _ in range(half)]}[order]
    g = torch.Generator(device="cuda").manual_seed(2)
    wide = torch.randint(-2000, 100000, (axes, rows + 5), generator=g, device="cuda", dtype=torch.int32)
    positions = wide[:, :rows]   # rows further apart than they are long
    freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
    before = [bits(x).clone() for x in (c.k, c.v)]
    out = torch.full((rows, 6, dim), 7.0, dtype=F[dtype], device="cuda")
    got = ar.ar_kv_append(c.k, c.v, c.table, c.n, k, v, q=q, q_out=out, seq_start=_ints(start), positions=positions, pair_axis=pair_axis,
                          inv_freq=freq, interleaved=interleaved, rotary_scale=1.25, **c.kw)
    assert got is out
    mine = slice(start[0], start[-1])
    turn = lambda x: _turned(x.double(), positions, pair_axis, freq, interleaved, 1.25)  # noqa: E731
    # cosine and sine in fp32 (2 steps each), two products and a sum, and the angle's own error, below 2^-40 here
    room = lambda x: 12 * U32 * 1.25 * 2 * x.double().abs().amax(-1, keepdim=True) + 0 * x.double()  # noqa: E731
    want = turn(q)
    check(out[mine], want[mine], (room(q) + half_step(want, F[dtype]))[mine], "q")
    assert bool((out[: start[0]] == 7).all()) and bool((out[start[-1]:] == 7).all())
    keys, values, r_k = turn(k) / scales[0], v.double() / scales[1], room(k) / scales[0]
    if cache == "e4m3":
        keys, values = keys.clamp(-448, 448), values.clamp(-448, 448)
    for b, n in enumerate(news):
        at = list(range(lengths[b] - n, lengths[b]))
        rows_b = slice(start[b], start[b + 1])
        if n:
            ct = TORCH[cache]
            check(c.tokens(c.k, b, at).double(), keys[rows_b], (r_k + half_step(keys, ct))[rows_b], "k")
            check(c.tokens(c.v, b, at).double(), values[rows_b], (half_step(values, ct) + 2 * U32 * values.abs())[rows_b], "v")
        old = list(range(lengths[b] - n))
        if old:
            page = c.table[b].long()[torch.tensor(old, device="cuda") // 16]
            for x, y in zip((c.k, c.v), before):
                assert torch.equal(bits(x)[page, torch.tensor(old) % 16], y[page, torch.tensor(old) % 16])


def test_one_axis_for_all_pairs_is_ar_kv_append():
    """The same bits, whichever axis holds the positions, over many rows a block too."""
    for rows in (5, 3000):
        a, b = (Cache([rows], 1, 128, 64, "bf16", "NHD", 3) for _ in range(2))
        qkv = _randn(5, rows, 4, 128).bfloat16()
        q, k, v = qkv.split([2, 1, 1], 1)
        freq = (10000.0 ** (-torch.arange(64, device="cuda") / 64)).float()
        pos = torch.randint(0, 1 << 20, (rows,), device="cuda", dtype=torch.int32)
        start = _ints([0, rows])
        x = ar.ar_kv_append(a.k, a.v, a.table, a.n, k, v, q=q, seq_start=start, positions=pos, inv_freq=freq)
        other = torch.stack([pos.flip(0), pos, torch.zeros_like(pos)])
        y = ar.ar_kv_append(b.k, b.v, b.table, b.n, k, v, q=q, seq_start=start, positions=other, pair_axis=[1] * 64, inv_freq=freq)
        assert torch.equal(x, y)
        assert torch.equal(a.k.view(torch.int16), b.k.view(torch.int16)) and torch.equal(a.v.view(torch.int16), b.v.view(torch.int16))


def test_positions_on_axes_in_a_captured_step():
    c = Cache([8, 3], 1, 64, 16, "fp16", "NHD", 3)
    q, k, v = (_randn(s, 2, 1, 64).half() for s in (1, 2, 3))
    freq = torch.ones(32, device="cuda")
    pos = _ints([[1, 2], [3, 4]])
    out = torch.empty_like(q)
    axis = [0] * 16 + [1] * 16
    call = lambda: ar.ar_kv_append(c.k, c.v, c.table, c.n, k, v, q=q, q_out=out, positions=pos, pair_axis=axis, inv_freq=freq)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    axis[:] = [1] * 32   # the list is read during the call only
    pos.copy_(_ints([[5, 6], [7, 8]]))
    graph.replay()
    torch.cuda.synchronize()
    want = _turned(q.double(), pos, [0] * 16 + [1] * 16, freq, False, 1.0)
    check(out, want, 24 * U32 * q.double().abs().amax() + half_step(want, torch.float16), "q")


# ------------------------------------------------------------------ compacting

def _kept_of(row, n):
    got, before = [], -1
    for x in row:
        if x <= before or x >= n:
            break
        got.append(x)
        before = x
    return got


def _compacted(cache, layers, kept, news):
    """The layers' pages and lengths after the moves, one token at a time; row bits."""
    pages = [bits(p).clone() for p in layers]
    table, lengths = cache.table.tolist(), []
    for b, length in enumerate(cache.lengths):
        n, context = news[b], length - news[b]
        if n <= 0 or context < 0:
            lengths.append(length)
            continue
        mine = _kept_of(kept[b], n)
        lengths.append(context + len(mine))
        for j, x in enumerate(mine):
            ends = []
            for at in (context + x, context + j):
                ok = at < len(table[b]) * cache.page and 0 <= table[b][at // cache.page] < layers[0].shape[0]
                ends.append((table[b][at // cache.page], at % cache.page) if ok else None)
            if x != j and None not in ends:
                for p in pages:
                    t = by_token(p, cache.layout)
                    t[ends[1]] = t[ends[0]].clone()
    return pages, lengths


def _same_bits(a, b):
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


@pytest.mark.parametrize("cache", ["fp32", "fp16", "bf16", "e4m3"])
@pytest.mark.parametrize("layers,heads,dim,page,layout,joint", [
    (1, 1, 128, 16, "NHD", False), (3, 2, 80, 17, "HND", True), (2, 3, 5, 4, "NHD", False), (40, 1, 64, 16, "HND", False), (128, 1, 8, 2, "NHD", True)])
def test_compacting(cache, layers, heads, dim, page, layout, joint):
    news, context = [7, 1, 0, 20, 3, 150], [0, 31, 4, 15, 16, 2]
    lengths = [c + n for c, n in zip(context, news)]
    caches = [Cache(lengths, heads, dim, page, cache, layout, 3, joint=joint) for _ in range(layers)]
    c = caches[0]
    for i, x in enumerate(caches):   # each layer's values are its own
        for p in (x.k, x.v):
            p.copy_((_randn(50 + i, *p.shape) * 3).to(p.dtype))
    r = random.Random(layers)
    most = 140
    kept = [[1, 2, 5, 6], [0], [], [0, 1, 2, 3, 4], [2], sorted(r.sample(range(150), 137))]
    kept = [x + [-1] * (most - len(x)) for x in kept]
    kept[3][5:9] = [9, 9, 10, 11]   # ends at the second 9
    wide = torch.full((len(news), most + 3), 0, dtype=torch.int32)
    wide[:, :most] = torch.tensor(kept)
    start = [sum(news[:b]) for b in range(len(news) + 1)]
    flat = [x.k for x in caches] + [x.v for x in caches]
    want, lengths_after = _compacted(c, flat, kept, news)
    got = ar.ar_kv_compact([x.k for x in caches], [x.v for x in caches], c.table, c.n, wide.cuda()[:, :most], seq_start=_ints(start), layout=layout)
    assert got.tolist() == lengths_after and got.dtype == torch.int32
    assert c.n.tolist() == lengths
    for x, y in zip(flat, want):
        assert _same_bits(bits(x), y)


@pytest.mark.parametrize("cache,page", [("bf16", 16), ("e4m3", 3)])
def test_compacting_idle_sequences_bad_pages_and_lists(cache, page):
    """Lengths below the drafts and beyond the table, entries that are no page, lists that begin with their end or name too much."""
    lengths = [3, 0, 40, 30, 30, 30, 30]
    c = Cache(lengths, 2, 64, page, cache, "NHD", 3)
    c.table[3, 20 // page] = -1
    c.table[4, 29 // page] = c.k.shape[0] + 5
    c.lengths = [3, -4, 40 + 3, 30, 30, 30, 2 ** 31 - 1]
    n = 12
    kept = [[0, 2, 3], [0, 1, 2], [1, 5, 11], [3, 7, 11], [2, 4, 11], [-1, 0, 1], [1, 2, 3]]
    flat = [c.k, c.v]
    want, lengths_after = _compacted(c, flat, kept, [n] * 7)
    out = torch.full((7,), 77, dtype=torch.int32, device="cuda")
    got = ar.ar_kv_compact(c.k, c.v, c.table, _ints(c.lengths), _ints(kept), drafted=n, new_lengths=out)
    assert got.data_ptr() == out.data_ptr() and out.tolist() == lengths_after
    assert all(_same_bits(bits(x), y) for x, y in zip(flat, want))
    before = [bits(x).clone() for x in flat]
    for most, drafted in ((0, 3), (2, 0)):   # nothing to keep, nothing drafted
        got = ar.ar_kv_compact(c.k, c.v, c.table, _ints([30] * 7), torch.zeros(7, most, dtype=torch.int32, device="cuda"), drafted=drafted)
        assert got.tolist() == [30 - drafted] * 7
    assert all(_same_bits(bits(x), y) for x, y in zip(flat, before))


def test_compacting_in_a_captured_step():
    c = Cache([40, 50], 1, 128, 16, "bf16", "NHD", 3)
    kept = _ints([[1, 3, -1], [0, 2, 4]])
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    call = lambda: ar.ar_kv_compact(c.k, c.v, c.table, c.n, kept, drafted=5, new_lengths=out)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rows in ([[1, 3, -1], [0, 2, 4]], [[4, -1, -1], [-1, 2, 3]]):
        kept.copy_(_ints(rows))
        want, lengths = _compacted(c, [c.k, c.v], rows, [5, 5])
        graph.replay()
        torch.cuda.synchronize()
        assert out.tolist() == lengths and _same_bits(c.k, want[0]) and _same_bits(c.v, want[1])


# ------------------------------------------------------------------ copying pages

def _copied(pages, src, dst):
    count = pages[0].shape[0]
    moves = [(s, d) for s, d in zip(src, dst) if s != d and 0 <= s < count and 0 <= d < count]
    got = [p.clone() for p in pages]
    for i, (s, d) in enumerate(moves):
        if any(d2 == s for _, d2 in moves) or any(d2 == d for _, d2 in moves[i + 1:]):
            continue
        for x, y in zip(got, pages):
            x[d] = y[s]
    return got


@pytest.mark.parametrize("cache", ["fp32", "fp16", "bf16", "e4m3"])
@pytest.mark.parametrize("layers,shape,joint", [(1, (40, 16, 1, 128), False), (3, (40, 2, 17, 80), True), (2, (40, 3, 5, 7), False),
                                                (16, (300, 4, 2, 64), False), (128, (9, 1, 1, 3), True)])
def test_copying_pages(cache, layers, shape, joint):
    pages = []
    for i in range(2 * layers):
        x = (_randn(i, shape[0], 2, *shape[1:]) * 3).to(TORCH[cache])
        pages.append(x[:, 1] if joint else x[:, 1].contiguous())
    r = random.Random(layers)
    order = r.sample(range(shape[0]), shape[0])
    n = shape[0] // 3
    src, dst = [order[r.randrange(n)] for _ in range(n)], order[n:2 * n]
    if shape[0] > 20:   # a page twice, none, the same, two with one destination, a chain, a swap
        src += [-1, shape[0], src[0], dst[2], order[-1], order[-1], dst[3], order[-3], order[-4], 5]
        dst += [order[-2], order[-2], -2 ** 31, dst[2], dst[0], dst[0], order[-2], order[-4], order[-3], 2 ** 31 - 1]
    want = _copied([bits(p) for p in pages], src, dst)
    ar.ar_kv_copy_pages(pages[:layers], pages[layers:], _ints(src), _ints(dst))
    for x, y in zip(pages, want):
        assert _same_bits(bits(x), y)


def test_copying_many_small_pages_and_views_of_heads():
    """More pairs than a block has threads; pages whose heads lie apart, whose tokens do, and both."""
    x = _randn(1, 5000, 2, 3, 8)
    want = _copied([x, x], list(range(0, 2000)), list(range(2500, 4500)))[0]
    y = x.clone()
    ar.ar_kv_copy_pages(x, y, torch.arange(2000, device="cuda", dtype=torch.int32), torch.arange(2500, 4500, device="cuda", dtype=torch.int32))
    assert torch.equal(x, want) and torch.equal(y, want)
    big = _randn(2, 30, 6, 8, 40).half()
    for view in (lambda t: t[:, :, ::2], lambda t: t[:, ::2], lambda t: t[:, ::3, 1::3], lambda t: t.transpose(1, 2), lambda t: t[:, :, :, 8:24],
                 lambda t: t[:, ::2, :, 3:10].transpose(1, 2)):
        a, b = big.clone(), big.clone()
        want = big.clone()
        view(want)[torch.tensor([3, 9, 20])] = view(big)[torch.tensor([1, 1, 7])]
        ar.ar_kv_copy_pages(view(a), view(b), _ints([1, 1, 7]), _ints([3, 9, 20]))
        assert torch.equal(a, want) and torch.equal(b, want)   # nothing beside the view's elements


def test_copying_in_a_captured_step():
    x, y = _randn(1, 10, 4, 2, 64).bfloat16(), _randn(2, 10, 4, 2, 64).bfloat16()
    src, dst = _ints([1, 2]), _ints([8, 9])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ar.ar_kv_copy_pages(x, y, src, dst)
    src.copy_(_ints([3, 4]))
    dst.copy_(_ints([5, -1]))
    want = _copied([x, y], [3, 4], [5, -1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,cache", TYPES)
def test_a_decoding_step_with_drafts(dtype, cache):
    """Fork, append a tree at its depths, attend, keep a path, and decode on: the same as if the path had been decoded plainly."""
    dim, heads, kv_heads, page, layers = 64, 8, 2, 16, 2
    scales = (0.05, 0.02) if cache == "e4m3" else (1.0, 1.0)
    freq = (10000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))).float()
    context, parents = 37, [-1, 0, 0, 1, 3, 2]   # two sequences, the second a fork of the first
    n = len(parents)
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    masks = model.tree_masks(n, 0)
    for i, p in enumerate(parents):
        masks[i] = (masks[p] if p >= 0 else 0) | 1 << i
    kept, path = [[0, 1, 3, 4], [0, 2]], 5
    caches = [Cache([context, context], kv_heads, dim, page, cache, "NHD", 20, scales, room=2) for i in range(layers)]
    first = caches[0]
    caches[1].k.copy_(-first.k.float())   # the same pages in every layer, with values of its own
    caches[1].v.copy_(first.v.float() / 2)
    kw = dict(k_scale=scales[0], v_scale=scales[1])
    # the fork: whole pages shared, the one being filled copied, new ones for what comes
    table = torch.full((2, 5), -1, dtype=torch.int32)
    full = context // page
    table[0, : full + 1] = first.table[0, : full + 1].cpu()
    table[1, :full] = table[0, :full]
    unused = [int(x) for x in first.table[1].tolist() if x >= 0] + first.free
    table[1, full], table[0, full + 1], table[1, full + 1] = unused[:3]
    table = table.cuda()
    ar.ar_kv_copy_pages([c.k for c in caches], [c.v for c in caches], table[0, full:full + 1].clone(), table[1, full:full + 1].clone())
    plain = [[bits(p).clone().view(p.dtype) for p in (c.k, c.v)] for c in caches]   # for decoding plainly
    q, k, v = (_randn(30 + i, 2 * n, h, dim).to(F[dtype]) for i, h in enumerate((heads, kv_heads, kv_heads)))
    start, lengths = _ints([0, n, 2 * n]), _ints([context + n] * 2)
    positions = _ints([context + d for d in depth] * 2)
    axes = torch.stack([positions, torch.zeros_like(positions)])   # one axis in use: the same as plain positions
    got = []
    for c in caches:
        turned = ar.ar_kv_append(c.k, c.v, table, lengths, k, v, q=q, seq_start=start, positions=axes, pair_axis=[0] * (dim // 2), inv_freq=freq, **kw)
        got.append(ar.ar_tree_attention(turned, c.k, c.v, table, lengths, mask=model.words_of(masks * 2, 1), seq_start=start, **kw))
    wide = _ints([x + [-1] * (n - len(x)) for x in kept])
    after = ar.ar_kv_compact([c.k for c in caches], [c.v for c in caches], table, lengths, wide, drafted=n)
    assert after.tolist() == [context + 4, context + 2]
    for b in range(2):
        rows = [b * n + x for x in kept[b]]
        for i, (c, (pk, pv)) in enumerate(zip(caches, plain)):
            for step, row in enumerate(rows):   # token after token
                one = slice(row, row + 1)
                length = _ints([context + step + 1])
                turned = ar.ar_kv_append(pk, pv, table[b:b + 1], length, k[one], v[one], q=q[one], inv_freq=freq, **kw)
                alone, lse = ar.ar_paged_attention(turned, pk, pv, table[b:b + 1], length, return_lse=True, **kw)
                # two kernels' roundings of the same weighted mean of values of at most 5 times their scale's steps
                room = 2 * half_step(alone.double(), F[dtype]) + 2.0 ** -14 * 5
                check(got[i][row], alone[0].double(), room[0], f"layer {i} row {row}")
            at = torch.arange(context + len(rows), device="cuda")
            place = table[b].long()[at // page], at % page
            assert _same_bits(bits(c.k)[place], bits(pk)[place]) and _same_bits(bits(c.v)[place], bits(pv)[place])
