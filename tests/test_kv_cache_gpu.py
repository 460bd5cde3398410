"""The paged key-value cache calls on the GPU against their formulas in 64 bits: ar_kv_append, ar_paged_attention and
ar_attention_join, over types, layouts, strides, lengths and masks, alone and together."""
import math

import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build
from tests import kv_cache_model as model
from tests.kv_cache_model import TORCH, U32, check, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    _build.build()
    ar.lib()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


class Cache:
    """Pages filled with values, every element that no sequence owns with NaN."""

    def __init__(self, lengths, kv_heads, dim, page, dtype, layout="NHD", seed=0, joint=False, columns=0, scales=(1.0, 1.0)):
        g = _gen(seed)
        self.lengths, self.page, self.layout, self.scales = lengths, page, layout, scales
        need = [max(0, -(-n // page)) for n in lengths]
        columns = max(columns, max(need, default=0), 1)
        pages = sum(need) + 3
        shape = (pages, page, kv_heads, dim) if layout == "NHD" else (pages, kv_heads, page, dim)
        order = torch.randperm(pages, generator=g, device="cuda").tolist()
        wide = torch.full((len(lengths), columns + 2), 1 << 30, dtype=torch.int32)   # behind the length: never read
        self.owned = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lengths):
            for c in range(need[b]):
                wide[b, c] = order.pop()
                self.owned[wide[b, c], : min(page, n - c * page)] = True
        self.table = wide.cuda()[:, :columns]   # rows further apart than they are long
        room = (pages, 2) + shape[1:] if joint else (2, pages) + shape[1:]
        both = torch.full(room, math.nan, device="cuda")
        halves = (both[:, 0], both[:, 1]) if joint else (both[0], both[1])
        for half, scale in zip(halves, scales):
            x = _normal(g, *shape) / scale
            if dtype == "e4m3":
                x = x.clamp(-448, 448)
            model.by_token(half, layout)[self.owned.cuda()] = model.by_token(x, layout)[self.owned.cuda()]
        both = both.to(TORCH[dtype])
        self.k, self.v = (both[:, 0], both[:, 1]) if joint else (both[0], both[1])
        self.n = torch.tensor(lengths, dtype=torch.int32, device="cuda")

    @property
    def args(self):
        return self.k, self.v, self.table, self.n

    @property
    def named(self):
        return {"layout": self.layout, "k_scale": self.scales[0], "v_scale": self.scales[1]}


def _attend(c, q, what, **kw):
    """One call, checked; returns (out, lse)."""
    dim = q.shape[2]
    out, lse = ar.ar_paged_attention(q, *c.args, return_lse=True, **c.named, **kw)
    scale = kw.pop("scale", None)
    kw = {k: v for k, v in kw.items() if k in ("window", "softcap")}
    ref, ref_lse, room, room_lse = model.attention(q, c.k, c.v, c.table, c.lengths, scale=dim ** -0.5 if scale is None else scale,
                                                   **kw, **c.named)
    check(out, ref, room + half_step(ref, out.dtype), f"{what} out")
    check(lse, ref_lse, room_lse, f"{what} lse")
    return out, lse


# ------------------------------------------------------------------ attention

# tile and page edges, nothing at all, one token
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 200, 0]


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 3), (8, 1), (18, 2), (34, 2)])
def test_attention_edges(dtype, cache, layout, heads, kv_heads):
    scales = (0.03125, 0.5) if cache == "e4m3" else (1.0, 1.0)
    c = Cache(EDGES, kv_heads, 128, 16, cache, layout, seed=heads, scales=scales)
    q = _normal(_gen(1), len(EDGES), heads, 128, std=2.0).to(TORCH[dtype])
    _attend(c, q, f"{dtype} {cache} {layout} {heads}/{kv_heads}")


@pytest.mark.parametrize("dtype,cache,dim", [("bf16", "bf16", d) for d in (8, 40, 64, 72, 80, 96, 104, 136, 192, 200, 256)]
                         + [("fp16", "fp16", d) for d in (16, 120, 160, 256)]
                         + [("fp32", "fp32", d) for d in (4, 12, 64, 80, 100, 160, 192, 196, 256)]
                         + [("bf16", "e4m3", d) for d in (16, 48, 64, 80, 112, 192, 256)])
@pytest.mark.parametrize("heads", [2, 10, 16])
def test_attention_head_sizes(dtype, cache, dim, heads):
    lengths = [70, 1, 0, 131, 64]
    c = Cache(lengths, 1, dim, 16, cache, "HND", seed=dim)
    q = _normal(_gen(dim), len(lengths), heads, dim).to(TORCH[dtype])
    _attend(c, q, f"{dtype} {cache} dim {dim}")


@pytest.mark.parametrize("page", [1, 3, 8, 17, 24, 32, 64, 100, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_page_sizes(page, dtype):
    lengths = [page, page - 1, page + 1, 3 * page + 2, 257]
    c = Cache(lengths, 2, 64, page, dtype, "NHD", seed=page)
    q = _normal(_gen(page), len(lengths), 10, 64).to(TORCH[dtype])
    _attend(c, q, f"page {page}")


@pytest.mark.parametrize("window", [1, 2, 31, 64, 65, 100, 1000])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "e4m3"), ("fp32", "fp32")])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_attention_window_and_softcap(window, dtype, cache, softcap):
    lengths = [0, 1, 64, 65, 129, 300, 777]
    c = Cache(lengths, 2, 64, 16, cache, "HND", seed=window)
    q = _normal(_gen(window), len(lengths), 8, 64, std=3.0).to(TORCH[dtype])
    _attend(c, q, f"window {window}", window=window, softcap=softcap, scale=0.25)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "e4m3"), ("fp32", "fp32")])
def test_attention_many_blocks_share_rows(dtype, cache):
    """Few long rows (each split over many blocks), many rows (several a block), and a mix, the longest first and last."""
    for lengths in ([9001], [5000, 1, 7777], [700] * 140, [4000] + [3] * 300 + [4500], [0] * 129 + [2000]):
        c = Cache(lengths, 1, 64, 32, cache, "NHD", seed=len(lengths))
        q = _normal(_gen(3), len(lengths), 4, 64).to(TORCH[dtype])
        _attend(c, q, f"{len(lengths)} rows")


def test_attention_strides_and_given_buffers():
    """k and v in one buffer, q as a part of a projection, a table cut from a wider one, buffers of the caller's."""
    lengths = [100, 0, 33, 64]
    c = Cache(lengths, 2, 96, 16, "bf16", "NHD", joint=True, columns=12)
    qkv = _normal(_gen(5), 4, 12, 96).to(torch.bfloat16)
    q = qkv[:, :8]
    out, lse = torch.full((4, 8, 96), math.nan, device="cuda", dtype=torch.bfloat16), torch.full((4, 8), math.nan, device="cuda")
    nbytes = ar.ar_paged_attention_workspace_size(*c.args, 8)
    ws = torch.full((nbytes // 4,), math.nan, device="cuda")
    got = _attend(c, q, "strided", out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse
    again = ar.ar_paged_attention(q, *c.args, workspace=ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32")])
def test_attention_holes_and_bad_lengths(dtype, cache):
    """Table entries that are no page leave their tokens out; lengths outside the table's room are cut to it."""
    c = Cache([80, 80, 80, 48, 48], 1, 64, 16, cache, "NHD", columns=5)
    t = c.table.clone()
    t[0, 1], t[0, 3] = -1, c.k.shape[0]
    t[1, :] = -7
    t[2, 4] = 1 << 30
    c.table = t
    c.n = torch.tensor([80, 80, 1 << 30, -5, 48], dtype=torch.int32, device="cuda")
    c.lengths = [80, 80, 80, 0, 48]
    q = _normal(_gen(2), 5, 8, 64).to(TORCH[dtype])
    out, lse = _attend(c, q, "holes")
    assert not out[1].any() and not out[3].any() and bool((lse[1] == -math.inf).all()) and bool((lse[3] == -math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_attention_of_infinite_and_nan_values(dtype):
    """A NaN key or value reaches its own rows only; scores of minus infinity weigh nothing."""
    c = Cache([70, 70, 70, 70], 2, 64, 16, dtype)
    clean = ar.ar_paged_attention(q := _normal(_gen(8), 4, 4, 64).abs().to(TORCH[dtype]), *c.args)
    at = lambda b, j: (int(c.table[b, j // 16]), j % 16)  # noqa: E731
    c.k[at(0, 5)][0] = math.nan          # sequence 0, head 0
    c.v[at(1, 69)][1, 3] = math.inf      # sequence 1, head 1
    c.k[at(2, 0)][0] = -math.inf         # q > 0: the score is minus infinity
    out, lse = ar.ar_paged_attention(q, *c.args, return_lse=True)
    assert bool(out[0, :2].isnan().all()) and bool(lse[0, :2].isnan().all()) and torch.equal(out[0, 2:], clean[0, 2:])
    assert not bool(out[1, 2:, 3].isfinite().any()) and torch.equal(out[1, :2], clean[1, :2])
    assert bool(out[2].isfinite().all()) and bool(lse[2].isfinite().all())
    c.lengths = [0, 0, 70, 70]
    c.n = torch.tensor(c.lengths, dtype=torch.int32, device="cuda")
    c.k[at(2, 0)][0] = -1e30 if dtype != "fp16" else -65504
    _attend(c, q, "lowest values")


def test_attention_large_scores_and_peaks():
    """Scores far apart and far from zero: the running maximum moves, small weights vanish."""
    for dtype in ("bf16", "fp16", "fp32"):
        c = Cache([300, 1500], 1, 128, 16, dtype, seed=4)
        c.k[int(c.table[0, 18]), 3] = 8.0
        q = (_normal(_gen(4), 2, 8, 128).abs() * 3).to(TORCH[dtype])
        _attend(c, q, f"peak {dtype}", scale=1.0)
        _attend(c, -q, f"lowest at the end {dtype}", scale=1.0)


def test_attention_tiny_and_huge_queries_on_an_8_bit_cache():
    c = Cache([200], 1, 128, 16, "e4m3", seed=9)
    for std, scale in ((1e-30, 1e29), (1e30, 1e-31)):
        q = _normal(_gen(4), 1, 8, 128, std=std).to(torch.bfloat16)
        _attend(c, q, f"queries of {std}", scale=scale)


def test_attention_repeats_bit_for_bit_and_follows_a_captured_graph():
    lengths = [3000, 5, 0, 900]
    c = Cache(lengths, 2, 128, 16, "bf16")
    q = _normal(_gen(1), 4, 16, 128).to(torch.bfloat16)
    first = ar.ar_paged_attention(q, *c.args, return_lse=True)
    again = ar.ar_paged_attention(q, *c.args, return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    ws = [torch.empty(ar.ar_paged_attention_workspace_size(*c.args, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for w, out in zip(ws, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ar.ar_paged_attention(q, *c.args, out=out, workspace=w)
        graphs.append(g)
    for n in (lengths, [10, 5, 0, 1], [2999, 1, 0, 64]):   # the graphs read the lengths as they are
        c.n.copy_(torch.tensor(n, dtype=torch.int32))
        want = ar.ar_paged_attention(q, *c.args)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_calls_on_another_stream():
    c = Cache([500, 20], 1, 64, 16, "fp16")
    q = _normal(_gen(1), 2, 4, 64).half()
    want, want_lse = ar.ar_paged_attention(q, *c.args, return_lse=True)
    joined = ar.ar_attention_join([want, want], [want_lse, want_lse])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        out, lse = ar.ar_paged_attention(q, *c.args, return_lse=True, stream=handle)
        both = ar.ar_attention_join([out, out], [lse, lse], stream=handle)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(both, joined)


def test_offsets_past_32_bits():
    """Pages beyond 2^32 elements of the pool: written, read back and attended to."""
    page, heads, dim = 64, 8, 128
    pages = (1 << 32) // (page * heads * dim) + 3
    k = torch.empty(pages, page, heads, dim, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[pages - 1, 0], [1, pages - 2]], dtype=torch.int32, device="cuda")
    for p in (0, 1, pages - 1, pages - 2):
        k[p].view(torch.uint8).fill_(0x7f)   # NaN
        v[p].view(torch.uint8).fill_(0x7f)
    g = _gen(6)
    n = 100
    new_k, new_v = (_normal(g, 2 * n, heads, dim).to(torch.bfloat16) for _ in range(2))
    lengths = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    ar.ar_kv_append(k, v, table, lengths, new_k, new_v, seq_start=start)
    want = new_k[:n].float().clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(k[pages - 1].view(torch.uint8), want[:64].view(torch.uint8))
    assert torch.equal(k[0, :36].view(torch.uint8), want[64:].view(torch.uint8))
    assert bool((k[0, 36:].view(torch.uint8) == 0x7f).all())
    q = _normal(g, 2, 16, dim).to(torch.bfloat16)
    out, lse = ar.ar_paged_attention(q, k, v, table, lengths, return_lse=True)
    ref, ref_lse, room, room_lse = model.attention(q, k, v, table, [n, n], scale=dim ** -0.5)
    check(out, ref, room + half_step(ref, out.dtype), "out")
    check(lse, ref_lse, room_lse, "lse")


# ------------------------------------------------------------------ append

def _append_and_check(lengths, new, heads, kv_heads, dim, rotary, page, dtype, cache, layout, *, interleaved=False, scale=1.0,
                      padding=0, positions=None, in_place=False, with_q=True, scales=(1.0, 1.0), offset=0, holes=(), seed=0):
    """`new`: new tokens of each sequence, or None for one each without seq_start.  `offset`: elements the rows are moved
    by, off any vector's alignment."""
    c = Cache(lengths, kv_heads, dim, page, cache, layout, seed=seed, scales=scales, columns=max(1, -(-max(lengths) // page)))
    for b, column in holes:
        c.table[b, column] = -1
    g = _gen(seed + 1)
    start = None
    tokens = len(lengths)
    if new is not None:
        start = [padding // 2]
        for n in new:
            start.append(start[-1] + n)
        tokens = start[-1] + padding - padding // 2
    qkv = _normal(g, tokens, (heads + 2 * kv_heads) * dim + offset).to(TORCH[dtype])[:, offset:]
    q, k, v = (x.reshape(tokens, -1, dim) if offset == 0 else x.unflatten(1, (-1, dim))
               for x in qkv.split([heads * dim, kv_heads * dim, kv_heads * dim], 1))
    freq = (10000.0 ** (-2 * torch.arange(rotary // 2, device="cuda", dtype=torch.float64) / max(rotary, 1))).float() if rotary else None
    pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
    before_k, before_v, before_q = c.k.clone(), c.v.clone(), q.clone()
    q_out = None if not with_q else q if in_place else torch.full_like(before_q, 7.0)
    start_t = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    got_q = ar.ar_kv_append(c.k, c.v, c.table, c.n, k, v, q=q if with_q else None, q_out=q_out, seq_start=start_t, positions=pos,
                            inv_freq=freq, interleaved=interleaved, rotary_scale=scale, **c.named)
    rows = model.rows_of(lengths, start, tokens)
    at = torch.tensor([positions[t] if positions is not None else p for t, _, p in rows], device="cuda")
    t = torch.tensor([r[0] for r in rows], device="cuda", dtype=torch.long)
    f64 = freq if rotary else torch.zeros(0, device="cuda")
    # The angle is off by pi 2^-25 for its rounding (at positions near 2^31 the 64-bit reference itself by 2^-22), sine and
    # cosine by two steps: each result within 2 * 2^-22 of |x| + |y|, which twice the largest element of the head bounds, the
    # products' and the sum's own roundings included.
    room = lambda x: 4 * 2.0 ** -22 * scale * x.double().abs().amax(-1, keepdim=True).expand(x.shape)  # noqa: E731
    if with_q:
        want = before_q.double()
        if not in_place:
            want = torch.full_like(want, 7.0)
        want[t] = model.rotate(before_q[t].double(), at, f64, interleaved, scale)
        slack = torch.zeros_like(want)
        slack[t] = room(before_q[t]) + half_step(want[t], got_q.dtype)
        check(got_q, want, slack, "q")
    else:
        assert got_q is None
    keys = model.rotate(k.double(), torch.zeros(tokens, device="cuda"), f64, interleaved, 1.0)
    keys[t] = model.rotate(k[t].double(), at, f64, interleaved, scale)
    table = c.table.tolist()
    for pages, before, x, s, what in ((c.k, before_k, keys, scales[0], "k"), (c.v, before_v, v.double(), scales[1], "v")):
        want, slack = model.by_token(before.double(), layout).clone(), None
        slack = torch.zeros_like(want)
        for row, b, p in rows:
            if 0 <= p < len(table[b]) * page and 0 <= table[b][p // page] < pages.shape[0]:
                y = x[row] / s
                y = y.clamp(-448, 448) if cache == "e4m3" else y
                want[table[b][p // page], p % page] = y
                slack[table[b][p // page], p % page] = (room(k[row:row + 1])[0] / s if what == "k" else 2 * U32 * y.abs()) + half_step(y, pages.dtype)
        got = model.by_token(pages, layout).double()
        clear = ~want.isnan()
        check(torch.where(clear, got, 0.0), torch.where(clear, want, 0.0), slack, what)
        assert bool(got[~clear].isnan().all()), f"{what}: written where nothing belongs"


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_steps_and_prompts(dtype, cache, layout, interleaved):
    scales = (0.25, 0.125) if cache == "e4m3" else (1.0, 1.0)
    _append_and_check([1, 16, 17, 100, 33], None, 8, 2, 128, 128, 16, dtype, cache, layout, interleaved=interleaved, scales=scales)
    _append_and_check([40, 5, 9, 64], [40, 0, 3, 17], 6, 3, 64, 32, 8, dtype, cache, layout, interleaved=interleaved, scale=1.25, scales=scales)


@pytest.mark.parametrize("dim,rotary", [(1, 0), (2, 2), (7, 4), (33, 32), (80, 40), (80, 80), (96, 64), (100, 100), (256, 256), (1000, 500)])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "e4m3")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_head_sizes(dim, rotary, dtype, cache, interleaved):
    _append_and_check([3, 20], [3, 6], 5, 1, dim, rotary, 7, dtype, cache, "NHD", interleaved=interleaved, seed=dim)


@pytest.mark.parametrize("offset", [1, 4, 8])
def test_append_rows_off_alignment(offset):
    _append_and_check([9, 2], None, 4, 2, 64, 64, 16, "bf16", "bf16", "HND", offset=offset)
    _append_and_check([9, 2], [5, 2], 4, 2, 64, 64, 16, "fp32", "fp32", "NHD", offset=offset)


def test_append_padding_idle_sequences_and_holes():
    """Rows outside seq_start, sequences of length 0, lengths shorter than their rows, tables with holes."""
    _append_and_check([0, 5, 0, 1], None, 4, 1, 64, 64, 4, "bf16", "bf16", "NHD")
    _append_and_check([12, 4, 30], [12, 0, 7], 4, 1, 64, 64, 4, "fp16", "fp16", "NHD", padding=9)
    _append_and_check([12, 3, 30], [12, 8, 7], 4, 1, 64, 64, 4, "bf16", "e4m3", "HND", padding=4)
    _append_and_check([12, 9, 30], [12, 8, 30], 4, 1, 64, 64, 4, "fp32", "fp32", "HND", padding=1, holes=[(0, 1), (2, 0), (2, 7)])


def test_append_in_place_without_queries_and_at_given_positions():
    _append_and_check([12, 9], [4, 9], 4, 2, 128, 128, 16, "bf16", "bf16", "NHD", in_place=True)
    _append_and_check([12, 9], [4, 9], 4, 2, 80, 40, 16, "fp16", "fp16", "NHD", in_place=True, interleaved=True)
    _append_and_check([12, 9], None, 4, 2, 128, 64, 16, "bf16", "bf16", "NHD", with_q=False)
    _append_and_check([4, 9, 3], None, 4, 2, 128, 128, 16, "fp32", "fp32", "NHD", positions=[1 << 20, 0, 131071])
    _append_and_check([4, 9, 3], None, 4, 2, 128, 128, 16, "fp32", "fp32", "NHD", positions=[(1 << 31) - 1, -1, -(1 << 31)])


def test_append_many_rows_and_sequences():
    _append_and_check([n % 50 for n in range(700)], None, 4, 1, 64, 64, 16, "bf16", "bf16", "NHD")
    new = [(7 * n) % 23 for n in range(300)]
    _append_and_check([n + 2 for n in new], new, 3, 1, 64, 64, 16, "bf16", "e4m3", "NHD", padding=5)


@pytest.mark.parametrize("rows", [7300, 19999])   # a block takes three and eight rows of 16 bits
@pytest.mark.parametrize("dtype,cache,dim,rotary", [("bf16", "bf16", 16, 16), ("fp16", "e4m3", 9, 6), ("fp32", "fp32", 16, 8)])
def test_append_many_short_rows(rows, dtype, cache, dim, rotary):
    new = [1, 0, rows // 3, 2, 0, 0, rows // 2, 5]
    new.append(rows - sum(new))
    _append_and_check([n + 3 for n in new], new, 2, 1, dim, rotary, 64, dtype, cache, "HND", padding=4)


def test_append_saturates_and_keeps_nan():
    c = Cache([2], 1, 16, 4, "e4m3")
    k = torch.tensor([[1e4, -1e4, math.inf, -math.inf, math.nan] + [448.0, 464.0, 500.0, -465.0, 0.0, -0.0] + [2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 2.0 ** -11, 17.0]],
                     device="cuda").view(1, 1, 16).to(torch.bfloat16)
    ar.ar_kv_append(c.k, c.v, c.table, c.n, k, k)
    page = int(c.table[0, 0])
    want = [448, -448, 448, -448, math.nan, 448, 448, 448, -448, 0, 0, 2.0 ** -9, 0, 2.0 ** -8, 0, 16]
    for pages in (c.k, c.v):
        got = pages[page, 1, 0].float().tolist()
        assert all(x == y or (x != x and y != y) for x, y in zip(got, want)), got


# ------------------------------------------------------------------ join

def _join_room(o, lse):
    """64-bit result and what fp32 leaves: a weight is off by 4 u max(1, |lse - max|), weights, products and sums over R by
    (R + 4) u each of the weighted sizes."""
    L = torch.stack(lse).double()
    top = L.amax(0)
    base = torch.where(top == -math.inf, 0.0, top)
    w = torch.exp(L - base)
    total = w.sum(0)
    safe = torch.where(total == 0, 1.0, total)
    x = torch.where((w == 0)[..., None], 0.0, torch.stack(o).double())
    ref = (w[..., None] * x).sum(0) / safe[..., None]
    size = (w[..., None] * x.abs()).sum(0) / safe[..., None]
    far = torch.where(L == -math.inf, 0.0, (L - base).abs()).amax(0).clamp(min=1) + base.abs()
    room = size * ((8 * far + 2 * (len(o) + 4)) * U32)[..., None]
    ref_lse = torch.where(total == 0, -math.inf, base + torch.log(safe))
    return ref, ref_lse, room, (8 * far + len(o) + 4 + 4 * ref_lse.abs().clamp(max=1e30)) * U32


@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 8, 11, 16])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("rows,dim", [((5,), 128), ((3, 7), 64), ((2, 3), 33), ((1,), 1), ((1000,), 40)])
def test_join(R, dtype, rows, dim):
    g = _gen(R * dim)
    o = [_normal(g, *rows, dim).to(TORCH[dtype]) for _ in range(R)]
    lse = [_normal(g, *rows, std=4.0) + 3 for _ in range(R)]
    for r in range(R):   # ranks without a key of some rows, whatever their rows hold
        off = torch.rand(rows, generator=g, device="cuda") < 0.3
        lse[r][off] = -math.inf
        o[r][off] = math.nan
    for x, y in zip(o, lse):   # the last row: no rank has any
        y.view(-1)[-1] = -math.inf
        x.view(-1, dim)[-1] = math.nan
    ref, ref_lse, room, room_lse = _join_room(o, lse)
    out, got = ar.ar_attention_join(o, lse, return_lse=True)
    check(out, ref, room + half_step(ref, out.dtype), "out")
    check(got, ref_lse, room_lse, "lse")
    assert not out.view(-1, dim)[-1].any() and float(got.view(-1)[-1]) == -math.inf
    again = ar.ar_attention_join(o, lse, out=o[-1])   # in place
    assert again is o[-1] and torch.equal(again, out)


def test_join_passes_nan_and_takes_unaligned_rows():
    g = _gen(1)
    o = [_normal(g, 4 * 64 + 1).half()[1:].view(4, 64) for _ in range(3)]
    lse = [_normal(g, 4) for _ in range(3)]
    ref, ref_lse, room, room_lse = _join_room(o, lse)
    out = ar.ar_attention_join(o, lse)
    check(out, ref, room + half_step(ref, out.dtype), "out")
    lse[1][2] = math.nan
    out = ar.ar_attention_join(o, lse)
    assert bool(out[2].isnan().all()) and bool(out[[0, 1, 3]].isfinite().all())


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("ranks", [1, 3])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_layers_steps_over_ranks(ranks, cache):
    """Prompts and then single steps of a layer whose cache is spread over ranks by token: append on every rank, attention
    on every rank, the join, the row-parallel projection's partials, and their reduction with residual and norm."""
    B, H, K, D, page, hidden = 3, 8, 2, 64, 8, 256
    prompts = [19, 1, 40]
    steps = 3
    scales = (0.0625, 0.0625) if cache == "e4m3" else (1.0, 1.0)
    g = _gen(ranks)
    total = [n + steps for n in prompts]
    qkv = [_normal(g, n, H + 2 * K, D).to(torch.bfloat16) for n in total]
    freq = (10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2))).float()
    weight = [_normal(g, H * D, hidden, std=0.05).to(torch.bfloat16) for _ in range(2)]   # two shards of the projection
    residual = _normal(g, B, hidden).to(torch.bfloat16)
    norm = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
    owner = lambda j: j % ranks  # noqa: E731 - rank of token j
    parts = []
    for r in range(ranks):
        own = [len([j for j in range(n) if owner(j) == r]) for n in total]
        c = Cache([0] * B, K, D, page, cache, "HND", columns=8, scales=scales)
        need = [max(1, -(-n // page)) for n in own]
        pool = torch.empty(2, sum(need), K, page, D, device="cuda").to(TORCH[cache])
        pool.view(torch.uint8 if cache == "e4m3" else torch.int16).fill_(127 if cache == "e4m3" else -1)   # NaN
        c.k, c.v = pool[0], pool[1]
        c.table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            c.table[b, : need[b]] = torch.arange(sum(need[:b]), sum(need[: b + 1]), dtype=torch.int32, device="cuda")
        parts.append(c)

    def append(r, c, take):
        """take[b]: the positions of sequence b's tokens that go to this rank now."""
        rows = torch.cat([qkv[b][take[b]] for b in range(B)])
        start = torch.tensor([sum(len(x) for x in take[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        c.n = c.n + torch.tensor([len(x) for x in take], dtype=torch.int32, device="cuda")
        pos = torch.tensor(sum(take, []), dtype=torch.int32, device="cuda")
        ar.ar_kv_append(c.k, c.v, c.table, c.n, rows[:, H:H + K], rows[:, H + K:], seq_start=start, positions=pos, inv_freq=freq, **c.named)

    for r, c in enumerate(parts):
        append(r, c, [[j for j in range(n) if owner(j) == r] for n in prompts])
    for step in range(steps):
        at = [n + step for n in prompts]
        for r, c in enumerate(parts):
            append(r, c, [[j] if owner(j) == r else [] for j in at])
        now = torch.stack([qkv[b][at[b]] for b in range(B)])
        scratch = Cache([n + 1 for n in at], K, D, page, "bf16", columns=8)   # turns the queries, its cache is not used
        q = ar.ar_kv_append(*scratch.args, now[:, H:H + K], now[:, H + K:], q=now[:, :H], inv_freq=freq)
        got = [ar.ar_paged_attention(q, *c.args, return_lse=True, **c.named) for c in parts]
        out = ar.ar_attention_join([x for x, _ in got], [x for _, x in got])
        for b in range(B):
            n = at[b] + 1
            pos = torch.arange(n, device="cuda")
            cached = []
            for kind, s in (("k", scales[0]), ("v", scales[1])):   # token j is the (j // ranks)-th of its rank
                x = torch.stack([getattr(parts[owner(j)], kind)[int(parts[owner(j)].table[b, j // ranks // page]), :, j // ranks % page].double()
                                 for j in range(n)]) * s
                want = qkv[b][:n, H:H + K].double() if kind == "k" else qkv[b][:n, H + K:].double()
                slack = 0.0
                if kind == "k":
                    slack = 8 * 2.0 ** -22 * want.abs().amax(-1, keepdim=True)
                    want = model.rotate(want, pos, freq, False, 1.0)
                check(x, want, slack + half_step(want / s, TORCH[cache]) * s, f"step {step} {kind}")
                cached.append(x.repeat_interleave(H // K, 1))
            k, v = cached
            z = torch.einsum("hd,jhd->hj", q[b].double(), k) * D ** -0.5
            want = torch.einsum("hj,jhd->hd", torch.softmax(z, 1), v)
            size = torch.einsum("hj,jhd->hd", torch.softmax(z, 1), v.abs())
            mass = torch.einsum("hd,jhd->hj", q[b].double().abs(), k.abs()).amax(1, keepdim=True) * D ** -0.5
            delta = (2 * (D + 2) * mass + 8 * z.abs().amax(1, keepdim=True).clamp(min=1)) * U32
            # the parts are rounded to bf16 before the join (2^-8 of size at the most), the whole once more
            check(out[b], want, size * (2.0 ** -8 + 8 * delta + 2.0 ** -15) + half_step(want, torch.bfloat16), f"step {step}")
        partials = [(out.view(B, -1)[:, : H * D // 2].contiguous() @ weight[0][: H * D // 2]), (out.view(B, -1)[:, H * D // 2:].contiguous() @ weight[1][H * D // 2:])]
        y, res = ar.ar_residual_rmsnorm(partials, residual, norm, 1e-6)
        x = sum(p.double() for p in partials) + residual.double()
        check(res, x, 4 * U32 * (sum(p.double().abs() for p in partials) + residual.double().abs()) + half_step(x, torch.bfloat16), "residual")
        y_ref = x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt()
        check(y, y_ref, y_ref.abs() * 2.0 ** -16 + 2 * half_step(y_ref, torch.bfloat16), "norm")
        residual = res


# ------------------------------------------------------------------ refusals, empty calls, threads

def test_calls_refuse_tensors_that_do_not_fit():
    c = Cache([20, 5], 2, 64, 16, "bf16", columns=2)
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    kv = torch.zeros(2, 2, 64, device="cuda", dtype=torch.bfloat16)
    good = dict(q=q, k_pages=c.k, v_pages=c.v, page_table=c.table, lengths=c.n)
    for change in (dict(q=q.half()), dict(q=q[:1]), dict(q=q[..., :32]), dict(q=q.transpose(0, 1)), dict(q=q.cpu()), dict(v_pages=c.v[:, :8]),
                   dict(v_pages=c.v.half()), dict(k_pages=c.k[0], v_pages=c.v[0]), dict(k_pages=c.k.cpu(), v_pages=c.v.cpu()),
                   dict(page_table=c.table.long()), dict(page_table=c.table[:1]), dict(page_table=c.table.cpu()), dict(lengths=c.n.long()),
                   dict(lengths=c.n[:1]), dict(out=torch.empty_like(q)[:1]), dict(out=torch.empty(2, 4, 64, device="cuda")),
                   dict(lse=torch.empty(2, 4)), dict(lse=torch.empty(4, 2, device="cuda").t()), dict(layout="nhd"),
                   dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises((ValueError, ar.ARError)):
            ar.ar_paged_attention(**{**good, **change})
    for change, status in ((dict(q=q[:, :3]), ar.AR_ERR_INVALID_ARG), (dict(window=-1), ar.AR_ERR_INVALID_ARG), (dict(softcap=math.nan), ar.AR_ERR_INVALID_ARG),
                           (dict(k_scale=0.0), ar.AR_ERR_INVALID_ARG), (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), ar.AR_ERR_WORKSPACE)):
        with pytest.raises(ar.ARError) as e:
            ar.ar_paged_attention(**{**good, **change})
        assert e.value.status == status
    wide = torch.zeros(3, 16, 2, 68, device="cuda", dtype=torch.bfloat16)   # rows that begin between vectors
    with pytest.raises(ar.ARError) as e:
        ar.ar_paged_attention(q, wide[..., 4:], wide[..., 4:], c.table, c.n)
    assert e.value.status == ar.AR_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        ar.ar_paged_attention(None, c.k, c.v, c.table, c.n)
    fine = dict(k_pages=c.k, v_pages=c.v, page_table=c.table, lengths=c.n, k=kv, v=kv)
    freq = torch.ones(32, device="cuda")
    for change in (dict(k=kv[:1]), dict(v=kv.half()), dict(k=kv.float(), v=kv.float()), dict(q=q, q_out=q[:, :2]), dict(q_out=q), dict(inv_freq=freq.half()),
                   dict(inv_freq=torch.ones(33, device="cuda")), dict(positions=c.n[:1]), dict(seq_start=c.n), dict(rotary_scale=math.inf)):
        with pytest.raises((ValueError, ar.ARError)):
            ar.ar_kv_append(**{**fine, **change})
    for parts, lse in (([q], [q]), ([q, q[:1]], [freq[:8].view(2, 4)] * 2), ([q, q.float()], [freq[:8].view(2, 4)] * 2), ([q] * 17, [freq[:8].view(2, 4)] * 17)):
        with pytest.raises(ValueError):
            ar.ar_attention_join(parts, lse)
    torch.cuda.synchronize()


def test_empty_calls():
    k = torch.zeros(1, 16, 2, 64, device="cuda", dtype=torch.float16)
    table, n = torch.zeros(0, 3, device="cuda", dtype=torch.int32), torch.zeros(0, device="cuda", dtype=torch.int32)
    none = torch.zeros(0, 4, 64, device="cuda", dtype=torch.float16)
    out, lse = ar.ar_paged_attention(none, k, k, table, n, return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    q = ar.ar_kv_append(k, k, table, n, none[:, :2], none[:, :2], q=none)
    assert q.shape == (0, 4, 64)
    out, lse = ar.ar_attention_join([none], [none[..., 0].float()], return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_a_captured_step_makes_its_own_scratch():
    """Append and attention captured together without given buffers, replayed as the cache grows."""
    lengths = [30, 1, 64]
    c = Cache([n + 3 for n in lengths], 2, 64, 16, "bf16", seed=3)
    g = _gen(3)
    qkv = _normal(g, 3, 12, 64).to(torch.bfloat16)
    q, k, v = qkv.split([8, 2, 2], dim=1)
    freq = torch.rand(32, generator=g, device="cuda")

    def step():
        turned = ar.ar_kv_append(*c.args, k, v, q=q, inv_freq=freq)
        return turned, *ar.ar_paged_attention(turned, *c.args, return_lse=True)

    c.n.copy_(torch.tensor(lengths, dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turned, out, lse = step()
    for i in range(1, 4):
        c.n.add_(1)
        qkv.copy_(_normal(g, 3, 12, 64))
        graph.replay()
        now = [n + i for n in lengths]
        ref, ref_lse, room, room_lse = model.attention(turned, c.k, c.v, c.table, now, scale=0.125)
        check(out, ref, room + half_step(ref, out.dtype), f"step {i}")
        check(lse, ref_lse, room_lse, f"step {i} lse")


def test_calls_of_several_threads():
    import threading
    c = [Cache([700, 3, 90], 1, 64, 16, "fp16", seed=s) for s in range(4)]
    q = [_normal(_gen(s), 3, 8, 64).half() for s in range(4)]
    want = [ar.ar_paged_attention(q[s], *c[s].args) for s in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def work(s):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                if not torch.equal(ar.ar_paged_attention(q[s], *c[s].args), want[s]):
                    wrong.append(s)
    threads = [threading.Thread(target=work, args=(s,)) for s in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32")])
def test_attention_of_thousands_of_rows(dtype, cache):
    """More rows than blocks, threads and a block's lengths by far; tokens of one page each, several rows on the same page."""
    B, K, D, page, pages = 6001, 2, 64, 4, 500
    g = _gen(12)
    k, v = (_normal(g, pages, page, K, D).to(TORCH[cache]) for _ in range(2))
    table = torch.randint(0, pages, (B, 1), generator=g, device="cuda", dtype=torch.int32)
    n = torch.randint(0, page + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    q = _normal(g, B, 2 * K, D).to(TORCH[dtype])
    out, lse = ar.ar_paged_attention(q, k, v, table, n, return_lse=True)
    kk, vv = (x[table[:, 0].long()].double().repeat_interleave(2, 2) for x in (k, v))   # [B, page, 2 K, D]
    z = torch.einsum("bhd,bjhd->bhj", q.double(), kk) / 8
    mass = (torch.einsum("bhd,bjhd->bhj", q.double().abs(), kk.abs()) / 8).amax(2)
    z = z.masked_fill(torch.arange(page, device="cuda")[None, None] >= n[:, None, None], -math.inf)
    p = torch.where(n[:, None, None] > 0, torch.softmax(z, 2), 0.0)
    want, size = torch.einsum("bhj,bjhd->bhd", p, vv), torch.einsum("bhj,bjhd->bhd", p, vv.abs())
    delta = (2 * (D + 2) * mass + 8 * z.masked_fill(z == -math.inf, 0).abs().amax(2).clamp(min=1)) * U32   # as in the model
    check(out, want, size * (4 * delta + 2.0 ** -16 + 4 * (page + 16) * U32)[..., None] + half_step(want, out.dtype), "out")
    check(lse, torch.logsumexp(z, 2), 2 * delta + 4 * (page + 24) * U32 * (1 + mass), "lse")


def test_sequences_that_share_pages_and_ranks_that_are_one():
    c = Cache([70, 70, 33], 2, 64, 16, "bf16")
    c.table = c.table.clone()
    c.table[1] = c.table[0]
    c.table[2, :3] = c.table[0, :3]
    q = _normal(_gen(4), 1, 8, 64).to(torch.bfloat16).expand(3, 8, 64).contiguous()
    out, lse = _attend(c, q, "shared")
    same = ar.ar_attention_join([out[:1], out[:1]], [lse[:1], lse[:1]])   # twice the same keys: the same mean
    check(same, out[:1].double(), half_step(out[:1].double(), out.dtype) * 2.0 ** -6, "twice")


def test_the_default_stream_by_its_handle():
    c = Cache([50], 1, 64, 16, "fp16")
    q = _normal(_gen(4), 1, 4, 64).half()
    want = ar.ar_paged_attention(q, *c.args)
    got = ar.ar_paged_attention(q, *c.args, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
