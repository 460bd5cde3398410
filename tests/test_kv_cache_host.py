"""Host-only checks of the paged key-value cache calls: refusals come back before anything is launched, empty calls
launch nothing, the ctypes mirrors match the C structures, workspace sizes follow the header, and the split of the work
over blocks (the kernels' integer arithmetic, restated) covers every tile once.  No test here reaches a launch."""
import ctypes
import os
import subprocess

import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ar.h")
FAKE = 0x10000  # never dereferenced: every call using it fails validation first


@pytest.fixture(scope="module")
def L():
    _build.build()
    return ar.lib()


def _cache(**kw):
    """A cache that every call takes (bf16, 16-token pages, 2 heads of 128)."""
    d = dict(k=FAKE, v=FAKE, dtype=ar.AR_BF16, pages=8, page_size=16, kv_heads=2, head_dim=128, page_stride=16 * 256,
             token_stride=256, head_stride=128, k_scale=1.0, v_scale=1.0, page_table=FAKE, batch=3, max_pages=4,
             table_stride=4, lengths=FAKE)
    d.update(kw)
    return ar.ArKVCache(**d)


def _append(L, cache=None, **kw):
    d = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, tokens=3, q_heads=8, dtype=ar.AR_BF16, q_stride=1024, k_stride=256, v_stride=256,
             q_out_stride=1024, seq_start=None, positions=None, inv_freq=FAKE, rotary_dim=128, interleaved=0, rotary_scale=1.0)
    d.update(kw)
    return L.ar_kv_append(cache if cache is not None else _cache(), ar.ArAppendParams(**d), None)


def _attend(L, cache=None, **kw):
    cache = cache if cache is not None else _cache()
    d = dict(q=FAKE, q_stride=1024, q_heads=8, scale=0.1, window=0, softcap=0.0, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40,
             dtype=ar.AR_BF16)
    d.update(kw)
    return L.ar_paged_attention(cache, *d.values(), None)


BAD_CACHES = [
    (dict(pages=0), "arg"), (dict(page_size=0), "arg"), (dict(kv_heads=0), "arg"), (dict(head_dim=0), "arg"), (dict(batch=-1), "arg"),
    (dict(max_pages=0), "arg"), (dict(table_stride=3), "arg"), (dict(k=None), "arg"), (dict(v=None), "arg"), (dict(page_table=None), "arg"),
    (dict(lengths=None), "arg"), (dict(k=FAKE + 1), "arg"), (dict(lengths=FAKE + 2), "arg"), (dict(page_stride=100), "arg"),
    (dict(token_stride=64), "arg"), (dict(head_stride=64), "arg"), (dict(k_scale=0.0), "arg"), (dict(v_scale=-1.0), "arg"),
    (dict(k_scale=float("nan")), "arg"), (dict(v_scale=float("inf")), "arg"), (dict(dtype=7), "no"), (dict(dtype=ar.AR_FP16), "no"),
    (dict(dtype=-1), "no"), (dict(kv_heads=1025), "no"), (dict(head_dim=1025, token_stride=2050, head_stride=1025, page_stride=1 << 20), "no"),
]
STATUS = {"arg": ar.AR_ERR_INVALID_ARG, "no": ar.AR_ERR_UNSUPPORTED, "ws": ar.AR_ERR_WORKSPACE}


@pytest.mark.parametrize("kw,kind", BAD_CACHES)
def test_bad_caches_are_refused(L, kw, kind):
    assert _append(L, _cache(**kw)) == STATUS[kind]
    if kw.get("kv_heads") != 1025:   # no number of query heads to go with them
        assert _attend(L, _cache(**kw)) in (STATUS[kind], ar.AR_ERR_UNSUPPORTED)


@pytest.mark.parametrize("kw,kind", [
    (dict(tokens=-1), "arg"), (dict(tokens=2), "arg"), (dict(q_heads=0), "arg"), (dict(q_heads=1025, q_stride=1 << 20, q_out_stride=1 << 20), "no"),
    (dict(q_out=None), "arg"), (dict(k=None), "arg"), (dict(v=None), "arg"), (dict(q=FAKE + 1), "arg"), (dict(positions=FAKE + 1), "arg"),
    (dict(seq_start=FAKE + 2), "arg"), (dict(q_stride=1023), "arg"), (dict(k_stride=255), "arg"), (dict(v_stride=0), "arg"),
    (dict(q_out_stride=8), "arg"), (dict(rotary_dim=3), "arg"), (dict(rotary_dim=130), "arg"), (dict(rotary_dim=-2), "arg"),
    (dict(inv_freq=None), "arg"), (dict(rotary_scale=float("nan")), "arg"), (dict(rotary_scale=float("inf")), "arg"),
    (dict(dtype=ar.AR_FP8_E4M3), "no"), (dict(dtype=9), "no"), (dict(dtype=ar.AR_FP32), "no")])
def test_append_refusals(L, kw, kind):
    assert _append(L, **kw) == STATUS[kind]


def test_append_dtype_pairs_null_and_empty(L):
    assert _append(L, _cache(dtype=ar.AR_FP8_E4M3), dtype=ar.AR_FP32) == ar.AR_ERR_UNSUPPORTED
    assert L.ar_kv_append(None, ar.ArAppendParams(), None) == ar.AR_ERR_INVALID_ARG
    assert L.ar_kv_append(_cache(), None, None) == ar.AR_ERR_INVALID_ARG
    assert _append(L, _cache(batch=0), tokens=0) == ar.AR_OK
    assert _append(L, tokens=0, seq_start=FAKE, k=None, v=None, q=None, q_out=None) == ar.AR_OK
    assert _append(L, _cache(batch=0), tokens=3, seq_start=FAKE) == ar.AR_ERR_INVALID_ARG   # rows of no sequence


@pytest.mark.parametrize("kw,kind", [
    (dict(q_heads=0), "arg"), (dict(q_heads=3), "arg"), (dict(q_heads=-2), "arg"), (dict(q_heads=2048, q_stride=1 << 20), "no"),
    (dict(scale=float("nan")), "arg"), (dict(scale=float("inf")), "arg"), (dict(window=-1), "arg"), (dict(softcap=-1.0), "arg"),
    (dict(softcap=float("inf")), "arg"), (dict(q=None), "arg"), (dict(out=None), "arg"), (dict(q_stride=1016), "arg"), (dict(lse=FAKE + 2), "arg"),
    (dict(q=FAKE + 8), "no"), (dict(out=FAKE + 2), "no"), (dict(q_stride=1028), "no"), (dict(dtype=ar.AR_FP16), "no"), (dict(dtype=3), "no"),
    (dict(ws=None), "ws"), (dict(ws=FAKE + 8), "ws"), (dict(ws_bytes=0), "ws")])
def test_attention_refusals(L, kw, kind):
    assert _attend(L, **kw) == STATUS[kind]


@pytest.mark.parametrize("cache,kw", [({}, dict(scale=3e38)), (dict(k_scale=1e20), dict(scale=-1e20)), ({}, dict(scale=2.0, softcap=1e-38)),
                                      ({}, dict(softcap=3e38))])
def test_attention_refuses_factors_that_overflow(L, cache, kw):
    assert _attend(L, _cache(**cache), **kw) == STATUS["arg"]


@pytest.mark.parametrize("kw", [dict(k=FAKE + 8), dict(v=FAKE + 2), dict(head_dim=120, token_stride=244), dict(head_dim=100, token_stride=256),
                                dict(head_dim=264, token_stride=528, head_stride=264, page_stride=16 * 528), dict(page_stride=16 * 256 + 4),
                                dict(head_stride=132, token_stride=264, page_stride=16 * 264),
                                dict(dtype=ar.AR_FP8_E4M3, head_dim=120, head_stride=128)])
def test_attention_refuses_what_is_not_whole_vectors(L, kw):
    c = _cache(**kw)
    assert _attend(L, c, q_stride=1 << 12) == ar.AR_ERR_UNSUPPORTED
    if "k" not in kw and "v" not in kw:
        assert L.ar_paged_attention_workspace_size(c, 8) == 0


def test_attention_null_and_empty(L):
    assert _attend(L, _cache(batch=0), q=None, out=None, ws=None, ws_bytes=0) == ar.AR_OK
    assert L.ar_paged_attention(None, FAKE, 1024, 8, 0.1, 0, 0.0, FAKE, None, FAKE, 1 << 40, ar.AR_BF16, None) == ar.AR_ERR_INVALID_ARG
    assert L.ar_paged_attention_workspace_size(None, 8) == 0
    need = L.ar_paged_attention_workspace_size(_cache(), 8)
    assert need > 0 and need % 256 == 0
    assert _attend(L, ws_bytes=need - 1) == ar.AR_ERR_WORKSPACE
    # strides that one page, token or head never uses refuse nothing: only the missing workspace does
    odd = _cache(pages=1, page_size=1, kv_heads=1, page_stride=1, token_stride=3, head_stride=0)
    assert _attend(L, odd, ws=None) == ar.AR_ERR_WORKSPACE


def test_workspace_size_does_not_depend_on_pointers_and_grows_no_further(L):
    bare = _cache(k=None, v=None, page_table=None, lengths=None)
    assert L.ar_paged_attention_workspace_size(bare, 8) == L.ar_paged_attention_workspace_size(_cache(), 8)
    sizes = [L.ar_paged_attention_workspace_size(_cache(batch=b, max_pages=m, table_stride=m), 8)
             for b, m in ((1, 1), (1, 100), (100, 100), (100, 2147483647), (1 << 20, 1 << 20), (2147483647, 2147483647))]
    assert sizes == sorted(sizes) and sizes[2] == sizes[3]   # from some length on, more of it needs no more
    assert L.ar_paged_attention_workspace_size(_cache(), 64) > L.ar_paged_attention_workspace_size(_cache(), 2)


def _join(L, R=2, partials=None, lse=None, rows=4, dim=128, out=FAKE, lse_out=None, dtype=ar.AR_BF16):
    arr = lambda v: (ctypes.c_void_p * max(R, 1))(*v)  # noqa: E731
    return L.ar_attention_join(arr(partials or [FAKE] * R), arr(lse or [FAKE] * R), R, rows, dim, out, lse_out, dtype, None)


def test_join_refusals(L):
    bad = ar.AR_ERR_INVALID_ARG
    assert _join(L, R=0, partials=[FAKE], lse=[FAKE]) == bad
    assert L.ar_attention_join(None, None, 17, 4, 128, FAKE, None, ar.AR_BF16, None) == bad
    assert L.ar_attention_join(None, None, 2, 4, 128, FAKE, None, ar.AR_BF16, None) == bad
    assert _join(L, rows=-1) == bad and _join(L, dim=0) == bad and _join(L, out=None) == bad and _join(L, out=FAKE + 1) == bad
    assert _join(L, partials=[FAKE, None]) == bad and _join(L, lse=[None, FAKE]) == bad and _join(L, lse=[FAKE, FAKE + 2]) == bad
    assert _join(L, lse=[FAKE, FAKE + 64], lse_out=FAKE + 64) == bad and _join(L, lse_out=FAKE + 66) == bad
    assert _join(L, dtype=ar.AR_FP8_E4M3) == ar.AR_ERR_UNSUPPORTED and _join(L, dtype=5) == ar.AR_ERR_UNSUPPORTED
    assert _join(L, rows=0, out=None) == ar.AR_OK


def test_other_calls_still_refuse_the_8_bit_type(L):
    ptrs = (ctypes.c_void_p * 2)(FAKE, FAKE)
    assert L.ar_sum(ptrs, 2, FAKE, 16, ar.AR_FP8_E4M3, ar.AR_ONESHOT, None) == ar.AR_ERR_UNSUPPORTED
    assert L.ar_rmsnorm(FAKE, FAKE, 1e-6, 16, 1, FAKE, ar.AR_FP8_E4M3, None) == ar.AR_ERR_UNSUPPORTED


@pytest.mark.parametrize("mirror,name", [(ar.ArKVCache, "ar_kv_cache"), (ar.ArAppendParams, "ar_append_params")])
def test_struct_layouts_match_c(tmp_path, mirror, name):
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "layout.c"
    prints = "".join(f'  printf("%zu ", offsetof({name}, {f}));\n' for f in fields)
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "{HEADER}"\nint main(void) {{\n  printf("%zu ", sizeof({name}));\n{prints}  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def test_python_calls_refuse_wrong_tensors():
    t = torch.zeros(2, 16, 2, 64)
    i = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pages must be a CUDA tensor"):
        ar.ar_kv_append(t, t, i, i[0, :1], t[0, :1], t[0, :1])
    with pytest.raises(ValueError, match="layout must be"):
        ar.ar_paged_attention(t[0], t, t, i, i[0, :1], layout="NDH")
    with pytest.raises(ValueError, match="CUDA tensors of the current device"):
        ar.ar_attention_join([t], [t[..., 0]])
    with pytest.raises(ValueError, match="at least one partial"):
        ar.ar_attention_join([], [])
    with pytest.raises(ValueError, match="one lse for each"):
        ar.ar_attention_join([t, t], [t[..., 0]])


def _run_of(total, blocks, c):
    q, r = divmod(total, blocks)
    return c * q + min(c, r), q + (c < r)


def _block_of(total, blocks, x):
    q, r = divmod(total, blocks)
    edge = r * (q + 1)
    return x // (q + 1) if x < edge else r + (x - edge) // q


@pytest.mark.parametrize("total,blocks", [(1, 304), (303, 304), (304, 304), (305, 304), (1000, 7), (12345, 304), (7, 1)])
def test_every_tile_has_one_block(total, blocks):
    runs = [_run_of(total, blocks, c) for c in range(blocks)]
    assert sum(n for _, n in runs) == total and max(n for _, n in runs) - min(n for _, n in runs) <= 1
    owner = [c for c, (lo, n) in enumerate(runs) for _ in range(n)]
    assert [lo for lo, n in runs if n] == [owner.index(c) for c in sorted(set(owner))]
    assert owner == [_block_of(total, blocks, x) for x in range(total)]


@pytest.mark.parametrize("tiles,heads,blocks", [([1, 5, 1, 9], 3, 4), ([1] * 50, 2, 7), ([40], 1, 13), ([3, 1, 7] * 9, 8, 304)])
def test_parts_of_a_row_lie_in_distinct_slots(tiles, heads, blocks):
    """A block's part of a row goes to slot 1 of the block when it begins the row and to slot 0 otherwise; the join looks
    for slot 1 in the row's first block and slot 0 in the rest."""
    total = sum(tiles) * heads
    items = [n for n in tiles for _ in range(heads)]
    start = [sum(items[:i]) for i in range(len(items))]
    written = {}
    for c in range(blocks):
        lo, n = _run_of(total, blocks, c)
        for item, (s, m) in enumerate(zip(start, items)):
            a, b = max(lo, s), min(lo + n, s + m)
            if a < b and (a, b) != (s, s + m):
                slot = (c, 1 if a == s else 0)
                assert slot not in written
                written[slot] = item
    for item, (s, m) in enumerate(zip(start, items)):
        c0, c1 = _block_of(total, blocks, s), _block_of(total, blocks, s + m - 1)
        want = [] if c0 == c1 else [(c, 1 if c == c0 else 0) for c in range(c0, c1 + 1)]
        assert sorted(k for k, v in written.items() if v == item) == want
