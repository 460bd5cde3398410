"""Host-only checks of the calls for drafted tokens: refusals come back before anything is launched, empty calls launch nothing, the
ctypes mirror matches the C structure, and workspace sizes cover what the kernels write.  No test here reaches a launch."""
import ctypes
import os
import subprocess

import pytest

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: every call using it fails validation first
STATUS = {"arg": ar.AR_ERR_INVALID_ARG, "no": ar.AR_ERR_UNSUPPORTED, "ws": ar.AR_ERR_WORKSPACE, "ok": ar.AR_OK}


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


def _tree(L, cache=None, ws=FAKE, ws_bytes=1 << 40, **kw):
    d = dict(q=FAKE, tokens=6, q_heads=8, dtype=ar.AR_BF16, q_stride=1024, seq_start=None, mask=FAKE, mask_words=1, scale=0.1, window=0,
             softcap=0.0, out=FAKE, lse=None)
    d.update(kw)
    return L.ar_tree_attention(cache if cache is not None else _cache(), ar.ArTreeParams(**d), ws, ws_bytes, None)


def _axes(L, axes=2, stride=3, pair_axis=bytes(64), cache=None, **kw):
    d = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, tokens=3, q_heads=8, dtype=ar.AR_BF16, q_stride=1024, k_stride=256, v_stride=256,
             q_out_stride=1024, seq_start=None, positions=FAKE, inv_freq=FAKE, rotary_dim=128, interleaved=0, rotary_scale=1.0)
    d.update(kw)
    return L.ar_kv_append_axes(cache if cache is not None else _cache(), ar.ArAppendParams(**d), axes, stride, pair_axis, None)


def _pointers(values):
    return (ctypes.c_void_p * len(values))(*values)


def _compact(L, cache=None, k=(FAKE, FAKE), v=(FAKE, FAKE), layers=2, kept=FAKE, kept_stride=5, most=5, seq_start=None, drafted=5, out=0x90000):
    return L.ar_kv_compact(cache if cache is not None else _cache(), _pointers(k) if k else None, _pointers(v) if v else None, layers, kept,
                           kept_stride, most, seq_start, drafted, out, None)


def _copy(L, cache=None, k=(FAKE, FAKE), v=(FAKE, FAKE), layers=2, src=FAKE, dst=FAKE, pairs=3):
    return L.ar_kv_copy_pages(cache if cache is not None else _cache(), _pointers(k) if k else None, _pointers(v) if v else None, layers, src, dst,
                              pairs, None)


BAD_PAGES = [(dict(pages=0), "arg"), (dict(page_size=0), "arg"), (dict(kv_heads=0), "arg"), (dict(head_dim=0), "arg"), (dict(page_stride=100), "arg"),
             (dict(token_stride=64), "arg"), (dict(head_stride=64), "arg"), (dict(dtype=7), "no"), (dict(dtype=-1), "no"), (dict(kv_heads=1025), "no"),
             (dict(head_dim=1025, token_stride=2050, head_stride=1025, page_stride=1 << 20), "no")]
BAD_TABLES = [(dict(batch=-1), "arg"), (dict(max_pages=0), "arg"), (dict(table_stride=3), "arg"), (dict(page_table=None), "arg"),
              (dict(lengths=None), "arg"), (dict(lengths=FAKE + 2), "arg"), (dict(page_table=FAKE + 1), "arg")]


@pytest.mark.parametrize("kw,kind", BAD_PAGES + BAD_TABLES)
def test_bad_caches_are_refused(L, kw, kind):
    assert _compact(L, _cache(**kw)) == STATUS[kind]
    if kw.get("kv_heads") != 1025:   # no number of query heads to go with them
        assert _tree(L, _cache(**kw)) in (STATUS[kind], ar.AR_ERR_UNSUPPORTED)
        assert _axes(L, cache=_cache(**kw)) in (STATUS[kind], ar.AR_ERR_UNSUPPORTED)
    if (kw, kind) in BAD_PAGES:
        assert _copy(L, _cache(**kw)) == STATUS[kind]


@pytest.mark.parametrize("kw,kind", [
    (dict(tokens=-1), "arg"), (dict(tokens=7), "arg"), (dict(q_heads=0), "arg"), (dict(q_heads=7), "arg"), (dict(q_heads=1026, q_stride=1 << 20), "no"),
    (dict(q=None), "arg"), (dict(out=None), "arg"), (dict(q=FAKE + 1), "arg"), (dict(q=FAKE + 2), "no"), (dict(out=FAKE + 8), "no"),
    (dict(lse=FAKE + 1), "arg"), (dict(seq_start=FAKE + 2), "arg"), (dict(mask=FAKE + 4), "arg"), (dict(mask_words=0), "arg"),
    (dict(mask_words=1025), "arg"), (dict(q_stride=1023), "arg"), (dict(q_stride=1025), "no"), (dict(window=-1), "arg"), (dict(softcap=-1.0), "arg"),
    (dict(softcap=float("inf")), "arg"), (dict(scale=float("nan")), "arg"), (dict(scale=3e38), "arg"), (dict(softcap=1e-38, scale=1e3), "arg"),
    (dict(dtype=ar.AR_FP32), "no"), (dict(dtype=ar.AR_FP8_E4M3), "no"), (dict(dtype=9), "no"), (dict(ws=None), "ws"), (dict(ws=FAKE + 8), "ws"),
    (dict(ws_bytes=100), "ws"), (dict(tokens=2 ** 31 - 1, seq_start=FAKE), "no")])
def test_tree_refusals(L, kw, kind):
    assert _tree(L, **kw) == STATUS[kind]


def test_tree_refuses_head_sizes_strides_and_null(L):
    assert _tree(L, _cache(head_dim=264, head_stride=264, token_stride=528, page_stride=528 * 16), q_stride=264 * 8) == ar.AR_ERR_UNSUPPORTED
    assert _tree(L, _cache(head_dim=124), q_stride=1024) == ar.AR_ERR_UNSUPPORTED
    assert _tree(L, _cache(token_stride=260, page_stride=260 * 16)) == ar.AR_ERR_UNSUPPORTED
    assert _tree(L, _cache(k=FAKE + 2)) == ar.AR_ERR_UNSUPPORTED
    assert L.ar_tree_attention(None, ar.ArTreeParams(), None, 0, None) == ar.AR_ERR_INVALID_ARG
    assert L.ar_tree_attention(_cache(), None, None, 0, None) == ar.AR_ERR_INVALID_ARG
    assert _tree(L, _cache(batch=0), seq_start=None, tokens=4) == ar.AR_ERR_INVALID_ARG


def test_empty_calls_launch_nothing(L):
    assert _tree(L, tokens=0, q=None, out=None, ws=None) == ar.AR_OK
    assert _tree(L, _cache(batch=0, page_table=None, lengths=None), tokens=0) == ar.AR_OK
    assert _tree(L, _cache(batch=0, page_table=None, lengths=None), tokens=5, seq_start=FAKE) == ar.AR_OK
    assert _axes(L, cache=_cache(batch=0), tokens=0, positions=None) == ar.AR_OK
    assert _compact(L, _cache(batch=0, page_table=None, lengths=None), k=None, v=None, out=None) == ar.AR_OK
    assert _copy(L, k=None, v=None, src=None, dst=None, pairs=0) == ar.AR_OK


@pytest.mark.parametrize("kw", [dict(axes=0), dict(axes=5), dict(axes=-1), dict(stride=2), dict(pair_axis=None), dict(pair_axis=bytes([0] * 63 + [2])),
                                dict(positions=None), dict(positions=FAKE + 1), dict(rotary_dim=130), dict(inv_freq=None), dict(tokens=-1)])
def test_axes_refusals(L, kw):
    assert _axes(L, **kw) == ar.AR_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,kind", [
    (dict(layers=0), "arg"), (dict(layers=-3), "arg"), (dict(layers=129), "no"), (dict(k=None), "arg"), (dict(v=None), "arg"), (dict(k=(FAKE, None)), "arg"),
    (dict(v=(FAKE + 1, FAKE)), "arg"), (dict(kept=None), "arg"), (dict(kept=FAKE + 2), "arg"), (dict(kept_stride=4), "arg"), (dict(most=-1), "arg"),
    (dict(drafted=-1), "arg"), (dict(seq_start=FAKE + 1), "arg"), (dict(out=None), "arg"), (dict(out=FAKE + 3), "arg"), (dict(out=FAKE), "arg"),
    (dict(out=0x20008, kept=0x20000), "arg"), (dict(out=0x20000, seq_start=0x1fff4), "arg")])
def test_compact_refusals(L, kw, kind):
    assert _compact(L, **kw) == STATUS[kind]


@pytest.mark.parametrize("kw,kind", [
    (dict(layers=0), "arg"), (dict(layers=129), "no"), (dict(k=None), "arg"), (dict(v=(None, FAKE)), "arg"), (dict(k=(FAKE, FAKE + 1)), "arg"),
    (dict(src=None), "arg"), (dict(dst=None), "arg"), (dict(src=FAKE + 2), "arg"), (dict(dst=FAKE + 1), "arg"), (dict(pairs=-1), "arg")])
def test_copy_refusals(L, kw, kind):
    assert _copy(L, **kw) == STATUS[kind]


def test_workspace_sizes(L):
    size = lambda heads=8, tokens=6, **kw: L.ar_tree_attention_workspace_size(_cache(**kw), heads, tokens)  # noqa: E731
    assert size() > 0 and size() % 256 == 0
    assert size(heads=7) == 0 and size(tokens=-1) == 0 and size(pages=0) == 0 and size(head_dim=300) == 0
    # two slots a block, a row of sums and two numbers for each row; no more rows than there are
    assert size(max_pages=10000, table_stride=10000, batch=300, tokens=3000) >= 2 * 152 * 64 * 130 * 4
    assert size(max_pages=10000, table_stride=10000, batch=64, tokens=64, heads=2) <= 2 * 304 * 64 * 130 * 4 + 304 * 32 + 512
    # no more blocks than tiles of the longest sequences: one page and four are both within a tile
    assert size(max_pages=1, table_stride=1) <= size(max_pages=4) < size(max_pages=400, table_stride=400)
    assert size(tokens=0) < 1 << 20


def test_ctypes_mirror_matches_the_header(tmp_path):
    fields = [f for f, _ in ar.ArTreeParams._fields_]
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include "ar.h"\nint main(void) { printf("%zu", sizeof(ar_tree_params));\n' +
                   "".join(f'printf(" %zu", offsetof(ar_tree_params, {f}));\n' for f in fields) +
                   'printf(" %d %d", AR_MAX_AXES, AR_MAX_LAYERS); return 0; }\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "probe")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "probe")], check=True, capture_output=True, text=True).stdout.split()]
    assert got[0] == ctypes.sizeof(ar.ArTreeParams)
    assert got[1:-2] == [getattr(ar.ArTreeParams, f).offset for f in fields]
    assert got[-2:] == [ar.AR_MAX_AXES, ar.AR_MAX_LAYERS]
