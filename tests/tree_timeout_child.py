"""Child process for test_tree_timeout_gpu.

`python -m tests.tree_timeout_child` (test build, libar_test.so): in every block of k_tree_mma that has three steps or more, no warp
hands the third one's weights over (AR_TEST_TREE_STALL=3, set by the parent), a flag that nothing sets.  The bounded waits run out,
the block lets what it has under way land and leaves, the call returns, ar_device_status reports it once, and calls of fewer steps
before and after are right.

`python -m tests.tree_timeout_child product` (libar.so, same environment): the library does not read the setting; the same calls
return with results that match the formulas, and no wait gives up."""
import sys
import time

import torch

import tensor_allreduce_residual_gb300 as ar
from tests import drafts_model as model
from tests.kv_cache_model import TORCH, check, half_step

# query type, cache type, heads, key-value heads, head size, page, new tokens: tensor copies and pages that do not fit their boxes, 8 bits
# with and without scaled queries, one group of softmax warps, 256 rows
FORMS = [("bf16", "bf16", 16, 2, 128, 64, 8), ("bf16", "bf16", 16, 2, 128, 17, 8), ("bf16", "e4m3", 16, 2, 64, 64, 8), ("fp16", "e4m3", 16, 2, 128, 17, 8),
         ("fp16", "fp16", 8, 1, 256, 16, 5), ("bf16", "bf16", 16, 1, 128, 32, 16)]


def _inputs(form, context, batch):
    dtype, cache, heads, kv_heads, dim, page, new = form
    scales = (0.05, 0.02) if cache == "e4m3" else (1.0, 1.0)
    c = model.Cache([context + new] * batch, kv_heads, dim, page, cache, "NHD", 3, scales)
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(batch * new, heads, dim, generator=g, device="cuda").to(TORCH[dtype])
    return c, q, [i * new for i in range(batch + 1)]


def _call(c, q):
    return ar.ar_tree_attention(q, c.k, c.v, c.table, c.n, return_lse=True, **c.kw)


def _right(form, context, batch):
    c, q, starts = _inputs(form, context, batch)
    out, lse = _call(c, q)
    ref, ref_lse, e_out, e_lse = model.attention(q, c, starts, None, scale=form[4] ** -0.5)
    check(lse, ref_lse, e_lse, "lse")
    check(out, ref, e_out + half_step(ref, TORCH[form[0]]), "out")


def main():
    product = sys.argv[1:] == ["product"]
    if not product:
        ar.use_test_library()
    torch.cuda.set_device(0)
    assert ar.ar_device_status() == ar.AR_OK
    for form in FORMS:
        _right(form, 40, 2)   # a tile of each item: fewer than three steps a block
        assert ar.ar_device_status() == ar.AR_OK, form
        if product:
            _right(form, 40000, 2)
            assert ar.ar_device_status() == ar.AR_OK, form
            continue
        c, q, _ = _inputs(form, 60000, 2)   # four tiles a block and more
        torch.cuda.synchronize()
        t0 = time.time()
        _call(c, q)
        torch.cuda.synchronize()
        took = time.time() - t0
        status = ar.ar_device_status()
        assert status == ar.AR_ERR_TIMEOUT, (form, status)
        assert ar.ar_device_status() == ar.AR_OK, form   # the record was cleared
        assert 0.5 < took < 10.0, (form, took)           # the waits ran out after about a second, all together
        for _ in range(3):
            _right(form, 40, 2)
        assert ar.ar_device_status() == ar.AR_OK, form
        print(f"{form}: {took:.2f} s", flush=True)
    print("product library ignores the test setting" if product else "tree timeout ok")


if __name__ == "__main__":
    sys.exit(main())
