"""What ar_kv_copy_pages and ar_kv_compact take as pages: either order of a page, of any number of tokens, and layers that share a cache."""
import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("shape", [(5, 2, 1025, 8), (5, 1025, 2, 8), (4, 1, 5000, 16), (4, 5000, 1, 16), (5, 1024, 3, 5), (5, 3, 1024, 5)])
def test_copying_pages_of_many_tokens_in_either_order(shape):
    """Heads are 1024 at the most, tokens of a page any number, and which of the two comes first does not matter."""
    x, y = _randn(1, *shape).half(), _randn(2, *shape).half()
    want = [t.clone() for t in (x, y)]
    for t in want:
        t[3] = t[0]
        t[2] = t[1]
    ar.ar_kv_copy_pages(x, y, _ints([0, 1]), _ints([3, 2]))
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_copying_refuses_pages_without_a_head_count():
    x = torch.zeros(3, 1025, 1025, 4, dtype=torch.float16, device="cuda")
    with pytest.raises(ar.ARError):
        ar.ar_kv_copy_pages(x, x.clone(), _ints([0]), _ints([1]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float8_e4m3fn])
def test_layers_that_share_a_cache_move_once(dtype):
    """The same buffers named by several layers, by keys and values at once, beside layers of their own: as if each was named once."""
    batch, n, context, page = 300, 20, 5, 16
    pages = batch * 2
    bits = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
    x = [(_randn(i, pages, page, 2, 64) * 3).to(dtype) for i in range(5)]
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(batch, 2)
    lengths = torch.full((batch,), context + n, dtype=torch.int32, device="cuda")
    kept = [sorted(torch.randperm(n, generator=torch.Generator().manual_seed(b))[: b % (n + 1)].tolist()) for b in range(batch)]
    wide = _ints([m + [-1] * (n - len(m)) for m in kept])
    want = []
    for t in x:
        flat = t.view(bits).clone().view(batch, 2 * page, 2, 64)
        for b, mine in enumerate(kept):
            flat[b, context: context + len(mine)] = flat[b, [context + j for j in mine]].clone()
        want.append(flat.view(pages, page, 2, 64))
    a, b, c, d, both = x
    got = ar.ar_kv_compact([a, c, a, both, a], [b, d, b, both, d], table, lengths, wide, drafted=n)
    assert got.tolist() == [context + len(m) for m in kept]
    for t, w in zip(x, want):
        assert torch.equal(t.view(bits), w)


def test_copying_in_layers_that_share_a_cache():
    a, b, c = (_randn(i, 9, 4, 2, 64) for i in range(3))
    want = [t.clone() for t in (a, b, c)]
    for t in want:
        t[7] = t[1]
    ar.ar_kv_copy_pages([a, a, c, c], [b, b, b, c], _ints([1]), _ints([7]))
    assert all(torch.equal(t, w) for t, w in zip((a, b, c), want))
