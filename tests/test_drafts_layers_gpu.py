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
