"""The model of k_tree_mma's hand-overs against the kernel's own shapes: those of every form that is launched, printed by a program that
nvcc compiles from ar_tree_mma.cuh, are the ones that the model runs."""
import random
import subprocess

import pytest

from tensor_allreduce_residual_gb300 import _build
from tests.test_tree_protocol_model import SHAPES, run

SOURCE = """
#include <cstdio>
#include "ar_tree_mma.cuh"
template <typename T, typename CT, int DIM, int NM>
void say(const char* types)
{
    using P = ar::TreeMmaShape<T, CT, DIM, NM>;
    std::printf("%s %d %d %d %d %d %d %d %d %d %d %d\\n", types, DIM, P::ROWS, NM, P::GROUPS, P::NS, P::QS, P::RS, P::TILES, int(P::SCALED),
                P::BUFFERS, P::EXPONENTS);
}
template <typename T, typename CT>
void all(const char* types)
{
    say<T, CT, 64, 1>(types);
    say<T, CT, 64, 2>(types);
    say<T, CT, 128, 1>(types);
    say<T, CT, 128, 2>(types);
    say<T, CT, 192, 1>(types);
    say<T, CT, 256, 1>(types);
}
int main()
{
    all<__half, __half>("16");
    all<__nv_bfloat16, __nv_bfloat16>("16");
    all<__half, __nv_fp8_e4m3>("8");
    all<__nv_bfloat16, __nv_fp8_e4m3>("8s");
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """(types, head size, rows) -> [arguments of the model's run]"""
    d = tmp_path_factory.mktemp("shapes")
    (d / "shapes.cu").write_text(SOURCE)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", f"-I{_build.INCLUDE}", f"-I{_build.CSRC}", str(d / "shapes.cu"), "-o", str(d / "shapes")], check=True)
    got = {}
    for line in subprocess.run([str(d / "shapes")], check=True, capture_output=True, text=True).stdout.splitlines():
        types, *numbers = line.split()
        dim, rows, NM, groups, NS, QS, RS, tiles, scaled, buffers, exponents = (int(x) for x in numbers)
        assert buffers == 2 and exponents == (4 if NM == 2 else 6) and bool(scaled) == (types == "8s")   # as the model has them
        assert got.setdefault((types, dim, rows), (NM, groups, NS, QS, RS, tiles, bool(scaled))) == (NM, groups, NS, QS, RS, tiles, bool(scaled))
    assert len(got) == 18
    return got


def test_the_model_runs_the_kernels_shapes(shapes):
    for name, shape in SHAPES.items():
        bits, _, dim, *rest = name.replace(",", "").split()
        rows = 256 if "256 rows" in name else 128
        types = "16" if bits == "16" else "8" if "fp16 queries" in name else "8s"
        assert shapes[types, int(dim), rows] == shape[:6] + (len(shape) > 6,), name


@pytest.mark.parametrize("boxes", [False, True])
@pytest.mark.parametrize("dim,rows", [(64, 128), (64, 256), (128, 128), (128, 256), (192, 128)])
def test_fp16_queries_on_8_bit_caches(shapes, dim, rows, boxes):
    """The shapes that the model's own list leaves out: as many descriptions of tiles as 16-bit caches have, and stages."""
    *shape, scaled = shapes["8", dim, rows]
    assert not scaled
    for seed in range(15):
        r = random.Random(100 + seed)
        items = [(r.choice([1, 1, 2, 3, 5, 9]), r.random() < 0.7) for _ in range(r.randint(1, 8))]
        stuck = run(*shape, items, seed, False, boxes)
        assert stuck is None, (items, stuck)
