"""The paged key-value cache calls from plain C: tests/kv_cache_c_example.c is compiled against include/ar.h, linked with
libar.so and the CUDA runtime, and run; its results are checked against the formulas in 64 bits."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from tensor_allreduce_residual_gb300 import _build
from tests import kv_cache_model as model

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
HEADS, KV_HEADS, DIM, LENGTHS = 4, 2, 64, (37, 5)


def test_c_program_appends_attends_and_joins(tmp_path):
    lib = _build.build()
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    exe = tmp_path / "kv_cache_c_example"
    subprocess.run(["gcc", "-std=c11", "-O2", os.path.join(HERE, "kv_cache_c_example.c"), f"-I{_build.INCLUDE}", f"-I{cuda}/include",
                    f"-L{os.path.dirname(lib)}", "-lar", f"-L{cuda}/lib64", "-lcudart", f"-Wl,-rpath,{os.path.dirname(lib)}",
                    f"-Wl,-rpath,{cuda}/lib64", "-o", str(exe)], check=True)
    g = torch.Generator().manual_seed(11)
    q = torch.randn(2, HEADS, DIM, generator=g)
    k, v = (torch.randn(sum(LENGTHS), KV_HEADS, DIM, generator=g) for _ in range(2))
    freq = 10000.0 ** (-torch.arange(DIM // 2) / (DIM // 2))
    inp, outp = tmp_path / "in.bin", tmp_path / "out.bin"
    torch.cat([x.reshape(-1) for x in (q, k, v, freq)]).numpy().astype(np.float32).tofile(inp)
    res = subprocess.run([str(exe), str(inp), str(outp)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and "kv_cache_c_example: ok" in res.stdout, res.stdout + res.stderr

    got = torch.from_numpy(np.fromfile(outp, dtype=np.float32)).view(2, 2, HEADS, DIM)
    at = 0
    for b, n in enumerate(LENGTHS):
        turned = model.rotate(k[at:at + n].double(), torch.arange(n), freq, False, 1.0).repeat_interleave(HEADS // KV_HEADS, 1)
        values = v[at:at + n].double().repeat_interleave(HEADS // KV_HEADS, 1)
        at += n
        z = torch.einsum("hd,jhd->hj", q[b].double(), turned) / 8
        p = torch.softmax(z, 1)
        want, size = torch.einsum("hj,jhd->hd", p, values), torch.einsum("hj,jhd->hd", p, values.abs())
        # The keys are off by 4 * 2^-22 of their row's largest element (angle, sine and cosine, products), which moves a score by
        # at most that times sum |q|; the products and sums add 2 (d + 2) u sum |q k|, the weights and their sums 64 u.
        keys = 4 * 2.0 ** -22 * turned.abs().amax() * q[b].double().abs().sum(1, keepdim=True) / 8
        mass = torch.einsum("hd,jhd->hj", q[b].double().abs(), turned.abs()).amax(1, keepdim=True) / 8
        delta = keys + 2 * (DIM + 2) * mass * model.U32
        room = size * (4 * delta + 4 * (n + 16) * model.U32 + 64 * model.U32)
        model.check(got[0, b], want, room, f"sequence {b}")
        model.check(got[1, b], want, 2 * room, f"sequence {b} joined")   # each half's weights and the join's are off likewise
