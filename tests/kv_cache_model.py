"""The paged key-value cache calls from their formulas, in 64-bit torch arithmetic with plain loops, and the errors
that fp32 arithmetic and one rounding may leave (shared by the GPU tests of those calls)."""
import math

import torch

TORCH = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
U32 = 2.0 ** -24   # half a step of fp32


def half_step(ref, dtype):
    """Half the spacing of `dtype` at the 64-bit values `ref`: what one rounding may be off by."""
    info = torch.finfo(dtype)
    e = torch.frexp(ref.abs().clamp(min=info.smallest_normal, max=2.0 ** 1000))[1].long() - 1
    # 2^e from its bits: torch.ldexp's power of two is a step short on a GPU, and a tie lies exactly half a step away.
    return ((e + 1023) << 52).view(torch.float64) * (info.eps / 2)


def rotate(x, pos, inv_freq, interleaved, scale):
    """x [rows, heads, dim] in 64 bits, each row turned at its position."""
    half = inv_freq.numel()
    angle = pos.double()[:, None, None] * inv_freq.double()
    c, s = torch.cos(angle) * scale, torch.sin(angle) * scale
    out = x.clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def by_token(pages, layout):
    """The pages as [pages, page_size, kv_heads, head_dim], a view."""
    return pages if layout == "NHD" else pages.transpose(1, 2)


def rows_of(lengths, seq_start, tokens):
    """(row, sequence, index in the sequence) of every row that belongs to a sequence."""
    got = []
    for b, n in enumerate(lengths):
        lo, hi = (b, b + 1) if seq_start is None else (seq_start[b], seq_start[b + 1])
        for t in range(lo, min(hi, tokens)):
            got.append((t, b, n - (hi - lo) + t - lo))
    return got


def attention(q, k_pages, v_pages, table, lengths, *, scale, window=0, softcap=0.0, layout="NHD", k_scale=1.0, v_scale=1.0):
    """out, lse in 64 bits, and how far fp32 arithmetic may leave each of them before out's own rounding.

    With u = 2^-24 and every product and sum rounded at most twice that far (a matrix unit may cut off where an adder
    rounds): a dot product of d terms is off by 2 (d + 2) u sum |q k|; the score, the exponent's base change and e^x add
    8 u max(1, |s|) more; softcap shrinks these, and adds 16 u |s| for its tanh: (e - 1) / (e + 1) of |x| >= 0.3 is off by
    e / (e - 1) <= 2.2 times e^(2x)'s 4 u, and by 5 u for its steps and the division.  A bf16 query on an 8-bit cache is
    scaled to fp16 with its largest element at 2^14 or more, so that elements are off by 2^-39 of the largest.
    So each weight is off by a factor e^(+-2 delta), relative to
    their sum 4 delta at the most.  Each weight is rounded to a pair of 16-bit numbers, to 2^-16 of it, or for bf16 queries
    on an 8-bit cache to one of fp16, to 2^-11; in fp16 the largest is 2^15, and a weight under 2^-29 of it is rounded to
    2^-40 of it, so that n of them add 2^-40 sum |v| to a sum of weights of 1 at least.  The sums of n weighted values and
    of n weights are off by 2 (n + 16) u each.
    """
    pages, ps = k_pages.shape[0], by_token(k_pages, layout).shape[1]
    B, H, D = q.shape
    K = by_token(k_pages, layout).shape[2]
    kd, vd = by_token(k_pages, layout), by_token(v_pages, layout)
    out = torch.zeros(B, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=q.device)
    e_out, e_lse = torch.zeros_like(out), torch.zeros_like(lse)
    rows = table.tolist()
    for b in range(B):
        n = max(0, min(int(lengths[b]), len(rows[b]) * ps))
        j = [x for x in range(max(0, n - window) if window else 0, n) if 0 <= rows[b][x // ps] < pages]
        if not j:
            continue
        page = torch.tensor([rows[b][x // ps] for x in j], device=q.device)
        slot = torch.tensor([x % ps for x in j], device=q.device)
        bits = (lambda x: x.view(torch.uint8)[page, slot].view(x.dtype)) if k_pages.dtype == TORCH["e4m3"] else (lambda x: x[page, slot])
        k = (bits(kd).double() * k_scale).repeat_interleave(H // K, 1)
        v = (bits(vd).double() * v_scale).repeat_interleave(H // K, 1)
        qb = q[b].double()
        s = torch.einsum("hd,jhd->hj", qb, k) * scale
        mass = torch.einsum("hd,jhd->hj", qb.abs(), k.abs()) * abs(scale)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        delta = 2 * (D + 2) * U32 * mass + (8 * s.abs().clamp(min=1) + (16 * s.abs() if softcap else 0)) * U32
        if q.dtype == torch.bfloat16 and k_pages.dtype == TORCH["e4m3"]:
            delta = delta + 2.0 ** -39 * abs(scale) * qb.abs().amax(1)[:, None] * k.abs().sum(2).T
        delta = delta.amax(1)
        p = torch.softmax(s, 1)
        out[b], lse[b] = torch.einsum("hj,jhd->hd", p, v), torch.logsumexp(s, 1)
        size = torch.einsum("hj,jhd->hd", p, v.abs())
        sums = 4 * (len(j) + 16) * U32
        once = q.dtype == torch.bfloat16 and k_pages.dtype == TORCH["e4m3"]
        e_out[b] = size * (4 * delta + 2.0 ** (-11 if once else -16) + sums)[:, None]
        if q.dtype == torch.float16 or k_pages.dtype == TORCH["e4m3"]:
            e_out[b] += 2.0 ** -40 * v.abs().sum(0)
        e_lse[b] = 2 * delta + sums + 4 * U32 * (1 + lse[b].abs())
    return out, lse, e_out, e_lse


def check(got, ref, room, what):
    """|got - ref| <= room everywhere, infinities equal."""
    got = got.double()
    same = (got == ref) | ((got - ref).abs() <= room)
    if not bool(same.all()):
        at = tuple(int(i) for i in (~same).nonzero()[0])
        raise AssertionError(f"{what}: {int((~same).sum())} of {same.numel()} values off; at {at}: {float(got[at])} "
                             f"against {float(ref[at])}, {float(room[at]) if torch.is_tensor(room) else room} allowed")
