"""Decoding with drafted tokens from its formulas, in 64-bit torch arithmetic with plain loops, and the errors that the kernels'
arithmetic may leave (shared by the GPU tests of ar_tree_attention, ar_kv_append_axes, ar_kv_compact and ar_kv_copy_pages)."""
import math
import random

import torch

from tests.kv_cache_model import TORCH, U32, by_token


def bits(pages):
    """Pages that torch can index: 8-bit ones as whole numbers."""
    return pages.view(torch.uint8) if pages.dtype == TORCH["e4m3"] else pages


class Cache:
    """Pages in no order that hold `lengths` tokens of each sequence; every element that no sequence owns is NaN."""

    def __init__(self, lengths, kv_heads, dim, page, dtype, layout="NHD", seed=0, scales=(1.0, 1.0), room=0, joint=False):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.lengths, self.page, self.layout, self.scales = lengths, page, layout, scales
        need = [-(-max(n, 0) // page) for n in lengths]
        columns = max(need + [1]) + room
        pages = sum(need) + 3
        shape = (pages, page, kv_heads, dim) if layout == "NHD" else (pages, kv_heads, page, dim)
        order = torch.randperm(pages, generator=g, device="cuda").tolist()
        wide = torch.full((len(lengths), columns + 1), -7, dtype=torch.int32)
        owned = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lengths):
            for c in range(need[b]):
                wide[b, c] = order.pop()
                owned[wide[b, c], : min(page, n - c * page)] = True
        self.free = order
        self.table = wide.cuda()[:, :columns]   # rows further apart than they are long
        both = torch.full((pages, 2) + shape[1:] if joint else (2, pages) + shape[1:], math.nan, device="cuda")
        halves = (both[:, 0], both[:, 1]) if joint else (both[0], both[1])
        for half, scale in zip(halves, scales):
            x = torch.randn(shape, generator=g, device="cuda") / scale
            x = x.clamp(-448, 448) if dtype == "e4m3" else x
            by_token(half, layout)[owned.cuda()] = by_token(x, layout)[owned.cuda()]
        both = both.to(TORCH[dtype])
        self.k, self.v = (both[:, 0], both[:, 1]) if joint else (both[0], both[1])
        self.n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.kw = dict(layout=layout, k_scale=scales[0], v_scale=scales[1])

    def tokens(self, pages, b, at):
        """Elements of tokens `at` of sequence b, [tokens, heads, dim]."""
        at = torch.as_tensor(at, dtype=torch.long, device="cuda")
        page = self.table[b].long()[at // self.page]
        return by_token(bits(pages), self.layout)[page, at % self.page].view(pages.dtype)


def tree_masks(n, seed, kind="tree"):
    """The rows' masks of a tree of n tokens as whole numbers; "any": bits of no order, some rows without one."""
    r, got = random.Random(seed), []
    for i in range(n):
        if kind == "any":
            got.append(0 if r.random() < 0.2 else r.getrandbits(n + 3))
        else:
            parent = r.randint(max(-1, i - 5), i - 1)
            got.append((got[parent] if parent >= 0 else 0) | 1 << i)
    return got


def words_of(masks, words):
    """Masks as an int64 tensor [rows, words]."""
    cut = [[(m >> 64 * i & (1 << 63) - 1) - (m >> 64 * i & 1 << 63) for i in range(words)] for m in masks]
    return torch.tensor(cut, dtype=torch.int64, device="cuda").view(len(masks), words)


def seen(i, n, length, window, mask):
    """Which tokens of its sequence row i of n new ones sees, before the cache's bounds."""
    context = length - n
    got = list(range(max(0, context)))
    got += [context + j for j in range(n) if (j <= i if mask is None else mask >> j & 1)]
    return [j for j in (got[-window:] if window else got) if j >= 0]


def attention(q, cache, starts, masks, *, scale, window=0, softcap=0.0):
    """out, lse in 64 bits and the room of each, over all rows of q; rows of no sequence are NaN.

    The bounds are those of kv_cache_model.attention (one dot product, exponential and weighted sum are the same arithmetic), but
    weights are taken against a reference that the largest may pass by 2^8 at the most, and are held in two 16-bit numbers: bf16
    leaves 2^-16 of a weight, fp16 the same, and where the second number runs out of bits 2^-25, of weights lifted by 2^7:
    2^-32 of the reference's, whose own weight of 1 is in the sum.
    """
    pages, page = cache.k.shape[0], cache.page
    T, H, D = q.shape
    K = by_token(cache.k, cache.layout).shape[2]
    out = torch.full((T, H, D), math.nan, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), math.nan, dtype=torch.float64, device="cuda")
    e_out, e_lse = torch.zeros_like(out), torch.zeros_like(lse)
    table = cache.table.tolist()
    for b, length in enumerate(cache.lengths):
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        ok = [j for j in range(max(0, min(length, len(table[b]) * page))) if 0 <= table[b][j // page] < pages]
        place = {j: x for x, j in enumerate(ok)}
        k = (cache.tokens(cache.k, b, ok).double() * cache.scales[0]).repeat_interleave(H // K, 1)
        v = (cache.tokens(cache.v, b, ok).double() * cache.scales[1]).repeat_interleave(H // K, 1)
        for i in range(n):
            row = starts[b] + i
            at = [place[j] for j in seen(i, n, max(length, 0), window, None if masks is None else masks[row]) if j in place]
            out[row], lse[row] = 0.0, -math.inf
            if not at:
                continue
            qb, kk, vv = q[row].double(), k[at], v[at]
            s = torch.einsum("hd,jhd->hj", qb, kk) * scale
            mass = torch.einsum("hd,jhd->hj", qb.abs(), kk.abs()) * abs(scale)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            delta = 2 * (D + 2) * U32 * mass + (8 * s.abs().clamp(min=1) + (16 * s.abs() if softcap else 0)) * U32
            if q.dtype == torch.bfloat16 and cache.k.dtype == TORCH["e4m3"]:
                delta = delta + 2.0 ** -39 * abs(scale) * qb.abs().amax(1)[:, None] * kk.abs().sum(2).T
            delta = delta.amax(1)
            p = torch.softmax(s, 1)
            out[row], lse[row] = torch.einsum("hj,jhd->hd", p, vv), torch.logsumexp(s, 1)
            size = torch.einsum("hj,jhd->hd", p, vv.abs())
            sums = 4 * (len(at) + 16) * U32
            e_out[row] = size * (4 * delta + 2.0 ** -16 + sums)[:, None]
            if q.dtype == torch.float16 or cache.k.dtype == TORCH["e4m3"]:
                e_out[row] += 2.0 ** -32 * vv.abs().sum(0)
            e_lse[row] = 2 * delta + sums + 4 * U32 * (1 + lse[row].abs())
    return out, lse, e_out, e_lse
