"""Cases of decoding with drafted tokens over the paged key-value cache: attention of a tree of drafted tokens, appending with
positions on several axes, compacting the accepted drafts, and copying pages.  `run` computes a case in plain torch operations, or
through the package's calls where `own` is true."""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZES = {"fp32": 4, "fp16": 2, "bf16": 2, "e4m3": 1}


def _tree(name, batch, new_lo, new_hi, lo, hi, heads, kv_heads, dim, page, dtype, cache, layout, window=0, softcap=0.0, chain=False):
    """new_lo..new_hi drafted tokens of each of `batch` sequences behind lo..hi tokens of context; `chain`: each sees all before it."""
    return {"op": "tree", "name": name, "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "cache": cache, "layout": layout, "window": window,
            "softcap": softcap, "chain": chain}


def _axes(name, batch, new, lo, hi, heads, kv_heads, dim, rotary, axes, turns, page, dtype, cache, layout, interleaved):
    """`new` tokens of each sequence (0: prompts of lo..hi tokens, whole), rotated by `axes` positions each; `turns`: the pairs take
    the axes in turn, or else in blocks."""
    return {"op": "axes", "name": name, "batch": batch, "new": new, "lo": lo, "hi": hi, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "axes": axes, "turns": turns, "page": page, "dtype": dtype, "cache": cache, "layout": layout,
            "interleaved": interleaved}


def _compact(name, layers, batch, new, lo, hi, kv_heads, dim, page, cache, layout):
    """`new` drafted tokens of each sequence, behind lo..hi tokens of context, of which some are kept."""
    return {"op": "compact", "name": name, "layers": layers, "batch": batch, "new": new, "lo": lo, "hi": hi, "kv_heads": kv_heads,
            "dim": dim, "page": page, "cache": cache, "layout": layout}


def _copy(name, layers, pairs, kv_heads, dim, page, cache):
    return {"op": "copy", "name": name, "layers": layers, "pairs": pairs, "kv_heads": kv_heads, "dim": dim, "page": page, "cache": cache}


def listed():
    return [
        # eight drafts behind one short sequence, one rank of eight at hidden 8192: all latency
        _tree("tree short bf16", 1, 8, 8, 503, 503, 8, 1, 128, 16, "bf16", "bf16", "NHD"),
        # sixteen drafts behind one long sequence: the length has to be split to fill the GPU
        _tree("tree long bf16", 1, 16, 16, 131056, 131056, 8, 1, 128, 64, "bf16", "bf16", "NHD"),
        # a ragged batch in steady decoding, trees of uneven sizes
        _tree("tree batch bf16", 64, 4, 32, 1, 8159, 32, 4, 128, 16, "bf16", "bf16", "NHD"),
        # a large ragged batch on an 8-bit cache, small trees of one size
        _tree("tree batch e4m3", 64, 8, 8, 1, 16376, 16, 2, 128, 64, "bf16", "e4m3", "HND"),
        # large trees, a sliding window, capped scores, small heads, pages that end inside a tile
        _tree("tree window fp16", 24, 64, 64, 1, 5000, 16, 8, 64, 24, "fp16", "fp16", "HND", 1024, 30.0),
        # 32-bit values, chains of five drafts, two query heads on each pair of keys and values
        _tree("chain batch fp32", 16, 5, 5, 1, 4096, 16, 8, 96, 32, "fp32", "fp32", "NHD", chain=True),
        # one decode step of a large batch behind images, into an 8-bit cache
        _axes("axes step e4m3", 256, 1, 1, 120, 32, 4, 128, 128, 3, False, 64, "fp16", "e4m3", "HND", True),
        # prompts of text and images with every head of hidden 8192, the axes in turn
        _axes("axes prompts bf16", 4, 0, 1000, 3000, 64, 8, 128, 128, 3, True, 64, "bf16", "bf16", "NHD", False),
        # what a small step accepted, one rank of eight: all latency
        _compact("compact step bf16", 8, 8, 8, 17, 2000, 1, 128, 16, "bf16", "NHD"),
        # what a large step accepted
        _compact("compact batch fp16", 4, 256, 32, 1, 500, 8, 128, 32, "fp16", "HND"),
        # the last pages of a few sequences that fork
        _copy("copy fork bf16", 16, 8, 1, 128, 16, "bf16"),
        # a pool's pages moved together
        _copy("copy pool e4m3", 4, 2000, 8, 128, 32, "e4m3"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tree", "axes", "compact", "copy"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp16", "fp32"])
    cache = "e4m3" if dtype != "fp32" and rng.random() < 0.35 else dtype
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
    page = rng.choice([1, 8, 16, 16, 17, 32, 64, 64, 128])
    layout = rng.choice(["NHD", "HND"])
    if op == "tree":
        hi = _spread(rng, 1, 100000)
        hi = min(hi, 64 * 8192 * 4 * 128 // 4 // (kv_heads * dim))  # cached values: a quarter of the largest listed case's room
        new_hi = _spread(rng, 1, 128)
        rows = 64 * 18 * 32 * 4096 * 128 // dim  # query rows times context of the largest listed case
        new_hi = max(1, min(new_hi, rows // (heads * hi)))
        most = min(64 * 8192 * 4 * 128 // 4 // (kv_heads * dim * hi), rows // (heads * hi * new_hi), 128)
        batch = _spread(rng, 1, max(1, most))
        case = _tree("", batch, rng.choice([1, new_hi, max(1, new_hi // 4)]), new_hi, rng.choice([0, 1, max(1, hi // 2)]), hi, heads, kv_heads,
                     dim, page, dtype, cache, layout, _spread(rng, 1, 8192) if rng.random() < 0.25 else 0,
                     rng.choice([0.0, 0.0, 0.0, 30.0]), rng.random() < 0.25)
    elif op == "axes":
        rotary = rng.choice([dim, dim, dim // 2, 16])
        most = 8192 * 80 * 128 // ((heads + 2 * kv_heads) * dim)  # tokens of the largest listed case
        if rng.random() < 0.5:
            batch = _spread(rng, 1, min(512, most))
            new, lo, hi = 1, 1, _spread(rng, 1, 4096)
            hi = max(1, min(hi, 40_000_000 // (batch * kv_heads * dim)))
        else:
            batch = rng.randint(1, 8)
            new, hi = 0, _spread(rng, 2, max(2, min(8192, most // batch)))
            lo = max(1, hi // 4)
        case = _axes("", batch, new, lo, hi, heads, kv_heads, dim, rotary, rng.choice([2, 3, 3, 4]), rng.random() < 0.5, page, dtype, cache,
                     layout, rng.random() < 0.4)
    elif op == "compact":
        layers, new = rng.choice([1, 2, 4, 8]), _spread(rng, 1, 64)
        batch = _spread(rng, 1, max(1, min(256, 4 * 256 * 32 * 8 * 128 // (layers * new * kv_heads * dim))))
        hi = _spread(rng, 1, max(1, min(2000, 150_000_000 // (layers * batch * kv_heads * dim))))
        case = _compact("", layers, batch, new, rng.choice([0, hi]), hi, kv_heads, dim, page, cache, layout)
    else:
        layers = rng.choice([1, 2, 4, 8])
        most = 4 * 2000 * 8 * 128 * 32 // (SIZES[cache] * layers * kv_heads * dim * page)
        case = _copy("", layers, _spread(rng, 1, max(1, min(4000, most))), kv_heads, dim, page, cache)
    return {k: v for k, v in case.items() if k != "name"}


def _rng(case):
    """Lengths and trees are the case's own, the same for every seed."""
    return random.Random("%s %d %d" % (case["op"], case["batch"], case["hi"]))


def _lengths(case):
    """Tokens of context of each sequence (prompts: of the whole sequence), the longest among them."""
    r = _rng(case)
    got = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    got[r.randrange(case["batch"])] = case["hi"]
    return got


def _news(case):
    """How many drafted tokens each sequence has."""
    r = random.Random("new %d %d" % (case["batch"], case["new_hi"]))
    got = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    got[r.randrange(case["batch"])] = case["new_hi"]
    return got


def _masks(case):
    """For each drafted token which of its sequence's it sees, as whole numbers: a tree's ancestors and the token itself."""
    r, got = random.Random("tree %d %d" % (case["batch"], case["new_hi"])), []
    for n in _news(case):
        mine = []
        for i in range(n):
            parent = i - 1 if case["chain"] else r.randint(max(-1, i - 6), i - 1)
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << i)
        got.append(mine)
    return got


def _kept(case):
    """Of each sequence's drafted tokens the ones that are kept, ascending."""
    r, got = random.Random("kept %d %d" % (case["batch"], case["new"])), []
    for _ in range(case["batch"]):
        mine, at = [], -1
        while True:
            at += 1 + (r.randint(0, 3) if r.random() < 0.6 else 0)
            if at >= case["new"] or r.random() < 0.1:
                break
            mine.append(at)
        got.append(mine)
    got[0] = list(range(1, case["new"], 2))  # one that moves in every case of two drafts or more
    return got


def work(case):
    c = SIZES[case["cache"]]
    if case["op"] == "copy":
        return {"bytes": 4 * case["layers"] * case["pairs"] * case["page"] * case["kv_heads"] * case["dim"] * c, "flops": 0}
    if case["op"] == "compact":
        moved = sum(sum(i != x for i, x in enumerate(mine)) for mine in _kept(case))
        return {"bytes": 4 * case["layers"] * moved * case["kv_heads"] * case["dim"] * c + 8 * case["batch"] * (1 + case["new"]), "flops": 0}
    e, w = SIZES[case["dtype"]], case.get("window", 0)
    if case["op"] == "axes":
        tokens = sum(_lengths(case)) if case["new"] == 0 else case["batch"] * case["new"]
        q, kv = case["heads"] * case["dim"], case["kv_heads"] * case["dim"]
        return {"bytes": tokens * ((2 * q + 2 * kv) * e + 2 * kv * c + 4 * case["axes"]),
                "flops": 3 * tokens * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    read = seen = rows = 0
    for context, masks in zip(_lengths(case), _masks(case)):
        counts = [bin(m).count("1") for m in masks]
        first = max(0, min(context, context - w + min(counts))) if w else 0  # the first token of context that a row sees
        read += context - first + len(masks)
        seen += sum(min(w, context + n) if w else context + n for n in counts)
        rows += len(masks)
    return {"bytes": read * case["kv_heads"] * case["dim"] * 2 * c + rows * case["heads"] * (2 * case["dim"] * e + 4),
            "flops": 4 * seen * case["heads"] * case["dim"]}


def _cache(case, g, layers, longest, scales):
    """Pages of `layers` layers and a table in no order."""
    batch, page, kv_heads, dim = case["batch"], case["page"], case["kv_heads"], case["dim"]
    per = -(-max(longest, 1) // page)
    pages = batch * per + 1
    table = torch.randperm(pages, generator=g, device="cuda")[: batch * per].to(torch.int32).view(batch, per)
    shape = (pages, page, kv_heads, dim) if case["layout"] == "NHD" else (pages, kv_heads, page, dim)
    return table, [[_pages(case, g, shape, scale) for _ in range(layers)] for scale in scales]


def _pages(case, g, shape, scale):
    got = torch.empty(shape, dtype=DTYPES[case["cache"]], device="cuda")
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, shape[0], step):  # 64 Mi values at a time
        x = torch.randn((min(step, shape[0] - i),) + shape[1:], generator=g, device="cuda")
        got[i:i + step] = (x / scale).clamp(-448, 448).to(got.dtype) if case["cache"] == "e4m3" else x.to(got.dtype)
    return got


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    scales = (0.03125, 0.015625) if case["cache"] == "e4m3" else (1.0, 1.0)
    if case["op"] == "copy":
        shape = (2 * case["pairs"] + 3, case["page"], case["kv_heads"], case["dim"])
        order = torch.randperm(shape[0], generator=g, device="cuda").to(torch.int32)
        src = order[case["pairs"]:2 * case["pairs"]].clone()
        src[::5] = src[0].clone()  # a page that several sequences share is copied for each
        return {"case": case, "src": src, "dst": order[: case["pairs"]].clone(),
                "k_pages": [_pages(case, g, shape, scales[0]) for _ in range(case["layers"])],
                "v_pages": [_pages(case, g, shape, scales[1]) for _ in range(case["layers"])]}
    context = _lengths(case)
    if case["op"] == "compact":
        kept = _kept(case)
        table, (k, v) = _cache(case, g, case["layers"], max(context) + case["new"], scales)
        wide = [mine + [-1] * (case["new"] - len(mine)) for mine in kept]
        return {"case": case, "page_table": table, "k_pages": k, "v_pages": v, "lengths": _ints([n + case["new"] for n in context]),
                "kept": _ints(wide)}
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "tree":
        news = _news(case)
        table, (k, v) = _cache(case, g, 1, max(c + n for c, n in zip(context, news)), scales)
        words = -(-max(news) // 64)
        flat = [m for mine in _masks(case) for m in mine]
        signed = [[(m >> 64 * i & (1 << 63) - 1) - (m >> 64 * i & 1 << 63) for i in range(words)] for m in flat]
        q = 2 * torch.randn(sum(news), case["heads"], case["dim"], generator=g, device="cuda")
        return {"case": case, "page_table": table, "k_pages": k[0], "v_pages": v[0], "lengths": _ints([c + n for c, n in zip(context, news)]),
                "k_scale": scales[0], "v_scale": scales[1], "q": q.to(dtype), "longest": max(news),
                "mask": None if case["chain"] else torch.tensor(signed, dtype=torch.int64, device="cuda"),
                "seq_start": None if min(news) == max(news) else _ints([sum(news[:b]) for b in range(len(news) + 1)])}
    table, (k, v) = _cache(case, g, 1, max(context), scales)
    new = context if case["new"] == 0 else [case["new"]] * case["batch"]
    tokens = sum(new)
    qkv = torch.randn(tokens, case["heads"] + 2 * case["kv_heads"], case["dim"], generator=g, device="cuda").to(dtype)
    s = {"case": case, "page_table": table, "k_pages": k[0], "v_pages": v[0], "lengths": _ints(context), "k_scale": scales[0], "v_scale": scales[1]}
    s["q"], s["k"], s["v"] = qkv.split([case["heads"], case["kv_heads"], case["kv_heads"]], dim=1)  # as one projection gives them
    s["seq_start"] = None if case["new"] == 1 else _ints([sum(new[:b]) for b in range(case["batch"] + 1)])
    half = case["rotary"] // 2
    j = torch.arange(half, device="cuda", dtype=torch.float64)
    s["inv_freq"] = (500000.0 ** (-2 * j / case["rotary"])).float()
    # frames of 24 rows of 32 patches, each sequence's with a start of its own
    t = torch.arange(tokens, device="cuda")
    base = torch.randint(0, 5000, (1,), generator=g, device="cuda")
    steps = [t // 768, t // 32 % 24, t % 32, t][: case["axes"]]
    s["positions"] = torch.stack([base + x for x in steps]).to(torch.int32)
    s["pair_axis"] = [x % case["axes"] if case["turns"] else x * case["axes"] // half for x in range(half)]
    return s


def _visible(s):
    """[batch, drafted, tokens] which tokens of its sequence each drafted token sees, and [batch, drafted] the tokens' rows."""
    case, n = s["case"], s["lengths"].long()[:, None]
    tokens = s["q"].shape[0]
    if s["seq_start"] is None:
        first = torch.arange(case["batch"], device="cuda")[:, None] * s["longest"]
        many = torch.full_like(first, s["longest"])
    else:
        first, many = s["seq_start"].long()[:-1, None], s["seq_start"].long().diff()[:, None]
    i = torch.arange(s["longest"], device="cuda")
    row = (first + i).clamp(max=tokens - 1)
    at = torch.arange(s["page_table"].shape[1] * case["page"], device="cuda")[None, None]
    draft = at - (n - many)[:, :, None]  # which drafted token a token of the sequence is, below 0 for context
    if s["mask"] is None:
        mine = draft <= i[None, :, None]
    else:
        word = s["mask"][row].gather(2, (draft.clamp(min=0) // 64).clamp(max=s["mask"].shape[1] - 1).expand(-1, s["longest"], -1))
        mine = (word >> (draft.clamp(min=0) % 64) & 1).bool()
    see = (draft < 0) | (mine & (draft < many[:, :, None]))
    see = see & (at < n[:, :, None]) & (i[None] < many)[:, :, None]
    if case["window"]:
        see = see & (see.sum(2, keepdim=True) - see.cumsum(2) < case["window"])  # the last ones of those it sees
    return see, row, (i[None] < many)


def _gathered(s, kind, keep):
    """[batch, kv_heads, length, dim] values of the cache in 32 bits, zeros behind each sequence."""
    case, pages = s["case"], s[kind + "_pages"]
    got = (pages.view(torch.uint8) if case["cache"] == "e4m3" else pages)[s["page_table"].long()]
    got = got.movedim(3, 1) if case["layout"] == "NHD" else got.movedim(2, 1)
    got = got.flatten(2, 3)
    got = (got.contiguous().view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else got).float()
    return torch.where(keep[:, None, :, None], got * s[kind + "_scale"], 0.0)


def _plain_tree(s):
    case = s["case"]
    see, row, mine = _visible(s)
    heads, dim, kv_heads, batch = case["heads"], case["dim"], case["kv_heads"], case["batch"]
    keep = torch.arange(see.shape[2], device="cuda")[None] < s["lengths"].long()[:, None]
    q = s["q"].float()[row].view(batch, -1, kv_heads, heads // kv_heads, dim).movedim(1, 3)  # [batch, kv_heads, group, drafted, dim]
    shape = q.shape
    scores = (q.reshape(batch, kv_heads, -1, dim) @ _gathered(s, "k", keep).transpose(2, 3)).view(*shape[:4], -1) * dim ** -0.5
    if case["softcap"]:
        scores = case["softcap"] * torch.tanh(scores / case["softcap"])
    scores = torch.where(see[:, None, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ _gathered(s, "v", keep)).view(shape) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.movedim(3, 1).flatten(2, 3)[mine].to(s["q"].dtype), "lse": lse.movedim(3, 1).flatten(2, 3)[mine]}


def _rotated(x, angle, interleaved):
    half = angle.shape[1]
    x = x.float()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _stored(x, scale, pages):
    if pages.dtype == torch.float8_e4m3fn:
        return (x / scale).clamp(-448, 448).to(pages.dtype).view(torch.uint8)
    return x.to(pages.dtype)


def _bits(pages):
    return pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages


def _plain_axes(s):
    case, lengths = s["case"], s["lengths"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    if s["seq_start"] is None:
        seq, pos = t, lengths - 1
    else:
        start = s["seq_start"].long()
        seq = torch.searchsorted(start, t, right=True) - 1
        pos = lengths[seq] - (start[1:] - start[:-1])[seq] + t - start[seq]
    angle = s["positions"].double()[torch.tensor(s["pair_axis"], device="cuda")].T * s["inv_freq"].double()
    page, slot = s["page_table"].long()[seq, pos // case["page"]], pos % case["page"]
    at = (page, slot) if case["layout"] == "NHD" else (page, slice(None), slot)
    _bits(s["k_pages"])[at] = _stored(_rotated(s["k"], angle, case["interleaved"]), s["k_scale"], s["k_pages"])
    _bits(s["v_pages"])[at] = _stored(s["v"].float(), s["v_scale"], s["v_pages"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q": _rotated(s["q"], angle, case["interleaved"]).to(s["q"].dtype)}


def _plain_compact(s):
    case, kept = s["case"], s["kept"].long()
    context = s["lengths"].long() - case["new"]
    mine = kept >= 0
    seq, to = mine.nonzero(as_tuple=True)
    table = s["page_table"].long()

    def moved(pages):
        def place(at):
            page, slot = table[seq, at // case["page"]], at % case["page"]
            return (page, slot) if case["layout"] == "NHD" else (page, slice(None), slot)

        pages[place(context[seq] + to)] = pages[place(context[seq] + kept[seq, to])]

    [moved(_bits(p)) for p in s["k_pages"] + s["v_pages"]]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "lengths": (context + mine.sum(1)).to(torch.int32)}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    [_bits(p).index_copy_(0, dst, _bits(p)[src]) for p in s["k_pages"] + s["v_pages"]]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def run(s):
    case = s["case"]
    if own:
        import tensor_allreduce_residual_gb300 as ar

        if case["op"] == "tree":
            out, lse = ar.ar_tree_attention(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["lengths"], mask=s["mask"],
                                            seq_start=s["seq_start"], window=case["window"], softcap=case["softcap"], layout=case["layout"],
                                            k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
            return {"out": out, "lse": lse}
        if case["op"] == "axes":
            q = ar.ar_kv_append(s["k_pages"], s["v_pages"], s["page_table"], s["lengths"], s["k"], s["v"], q=s["q"], seq_start=s["seq_start"],
                                positions=s["positions"], pair_axis=s["pair_axis"], inv_freq=s["inv_freq"], interleaved=case["interleaved"],
                                layout=case["layout"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q": q}
        if case["op"] == "compact":
            lengths = ar.ar_kv_compact(s["k_pages"], s["v_pages"], s["page_table"], s["lengths"], s["kept"], drafted=case["new"],
                                       layout=case["layout"])
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "lengths": lengths}
        ar.ar_kv_copy_pages(s["k_pages"], s["v_pages"], s["src"], s["dst"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return {"tree": _plain_tree, "axes": _plain_axes, "compact": _plain_compact, "copy": _plain_copy}[case["op"]](s)


def exact(case, seed):
    s = prepare(case, seed)

    def tree():
        heads, kv_heads, dim, w = case["heads"], case["kv_heads"], case["dim"], case["window"]
        outs, lses, row = [], [], 0
        for b, (context, masks) in enumerate(zip(_lengths(case), _masks(case))):
            n, many = context + len(masks), len(masks)
            used = s["page_table"][b, : -(-n // case["page"])].long()
            both = []
            for kind in ("k", "v"):
                pages = s[kind + "_pages"]
                x = _bits(pages)[used].view(pages.dtype).double() * s[kind + "_scale"]
                x = x.transpose(1, 2) if case["layout"] == "HND" else x
                both.append(x.reshape(-1, kv_heads, dim)[:n])
            q = s["q"][row:row + many].double().view(many, kv_heads, -1, dim)
            z = torch.einsum("thgd,jhd->thgj", q, both[0]) / math.sqrt(dim)
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            hide = torch.zeros(many, n, dtype=torch.bool)
            for t, m in enumerate(masks):
                left = w or n
                for i in range(many - 1, -1, -1):
                    left -= m >> i & 1
                    hide[t, context + i] = not (m >> i & 1) or left < 0
                hide[t, : max(0, context - max(left, 0))] = True
            z = z.masked_fill(hide.cuda()[:, None, None], -math.inf)
            lses.append(torch.logsumexp(z, 3).view(many, heads))
            outs.append(torch.einsum("thgj,jhd->thgd", torch.softmax(z, 3), both[1]).reshape(many, heads, dim))
            row += many
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}

    def axes():
        lengths, page, table = _lengths(case), case["page"], s["page_table"].tolist()
        k_pages, v_pages, half = s["k_pages"].double(), s["v_pages"].double(), case["rotary"] // 2
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        angle = torch.stack([s["positions"][a].double() * f for a, f in zip(s["pair_axis"], s["inv_freq"].double())], 1)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]

        def turned(x):
            head = x[..., : 2 * half]
            pair = head.unflatten(-1, (half, 2)) if case["interleaved"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            return torch.cat([(z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2), x[..., 2 * half:]], -1)

        q_out, keys, values, row = turned(q), turned(k) / s["k_scale"], v / s["v_scale"], 0
        if case["cache"] == "e4m3":
            keys, values = keys.clamp(-448, 448), values.clamp(-448, 448)
        for b, n in enumerate(lengths):
            at, many = n - (n if case["new"] == 0 else case["new"]), n if case["new"] == 0 else case["new"]
            done = 0
            while done < many:  # a page at a time
                p, lo = table[b][(at + done) // page], (at + done) % page
                take = min(page - lo, many - done)
                for pages, x in ((k_pages, keys), (v_pages, values)):
                    part = x[row + done:row + done + take]
                    if case["layout"] == "NHD":
                        pages[p, lo:lo + take] = part
                    else:
                        pages[p, :, lo:lo + take] = part.transpose(0, 1)
                done += take
            row += many
        return {"k_pages": k_pages, "v_pages": v_pages, "q": q_out}

    def compact():
        page, table, context, kept = case["page"], s["page_table"].tolist(), _lengths(case), _kept(case)
        moves = [(table[b], c + i, c + x) for b, (c, mine) in enumerate(zip(context, kept)) for i, x in enumerate(mine) if x != i]
        to = torch.tensor([(t[i // page], i % page) for t, i, _ in moves], dtype=torch.long, device="cuda").view(-1, 2)
        come = torch.tensor([(t[i // page], i % page) for t, _, i in moves], dtype=torch.long, device="cuda").view(-1, 2)
        got = {}
        for kind in ("k_pages", "v_pages"):
            got[kind] = [p.double() for p in s[kind]]
            for x in got[kind]:
                x = x if case["layout"] == "NHD" else x.transpose(1, 2)
                x[to[:, 0], to[:, 1]] = x[come[:, 0], come[:, 1]].clone()
        return {**got, "lengths": None}

    def copy():
        got = {}
        for kind in ("k_pages", "v_pages"):
            got[kind] = [p.double() for p in s[kind]]
            for x in got[kind]:
                x[s["dst"].long()] = x[s["src"].long()].clone()
        return got

    return {"tree": tree, "axes": axes, "compact": compact, "copy": copy}[case["op"]]()
