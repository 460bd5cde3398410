"""Cases of the paged key-value cache operators: appending with rotation, attention of one new token, and the join of
partial attentions.  `run` computes a case in plain torch operations, or through the package's calls where `own` is true."""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZES = {"fp32": 4, "fp16": 2, "bf16": 2, "e4m3": 1}


def _append(name, batch, new, lo, hi, heads, kv_heads, dim, rotary, page, dtype, cache, layout, interleaved):
    """`new` tokens of each of `batch` sequences (0: prompts of lo..hi tokens, whole) that then hold lo..hi tokens."""
    return {"op": "append", "name": name, "batch": batch, "new": new, "lo": lo, "hi": hi, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "rotary": rotary, "page": page, "dtype": dtype, "cache": cache, "layout": layout, "interleaved": interleaved}


def _attend(name, batch, lo, hi, heads, kv_heads, dim, page, dtype, cache, layout, window=0, softcap=0.0):
    return {"op": "attend", "name": name, "batch": batch, "lo": lo, "hi": hi, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "dtype": dtype, "cache": cache, "layout": layout, "window": window, "softcap": softcap}


def _join(name, ranks, rows, dim, dtype):
    return {"op": "join", "name": name, "ranks": ranks, "rows": rows, "dim": dim, "dtype": dtype}


def listed():
    return [
        # one decode step of a small batch, one rank of eight at hidden 8192: all latency
        _append("append step bf16", 8, 1, 17, 2000, 8, 1, 128, 128, 16, "bf16", "bf16", "NHD", False),
        # one decode step of a large batch into an 8-bit cache
        _append("append step e4m3", 256, 1, 1, 120, 32, 4, 128, 128, 64, "fp16", "e4m3", "HND", True),
        # a few prompts at once with every head of hidden 8192
        _append("append prompts bf16", 4, 0, 1000, 3000, 64, 8, 128, 128, 64, "bf16", "bf16", "NHD", False),
        # prompts with a head size and a part of it rotated that fill no 16-byte vectors evenly
        _append("append prompts fp32", 7, 0, 1, 700, 12, 3, 80, 40, 17, "fp32", "fp32", "HND", False),
        # one short sequence, one rank of eight: all latency
        _attend("attend short bf16", 1, 511, 511, 8, 1, 128, 16, "bf16", "bf16", "NHD"),
        # one long sequence, one rank of eight: the length has to be split to fill the GPU
        _attend("attend long bf16", 1, 131072, 131072, 8, 1, 128, 64, "bf16", "bf16", "NHD"),
        # a ragged batch in steady decoding
        _attend("attend batch bf16", 64, 1, 8191, 32, 4, 128, 16, "bf16", "bf16", "NHD"),
        # a large ragged batch on an 8-bit cache
        _attend("attend batch e4m3", 128, 1, 16384, 16, 2, 128, 64, "bf16", "e4m3", "HND"),
        # a sliding window, capped scores, small heads, pages that end inside a tile
        _attend("attend window fp16", 48, 1, 5000, 16, 8, 64, 24, "fp16", "fp16", "HND", 1024, 30.0),
        # 32-bit values, two query heads on each pair of keys and values
        _attend("attend batch fp32", 16, 1, 4096, 16, 8, 96, 32, "fp32", "fp32", "NHD"),
        # two ranks' parts of a small step
        _join("join step fp16", 2, 64, 128, "fp16"),
        # eight ranks' parts of many rows
        _join("join rows bf16", 8, 65536, 128, "bf16"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "join"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp16", "fp32"])
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    if op == "join":
        return {k: v for k, v in _join("", rng.randint(1, 16), _spread(rng, 1, 32768), rng.choice([dim, dim, 100, 33]), dtype).items() if k != "name"}
    cache = "e4m3" if dtype != "fp32" and rng.random() < 0.35 else dtype
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
    page = rng.choice([1, 8, 16, 16, 17, 32, 64, 64, 128])
    layout = rng.choice(["NHD", "HND"])
    if op == "append":
        rotary = rng.choice([dim, dim, dim // 2, 16])
        most = 8192 * 80 * 128 // ((heads + 2 * kv_heads) * dim)  # tokens of the largest listed case
        if rng.random() < 0.5:
            batch = _spread(rng, 1, min(512, most))
            new, hi = 1, _spread(rng, 1, 4096)
            hi = max(1, min(hi, 40_000_000 // (batch * kv_heads * dim)))
            lo = 1
        else:
            batch = rng.randint(1, 8)
            new, hi = 0, _spread(rng, 2, max(2, min(8192, most // batch)))
            lo = max(1, hi // 4)
        case = _append("", batch, new, lo, hi, heads, kv_heads, dim, rotary, page, dtype, cache, layout, rng.random() < 0.4)
    else:
        hi = _spread(rng, 1, 131072)
        most = 128 * 16384 * 2 * 128 // 6 // (kv_heads * dim)  # cached values: a sixth of the largest listed case's room
        hi = min(hi, most)
        batch = _spread(rng, 1, max(1, min(256, most // hi)))
        window = _spread(rng, 1, 8192) if rng.random() < 0.25 else 0
        case = _attend("", batch, rng.choice([0, 1, max(1, hi // 2)]), hi, heads, kv_heads, dim, page, dtype, cache, layout, window,
                       rng.choice([0.0, 0.0, 0.0, 30.0]))
    return {k: v for k, v in case.items() if k != "name"}


def _lengths(case):
    """The sequences' lengths: the case's own, the same for every seed, the longest among them."""
    r = random.Random(1000003 * case["batch"] + case["hi"])
    got = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    got[r.randrange(case["batch"])] = case["hi"]
    return got


def _attended(case):
    w = case["window"]
    return [min(n, w) if w else n for n in _lengths(case)]


def work(case):
    if case["op"] == "join":
        n, e = case["rows"] * case["dim"], SIZES[case["dtype"]]
        return {"bytes": (case["ranks"] + 1) * (n * e + case["rows"] * 4), "flops": 2 * case["ranks"] * n}
    e, c = SIZES[case["dtype"]], SIZES[case["cache"]]
    if case["op"] == "append":
        tokens = sum(_lengths(case)) if case["new"] == 0 else case["batch"] * case["new"]
        q, kv = case["heads"] * case["dim"], case["kv_heads"] * case["dim"]
        return {"bytes": tokens * ((2 * q + 2 * kv) * e + 2 * kv * c), "flops": 3 * tokens * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    keys = sum(_attended(case))
    out = case["batch"] * case["heads"]
    return {"bytes": keys * case["kv_heads"] * case["dim"] * 2 * c + out * (2 * case["dim"] * e + 4), "flops": 4 * keys * case["heads"] * case["dim"]}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    if case["op"] == "join":
        lse = [4 + 2 * torch.randn(case["rows"], generator=g, device="cuda") for _ in range(case["ranks"])]
        for r, x in enumerate(lse[1:]):  # some ranks hold none of a row's keys
            x[r::7] = -math.inf
        return {"case": case, "partials": [normal(case["rows"], case["dim"]) for _ in range(case["ranks"])], "lse": lse}
    lengths = _lengths(case)
    batch, page, kv_heads, dim = case["batch"], case["page"], case["kv_heads"], case["dim"]
    per = -(-max(case["hi"], 1) // page)
    pages = batch * per + 1
    table = torch.randperm(pages, generator=g, device="cuda")[: batch * per].to(torch.int32).view(batch, per)
    shape = (pages, page, kv_heads, dim) if case["layout"] == "NHD" else (pages, kv_heads, page, dim)
    small = case["cache"] == "e4m3"
    s = {"case": case, "page_table": table, "lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda"),
         "k_scale": 0.03125 if small else 1.0, "v_scale": 0.015625 if small else 1.0}
    for kind in ("k", "v"):
        s[kind + "_pages"] = torch.empty(shape, dtype=DTYPES[case["cache"]], device="cuda")
        step = max(1, (1 << 26) // (page * kv_heads * dim))
        for i in range(0, pages, step):  # 64 Mi values at a time
            x = torch.randn((min(step, pages - i),) + shape[1:], generator=g, device="cuda")
            s[kind + "_pages"][i:i + step] = (x / s[kind + "_scale"]).clamp(-448, 448).to(DTYPES["e4m3"]) if small else x.to(dtype)
    if case["op"] == "attend":
        s["q"] = normal(batch, case["heads"], dim, std=2.0)
        return s
    new = lengths if case["new"] == 0 else [case["new"]] * batch
    tokens = sum(new)
    qkv = normal(tokens, case["heads"] + 2 * kv_heads, dim)  # as one projection gives them
    s["q"], s["k"], s["v"] = qkv.split([case["heads"], kv_heads, kv_heads], dim=1)
    s["seq_start"] = None
    if case["new"] != 1:
        s["seq_start"] = torch.tensor([sum(new[:b]) for b in range(batch + 1)], dtype=torch.int32, device="cuda")
    j = torch.arange(case["rotary"] // 2, device="cuda", dtype=torch.float64)
    s["inv_freq"] = (500000.0 ** (-2 * j / case["rotary"])).float()
    return s


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


def _plain_append(s):
    case, lengths = s["case"], s["lengths"].long()
    tokens = s["q"].shape[0]
    t = torch.arange(tokens, device="cuda")
    if s["seq_start"] is None:
        seq, pos = t, lengths - 1
    else:
        start = s["seq_start"].long()
        seq = torch.searchsorted(start, t, right=True) - 1
        pos = lengths[seq] - (start[1:] - start[:-1])[seq] + t - start[seq]
    angle = pos.double()[:, None] * s["inv_freq"].double()
    page, slot = s["page_table"].long()[seq, pos // case["page"]], pos % case["page"]
    k = _stored(_rotated(s["k"], angle, case["interleaved"]), s["k_scale"], s["k_pages"])
    v = _stored(s["v"].float(), s["v_scale"], s["v_pages"])
    bits = (lambda x: x.view(torch.uint8)) if case["cache"] == "e4m3" else (lambda x: x)
    at = (page, slot) if case["layout"] == "NHD" else (page, slice(None), slot)
    bits(s["k_pages"])[at] = k
    bits(s["v_pages"])[at] = v
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q": _rotated(s["q"], angle, case["interleaved"]).to(s["q"].dtype)}


def _gathered(s, kind, keep):
    """[batch, kv_heads, length, dim] values of the cache in 32 bits, zeros behind each sequence."""
    case, pages = s["case"], s[kind + "_pages"]
    got = (pages.view(torch.uint8) if case["cache"] == "e4m3" else pages)[s["page_table"].long()]
    if case["layout"] == "NHD":
        got = got.movedim(3, 1)
    else:
        got = got.movedim(2, 1)
    got = got.flatten(2, 3)
    got = (got.contiguous().view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else got).float()
    return torch.where(keep[:, None, :, None], got * s[kind + "_scale"], 0.0)


def _plain_attend(s):
    case, n = s["case"], s["lengths"].long()[:, None]
    batch, heads, dim = s["q"].shape
    at = torch.arange(s["page_table"].shape[1] * case["page"], device="cuda")[None]
    keep = at < n
    if case["window"]:
        keep = keep & (at >= n - case["window"])
    q = s["q"].float().view(batch, case["kv_heads"], -1, dim)
    scores = q @ _gathered(s, "k", keep).transpose(2, 3) * dim ** -0.5
    if case["softcap"]:
        scores = case["softcap"] * torch.tanh(scores / case["softcap"])
    scores = torch.where(keep[:, None, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = p @ _gathered(s, "v", keep) / torch.where(total == 0, 1.0, total)
    return {"out": out.view(batch, heads, dim).to(s["q"].dtype), "lse": (top + torch.log(total)).view(batch, heads)}


def _plain_join(s):
    lse = torch.stack(s["lse"])
    top = lse.amax(0)
    w = torch.exp(lse - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(0)
    x = torch.where((w == 0)[..., None], 0.0, torch.stack(s["partials"]).float())
    out = (x * w[..., None]).sum(0) / torch.where(total == 0, 1.0, total)[:, None]
    return {"out": out.to(s["partials"][0].dtype), "lse": top + torch.log(total)}


def run(s):
    case = s["case"]
    if own:
        import tensor_allreduce_residual_gb300 as ar

        if case["op"] == "append":
            q = ar.ar_kv_append(s["k_pages"], s["v_pages"], s["page_table"], s["lengths"], s["k"], s["v"], q=s["q"], seq_start=s["seq_start"],
                                inv_freq=s["inv_freq"], interleaved=case["interleaved"], layout=case["layout"], k_scale=s["k_scale"],
                                v_scale=s["v_scale"])
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q": q}
        if case["op"] == "attend":
            out, lse = ar.ar_paged_attention(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["lengths"], window=case["window"],
                                             softcap=case["softcap"], layout=case["layout"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                             return_lse=True)
        else:
            out, lse = ar.ar_attention_join(s["partials"], s["lse"], return_lse=True)
        return {"out": out, "lse": lse}
    return {"append": _plain_append, "attend": _plain_attend, "join": _plain_join}[case["op"]](s)


def exact(case, seed):
    s = prepare(case, seed)

    def turned(row, pos, freq, interleaved):
        """Heads' rows [n, dim], each turned at its position [n, 1], as complex numbers."""
        half = freq.numel()
        pair = row[:, : 2 * half].reshape(-1, half, 2) if interleaved else row[:, : 2 * half].reshape(-1, 2, half).transpose(1, 2)
        z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(pos * freq), pos * freq)
        flat = torch.view_as_real(z) if interleaved else torch.view_as_real(z).transpose(1, 2)
        return torch.cat([flat.reshape(-1, 2 * half), row[:, 2 * half:]], 1)

    def append():
        lengths, page, table = _lengths(case), case["page"], s["page_table"].tolist()
        k_pages, v_pages, freq = s["k_pages"].double(), s["v_pages"].double(), s["inv_freq"].double()
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        q_out, row = torch.empty_like(q), 0
        for b, n in enumerate(lengths):
            first = 0 if case["new"] == 0 else n - case["new"]
            many = n - first
            pos = torch.arange(first, n, dtype=torch.float64, device="cuda")
            got = []
            for x in (q, k):
                heads = x.shape[1]
                flat = x[row:row + many].transpose(0, 1).reshape(heads * many, -1)
                got.append(turned(flat, pos.repeat(heads)[:, None], freq, case["interleaved"]).view(heads, many, -1).transpose(0, 1))
            q_out[row:row + many] = got[0]
            keys, values = got[1] / s["k_scale"], v[row:row + many] / s["v_scale"]
            if case["cache"] == "e4m3":
                keys, values = keys.clamp(-448, 448), values.clamp(-448, 448)
            done = 0
            while done < many:  # a page at a time
                at, lo = table[b][(first + done) // page], (first + done) % page
                take = min(page - lo, many - done)
                for pages, x in ((k_pages, keys), (v_pages, values)):
                    if case["layout"] == "NHD":
                        pages[at, lo:lo + take] = x[done:done + take]
                    else:
                        pages[at, :, lo:lo + take] = x[done:done + take].transpose(0, 1)
                done += take
            row += many
        return {"k_pages": k_pages, "v_pages": v_pages, "q": q_out}

    def attend():
        heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
        out = torch.zeros(case["batch"], heads, dim, dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], heads), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(case)):
            if n == 0:
                continue
            used = s["page_table"][b, : -(-n // case["page"])].long()
            first = max(0, n - case["window"]) if case["window"] else 0
            both = []
            for kind in ("k", "v"):
                pages = s[kind + "_pages"]
                x = pages.view(torch.uint8)[used].view(pages.dtype) if case["cache"] == "e4m3" else pages[used]
                x = x.double() * s[kind + "_scale"]
                x = x.transpose(1, 2) if case["layout"] == "HND" else x
                both.append(x.reshape(-1, kv_heads, dim)[first:n])
            z = torch.einsum("hgd,jhd->hgj", s["q"][b].double().view(kv_heads, -1, dim), both[0]) / math.sqrt(dim)
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            lse[b] = torch.logsumexp(z, 2).view(-1)
            out[b] = torch.einsum("hgj,jhd->hgd", torch.softmax(z, 2), both[1]).reshape(heads, dim)
        return {"out": out, "lse": lse}

    def join():
        lse = torch.stack(s["lse"], 1).double()
        share = torch.softmax(torch.where(lse == -math.inf, torch.finfo(torch.float64).min, lse), 1)
        return {"out": torch.einsum("nr,rnd->nd", share, torch.stack(s["partials"]).double()), "lse": torch.logsumexp(lse, 1)}

    return {"append": append, "attend": attend, "join": join}[case["op"]]()
