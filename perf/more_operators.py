"""Workloads of the operators in front of and around an 8-bit paged key-value cache.

Four operators that the full-attention layers of a hybrid model need: page
tables, positions and slots built on the GPU from request lengths; the norms of
queries and keys with the position rotation (and their gradients); new keys and
values into e4m3 pages with one scale per page and head; and the attention of
one new token over such a cache. Where ``own`` is false each runs in its plain
form (elementary torch operations in 32 bits, rounded once at the end; angles
in 64); where it is true the package's kernels run.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # every running sequence gets one token; a few have finished
        {"name": "plan step", "op": "plan", "b": 256, "page": 64, "width": 256, "new": 256,
         "step": True, "release": True},
        # ragged prompts join, some in the slots of sequences that have just finished
        {"name": "plan prompts", "op": "plan", "b": 64, "page": 16, "width": 2048, "new": 65536,
         "step": False, "release": True},
        # one token of one sequence, small model: latency
        {"name": "heads token", "op": "heads", "t": 1, "hq": 32, "hk": 8, "dim": 128, "rot": 128,
         "pairs": False, "seqs": 1, "far": 131072},
        # slices of a fused projection, an ordinary prompt
        {"name": "heads prompt", "op": "heads", "t": 8192, "hq": 64, "hk": 8, "dim": 128, "rot": 128,
         "pairs": False, "seqs": 1, "far": 0},
        # a training step on that prompt
        {"name": "heads gradient", "op": "heads_backward", "t": 8192, "hq": 64, "hk": 8, "dim": 128,
         "rot": 128, "pairs": False, "seqs": 1, "far": 0, "dout32": False},
        # a ragged batch, a quarter of the channels rotated in pairs, gradients in fp32
        {"name": "heads gradient ragged", "op": "heads_backward", "t": 5003, "hq": 16, "hk": 2,
         "dim": 64, "rot": 16, "pairs": True, "seqs": 16, "far": 100000, "dout32": True},
        # one token for each of 256 running sequences
        {"name": "append step", "op": "append", "b": 256, "t": 256, "step": True, "hkv": 8, "dim": 128,
         "page": 64, "longest": 1024, "heads_first": False},
        # ragged prompts, some continued in the middle of a page
        {"name": "append prompts", "op": "append", "b": 16, "t": 8191, "step": False, "hkv": 8,
         "dim": 128, "page": 64, "longest": 2048, "heads_first": True},
        # a long document
        {"name": "append long", "op": "append", "b": 1, "t": 65536, "step": False, "hkv": 8, "dim": 128,
         "page": 32, "longest": 0, "heads_first": False},
        # one sequence, a short cache: latency
        {"name": "attention short", "op": "attention", "b": 1, "hq": 32, "hkv": 8, "dim": 128,
         "page": 16, "longest": 700, "ragged": False, "heads_first": False},
        # a serving batch with lengths spread over a factor of thousands, one slot unused
        {"name": "attention ragged", "op": "attention", "b": 64, "hq": 64, "hkv": 8, "dim": 128,
         "page": 64, "longest": 16384, "ragged": True, "heads_first": True},
        # two long documents: few rows, a long axis
        {"name": "attention long", "op": "attention", "b": 2, "hq": 32, "hkv": 8, "dim": 128,
         "page": 32, "longest": 131072, "ragged": False, "heads_first": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


PAGES = [1, 8, 16, 17, 32, 64, 64, 100, 128]


def draw(rng):
    op = rng.choice(["plan", "heads", "heads_backward", "append", "append", "attention",
                     "attention", "attention"])
    if op == "plan":
        b = _log(rng, 1, 4096)
        page, width = rng.choice(PAGES), _log(rng, 1, (1 << 20) // b)
        step = rng.random() < 0.5
        return {"op": op, "b": b, "page": page, "width": width, "step": step,
                "new": b if step else _log(rng, 1, min(1 << 17, max(1, b * page * width // 4))),
                "release": rng.random() < 0.7}
    if op in ("heads", "heads_backward"):
        dim = rng.choice([64, 128, 128, 256])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 3, 4, 6, 8, 8])
        t = _log(rng, 1, min(16384, (1 << 26) // ((hq + hk) * dim)))
        c = {"op": op, "t": t, "hq": hq, "hk": hk, "dim": dim,
             "rot": rng.choice([dim, dim, dim // 2, dim // 4, 16 * rng.randint(1, dim // 16)]),
             "pairs": rng.random() < 0.4, "seqs": rng.choice([1, 1, rng.randint(2, 24)]),
             "far": rng.choice([0, 0, _log(rng, 1, 1 << 20)])}
        if op == "heads_backward":
            c["dout32"] = rng.random() < 0.5
        return c
    hkv, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]), rng.choice(PAGES)
    c = {"op": op, "hkv": hkv, "dim": dim, "page": page, "heads_first": rng.random() < 0.5}
    if op == "append":
        c["step"] = rng.random() < 0.5
        c["b"] = _log(rng, 1, 512 if c["step"] else 32)
        c["t"] = c["b"] if c["step"] else _log(rng, c["b"], (1 << 26) // (hkv * dim * 2))
        c["longest"] = _log(rng, 1, min(8192, (1 << 18) // c["b"]))
        return c
    longest = _log(rng, 1, 131072)
    c["b"] = _log(rng, 1, max(1, min(256, (1 << 21) // (longest * hkv))))
    return {**c, "hq": hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16]), "longest": longest,
            "ragged": rng.random() < 0.7}


# ----------------------------------------------------------------- the inputs

def _lengths(total, n, gen):
    """n ragged lengths with the given sum, some of them perhaps zero."""
    cuts = torch.sort(torch.randint(0, total + 1, (n - 1,), generator=gen)).values
    return torch.diff(torch.cat([torch.zeros(1, dtype=torch.int64), cuts,
                                 torch.full((1,), total, dtype=torch.int64)]))


def _i32(t):
    return t.to(torch.int32).to(DEV)


def _deal(need, width, extra, gen):
    """A table that deals ids out in no order: ([n, width] on the host, ids left over)."""
    order = torch.randperm(int(need.sum()) + extra, generator=gen).to(torch.int32)
    table = torch.zeros(len(need), width, dtype=torch.int32)
    held = torch.arange(width) < need[:, None]
    table[held] = order[:int(need.sum())]
    return table, order[int(need.sum()):]


def prepare(case, seed):
    gen = torch.Generator(device="cpu").manual_seed(seed)
    dgen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=dgen, device=DEV, dtype=torch.float32) * scale).to(dtype)

    def cache_of(pages):
        """Pages that hold keys beside values, with their scales: numbers around 1, in e4m3 at
        scales that are powers of two."""
        h, p, d = case["hkv"], case["page"], case["dim"]
        shape = (pages, 2, h, p, d) if case["heads_first"] else (pages, 2, p, h, d)
        cache = torch.empty(shape, dtype=F8, device=DEV)
        scale = torch.exp2(torch.randint(-8, -5, (pages, 2, h), generator=dgen, device=DEV).float())
        per = scale[:, :, :, None, None] if case["heads_first"] else scale[:, :, None, :, None]
        for i in range(0, pages, 4096):
            part = randn(*cache[i:i + 4096].shape, dtype=torch.float32) / per[i:i + 4096]
            cache[i:i + 4096] = part.clamp(-448, 448).to(F8)
        if case["heads_first"]:
            cache = cache.transpose(2, 3)
        return {"k_cache": cache[:, 0], "v_cache": cache[:, 1], "k_scale": scale[:, 0],
                "v_scale": scale[:, 1]}

    op, s = case["op"], {"case": case}
    if op == "plan":
        b, page, width = case["b"], case["page"], case["width"]
        most = page * width
        new = torch.ones(b, dtype=torch.int64) if case["step"] else _lengths(case["new"], b, gen)
        new = new.clamp(max=most)
        lens = (torch.rand(b, generator=gen, dtype=torch.float64) * (most - new + 1)).long()
        gone = torch.rand(b, generator=gen) < 0.1
        if not case["release"]:
            gone = torch.zeros(b, dtype=torch.bool)
        if case["step"]:
            new[gone & (torch.rand(b, generator=gen) < 0.5)] = 0
        have = (lens + page - 1) // page
        pool = b * width + 5
        table, free = _deal(have, width, pool - int(have.sum()), gen)
        stack = torch.zeros(pool, dtype=torch.int32)
        stack[:len(free)] = free
        s.update(table=table.to(DEV), lens=_i32(lens), new=_i32(new), gone=gone.to(DEV),
                 free=stack.to(DEV), count=_i32(torch.tensor([len(free)])),
                 tokens=case["new"] if case["step"] else case["new"] + 7)
        return s
    if op in ("heads", "heads_backward"):
        t, hq, hk, d, rot = case["t"], case["hq"], case["hk"], case["dim"], case["rot"]
        whole = randn(t, (hq + 2 * hk) * d)   # q, k and v from one projection
        s["q"] = whole[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = whole[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["q_weight"] = 1 + 0.2 * randn(d, dtype=torch.float32)
        s["k_weight"] = 1 + 0.2 * randn(d, dtype=torch.float32)
        lens = _lengths(t, case["seqs"], gen)
        past = torch.randint(0, case["far"] + 1, (case["seqs"],), generator=gen)
        first = lens.cumsum(0) - lens
        pos = torch.arange(t) + torch.repeat_interleave(past - first, lens)
        s["positions"] = _i32(pos)
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(DEV)
        if op == "heads_backward":
            dtype = torch.float32 if case["dout32"] else torch.bfloat16
            s["dq_out"], s["dk_out"] = randn(t, hq, d, dtype=dtype), randn(t, hk, d, dtype=dtype)
        return s
    b, page, longest = case["b"], case["page"], case["longest"]
    if op == "append":
        new = torch.ones(b, dtype=torch.int64) if case["step"] else _lengths(case["t"], b, gen)
        past = torch.randint(0, longest + 1, (b,), generator=gen)
        if not case["step"]:   # half of the prompts are new
            past[torch.rand(b, generator=gen) < 0.5] = 0
        lens = past + new
        s["cu"] = None if case["step"] else _i32(torch.cat([torch.zeros(1, dtype=torch.int64),
                                                           new.cumsum(0)]))
        x = randn(case["t"], 3, case["hkv"], case["dim"])   # k and v out of a wider projection
        s["k"], s["v"] = x[:, 1], x[:, 2]
        s["k"].mul_(4 ** torch.rand(case["t"], 1, 1, generator=dgen, device=DEV))
    else:
        lens = torch.full((b,), longest, dtype=torch.int64)
        if case["ragged"]:
            lens = torch.exp(torch.rand(b, generator=gen) * math.log(longest)).round().to(torch.int64)
            lens[torch.randint(0, b, (1,), generator=gen)] = longest
            if b > 2:  # a slot with nothing in it
                lens[int((lens == lens.min()).nonzero()[0])] = 0
        s["q"] = randn(b, case["hq"], case["dim"])
    need = (lens + page - 1) // page
    pages = int(need.sum()) + 3
    if op == "append":   # as many as the longest pasts would need
        pages = (case["t"] + b * longest) // page + 2 * b + 3
    table, _ = _deal(need, max(1, int(need.max())), pages - int(need.sum()), gen)
    s.update(table=table.to(DEV), lens=_i32(lens), lens_host=lens.tolist(), **cache_of(pages))
    return s


# ------------------------------------------------------------ the plain forms

def _plain_plan(s):
    page, b, tokens = s["case"]["page"], s["case"]["b"], s["tokens"]
    lens, new, gone = s["lens"].long(), s["new"].long(), s["gone"]
    width, count = s["table"].shape[1], s["count"].long()
    at = torch.arange(width, device=DEV)
    # pages of finished sequences go on top of the stack
    drop = gone[:, None] & (at < ((lens + page - 1) // page)[:, None])
    rank = drop.reshape(-1).cumsum(0).reshape(b, width) - 1
    size = s["free"].shape[0]
    free = torch.cat([s["free"], s["free"].new_zeros(1)])   # one place for what is not pushed
    free[torch.where(drop, count + rank, size).reshape(-1)] = s["table"].reshape(-1)
    free = free[:size]
    top = count + drop.sum()
    lens = torch.where(gone, 0, lens)
    have, end = (lens + page - 1) // page, (lens + new + page - 1) // page
    fresh = (at >= have[:, None]) & (at < end[:, None])
    order = fresh.reshape(-1).cumsum(0).reshape(b, width) - 1
    table = torch.where(fresh, free[torch.where(fresh, top - 1 - order, 0)], s["table"])
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    row = torch.arange(tokens, device=DEV)
    live = row < cu[-1]
    seq = torch.searchsorted(cu[1:], row, right=True).clamp(max=b - 1)
    pos = torch.where(live, lens[seq] + row - cu[seq], 0)
    slot = table[seq, pos // page].long() * page + pos % page
    return {"table": table, "lens": (lens + new).to(torch.int32), "free": free,
            "count": (top - fresh.sum()).to(torch.int32), "cu": cu.to(torch.int32),
            "positions": pos.to(torch.int32), "slots": torch.where(live, slot, -1)}


EPS = 1e-6


def _angles(s):
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _turn(x, cos, sin, pairs):
    """The first channels turned by the angles: (i, i + n) together, or (2i, 2i + 1)."""
    n = cos.shape[-1]
    if pairs:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _plain_heads(s):
    cos, sin = _angles(s)
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s[name + "_weight"]
        out[name] = _turn(x, cos, sin, s["case"]["pairs"]).to(torch.bfloat16)
    return out


def _plain_heads_backward(s):
    cos, sin = _angles(s)
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        g = _turn(s["d%s_out" % name].float(), cos, -sin, s["case"]["pairs"])
        u = x * r
        out["d%s_weight" % name] = (g * u).sum((0, 1))
        g = g * s[name + "_weight"]
        out["d" + name] = (r * (g - u * (g * u).mean(-1, keepdim=True))).to(torch.bfloat16)
    return out


def _scale_for(top):
    """The least power of two that brings `top` to 448 or below, from 2^-126 on."""
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(top == 0, -126, e.clamp(min=-126))
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_append(s):
    page = s["case"]["page"]
    t = s["k"].shape[0]
    lens = s["lens"].long()
    b = lens.shape[0]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(b + 1, device=DEV)
    row = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    new = cu[1:] - cu[:-1]
    first = lens - new
    pos = first[seq] + row - cu[seq]
    ids, off = s["table"][seq, pos // page].long(), pos % page
    # the pages that go on from rows they hold
    cont = (new > 0) & (first % page > 0)
    old = s["table"][torch.arange(b, device=DEV), (first // page).clamp(max=s["table"].shape[1] - 1)].long()[cont]
    for x, name in ((s["k"], "k"), (s["v"], "v")):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        x = x.float()
        pages, h = scale.shape
        top = torch.zeros(pages, h, device=DEV).scatter_reduce(
            0, ids[:, None].expand(t, h), x.abs().amax(-1), "amax")
        now = torch.zeros_like(scale)
        now[ids] = _scale_for(top)[ids]
        now[old] = torch.maximum(now[old], scale[old])
        held = cache[old].float() * (scale[old] / now[old])[:, None, :, None]
        cache[old] = held.clamp(-448, 448).to(F8)
        cache.view(torch.uint8)[ids, off] = (x * (1 / now[ids])[:, :, None]).clamp(-448, 448).to(F8).view(torch.uint8)
        scale[ids] = now[ids]
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_attention(s):
    b, hq, dim = s["q"].shape
    hkv = s["k_cache"].shape[2]
    table = s["table"].long()
    k, v = ((s[n + "_cache"][table].float() * s[n + "_scale"][table][:, :, None, :, None]).flatten(1, 2)
            for n in ("k", "v"))  # [b, token, hkv, dim]
    q = s["q"].float().view(b, hkv, hq // hkv, dim)
    score = torch.einsum("bhrd,bthd->bhrt", q, k) / math.sqrt(dim)
    live = torch.arange(k.shape[1], device=DEV) < s["lens"][:, None]
    score = score.masked_fill(~live[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("bhrt,bthd->bhrd", e, v) / torch.where(total == 0, 1.0, total)
    lse = torch.log(total) + top
    return {"out": o.reshape(b, hq, dim).to(torch.bfloat16), "lse": lse.reshape(b, hq)}


# -------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "heads": _plain_heads, "heads_backward": _plain_heads_backward,
                "append": _plain_append, "attention": _plain_attention}[op](s)
    import prefill_kda_chunk_gb300 as K
    if op == "plan":
        table, lens, free, count, cu, positions, slots = K.page_plan(
            s["table"], s["lens"], s["new"], s["free"], s["count"], s["case"]["page"], s["tokens"],
            release=s["gone"])
        return {"table": table, "lens": lens, "free": free, "count": count, "cu": cu,
                "positions": positions, "slots": slots}
    if op == "heads":
        q, k = K.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"],
                              s["positions"], eps=EPS, interleaved=s["case"]["pairs"])
        return {"q": q, "k": k}
    if op == "heads_backward":
        dq, dk, dqw, dkw = K.qk_norm_rope_backward(
            s["q"], s["k"], s["dq_out"], s["dk_out"], s["q_weight"], s["k_weight"], s["inv_freq"],
            s["positions"], eps=EPS, interleaved=s["case"]["pairs"])
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    if op == "append":
        K.paged_append_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                           s["table"], s["lens"], cu_seqlens=s["cu"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    out, lse = K.paged_decode_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                  s["table"], s["lens"])
    return {"out": out, "lse": lse}


def work(case):
    op = case["op"]
    if op == "plan":
        b, cells = case["b"], case["b"] * case["width"]
        # table and stack in and out, lengths, rows
        return {"bytes": 16 * cells + 17 * b + 12 * case["new"], "flops": 0}
    if op in ("heads", "heads_backward"):
        n = case["t"] * (case["hq"] + case["hk"]) * case["dim"]
        small = 4 * case["t"] + 2 * case["rot"] + 8 * case["dim"]
        if op == "heads":
            return {"bytes": 4 * n + small, "flops": 8 * n}
        return {"bytes": n * (8 if case["dout32"] else 6) + small + 8 * case["dim"], "flops": 16 * n}
    hkv, dim = case["hkv"], case["dim"]
    if op == "append":
        n = case["t"] * hkv * dim * 2
        return {"bytes": 3 * n + 8 * case["b"] + 16 * hkv * max(case["b"], case["t"] // case["page"]),
                "flops": 2 * n}
    b, hq = case["b"], case["hq"]
    # ragged lengths are spread evenly over the logarithm
    tokens = case["longest"] * b
    if case["ragged"] and case["longest"] > 1:
        tokens = case["longest"] + (b - 1) * (case["longest"] - 1) / math.log(case["longest"])
    return {"bytes": 2 * tokens * hkv * dim + 8 * hkv * tokens / case["page"] + b * hq * (4 * dim + 4),
            "flops": 4 * tokens * hq * dim}


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    if case["op"] == "plan":   # whole numbers
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attention":
        return _exact_attention(s)
    return _exact_heads(s)


def _exact_heads(s):
    """By complex numbers: a pair of channels times e^(i angle); the gradient as the transposed
    derivative of x / |x|."""
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None, None] * s["inv_freq"].double())
    n = turn.shape[-1]

    def rotated(x, by):
        if s["case"]["pairs"]:
            z = torch.complex(x[..., 0:2 * n:2].contiguous(), x[..., 1:2 * n:2].contiguous()) * by
            return torch.cat([torch.view_as_real(z).flatten(-2), x[..., 2 * n:]], -1)
        z = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous()) * by
        return torch.cat([z.real, z.imag, x[..., 2 * n:]], -1)

    out = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_weight"].double()
        d = x.shape[-1]
        size = torch.sqrt((x.square().sum(-1, keepdim=True) + d * EPS) / d)
        if s["case"]["op"] == "heads":
            out[name] = rotated(x / size * w, turn)
            continue
        g = rotated(s["d%s_out" % name].double(), turn.conj())
        out["d%s_weight" % name] = torch.einsum("thd,thd->d", g, x / size)
        gw = g * w
        out["d" + name] = gw / size - x * torch.einsum("thd,thd->th", gw, x)[..., None] / (d * size ** 3)
    return out


def _e4m3(y):
    """The nearest e4m3 numbers, ties to even."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(y.abs() >= torch.exp2(e + 1), e + 1, torch.where(y.abs() < torch.exp2(e), e - 1, e))
    step = torch.exp2(e.clamp(min=-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_append(s):
    """Sequence by sequence and page by page."""
    page = s["case"]["page"]
    out = {}
    cu = s["cu"].tolist() if s["cu"] is not None else list(range(len(s["lens_host"]) + 1))
    table = s["table"].cpu()
    runs = []   # (page, first row in it, first token, tokens)
    for i, end in enumerate(s["lens_host"]):
        at, pos = cu[i], end - (cu[i + 1] - cu[i])
        while pos < end:
            m = min(end - pos, page - pos % page)
            runs.append((int(table[i, pos // page]), pos % page, at, m))
            at, pos = at + m, pos + m
    if len(runs) > 20000:
        return None
    for name in ("k", "v"):
        x = s[name].double()
        cache, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        for p, row, at, m in runs:
            new = x[at:at + m]
            top, e = torch.frexp(new.abs().amax((0, 2)) / 448)
            e = torch.where(top == 0, -126, torch.where(top == 0.5, e - 1, e).clamp(min=-126))
            want = ((e.long() + 1023) << 52).view(torch.float64)
            if row > 0:
                want = torch.maximum(want, scale[p])
                cache[p, :] = _e4m3(cache[p] * (scale[p] / want)[:, None])
            cache[p, row:row + m] = _e4m3(new / want[:, None])
            scale[p] = want
        out[name + "_cache"], out[name + "_scale"] = cache, scale
    return out


def _exact_attention(s):
    q, hkv, page = s["q"].double(), s["k_cache"].shape[2], s["k_cache"].shape[1]
    b, hq, dim = q.shape
    out = torch.zeros(b, hq, dim, dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        ids = s["table"][i, :-(-n // page)].long()
        k, v = (s[c + "_cache"][ids].double() * s[c + "_scale"][ids].double()[:, None, :, None]
                for c in ("k", "v"))
        k, v = (x.reshape(-1, hkv, dim)[:n] for x in (k, v))
        for g in range(hkv):
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            score = q[i, heads] @ k[:, g].t() / math.sqrt(dim)
            lse[i, heads] = torch.logsumexp(score, -1)
            out[i, heads] = torch.softmax(score, -1) @ v[:, g]
    return {"out": out, "lse": lse}
