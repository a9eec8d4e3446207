"""Workloads of the operators that a hybrid model needs next to KDA.

Three operators are covered: the short causal convolution (prompt, single
token, gradient), the selective state space scan (prompt, single token) and
the attention of one new token over a paged key-value cache. Where ``own`` is
false each runs in its plain form (elementary torch operations in 32 bits,
rounded once at the end); where it is true the package's kernels run.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the q slice of a fused q/k/v projection of 64 heads x 128, one prompt
        {"name": "conv prompt", "op": "conv", "t": 8192, "d": 8192, "w": 4, "seqs": 1, "fused": 3,
         "bias": False, "silu": True, "state": False},
        # x, B and C of a state space layer (64 heads x 64 and 2 x 8 groups x 128), a packed batch
        # of ragged prompts that continue from their histories
        {"name": "conv ragged", "op": "conv", "t": 5003, "d": 6144, "w": 4, "seqs": 16, "fused": 1,
         "bias": True, "silu": True, "state": True},
        # one new token for each of 256 running sequences, q, k and v of 64 heads at once
        {"name": "conv step", "op": "conv_step", "n": 256, "d": 24576, "w": 4, "bias": False,
         "silu": True},
        # a training step: the gradient after KDA's own, which is in fp32
        {"name": "conv gradient", "op": "conv_backward", "t": 8192, "d": 8192, "w": 4, "seqs": 1,
         "bias": True, "silu": True, "state": False, "dout32": True},
        # a short question to a small model: latency
        {"name": "scan short", "op": "scan", "t": 37, "h": 8, "p": 64, "n": 128, "g": 1, "seqs": 1,
         "state": False},
        # the ordinary prompt
        {"name": "scan prompt", "op": "scan", "t": 8192, "h": 64, "p": 64, "n": 128, "g": 8, "seqs": 1,
         "state": False},
        # 16 ragged prompts in one packed batch, continued from earlier states
        {"name": "scan ragged", "op": "scan", "t": 8191, "h": 64, "p": 64, "n": 128, "g": 1, "seqs": 16,
         "state": True},
        # a long document, wide heads, few of them
        {"name": "scan long", "op": "scan", "t": 131072, "h": 32, "p": 128, "n": 128, "g": 1, "seqs": 1,
         "state": True},
        # one new token for each of 256 running sequences
        {"name": "scan step", "op": "scan_step", "n_seqs": 256, "h": 64, "p": 64, "n": 128, "g": 8},
        # one sequence, a short cache: latency
        {"name": "attention short", "op": "attention", "b": 1, "hq": 32, "hkv": 8, "dim": 128,
         "page": 16, "longest": 700, "ragged": False},
        # a serving batch with lengths spread over a factor of hundreds, one slot unused
        {"name": "attention ragged", "op": "attention", "b": 64, "hq": 64, "hkv": 8, "dim": 128,
         "page": 64, "longest": 16384, "ragged": True},
        # two long documents: few rows, a long axis
        {"name": "attention long", "op": "attention", "b": 2, "hq": 32, "hkv": 8, "dim": 128,
         "page": 32, "longest": 131072, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "conv_backward", "scan", "scan", "scan_step",
                     "attention", "attention"])
    if op in ("conv", "conv_backward"):
        t = _log(rng, 1, 16384)
        d = _log(rng, 32, min(16384, (1 << 26) // t))
        if rng.random() < 0.7:
            d = max(8, d // 8 * 8)
        c = {"op": op, "t": t, "d": d, "w": rng.choice([2, 3, 4, 4]),
             "seqs": rng.choice([1, 1, rng.randint(2, 24)]), "bias": rng.random() < 0.5,
             "silu": rng.random() < 0.8, "state": rng.random() < 0.5}
        if op == "conv":
            c["fused"] = rng.choice([1, 1, 3])
        else:
            c["dout32"] = rng.random() < 0.5
        return c
    if op == "conv_step":
        d = _log(rng, 32, 32768)
        if rng.random() < 0.7:
            d = max(8, d // 8 * 8)
        return {"op": op, "n": _log(rng, 1, 512), "d": d, "w": rng.choice([2, 3, 4, 4]),
                "bias": rng.random() < 0.5, "silu": rng.random() < 0.8}
    if op == "scan":
        g = rng.choice([1, 1, 2, 4, 8])
        h = g * rng.randint(1, max(1, 96 // g))
        t = _log(rng, 1, min(65536, (1 << 20) // h))
        return {"op": op, "t": t, "h": h, "p": rng.choice([64, 64, 128]),
                "n": rng.choice([64, 128, 128]), "g": g,
                "seqs": rng.choice([1, 1, rng.randint(2, 24)]), "state": rng.random() < 0.5}
    if op == "scan_step":
        g = rng.choice([1, 1, 2, 4, 8])
        h = g * rng.randint(1, max(1, 96 // g))
        return {"op": op, "n_seqs": _log(rng, 1, max(1, 16384 // h)), "h": h,
                "p": rng.choice([64, 64, 128]), "n": rng.choice([64, 128, 128]), "g": g}
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    longest = _log(rng, 1, 131072)
    b = _log(rng, 1, max(1, min(256, (1 << 21) // (longest * hkv))))
    return {"op": op, "b": b, "hq": hq, "hkv": hkv, "dim": rng.choice([64, 128, 128]),
            "page": rng.choice([1, 8, 16, 17, 32, 64, 64, 100, 128]), "longest": longest,
            "ragged": rng.random() < 0.7}


# ----------------------------------------------------------------- the inputs

def _lengths(total, n, gen):
    """n ragged lengths with the given sum, some of them perhaps zero."""
    cuts = torch.sort(torch.randint(0, total + 1, (n - 1,), generator=gen)).values
    return torch.diff(torch.cat([torch.zeros(1, dtype=torch.int64), cuts,
                                 torch.full((1,), total, dtype=torch.int64)])).tolist()


def _cu(lengths):
    return torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cpu").manual_seed(seed)
    dgen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=dgen, device=DEV, dtype=torch.float32) * scale).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=dgen, device=DEV, dtype=torch.float32)

    op, s = case["op"], {"case": case}
    if op in ("conv", "conv_backward", "conv_step"):
        d, w = case["d"], case["w"]
        s["weight"] = randn(d, w, dtype=torch.float32, scale=w ** -0.5)
        s["bias"] = randn(d, dtype=torch.float32, scale=0.1) if case["bias"] else None
        s["activation"] = "silu" if case["silu"] else None
        if op == "conv_step":
            s["x"] = randn(case["n"], d)
            s["history"] = randn(case["n"], w - 1, d)
            return s
        n, t, f = case["seqs"], case["t"], case.get("fused", 1)
        whole = randn(t, f * d)
        s["x"] = whole[:, :d]  # one slice of a fused projection
        s["lengths"] = _lengths(t, n, gen)
        s["cu"] = _cu(s["lengths"]).to(DEV) if n > 1 else None
        s["history"] = randn(n, w - 1, d) if case["state"] else None
        if op == "conv_backward":
            s["d_out"] = randn(t, d, dtype=torch.float32 if case["dout32"] else torch.bfloat16)
            s["d_final"] = randn(n, w - 1, d, dtype=torch.float32) if case["state"] else None
        return s
    if op in ("scan", "scan_step"):
        h, p, ns, g = case["h"], case["p"], case["n"], case["g"]
        rows = case["t"] if op == "scan" else case["n_seqs"]
        seqs = case["seqs"] if op == "scan" else rows
        # x, B and C as slices of the convolution's output; dt as the projection gives it
        xbc = randn(rows, h * p + 2 * g * ns)
        s["x"] = xbc[:, :h * p].view(rows, h, p)
        s["b"] = xbc[:, h * p:h * p + g * ns].view(rows, g, ns)
        s["c"] = xbc[:, h * p + g * ns:].view(rows, g, ns)
        s["dt"] = randn(rows, h, dtype=torch.float32, scale=0.5)
        step = torch.exp(rand(h) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus gives `step` again
        s["a"] = -(1 + 15 * rand(h))
        s["d"] = 1 + 0.1 * randn(h, dtype=torch.float32)
        if op == "scan":
            s["lengths"] = _lengths(rows, seqs, gen)
            s["cu"] = _cu(s["lengths"]).to(DEV) if seqs > 1 else None
        s["state"] = (randn(seqs, h, ns, p, dtype=torch.float32, scale=0.5)
                      if op == "scan_step" or case["state"] else None)
        return s
    b, hkv, dim, page, longest = case["b"], case["hkv"], case["dim"], case["page"], case["longest"]
    lens = torch.full((b,), longest, dtype=torch.int64)
    if case["ragged"]:
        lens = torch.exp(torch.rand(b, generator=gen) * math.log(longest)).round().to(torch.int64)
        lens[torch.randint(0, b, (1,), generator=gen)] = longest
        if b > 2:  # a slot with nothing in it
            lens[int((lens == lens.min()).nonzero()[0])] = 0
    need = (lens + page - 1) // page
    most = int(need.max())
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.zeros(b, max(1, most), dtype=torch.int32)
    at = 0
    for i in range(b):
        k = int(need[i])
        table[i, :k] = order[at:at + k]
        at += k
    s["lens_host"] = lens.tolist()
    s["lens"] = lens.to(torch.int32).to(DEV)
    s["table"] = table.to(DEV)
    cache = torch.empty(pages, 2, page, hkv, dim, dtype=torch.bfloat16, device=DEV)
    for i in range(0, pages, 4096):  # keys and values of one page lie side by side
        cache[i:i + 4096] = randn(*cache[i:i + 4096].shape)
    s["k_cache"], s["v_cache"] = cache[:, 0], cache[:, 1]
    s["q"] = randn(b, case["hq"], dim)
    return s


# ------------------------------------------------------------ the plain forms

def _silu(z):
    return z / (1 + torch.exp(-z))


def _taps(s, w):
    """[t, w, d]: row t and the w - 1 rows before it, from the history where the sequence starts."""
    x, n = s["x"].float(), len(s["lengths"])
    t, d = x.shape
    hist = s["history"].float() if s["history"] is not None else x.new_zeros(n, w - 1, d)
    pos, seq = _places(s)
    back = torch.arange(w - 1, -1, -1, device=x.device)
    src = torch.arange(t, device=x.device)[:, None] - back
    inside = pos[:, None] >= back
    early = t + seq[:, None] * (w - 1) + (w - 1) + pos[:, None] - back
    return torch.cat([x, hist.reshape(n * (w - 1), d)])[torch.where(inside, src, early)]


def _places(s):
    """Each token's position in its sequence, and its sequence."""
    t = s["x"].shape[0]
    at = torch.arange(t, device=DEV)
    if s["cu"] is None:
        return at, torch.zeros_like(at)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu[1:], at, right=True)
    return at - cu[seq], seq


def _last_rows(s, w):
    """[n, w - 1] indices into (x rows, then history rows) of the history after the call."""
    t, n = s["x"].shape[0], len(s["lengths"])
    cu = s["cu"].long() if s["cu"] is not None else torch.tensor([0, t], device=DEV)
    lens = cu[1:] - cu[:-1]
    back = torch.arange(w - 1, 0, -1, device=DEV)
    pos = lens[:, None] - back
    early = t + torch.arange(n, device=DEV)[:, None] * (w - 1) + (w - 1) + pos
    return torch.where(pos >= 0, cu[:-1, None] + pos, early)


def _plain_conv(s):
    w = s["case"]["w"]
    z = torch.einsum("twd,dw->td", _taps(s, w), s["weight"])
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _silu(z) if s["activation"] else z
    n, d = len(s["lengths"]), s["x"].shape[1]
    hist = s["history"] if s["history"] is not None else s["x"].new_zeros(n, w - 1, d)
    rows = torch.cat([s["x"], hist.reshape(n * (w - 1), d)])
    return {"out": y.to(torch.bfloat16), "history": rows[_last_rows(s, w)]}


def _plain_conv_step(s):
    rows = torch.cat([s["history"], s["x"][:, None]], 1)
    z = (rows.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _silu(z) if s["activation"] else z
    return {"out": y.to(torch.bfloat16), "history": rows[:, 1:].contiguous()}


def _plain_conv_backward(s):
    w, d = s["case"]["w"], s["x"].shape[1]
    t, n = s["x"].shape[0], len(s["lengths"])
    taps = _taps(s, w)
    dz = s["d_out"].float()
    if s["activation"]:
        z = torch.einsum("twd,dw->td", taps, s["weight"])
        z = z + s["bias"] if s["bias"] is not None else z
        sig = 1 / (1 + torch.exp(-z))
        dz = dz * (sig * (1 + z * (1 - sig)))
    # the gradient of row r (of x, then of the histories) gathers dz of the w rows it reaches
    pos, seq = _places(s)
    cu = s["cu"].long() if s["cu"] is not None else torch.tensor([0, t], device=DEV)
    lens = cu[1:] - cu[:-1]
    hist_pos = torch.arange(-(w - 1), 0, device=DEV).repeat(n)
    hist_seq = torch.arange(n, device=DEV).repeat_interleave(w - 1)
    pos, seq = torch.cat([pos, hist_pos]), torch.cat([seq, hist_seq])
    ahead = torch.arange(w, device=DEV)
    to = pos[:, None] + ahead
    ok = (to >= 0) & (to < lens[seq][:, None])
    at = torch.where(ok, cu[seq][:, None] + to, 0)
    reach = dz[at] * ok[:, :, None]
    grad = torch.einsum("rwd,dw->rd", reach, s["weight"].flip(1))
    if s["d_final"] is not None:
        grad[_last_rows(s, w).reshape(-1)] += s["d_final"].reshape(n * (w - 1), d)
    out = {"dx": grad[:t].to(torch.bfloat16), "dweight": torch.einsum("twd,td->dw", taps, dz)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum(0)
    if s["history"] is not None:
        out["d_history"] = grad[t:].reshape(n, w - 1, d)
    return out


def _softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-torch.abs(z)))


def _spans(v):
    """[..., m] -> [..., m + 1, m + 1]: entry (j, i) is the sum of v[i:j], -inf above the diagonal."""
    m = v.shape[-1]
    k = torch.arange(m + 1, device=v.device)
    v = torch.cat([torch.zeros_like(v[..., :1]), v], -1)
    spread = v[..., :, None] * (k[:, None] > k)
    return spread.cumsum(-2).masked_fill(k[:, None] < k, -math.inf)


def _plain_scan(s):
    size = 64
    x, b, c = s["x"].float(), s["b"].float(), s["c"].float()
    dt = _softplus(s["dt"] + s["dt_bias"])
    t, h, p = x.shape
    g, ns, seqs = b.shape[1], b.shape[2], len(s["lengths"])
    r = h // g
    pos, seq = _places(s)
    most = -(-max(s["lengths"]) // size) * size
    nc = most // size

    def padded(v):
        return v.new_zeros(seqs, most, *v.shape[1:]).index_put((seq, pos), v)

    xs = padded(x).view(seqs, nc, size, g, r, p)
    bs = padded(b).view(seqs, nc, size, g, ns)
    cs = padded(c).view(seqs, nc, size, g, ns)
    dts = padded(dt).view(seqs, nc, size, g, r).permute(0, 1, 3, 4, 2)  # [seq, chunk, g, r, token]
    log = dts * s["a"].view(g, r, 1)
    span = _spans(log)  # sums over tokens i .. j - 1 of a chunk
    inside = torch.exp(span[..., 1:, 1:])
    score = torch.einsum("zklgn,zkmgn->zkglm", cs, bs)[:, :, :, None] * inside * dts[..., None, :]
    y = torch.einsum("zkgrlm,zkmgrp->zklgrp", score, xs)
    to_end = torch.exp(span[..., size, 1:]) * dts
    add = torch.einsum("zkgrm,zkmgn,zkmgrp->zkgrnp", to_end, bs, xs)
    first = s["state"] if s["state"] is not None else x.new_zeros(seqs, h, ns, p)
    add = torch.cat([first.view(seqs, 1, g, r, ns, p), add], 1)
    carry = torch.exp(_spans(log.sum(-1).permute(0, 2, 3, 1)))  # [seq, g, r, chunk + 1, chunk + 1]
    entry = torch.einsum("zgrji,zigrnp->zjgrnp", carry, add)
    from_start = torch.exp(span[..., 1:, 0])
    y = y + torch.einsum("zklgn,zkgrnp,zkgrl->zklgrp", cs, entry[:, :nc], from_start)
    y = y.reshape(seqs, most, h, p)[seq, pos] + s["d"][:, None] * x
    return {"out": y.to(torch.bfloat16), "state": entry[:, nc].reshape(seqs, h, ns, p)}


def _plain_scan_step(s):
    x, b, c = s["x"].float(), s["b"].float(), s["c"].float()
    r = x.shape[1] // b.shape[1]
    dt = _softplus(s["dt"] + s["dt_bias"])
    b, c = b.repeat_interleave(r, 1), c.repeat_interleave(r, 1)
    new = s["state"] * torch.exp(dt * s["a"])[..., None, None]
    new = new + (dt[..., None] * b)[..., None] * x[:, :, None, :]
    y = (c[..., None] * new).sum(2) + s["d"][:, None] * x
    return {"out": y.to(torch.bfloat16), "state": new}


def _plain_attention(s):
    b, hq, dim = s["q"].shape
    hkv = s["k_cache"].shape[2]
    table = s["table"].long()
    k = s["k_cache"][table].float().flatten(1, 2)  # [b, token, hkv, dim]
    v = s["v_cache"][table].float().flatten(1, 2)
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
        return {"conv": _plain_conv, "conv_step": _plain_conv_step,
                "conv_backward": _plain_conv_backward, "scan": _plain_scan,
                "scan_step": _plain_scan_step, "attention": _plain_attention}[op](s)
    import prefill_kda_chunk_gb300 as K
    if op == "conv":
        out, hist = K.short_conv(s["x"], s["weight"], s["bias"], initial_state=s["history"],
                                 cu_seqlens=s["cu"], activation=s["activation"])
        return {"out": out, "history": hist}
    if op == "conv_step":
        out, hist = K.short_conv_step(s["x"], s["weight"], s["history"], s["bias"],
                                      activation=s["activation"])
        return {"out": out, "history": hist}
    if op == "conv_backward":
        dx, dw, db, dh = K.short_conv_backward(
            s["x"], s["weight"], s["d_out"], s["bias"], initial_state=s["history"],
            cu_seqlens=s["cu"], activation=s["activation"], d_final_state=s["d_final"],
            d_initial_state=s["history"] is not None)
        out = {"dx": dx, "dweight": dw}
        if db is not None:
            out["dbias"] = db
        if dh is not None:
            out["d_history"] = dh
        return out
    if op == "scan":
        out, state = K.ssm_prefill(s["x"], s["dt"], s["a"], s["b"], s["c"], s["d"], s["dt_bias"],
                                   initial_state=s["state"], cu_seqlens=s["cu"], dt_softplus=True)
        return {"out": out, "state": state}
    if op == "scan_step":
        out, state = K.ssm_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["state"], s["d"],
                                s["dt_bias"], dt_softplus=True)
        return {"out": out, "state": state}
    out, lse = K.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])
    return {"out": out, "lse": lse}


def work(case):
    op = case["op"]
    if op in ("conv", "conv_backward"):
        td, d, w = case["t"] * case["d"], case["d"], case["w"]
        hist = case["seqs"] * (w - 1) * d
        params = 4 * d * (w + case["bias"])
        if op == "conv":
            return {"bytes": 4 * td + 2 * hist * (1 + case["state"]) + params,
                    "flops": td * (2 * w + 4 * case["silu"])}
        return {"bytes": td * (2 + 2 + (4 if case["dout32"] else 2)) + 2 * params
                + 10 * hist * case["state"], "flops": td * (6 * w + 8 * case["silu"])}
    if op == "conv_step":
        nd, w = case["n"] * case["d"], case["w"]
        return {"bytes": 4 * nd * w + 4 * case["d"] * (w + case["bias"]),
                "flops": nd * (2 * w + 4 * case["silu"])}
    if op in ("scan", "scan_step"):
        h, p, n, g = case["h"], case["p"], case["n"], case["g"]
        rows = case["t"] if op == "scan" else case["n_seqs"]
        seqs, states = (case["seqs"], 1 + case["state"]) if op == "scan" else (rows, 2)
        return {"bytes": rows * (4 * h * p + 4 * h + 4 * g * n) + 4 * states * seqs * h * n * p,
                "flops": 4 * rows * h * n * p}
    b, hq, hkv, dim = case["b"], case["hq"], case["hkv"], case["dim"]
    # ragged lengths are spread evenly over the logarithm
    tokens = case["longest"] * b
    if case["ragged"] and case["longest"] > 1:
        tokens = case["longest"] + (b - 1) * (case["longest"] - 1) / math.log(case["longest"])
    return {"bytes": 4 * tokens * hkv * dim + b * hq * (4 * dim + 4),
            "flops": 4 * tokens * hq * dim}


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attention":
        return _exact_attention(s)
    if op in ("scan", "scan_step"):
        return _exact_scan(s)
    return _exact_conv(s)


def _exact_conv(s):
    """Sequence by sequence: shifted copies of the rows, history in front."""
    case = s["case"]
    w, op = case["w"], case["op"]
    wt = s["weight"].double()
    if op == "conv_step":
        pieces = [(s["x"].double(), s["history"].double().transpose(0, 1))]
    else:
        pieces, at = [], 0
        for i, n in enumerate(s["lengths"]):
            x = s["x"][at:at + n].double()
            hist = (s["history"][i].double() if s["history"] is not None
                    else x.new_zeros(w - 1, x.shape[1]))
            pieces.append((x, hist, at, n))
            at += n
    if op == "conv_step":
        x, hist = pieces[0]
        rows = [hist[j] for j in range(w - 1)] + [x]
        z = sum(wt[:, j] * rows[j] for j in range(w))
        z = z + s["bias"].double() if s["bias"] is not None else z
        return {"out": z * torch.sigmoid(z) if case["silu"] else z, "history": torch.stack(rows[1:], 1)}
    if op == "conv":
        outs, hists = [], []
        for x, hist, at, n in pieces:
            full = torch.cat([hist, x])
            z = sum(wt[:, j] * full[j:j + n] for j in range(w))
            z = z + s["bias"].double() if s["bias"] is not None else z
            outs.append(z * torch.sigmoid(z) if case["silu"] else z)
            hists.append(full[n:])
        return {"out": torch.cat(outs), "history": torch.stack(hists)}
    dw = torch.zeros_like(wt)
    db = torch.zeros_like(wt[:, 0])
    dxs, dhs = [], []
    for i, (x, hist, at, n) in enumerate(pieces):
        full = torch.cat([hist, x])
        dz = s["d_out"][at:at + n].double()
        if case["silu"]:
            z = sum(wt[:, j] * full[j:j + n] for j in range(w))
            z = z + s["bias"].double() if s["bias"] is not None else z
            sig = torch.sigmoid(z)
            dz = dz * sig * (1 + z * (1 - sig))
        dfull = torch.zeros_like(full)
        for j in range(w):
            dfull[j:j + n] += wt[:, j] * dz
            dw[:, j] += (dz * full[j:j + n]).sum(0)
        db += dz.sum(0)
        if s["d_final"] is not None:
            dfull[n:] += s["d_final"][i].double()
        dxs.append(dfull[w - 1:])
        dhs.append(dfull[:w - 1])
    out = {"dx": torch.cat(dxs), "dweight": dw}
    if s["bias"] is not None:
        out["dbias"] = db
    if s["history"] is not None:
        out["d_history"] = torch.stack(dhs)
    return out


def _exact_scan(s):
    """The recurrence, token by token, every sequence side by side."""
    x, b, c = s["x"], s["b"], s["c"]
    rows, h, p = x.shape
    r = h // b.shape[1]
    raw = s["dt"].double() + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    decay = torch.exp(dt * s["a"].double())
    if s["case"]["op"] == "scan_step":
        starts, lens = torch.arange(rows), torch.ones(rows, dtype=torch.int64)
    else:
        lens = torch.tensor(s["lengths"])
        starts = lens.cumsum(0) - lens
    order = torch.argsort(lens, descending=True)  # at each position the live ones come first
    starts, lens = starts[order].to(DEV), lens[order]
    live = (lens[:, None] > torch.arange(int(lens[0]))).sum(0).tolist() if int(lens[0]) else []
    state = (s["state"].double()[order.to(DEV)] if s["state"] is not None
             else torch.zeros(len(lens), h, b.shape[2], p, dtype=torch.float64, device=DEV))
    y = torch.empty(rows, h, p, dtype=torch.float64, device=DEV)
    skip = s["d"].double()[:, None]
    for t, m in enumerate(live):
        at = starts[:m] + t
        xt = x[at].double()
        bt = b[at].double().repeat_interleave(r, 1) * dt[at][..., None]
        ct = c[at].double().repeat_interleave(r, 1)
        now = state[:m]
        now.mul_(decay[at][..., None, None]).addcmul_(bt[..., None], xt[:, :, None, :])
        y[at] = torch.matmul(ct[:, :, None, :], now)[:, :, 0] + skip * xt
    back = torch.empty_like(state)
    back[order.to(DEV)] = state
    return {"out": y, "state": back}


def _exact_attention(s):
    q, hkv, page = s["q"].double(), s["k_cache"].shape[2], s["k_cache"].shape[1]
    b, hq, dim = q.shape
    out = torch.zeros(b, hq, dim, dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        ids = s["table"][i, :-(-n // page)].long()
        k = s["k_cache"][ids].reshape(-1, hkv, dim)[:n]
        v = s["v_cache"][ids].reshape(-1, hkv, dim)[:n]
        for g in range(hkv):
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            score = q[i, heads] @ k[:, g].double().t() / math.sqrt(dim)
            lse[i, heads] = torch.logsumexp(score, -1)
            out[i, heads] = torch.softmax(score, -1) @ v[:, g].double()
    return {"out": out, "lse": lse}
