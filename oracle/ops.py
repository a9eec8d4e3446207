"""64-bit references of the operators around the KDA layers: the short causal
convolution and its gradient, the selective state space scan, and decode
attention over a paged cache. Written from the definitions, sequence by
sequence and token by token, on the CPU. Each returns its results together
with the same sums over absolute values, by which a rounding error is
measured.
"""
import math

import torch

F64 = torch.float64


def spans(tokens, n, cu):
    """[(start, end)] of n sequences in `tokens` rows."""
    if cu is None:
        step = tokens // n if n else 0
        return [(i * step, (i + 1) * step) for i in range(n)]
    cu = [int(v) for v in cu]
    return list(zip(cu[:-1], cu[1:]))


def _d(t):
    return None if t is None else t.detach().cpu().to(F64)


def silu(z):
    return z * torch.sigmoid(z)


def short_conv(x, weight, bias=None, state=None, cu=None, n=1, act=True):
    """x [tokens, D] -> (out, history, sum of absolute values of z)."""
    x, weight, bias, state = _d(x), _d(weight), _d(bias), _d(state)
    D, W = weight.shape
    out, size = torch.zeros_like(x), torch.zeros_like(x)
    hist = torch.zeros(n, W - 1, D, dtype=F64)
    for i, (a, b) in enumerate(spans(x.shape[0], n, cu)):
        rows = torch.cat([state[i] if state is not None else torch.zeros(W - 1, D, dtype=F64), x[a:b]])
        z = torch.zeros(b - a, D, dtype=F64)
        s = torch.zeros(b - a, D, dtype=F64)
        for j in range(W):
            z += weight[:, j] * rows[j:j + b - a]
            s += (weight[:, j] * rows[j:j + b - a]).abs()
        if bias is not None:
            z += bias
            s += bias.abs()
        out[a:b] = silu(z) if act else z
        size[a:b] = s
        hist[i] = rows[b - a:]
    return out, hist, size


def short_conv_backward(x, weight, d_out, bias=None, state=None, cu=None, n=1, act=True,
                        d_final=None):
    """-> dict of dx, dweight, dbias, dstate, each a pair (value, sum of absolute values)."""
    x, weight, bias, state, d_out, d_final = (_d(v) for v in (x, weight, bias, state, d_out, d_final))
    D, W = weight.shape
    dx, dx_s = torch.zeros_like(x), torch.zeros_like(x)
    dw, dw_s = torch.zeros_like(weight), torch.zeros_like(weight)
    db, db_s = torch.zeros(D, dtype=F64), torch.zeros(D, dtype=F64)
    dh, dh_s = torch.zeros(n, W - 1, D, dtype=F64), torch.zeros(n, W - 1, D, dtype=F64)
    for i, (a, b) in enumerate(spans(x.shape[0], n, cu)):
        T = b - a
        rows = torch.cat([state[i] if state is not None else torch.zeros(W - 1, D, dtype=F64), x[a:b]])
        z = sum(weight[:, j] * rows[j:j + T] for j in range(W))
        z_s = sum((weight[:, j] * rows[j:j + T]).abs() for j in range(W))
        if bias is not None:
            z, z_s = z + bias, z_s + bias.abs()
        g = d_out[a:b]
        if act:
            s = torch.sigmoid(z)
            g = g * (s * (1 + z * (1 - s)))
            # |silu''| <= 1/2: the error of z enters dz with at most this weight
            g_s = d_out[a:b].abs() * (1 + z_s)
        else:
            g_s = g.abs()
        dr = torch.zeros(T + W - 1, D, dtype=F64)
        dr_s = torch.zeros(T + W - 1, D, dtype=F64)
        for j in range(W):
            dr[j:j + T] += weight[:, j] * g
            dr_s[j:j + T] += weight[:, j].abs() * g_s
            dw[:, j] += (g * rows[j:j + T]).sum(0)
            dw_s[:, j] += (g_s * rows[j:j + T].abs()).sum(0)
        db += g.sum(0)
        db_s += g_s.sum(0)
        if d_final is not None:
            dr[T:] += d_final[i]
            dr_s[T:] += d_final[i].abs()
        dx[a:b], dx_s[a:b] = dr[W - 1:], dr_s[W - 1:]
        dh[i], dh_s[i] = dr[:W - 1], dr_s[:W - 1]
    return {"dx": (dx, dx_s), "dweight": (dw, dw_s), "dbias": (db, db_s), "dstate": (dh, dh_s)}


def ssm(x, dt, a, b, c, d=None, dt_bias=None, state=None, cu=None, n=1, softplus=False):
    """x [tokens, H, P] -> (out, state, absolute sums of out, absolute sums of state)."""
    x, dt, a, b, c, d, dt_bias, state = (_d(v) for v in (x, dt, a, b, c, d, dt_bias, state))
    tokens, H, P = x.shape
    G, N = b.shape[1:]
    delta = dt if dt_bias is None else dt + dt_bias
    if softplus:
        delta = torch.clamp(delta, min=0) + torch.log1p(torch.exp(-delta.abs()))
    b, c = b.repeat_interleave(H // G, 1), c.repeat_interleave(H // G, 1)
    out, size = torch.zeros_like(x), torch.zeros_like(x)
    final = torch.zeros(n, H, N, P, dtype=F64)
    final_s = torch.zeros(n, H, N, P, dtype=F64)
    for i, (lo, hi) in enumerate(spans(tokens, n, cu)):
        S = state[i].clone() if state is not None else torch.zeros(H, N, P, dtype=F64)
        A = S.abs()
        for t in range(lo, hi):
            decay = torch.exp(a * delta[t])[:, None, None]
            add = delta[t][:, None, None] * b[t][:, :, None] * x[t][:, None, :]
            S = decay * S + add
            A = decay * A + add.abs()
            out[t] = (c[t][:, :, None] * S).sum(1)
            size[t] = (c[t].abs()[:, :, None] * A).sum(1)
            if d is not None:
                out[t] += d[:, None] * x[t]
                size[t] += (d[:, None] * x[t]).abs()
        final[i], final_s[i] = S, A
    return out, final, size, final_s


def paged_attention(q, k_cache, v_cache, table, lens, scale=None):
    """-> (out, lse, sum of p |v|, largest sum of |q||k| scale of a row)."""
    q, table, lens = _d(q), table.cpu(), [int(v) for v in lens]
    B, Hq, D = q.shape
    ps, Hkv = k_cache.shape[1:3]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, size = torch.zeros(B, Hq, D, dtype=F64), torch.zeros(B, Hq, D, dtype=F64)
    lse = torch.full((B, Hq), -math.inf, dtype=F64)
    reach = torch.zeros(B, Hq, dtype=F64)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        ids = table[i, :-(-n // ps)].long().to(k_cache.device)
        k = _d(k_cache[ids]).reshape(-1, Hkv, D)[:n]
        v = _d(v_cache[ids]).reshape(-1, Hkv, D)[:n]
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            s = scale * (k[:, kv] @ q[i, h])
            p = torch.softmax(s, 0)
            out[i, h] = p @ v[:, kv]
            size[i, h] = p @ v[:, kv].abs()
            lse[i, h] = torch.logsumexp(s, 0)
            reach[i, h] = (abs(scale) * (k[:, kv].abs() @ q[i, h].abs())).max()
    return out, lse, size, reach
