"""64-bit references of the operators in front of and around an 8-bit paged cache:
page plans, norms of queries and keys with the rotation (and their gradients), new
tokens into the cache, and decode attention over it. Written from the definitions,
on the CPU, number by number where numbers are whole. Computed results come with the
same sums over absolute values, by which a rounding error is measured.
"""
import math

import torch

from . import ops

F64 = torch.float64


def page_plan(table, lens, news, free, count, page, tokens, release=None):
    """-> (table, lens, free, count, cu, positions, slots), lists; None where it cannot be."""
    table = [[int(v) for v in row] for row in table]
    lens, news, free = ([int(v) for v in x] for x in (lens, news, free))
    count, width = int(count), len(table[0]) if table else 0
    for i, row in enumerate(table):
        if release is not None and bool(release[i]):
            for j in range(-(-lens[i] // page)):
                free[count] = row[j]
                count += 1
            lens[i] = 0
    cu, positions, slots = [0], [], []
    for i, row in enumerate(table):
        for pos in range(lens[i], lens[i] + news[i]):
            if pos >= width * page:
                return None
            if pos % page == 0:
                if count == 0:
                    return None
                count -= 1
                row[pos // page] = free[count]
            positions.append(pos)
            slots.append(row[pos // page] * page + pos % page)
        lens[i] += news[i]
        cu.append(cu[-1] + news[i])
    rest = tokens - len(positions)
    if rest < 0:
        return None
    return table, lens, free, count, cu, positions + [0] * rest, slots + [-1] * rest


def _pairs(R, interleaved):
    i = torch.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def _turned(u, freq, pos, interleaved, sign=1.0):
    """u [T, H, D] and its absolute sums [T, H, D]: channel pairs by a rotation matrix."""
    y, size = u.clone(), u.abs()
    if freq is None:
        return y, size
    a, b = _pairs(2 * freq.numel(), interleaved)
    t = pos.to(F64)[:, None] * freq.to(F64)
    c, s = torch.cos(t)[:, None], sign * torch.sin(t)[:, None]
    y[..., a], y[..., b] = u[..., a] * c - u[..., b] * s, u[..., a] * s + u[..., b] * c
    size[..., a] = size[..., b] = u[..., a].abs() + u[..., b].abs()
    return y, size


def norm_rope(x, weight=None, freq=None, pos=None, eps=1e-6, interleaved=False):
    """x [T, H, D] -> (y, absolute sums of y)."""
    x = x.detach().cpu().to(F64)
    w = torch.ones(x.shape[-1], dtype=F64) if weight is None else weight.cpu().to(F64)
    u = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + eps) * w
    return _turned(u, None if freq is None else freq.cpu(), None if pos is None else pos.cpu(), interleaved)


def norm_rope_backward(x, dy, weight=None, freq=None, pos=None, eps=1e-6, interleaved=False):
    """-> ((dx, absolute sums), (dweight, absolute sums))."""
    x, dy = x.detach().cpu().to(F64), dy.detach().cpu().to(F64)
    D = x.shape[-1]
    w = torch.ones(D, dtype=F64) if weight is None else weight.cpu().to(F64)
    g, g_s = _turned(dy, None if freq is None else freq.cpu(), None if pos is None else pos.cpu(),
                     interleaved, -1.0)
    n = torch.sqrt((x ** 2).mean(-1, keepdim=True) + eps)
    u = x / n
    dw, dw_s = (g * u).sum((0, 1)), (g_s * u.abs()).sum((0, 1))
    h, h_s = g * w, g_s * w.abs()
    dx = (h - u * (h * u).mean(-1, keepdim=True)) / n
    dx_s = (h_s + u.abs() * (h_s * u.abs()).mean(-1, keepdim=True)) / n
    return (dx, dx_s), (dw, dw_s)


# the numbers that e4m3 codes 0 .. 126 stand for, rising
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(F64)


def e4m3(y):
    """Nearest numbers, ties to the even code, 448 beyond it, NaN for infinities and NaN."""
    a = y.abs().clamp(max=448)
    hi = torch.searchsorted(E4M3, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    out = torch.where(E4M3[hi] == a, a, E4M3[code]) * torch.sign(y)
    return torch.where(torch.isfinite(y), out, math.nan)


def scale_for(top):
    """The least power of two from 2^-126 on that brings `top` to 448 or below."""
    k = -126
    while top > 448 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append(x, cache, scale, table, lens, cu=None):
    """x [T, H, D] into (cache [pages, page, H, D], scale [pages, H]), both 64 bits, in place."""
    x = x.detach().cpu().to(F64)
    page, H = cache.shape[1:3]
    table, lens = table.cpu(), [int(v) for v in lens]
    cu = [int(v) for v in cu] if cu is not None else list(range(len(lens) + 1))
    for i, n in enumerate(lens):
        at, end = cu[i], cu[i + 1]
        if n == 0:
            continue
        pos = n - (end - at)
        while at < end:
            p, row = int(table[i, pos // page]), pos % page
            m = min(end - at, page - row)
            for h in range(H):
                new = x[at:at + m, h]
                fine = new.abs()[torch.isfinite(new)]
                want = scale_for(float(fine.max()) if fine.numel() else 0.0)
                if row > 0:
                    want = max(want, float(scale[p, h]))
                    if want > scale[p, h]:
                        cache[p, :, h] = e4m3(cache[p, :, h] * (scale[p, h] / want))
                cache[p, row:row + m, h] = e4m3(new / want)
                scale[p, h] = want
            at, pos = at + m, pos + m


def paged_attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale=None):
    """-> (out, lse, sum of p |v|, largest sum of |q||k| scale of a row, floor), as
    ops.paged_attention over the numbers that the cache stands for. floor: the largest weight
    times its value's scale, times the sum of the cached |v|: the terms that a weight is split
    into end at a fraction of the largest one."""
    numbers = [(c.detach().cpu().to(F64), s.detach().cpu().to(F64))
               for c, s in ((k_cache, k_scale), (v_cache, v_scale))]
    k, v = (c * s[:, None, :, None] for c, s in numbers)
    out, lse, size, reach = ops.paged_attention(q, k, v, table, lens, scale)
    q, table = q.detach().cpu().to(F64), table.cpu()
    page, H, D = k.shape[1:]
    scale = 1 / math.sqrt(D) if scale is None else scale
    floor = torch.zeros_like(out)
    for i, n in enumerate(int(x) for x in lens):
        ids = table[i, :-(-n // page)].long()
        kk, codes = k[ids].reshape(-1, H, D)[:n], numbers[1][0][ids].reshape(-1, H, D)[:n].abs().sum(0)
        vs = numbers[1][1][ids].repeat_interleave(page, 0)[:n]
        for h in range(q.shape[1] if n else 0):
            g = h // (q.shape[1] // H)
            p = torch.softmax(scale * (kk[:, g] @ q[i, h]), 0)
            floor[i, h] = (p * vs[:, g]).max() * codes[g]
    return out, lse, size, reach, floor
