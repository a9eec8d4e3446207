"""The 64-bit references of the convolution, scan and paged attention, on the
CPU: closed forms, invariants, and the gradient against central differences."""
import math

import pytest
import torch

from oracle import ops

F64 = torch.float64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, dtype=F64)


def test_conv_is_torch_conv1d():
    g = gen(0)
    x, w, b, h = randn(g, 9, 5), randn(g, 5, 4), randn(g, 5), randn(g, 1, 3, 5)
    out, hist, _ = ops.short_conv(x, w, b, h, act=False)
    full = torch.cat([h[0], x]).t()[None]
    ref = torch.nn.functional.conv1d(full, w[:, None], b, groups=5)[0].t()
    assert torch.allclose(out, ref, rtol=0, atol=1e-12)
    assert torch.equal(hist[0], x[-3:])


def test_conv_packed_is_separate_and_short_sequences_keep_history():
    g = gen(1)
    x, w, h = randn(g, 6, 3), randn(g, 3, 4), randn(g, 4, 3, 3)
    cu = [0, 1, 1, 5, 6]
    out, hist, _ = ops.short_conv(x, w, None, h, cu=cu, n=4)
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        o, f, _ = ops.short_conv(x[a:b], w, None, h[i:i + 1])
        assert torch.equal(out[a:b], o) and torch.equal(hist[i], f[0])
    assert torch.equal(hist[1], h[1])                                  # nothing came
    assert torch.equal(hist[0], torch.cat([h[0, 1:], x[:1]]))


@pytest.mark.parametrize("W,act", [(2, True), (3, False), (4, True)])
def test_conv_gradient_against_differences(W, act):
    g = gen(W)
    cu = [0, 2, 2, 9, 10]
    x, w, b, h = randn(g, 10, 3), randn(g, 3, W), randn(g, 3), randn(g, 4, W - 1, 3)
    dy, df = randn(g, 10, 3), randn(g, 4, W - 1, 3)

    def loss(x, w, b, h):
        o, f, _ = ops.short_conv(x, w, b, h, cu=cu, n=4, act=act)
        return float((o * dy).sum() + (f * df).sum())

    got = ops.short_conv_backward(x, w, dy, b, h, cu=cu, n=4, act=act, d_final=df)
    args = [x, w, b, h]
    for i, name in enumerate(("dx", "dweight", "dbias", "dstate")):
        u = randn(g, *args[i].shape)
        e = 1e-5
        hi, lo = ([v + s * e * u if k == i else v for k, v in enumerate(args)] for s in (1, -1))
        diff = (loss(*hi) - loss(*lo)) / (2 * e)
        assert abs(diff - float((got[name][0] * u).sum())) <= 1e-7 * (1 + abs(diff)), name


def test_scan_closed_forms():
    g = gen(3)
    x, b, c = randn(g, 5, 2, 3), randn(g, 5, 1, 4), randn(g, 5, 1, 4)
    dt, a, s0 = torch.rand(5, 2, generator=g, dtype=F64), -torch.rand(2, generator=g, dtype=F64), \
        randn(g, 1, 2, 4, 3)
    # without input only the decay is left
    y, s, _, _ = ops.ssm(torch.zeros_like(x), dt, a, b, c, state=s0)
    decay = torch.exp(a * dt.sum(0))
    assert torch.allclose(s[0], decay[:, None, None] * s0[0], rtol=0, atol=1e-12)
    # from a zero state, the quadratic form over pairs of tokens
    y, s, _, _ = ops.ssm(x, dt, a, b, c)
    for h in range(2):
        for t in range(5):
            ref = sum(float(c[t, 0] @ b[r, 0]) * math.exp(float(a[h] * dt[r + 1:t + 1, h].sum()))
                      * float(dt[r, h]) * x[r, h] for r in range(t + 1))
            assert torch.allclose(y[t, h], ref, rtol=0, atol=1e-12)
    # softplus of a large value is the value, of a very negative one its exponential
    big = torch.tensor([[30.0, -30.0]], dtype=F64)
    y, s, _, _ = ops.ssm(x[:1], big, a, b[:1], c[:1], softplus=True)
    y2, s2, _, _ = ops.ssm(x[:1], torch.tensor([[30.0 + math.exp(-30), math.log1p(math.exp(-30))]],
                                               dtype=F64), a, b[:1], c[:1])
    assert torch.allclose(s, s2, rtol=1e-12, atol=0)


def test_scan_state_passing_and_groups():
    g = gen(4)
    x, b, c = randn(g, 7, 4, 3), randn(g, 7, 2, 4), randn(g, 7, 2, 4)
    dt, a = torch.rand(7, 4, generator=g, dtype=F64), -torch.rand(4, generator=g, dtype=F64)
    y, s, _, _ = ops.ssm(x, dt, a, b, c)
    y1, s1, _, _ = ops.ssm(x[:3], dt[:3], a, b[:3], c[:3])
    y2, s2, _, _ = ops.ssm(x[3:], dt[3:], a, b[3:], c[3:], state=s1)
    assert torch.allclose(torch.cat([y1, y2]), y, rtol=0, atol=1e-12)
    assert torch.allclose(s2, s, rtol=0, atol=1e-12)
    # heads 2 and 3 use the second group
    y3, _, _, _ = ops.ssm(x[:, 2:], dt[:, 2:], a[2:], b[:, 1:], c[:, 1:])
    assert torch.equal(y3, y[:, 2:])


def test_attention_forms():
    g = gen(5)
    k, v = randn(g, 4, 2, 1, 8), randn(g, 4, 2, 1, 8)
    q = randn(g, 3, 2, 8)
    table = torch.tensor([[2, 0, 9], [3, 9, 9], [9, 9, 9]], dtype=torch.int32)
    out, lse, _, _ = ops.paged_attention(q, k, v, table, [3, 1, 0])
    rows_k, rows_v = torch.cat([k[2], k[0][:1]])[:, 0], torch.cat([v[2], v[0][:1]])[:, 0]
    ref = torch.nn.functional.scaled_dot_product_attention(q[0][:, None], rows_k[None].expand(2, 3, 8),
                                                           rows_v[None].expand(2, 3, 8))[:, 0]
    assert torch.allclose(out[0], ref, rtol=0, atol=1e-12)
    assert torch.equal(out[1], v[3, 0].expand(2, 8))          # one token: its value
    assert torch.allclose(lse[1], (q[1] @ k[3, 0, 0]) / math.sqrt(8), rtol=0, atol=1e-12)
    assert not out[2].any() and torch.isinf(lse[2]).all()
