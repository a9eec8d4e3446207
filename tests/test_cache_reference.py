"""The 64-bit references around the 8-bit cache against closed forms and other ways to
the same numbers."""
import math

import pytest
import torch

from oracle import cache as C

F64 = torch.float64


def test_plan_worked_by_hand():
    table = [[5, 6, 0], [7, 0, 0], [8, 9, 4]]
    # slot 1 gives 7 back and starts again with 3 tokens; slot 0 fills its page and takes one
    got = C.page_plan(table, [3, 2, 6], [2, 3, 0], [1, 2, 3, 0, 0], 3, 2, 7, release=[0, 1, 0])
    assert got[0] == [[5, 6, 7], [3, 2, 0], [8, 9, 4]]
    assert got[1] == [5, 3, 6] and got[3] == 1 and got[2] == [1, 2, 3, 7, 0]
    assert got[4] == [0, 2, 5, 5]
    assert got[5] == [3, 4, 0, 1, 2, 0, 0]
    assert got[6] == [13, 14, 6, 7, 4, -1, -1]
    assert C.page_plan(table, [3, 2, 6], [2, 9, 0], [1, 2, 3, 0, 0], 3, 2, 20) is None   # too long
    assert C.page_plan(table, [3, 2, 6], [2, 3, 0], [1, 2, 3], 1, 2, 7) is None          # no pages


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_depends_on_distance_alone(interleaved):
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(2, 1, 1, 64, generator=g, dtype=F64)
    freq = 10000.0 ** (-torch.arange(0, 64, 2, dtype=F64) / 64)
    dots = []
    for a, b in ((3, 1), (102, 100), (100000, 99998)):
        y = [C.norm_rope(x, None, freq, torch.tensor([p]), 0.0, interleaved)[0] for x, p in ((q, a), (k, b))]
        assert torch.allclose((y[0] ** 2).sum(), torch.tensor(64.0, dtype=F64))
        dots.append(float((y[0] * y[1]).sum()))
    assert max(dots) - min(dots) < 1e-9


@pytest.mark.parametrize("interleaved,R", [(False, 32), (True, 16), (False, 0)])
def test_norm_gradient_against_autograd(interleaved, R):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(5, 3, 64, generator=g, dtype=F64, requires_grad=True)
    w = torch.randn(64, generator=g, dtype=F64, requires_grad=True)
    dy = torch.randn(5, 3, 64, generator=g, dtype=F64)
    freq = torch.rand(R // 2, generator=g, dtype=F64) if R else None
    pos = torch.tensor([0, 1, 7, -3, 1000]) if R else None
    u = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + 1e-3) * w
    if R:
        t = (pos[:, None] * freq)[:, None]
        a, b = C._pairs(R, interleaved)
        z = torch.complex(u[..., a], u[..., b]) * torch.polar(torch.ones_like(t), t)
        y = u.clone()
        y[..., a], y[..., b] = z.real, z.imag
    else:
        y = u
    assert torch.allclose(y, C.norm_rope(x, w.detach(), freq, pos, 1e-3, interleaved)[0])
    y.backward(dy)
    (dx, _), (dw, _) = C.norm_rope_backward(x, dy, w.detach(), freq, pos, 1e-3, interleaved)
    assert torch.allclose(dx, x.grad) and torch.allclose(dw, w.grad)


def test_e4m3_against_torch():
    y = torch.cat([C.E4M3, (C.E4M3[1:] + C.E4M3[:-1]) / 2, torch.linspace(0, 448, 5000, dtype=F64)])
    y = torch.cat([y, -y])
    assert torch.equal(C.e4m3(y), y.float().to(torch.float8_e4m3fn).to(F64))
    assert torch.isnan(C.e4m3(torch.tensor([math.inf, -math.inf, math.nan], dtype=F64))).all()
    for top, k in ((448, 0), (449, 1), (224, -1), (1.75, -8), (1.76, -7), (0, -126), (1e-38, -126)):
        assert C.scale_for(top) == 2.0 ** k


def test_append_keeps_what_fits():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 2, 64, generator=g).to(torch.bfloat16)
    table = torch.tensor([[2, 0, 4]])
    whole, ws = torch.zeros(5, 16, 2, 64, dtype=F64), torch.zeros(5, 2, dtype=F64)
    C.append(x, whole, ws, table, [40], [0, 40])
    steps, ss = torch.zeros_like(whole), torch.zeros_like(ws)
    for t in range(40):
        C.append(x[t:t + 1], steps, ss, table, [t + 1])
    assert torch.equal(ws, ss)
    for i, p in enumerate((2, 0, 4)):
        rows = x[16 * i:16 * (i + 1)].to(F64)
        n = len(rows)
        got = whole[p, :n] * ws[p][:, None]
        # e4m3: half a step of 2^-4, or of the smallest numbers
        assert ((got - rows).abs() <= torch.maximum(rows.abs() * 2.0 ** -4, ws[p][:, None] * 2.0 ** -10)).all()
        assert (got.abs().amax((0, 2)) > 448 / 2 * ws[p] * (1 - 2.0 ** -4)).all()
        # token by token the page was scaled down in between: once more half a step below
        # 2^-6 (numbers of full precision are not touched)
        diff = (steps[p, :n] - whole[p, :n]).abs()
        assert (diff <= 2.0 ** -9).all() and (diff[whole[p, :n].abs() > 2.0 ** -6] == 0).all()


def test_attention_of_equal_keys_is_the_mean():
    g = torch.Generator().manual_seed(4)
    v = torch.randn(3, 4, 1, 64, generator=g).to(torch.float8_e4m3fn)
    k = torch.ones(3, 4, 1, 64).to(torch.float8_e4m3fn)
    vs = torch.tensor([[0.5], [2.0], [1.0]])
    out, lse, _, _, floor = C.paged_attention(torch.ones(1, 2, 64), k, v, torch.ones(3, 1), vs,
                                       torch.tensor([[2, 1]]), [6])
    rows = torch.cat([v[2].to(F64), 2 * v[1, :2].to(F64)])[:, 0]
    assert torch.allclose(out[0, 0], rows.mean(0)) and math.isclose(float(lse[0, 0]), 8 + math.log(6))
    assert torch.allclose(floor[0, 0], 2 / 6 * torch.cat([v[2], v[1, :2]]).to(F64)[:, 0].abs().sum(0))
