"""How exactly the norms with the rotation know a position's sines and cosines.

With a head of ones (its norm is 1), one token, and a gradient of ones for the first of each pair, the
gradient of the weights is the cosines and minus the sines themselves, in fp32.
"""
import pytest
import torch

import prefill_kda_chunk_gb300 as K
from test_gpu_cache import BF16, F32, I32, built  # noqa: F401

pytestmark = pytest.mark.gpu


def errors(farthest, pairs, n=150, D=256):
    x, w = torch.ones(1, 1, D, dtype=BF16, device="cuda"), torch.ones(D, device="cuda")
    first = torch.arange(0, D, 2) if pairs else torch.arange(D // 2)
    second = first + 1 if pairs else first + D // 2
    dy = torch.zeros(1, 1, D)
    dy[..., first] = 1.0
    g, dy, found = torch.Generator().manual_seed(farthest + pairs), dy.cuda(), []
    for i in range(n):
        freq = torch.rand(D // 2, generator=g)
        pos = torch.randint(0, farthest, (1,), generator=g).to(I32) * (-1) ** i
        _, _, dw, _ = K.qk_norm_rope_backward(x, None, dy, None, w, None, freq.cuda(), pos.cuda(), eps=0.0, interleaved=pairs)
        dw, t = dw.double().cpu(), pos.double() * freq.double()
        found += [dw[first] - torch.cos(t), dw[second] + torch.sin(t)]
    return torch.cat(found)


@pytest.mark.parametrize("pairs", [False, True])
def test_angles_of_near_positions(pairs):
    """Below position 4096 a turn's fraction is rounded once, to a multiple of 2^-25: off by 2^-26 / sqrt(3)
    of a turn in the root mean square, 2^-24.1 of a radian; the sine, the cosine and 1 / sqrt(1) add roundings of
    2^-25 to values that are one half in the mean square. Together below 2^-23.7."""
    e = errors(4096, pairs)
    assert float(e.square().mean().sqrt()) <= 2.0 ** -23.7


@pytest.mark.parametrize("pairs", [False, True])
def test_angles_of_far_positions(pairs):
    """Up to 2^24 two fractions are added, each step off by 2^-25 of a turn at most (2^-24 where a sum is
    above one half): 2^-23 of a turn, 2^-20.3 of a radian, and the roundings."""
    e = errors(1 << 24, pairs)
    assert float(e.abs().max()) <= 2.0 ** -20.2
    assert float(e.square().mean().sqrt()) <= 2.0 ** -23
