"""How exactly the attention over the 8-bit cache holds its weights.

Two tokens whose values nearly cancel show a weight's error beside a small output. The first
token's weight is its tile's largest, which the terms hold exactly. The second's, w >= 2^e: each e4m3 term
leaves half a step, 2^-4 2^e, of which the next one gets 32 times as much; after four 2^-19, and
2^-21 from rounding to half precision behind the second: 2^-18.68 of w. Its share of size, the sum of
p |v|, is at most 30 / 38 (r = 1, a = 8, b = 30). ex2, the scores (one product each, times the
scale) and the sum add 2^-21 of fp32. Together 2^-18.69 size, and bf16's rounding, 2^-8 of out.
"""
import pytest
import torch

import prefill_kda_chunk_gb300 as K
from oracle import cache as C
from test_gpu_cache import BF16, F8, I32, built, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,group,page", [(128, 8, 16), (64, 8, 16), (128, 16, 16), (64, 4, 17), (128, 16, 17)])
def test_weights_of_values_that_cancel(D, group, page):
    B, g = 512 // group, torch.Generator().manual_seed(D + group + page)
    q = torch.zeros(B, group, D)
    q[..., 0] = -0.7 * torch.rand(B, group, generator=g)
    q = q.to(BF16)
    k, v = torch.zeros(B, page, 1, D), torch.zeros(B, page, 1, D)
    k[:, 1, 0, 0] = 1.0   # scores 0 and q[0]
    # a in 8 .. 15, b in 8 .. 30: all ratios that e4m3 has, and what cancels at weights of 0.5 to 1
    a = torch.randint(8, 16, (B, D), generator=g).float()
    b = torch.randint(8, 16, (B, D), generator=g).float()
    v[:, 0, 0], v[:, 1, 0] = a, -torch.where(torch.rand(B, D, generator=g) < 0.3, 2 * b, b)
    one = torch.ones(B, 1)
    table, lens = torch.arange(B, dtype=I32)[:, None], [2] * B
    case = (q, k.to(F8), v.to(F8), one, one, table)
    out, _ = K.paged_decode_fp8(*(t.cuda() for t in case), i32(lens), scale=1.0)
    K.check_device_error()
    ref, _, size, _, _ = C.paged_attention(*case, lens, 1.0)
    small = ref.abs() <= 2.0 ** -9 * size
    assert small.sum() > 50, "nothing cancels"
    err = (out.double().cpu() - ref).abs() - 2.0 ** -8 * ref.abs()
    worst = float((err / size).max())
    assert worst <= 2.0 ** -18.6, f"a weight is off by more than its terms leave: {worst:.2e}"
