"""Bounded waits of the operators around the 8-bit cache: calls that take long are not cut off."""
import math

import pytest
import torch

import prefill_kda_chunk_gb300 as K
from test_gpu_cache import BF16, F8, I32, attention_close, built, i32, make  # noqa: F401

pytestmark = pytest.mark.gpu


def test_attention_for_seconds():
    """A call that works for three seconds or more, where the queries of later pieces wait for the end of
    one that takes nearly as long: 2^31 - 4096 tokens for each of 48 heads, one page again and again,
    and six short sequences behind them.

    Scores are zero and values whole numbers whose sum over 128 tokens is -1, 0 or 1, so that every sum of
    a piece's values and weights is a whole number below 2^24, exact in fp32. The pieces' values add up to
    less than 2^24 as well; their weights, to 2^31, are off by 2^-24 for each of the 20 additions at
    most. out = (-1, 0, 1) / 128, which bf16 holds, is less than half a step away."""
    page, H, D, pages, short = 4096, 48, 64, 7, [5, 1, 130, 7, 4096, 33]
    reps = (1 << 31) // page - 1
    r = make(4)
    k, v = (r(pages, page, H, D).to(F8) for _ in "kv")
    k.view(torch.uint8)[0] = 0
    c = torch.randint(-1, 2, (H, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).float()
    t = torch.arange(page, device="cuda") % 128
    sign = torch.where(t < 64, 1.0, -1.0)[:, None, None].expand(page, H, D)
    v[0] = torch.where((t == 127)[:, None, None], c - 1, sign).to(F8)
    one = torch.ones(pages, H, device="cuda")
    table = torch.zeros(1 + len(short), reps, dtype=I32, device="cuda")
    table[1:, 0] = torch.arange(1, 1 + len(short), dtype=I32, device="cuda")
    q = r(1 + len(short), H, D)
    began, ended = torch.cuda.Event(True), torch.cuda.Event(True)
    began.record()
    o, l = K.paged_decode_fp8(q, k, v, one, one, table, i32([reps * page] + short))
    ended.record()
    K.check_device_error()
    assert began.elapsed_time(ended) > 2200, "the call does not take long enough for what this test is for"
    assert torch.equal(o[0].float(), c / 128)
    assert ((l[0] - math.log(reps * page)).abs() <= 1e-5).all()
    attention_close(o[1:], l[1:], q[1:], k, v, one, one, table[1:, :1], short)


def stalled(batch, call):
    """Milliseconds that the call takes on the GPU when no warp gets more than so many batches and three."""
    began, ended = torch.cuda.Event(True), torch.cuda.Event(True)
    assert K.kda_test_stall_qk_norm_rope(batch) == 0
    try:
        began.record()
        call()
        ended.record()
        with pytest.raises(K.KdaError, match="TIMEOUT"):
            K.check_device_error()
    finally:
        assert K.kda_test_stall_qk_norm_rope(-1) == 0
    return began.elapsed_time(ended)


@pytest.mark.parametrize("batch", [0, 1, 4])
@pytest.mark.parametrize("weights", [True, False])
def test_norms_wait_once_and_no_more(weights, batch):
    """Warps with a dozen batches or more to come: the first wait that runs out, two seconds, is the last one (and a
    tenth for each of three places of the ring). The next call is right."""
    T, H, D = 12000, 40, 64
    r = make(3)
    q, k, dq, dk = r(T, H, D), r(T, 8, D), r(T, H, D), r(T, 8, D)
    w = [1 + 0.1 * r(D, dtype=torch.float32) if weights else None for _ in "qk"]
    pos = torch.arange(T, dtype=I32, device="cuda")
    freq = torch.rand(D // 2, device="cuda")
    for call in (lambda: K.qk_norm_rope(q, k, *w, freq, pos),
                 lambda: K.qk_norm_rope_backward(q, k, dq, dk, *w, freq, pos)):
        ref = call()
        K.check_device_error()
        assert stalled(batch, call) < 3500
        got = call()
        K.check_device_error()
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, ref))


def test_stall_hook_arguments():
    assert K.kda_test_stall_qk_norm_rope(-2) != 0
    assert K.kda_test_stall_qk_norm_rope(-1) == 0


def test_no_wait_runs_out_at_work():
    """Hundreds of calls whose roles wait for one another all the time: the clock that they share may be set
    between a wait's two readings of the time."""
    r, H, D, page = make(6), 8, 64, 64
    lens = [32768] * 8
    k, v = (r(4096, page, H, D).to(F8) for _ in "kv")
    one = torch.ones(4096, H, device="cuda")
    table = torch.arange(4096, dtype=I32, device="cuda").view(8, 512)
    q, n = r(8, 64, D), i32(lens)
    ref = K.paged_decode_fp8(q, k, v, one, one, table, n)
    for i in range(400):
        got = K.paged_decode_fp8(q, k, v, one, one, table, n)
        if i % 50 == 0:
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    K.check_device_error()


@pytest.mark.parametrize("page", [4096, 17])
def test_attention_leaves_a_long_piece(page):
    """A wait that runs out early in pieces of 110000 tiles: the roles come to their end in a second or two."""
    r, H, D = make(5), 1, 64
    reps = (1 << 31) // page - 1
    k, v = (r(2, page, H, D).to(F8) for _ in "kv")
    one = torch.ones(2, H, device="cuda")
    q, table, lens = r(1, 8, D), torch.zeros(1, reps, dtype=I32, device="cuda"), i32([reps * page])
    small = (q, k, v, one, one, table[:, :1].contiguous(), i32([page]))
    ref = K.paged_decode_fp8(*small)
    began, ended = torch.cuda.Event(True), torch.cuda.Event(True)
    assert K.kda_test_stall_paged_fp8(3) == 0
    try:
        began.record()
        K.paged_decode_fp8(q, k, v, one, one, table, lens)
        ended.record()
        with pytest.raises(K.KdaError, match="TIMEOUT"):
            K.check_device_error()
    finally:
        assert K.kda_test_stall_paged_fp8(-1) == 0
    assert began.elapsed_time(ended) < 6000
    got = K.paged_decode_fp8(*small)
    K.check_device_error()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
