"""The convolution, scan and paged attention entry points without a GPU: bad
arguments are refused before the device is touched."""
import pytest
import torch

import prefill_kda_chunk_gb300 as K
from prefill_kda_chunk_gb300 import build as B

A = 1 << 20  # an aligned fake address; validation fails before any dereference
M = 1 << 24


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return K.lib()


def conv(**kw):
    args = dict(x=A, weight=A + M, bias=A + 2 * M, initial_state=A + 3 * M, cu_seqlens=0, B=1,
                T=16, D=64, W=4, N=1, x_stride=64, flags=1, out=A + 4 * M, out_stride=64,
                final_state=A + 5 * M, stream=0)
    args.update(kw)
    return K.kda_short_conv(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=2), "KDA_ERR_BAD_FLAGS"),
    (dict(W=1), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(W=5), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(D=0), "KDA_ERR_BAD_SHAPE"),
    (dict(T=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(N=2), "KDA_ERR_BAD_SHAPE"),
    (dict(B=2, N=2, cu_seqlens=A + 6 * M), "KDA_ERR_BAD_SHAPE"),
    (dict(T=1 << 31), "KDA_ERR_BAD_SHAPE"),
    (dict(x_stride=63), "KDA_ERR_BAD_SHAPE"),
    (dict(out_stride=63), "KDA_ERR_BAD_SHAPE"),
    (dict(x=0), "KDA_ERR_NULL_ARG"),
    (dict(out=0), "KDA_ERR_NULL_ARG"),
    (dict(weight=0), "KDA_ERR_NULL_ARG"),
    (dict(x=A + 1), "KDA_ERR_MISALIGNED"),
    (dict(weight=A + M + 2), "KDA_ERR_MISALIGNED"),
    (dict(out=A), "KDA_ERR_ALIAS"),
    (dict(out=A + 64, out_stride=128, x_stride=128, D=65), "KDA_ERR_ALIAS"),
    (dict(final_state=A + 3 * M), "KDA_ERR_ALIAS"),
    (dict(final_state=A + 4 * M), "KDA_ERR_ALIAS"),
])
def test_conv_refusals(kw, code):
    assert conv(**kw) == K.STATUS_CODE[code]


def test_conv_slices_of_one_buffer_do_not_alias():
    # x and out are the two halves of each row of one buffer: past the checks of
    # the arguments (and stopped by those of the device or of the pointers)
    rc = conv(x=A, out=A + 128, x_stride=128, out_stride=128)
    assert rc not in (K.STATUS_CODE["KDA_ERR_ALIAS"], 0)


def conv_step(**kw):
    args = dict(x=A, weight=A + M, bias=0, state_in=A + 3 * M, N=4, D=64, W=4, x_stride=64,
                flags=0, out=A + 4 * M, out_stride=64, state_out=A + 3 * M, stream=0)
    args.update(kw)
    return K.kda_short_conv_step(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=2), "KDA_ERR_BAD_FLAGS"),
    (dict(W=5), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(N=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(x_stride=8), "KDA_ERR_BAD_SHAPE"),
    (dict(state_out=0), "KDA_ERR_NULL_ARG"),
    (dict(x=0), "KDA_ERR_NULL_ARG"),
    (dict(state_out=A + 3 * M + 2), "KDA_ERR_ALIAS"),
    (dict(out=A + 3 * M), "KDA_ERR_ALIAS"),
])
def test_conv_step_refusals(kw, code):
    assert conv_step(**kw) == K.STATUS_CODE[code]


def test_empty_batches_are_no_ops():
    assert K.kda_short_conv_step(0, 0, 0, 0, 0, 64, 4, 64, 0, 0, 64, 0, 0) == 0
    assert K.kda_ssm_step(0, 0, A, 0, 0, 0, 0, 0, 0, 4, 64, 1, 128, 256, 4, 128, 128, 0, 0, 0, 0) == 0
    assert K.kda_paged_decode(0, 0, 0, 0, 0, 0, 8, 8, 128, 0, 16, 0, 16 * 8 * 128, 16 * 8 * 128, 1.0,
                              0, 0, 0) == 0


def conv_backward(**kw):
    args = dict(x=A, weight=A + M, bias=A + 2 * M, initial_state=0, cu_seqlens=0, B=1, T=16, D=64,
                W=4, N=1, x_stride=64, flags=3, d_out=A + 4 * M, dout_stride=64, d_final_state=0,
                dx=A + 5 * M, dx_stride=64, dweight=A + 6 * M, dbias=A + 7 * M,
                d_initial_state=A + 8 * M, stream=0)
    args.update(kw)
    return K.kda_short_conv_backward(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=4), "KDA_ERR_BAD_FLAGS"),
    (dict(W=0), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(dout_stride=60), "KDA_ERR_BAD_SHAPE"),
    (dict(dx_stride=60), "KDA_ERR_BAD_SHAPE"),
    (dict(d_out=0), "KDA_ERR_NULL_ARG"),
    (dict(dx=0), "KDA_ERR_NULL_ARG"),
    (dict(dweight=0), "KDA_ERR_NULL_ARG"),
    (dict(d_out=A + 4 * M + 2), "KDA_ERR_MISALIGNED"),       # fp32 on a 2-byte boundary
    (dict(dweight=A + 6 * M + 2), "KDA_ERR_MISALIGNED"),
    (dict(dx=A), "KDA_ERR_ALIAS"),
    (dict(dx=A + 4 * M), "KDA_ERR_ALIAS"),
    (dict(dbias=A + 6 * M), "KDA_ERR_ALIAS"),
    (dict(d_initial_state=A + 5 * M), "KDA_ERR_ALIAS"),
])
def test_conv_backward_refusals(kw, code):
    assert conv_backward(**kw) == K.STATUS_CODE[code]


def ssm(**kw):
    args = dict(x=A, dt=A + M, a=A + 2 * M, b=A + 3 * M, c=A + 4 * M, d=0, dt_bias=0,
                initial_state=0, cu_seqlens=0, B=1, T=16, H=4, P=64, G=2, n=128, N=1,
                x_stride=256, dt_stride=4, b_stride=256, c_stride=256, flags=1, out=A + 5 * M,
                final_state=A + 6 * M, stream=0)
    args.update(kw)
    return K.kda_ssm_prefill(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=2), "KDA_ERR_BAD_FLAGS"),
    (dict(P=96), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(n=16), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(G=3), "KDA_ERR_BAD_SHAPE"),
    (dict(H=0), "KDA_ERR_BAD_SHAPE"),
    (dict(N=2), "KDA_ERR_BAD_SHAPE"),
    (dict(x_stride=248), "KDA_ERR_BAD_SHAPE"),
    (dict(dt_stride=3), "KDA_ERR_BAD_SHAPE"),
    (dict(b_stride=128), "KDA_ERR_BAD_SHAPE"),
    (dict(a=0), "KDA_ERR_NULL_ARG"),
    (dict(c=0), "KDA_ERR_NULL_ARG"),
    (dict(x=A + 8), "KDA_ERR_MISALIGNED"),
    (dict(x_stride=260), "KDA_ERR_MISALIGNED"),
    (dict(out=A), "KDA_ERR_ALIAS"),
    (dict(final_state=A + 5 * M), "KDA_ERR_ALIAS"),
    (dict(initial_state=A + 6 * M + 16), "KDA_ERR_ALIAS"),
])
def test_ssm_refusals(kw, code):
    assert ssm(**kw) == K.STATUS_CODE[code]


def ssm_step(**kw):
    args = dict(x=A, dt=A + M, a=A + 2 * M, b=A + 3 * M, c=A + 4 * M, d=0, dt_bias=0,
                state_in=A + 6 * M, N=2, H=4, P=64, G=2, n=128, x_stride=256, dt_stride=4,
                b_stride=256, c_stride=256, flags=0, out=A + 5 * M, state_out=A + 6 * M, stream=0)
    args.update(kw)
    return K.kda_ssm_step(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(P=32), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(state_out=0), "KDA_ERR_NULL_ARG"),
    (dict(state_out=A + 6 * M + 64), "KDA_ERR_ALIAS"),
    (dict(state_in=A + 6 * M + 4, state_out=A + 8 * M), "KDA_ERR_MISALIGNED"),
])
def test_ssm_step_refusals(kw, code):
    assert ssm_step(**kw) == K.STATUS_CODE[code]


def paged(**kw):
    args = dict(q=A, k_cache=A + M, v_cache=A + 3 * M, page_table=A + 5 * M, seq_lens=A + 6 * M,
                B=2, Hq=8, Hkv=2, D=128, pages=4, page_size=16, max_pages=3,
                k_page_stride=16 * 256, v_page_stride=16 * 256, scale=1.0, out=A + 7 * M,
                lse=A + 8 * M, stream=0)
    args.update(kw)
    return K.kda_paged_decode(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(B=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(Hq=7), "KDA_ERR_BAD_SHAPE"),
    (dict(Hq=1), "KDA_ERR_BAD_SHAPE"),
    (dict(page_size=0), "KDA_ERR_BAD_SHAPE"),
    (dict(max_pages=1 << 28), "KDA_ERR_BAD_SHAPE"),
    (dict(k_page_stride=16 * 256 - 8), "KDA_ERR_BAD_SHAPE"),
    (dict(q=0), "KDA_ERR_NULL_ARG"),
    (dict(page_table=0), "KDA_ERR_NULL_ARG"),
    (dict(v_cache=0), "KDA_ERR_NULL_ARG"),
    (dict(seq_lens=0), "KDA_ERR_NULL_ARG"),
    (dict(k_cache=A + M + 8), "KDA_ERR_MISALIGNED"),
    (dict(v_page_stride=16 * 256 + 4), "KDA_ERR_MISALIGNED"),
    (dict(out=A), "KDA_ERR_ALIAS"),
    (dict(lse=A + 7 * M), "KDA_ERR_ALIAS"),
])
def test_paged_refusals(kw, code):
    assert paged(**kw) == K.STATUS_CODE[code]


def test_python_front_refuses():
    """The binding's own checks, which need no library call."""
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        K.short_conv(x, w)                                  # not on a GPU
    with pytest.raises(ValueError):
        K.short_conv(x, w, activation="gelu")
    with pytest.raises(ValueError):
        K.short_conv_step(x, w, in_place=True)
    with pytest.raises(ValueError):
        K.ssm_prefill(torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 2),
                      torch.zeros(2), torch.zeros(4, 1, 64, dtype=torch.bfloat16),
                      torch.zeros(4, 1, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        K.paged_decode(torch.zeros(1, 2, 64, dtype=torch.bfloat16),
                       torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16),
                       torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16),
                       torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("d32", [False, True])
@pytest.mark.parametrize("off", [0, 4, 1])
def test_conv_gradient_scratch_holds_every_tile(off, d32):
    """Each form of the gradient (its channels per block follow from the width and the
    alignment) asks for the scratch that its own tiles write."""
    g = torch.Generator().manual_seed(10 * off + d32)
    cases = [(7180, 3841), (13766, 2112), (14400, 2050), (27712, 1026), (71708, 385),
             (87297, 800), (131072, 130), (126474, 150), (0, 5), (1, 1)]
    for _ in range(1000):
        u, v = torch.rand(2, generator=g, dtype=torch.float64).tolist()
        cases.append((int(2 ** (18 * u)), int(2 ** (14 * v))))
    forms = set()
    for T, D in cases:
        at, stride = A + 2 * off, -(-(D + off) // 8) * 8
        rc, (scratch, channels, cols, run, tiles) = K.kda_test_conv_backward_plan(
            at, A + (4 if d32 else 2) * off, at, T, D, 4, stride, stride, stride,
            K.CONV_DOUT_FP32 * d32)
        assert rc == 0
        forms.add(channels)
        assert channels == (32 if off == 1 or D % 4 else 128)
        assert (cols - 1) * channels < D <= cols * channels
        assert (tiles - 1) * 8 * run < max(T, 1) <= tiles * 8 * run   # every token, no empty tile
        assert scratch >= tiles * 5 * D * 4, (T, D, channels)
    assert forms == ({32} if off == 1 else {32, 128})
