"""Short convolution, state space scan and paged decode attention on the GPU
against the 64-bit references.

Tolerances, element by element. A bf16 output is rounded once, by at most
2^-9 of its value (2^-8 is allowed); before that it is a sum whose terms have
an absolute sum S, known from the reference, and whose fp32 or split-bf16
arithmetic errs by far less than 2^-12 S. An fp32 output is allowed 2^-17 S:
a few hundred roundings of 2^-24 along the longest chain of operations.
"""
import math

import pytest
import torch

import prefill_kda_chunk_gb300 as K
from oracle import ops

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from prefill_kda_chunk_gb300 import build
    build.build()
    K.lib()


def close(got, ref, size, tag):
    got = got.detach().cpu()
    coarse = got.dtype == BF16
    got = got.double()
    assert torch.isfinite(got).all(), f"{tag}: not finite"
    tol = (2.0 ** -8 * ref.abs() + 2.0 ** -12 * size) if coarse else 2.0 ** -17 * size
    worst = ((got - ref).abs() - tol).max() if got.numel() else torch.tensor(-1.0)
    assert worst <= 1e-30, f"{tag}: over the bound by {float(worst):.3e}"


def make(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=BF16, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
    return randn


def cu_of(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32)


# ------------------------------------------------------------ convolution

CONV = [
    # lens, D, W, bias, silu, state, columns of the buffer x is a slice of, offset of the slice
    ([1], 8, 4, True, True, True, 8, 0),
    ([5], 1, 2, False, False, False, 1, 0),
    ([0, 3, 0, 0, 1, 2, 0], 36, 4, True, True, True, 36, 0),
    ([300, 0, 1, 41, 700], 264, 4, True, True, True, 272, 8),
    ([257], 520, 3, False, True, False, 1040, 520),
    ([31, 33, 256], 7, 4, True, False, True, 9, 1),
    ([64] * 5, 1032, 2, True, True, False, 1032, 0),
    ([2] * 70, 260, 4, False, True, True, 264, 4),
    ([1000], 8200, 4, False, True, True, 8200, 0),
]


def conv_case(lens, D, W, bias, state, cols, off, seed=0):
    r = make(seed + D + W)
    T, N = sum(lens), len(lens)
    x = r(T, cols)[:, off:off + D]
    w = r(D, W, dtype=F32, scale=0.5)
    b = r(D, dtype=F32) if bias else None
    h = r(N, W - 1, D) if state else None
    return r, x, w, b, h, T, N


@pytest.mark.parametrize("lens,D,W,bias,silu,state,cols,off", CONV)
def test_conv(lens, D, W, bias, silu, state, cols, off):
    r, x, w, b, h, T, N = conv_case(lens, D, W, bias, state, cols, off)
    cu = cu_of(lens)
    out = torch.full((T, D + 8), float("nan"), dtype=BF16, device="cuda")[:, 8:]
    o, f = K.short_conv(x, w, b, initial_state=h, cu_seqlens=cu.cuda(), out=out,
                        activation="silu" if silu else None)
    K.check_device_error()
    ro, rf, size = ops.short_conv(x, w, b, h, cu=cu, n=N, act=silu)
    close(o, ro, size, "out")
    assert torch.equal(f.cpu().double(), rf), "history"


@pytest.mark.parametrize("silu", [True, False])
def test_conv_fixed_batch_and_no_tokens(silu):
    r = make(3)
    x, w, h = r(3, 45, 72), r(72, 4, dtype=F32), r(3, 3, 72)
    o, f = K.short_conv(x, w, None, initial_state=h, activation="silu" if silu else None)
    ro, rf, size = ops.short_conv(x.reshape(-1, 72), w, None, h, n=3, act=silu)
    close(o.reshape(-1, 72), ro, size, "out")
    assert torch.equal(f.cpu().double(), rf)
    o, f = K.short_conv(x[:, :0], w, None, initial_state=h)
    K.check_device_error()
    assert o.shape == (3, 0, 72) and torch.equal(f, h)
    o, f = K.short_conv(x, w, output_final_state=False)
    assert f is None


def test_conv_bad_cu_seqlens_is_reported_and_skips():
    r = make(4)
    x, w = r(20, 64), r(64, 4, dtype=F32)
    out = torch.zeros_like(x)
    cu = torch.tensor([0, 12, 8, 20], dtype=torch.int32, device="cuda")
    K.short_conv(x, w, cu_seqlens=cu, out=out)
    with pytest.raises(K.KdaError, match="CU_SEQLENS"):
        K.check_device_error()
    assert not out.any()
    K.short_conv(x, w, out=out)
    K.check_device_error()


@pytest.mark.parametrize("N,D,W,bias,silu,cols,off", [
    (1, 8, 4, True, True, 8, 0), (3, 1, 2, False, False, 1, 0), (37, 36, 3, True, True, 40, 4),
    (256, 1544, 4, False, True, 1544, 0), (5, 7, 4, True, True, 9, 1)])
def test_conv_step(N, D, W, bias, silu, cols, off):
    r, x, w, b, h, _, _ = conv_case([1] * N, D, W, bias, True, cols, off)
    act = "silu" if silu else None
    o, f = K.short_conv_step(x, w, h, b, activation=act)
    ro, rf, size = ops.short_conv(x, w, b, h, cu=range(N + 1), n=N, act=silu)
    close(o, ro, size, "out")
    assert torch.equal(f.cpu().double(), rf)
    # in place, the same bits; without a history it is zeros
    h2 = h.clone()
    o2, f2 = K.short_conv_step(x, w, h2, b, activation=act, in_place=True)
    assert f2.data_ptr() == h2.data_ptr() and torch.equal(o2, o) and torch.equal(h2, f)
    o3, f3 = K.short_conv_step(x, w, None, b, activation=act)
    o4, f4 = K.short_conv_step(x, w, torch.zeros_like(h), b, activation=act)
    assert torch.equal(o3, o4) and torch.equal(f3, f4)


def test_conv_steps_follow_the_prompt():
    r = make(8)
    x, w, b, h = r(6, 9, 40), r(40, 4, dtype=F32), r(40, dtype=F32), r(6, 3, 40)
    o, f = K.short_conv(x, w, b, initial_state=h)
    state = h.clone()
    for t in range(9):
        y, _ = K.short_conv_step(x[:, t], w, state, b, in_place=True)
        assert torch.equal(y, o[:, t]), t
    assert torch.equal(state, f)


@pytest.mark.parametrize("d32", [True, False])
@pytest.mark.parametrize("lens,D,W,bias,silu,state,cols,off", CONV)
def test_conv_gradient(lens, D, W, bias, silu, state, cols, off, d32):
    r, x, w, b, h, T, N = conv_case(lens, D, W, bias, state, cols, off)
    cu = cu_of(lens)
    dy = r(T, cols, dtype=F32 if d32 else BF16)[:, off:off + D]
    df = r(N, W - 1, D, dtype=F32) if state else None
    dx = torch.full((T, cols), float("nan"), dtype=BF16, device="cuda")[:, off:off + D]
    kw = dict(bias=b, initial_state=h, cu_seqlens=cu.cuda(), activation="silu" if silu else None,
              d_final_state=df)
    got = K.short_conv_backward(x, w, dy, dx=dx, **kw)
    K.check_device_error()
    ref = ops.short_conv_backward(x, w, dy, b, h, cu=cu, n=N, act=silu, d_final=df)
    for g, name in zip(got, ("dx", "dweight", "dbias", "dstate")):
        if g is None:
            assert name == "dbias" and not bias
        else:
            close(g, *ref[name], name)
    again = K.short_conv_backward(x, w, dy, **kw)
    for g, g2 in zip(got, again):
        assert g is None or torch.equal(g, g2), "not the same bits again"


def test_conv_gradient_against_differences():
    """Directional derivatives of the reference's forward pass; the bound is the
    reference's own truncation and the one rounding of dx to bf16."""
    r = make(12)
    lens = [3, 0, 50, 1]
    x, w, b, h = r(54, 16), r(16, 4, dtype=F32, scale=0.5), r(16, dtype=F32), r(4, 3, 16)
    dy, df, cu = r(54, 16, dtype=F32), r(4, 3, 16, dtype=F32), cu_of(lens)
    got = K.short_conv_backward(x, w, dy, bias=b, initial_state=h, cu_seqlens=cu.cuda(),
                                d_final_state=df)
    args = [t.cpu().double() for t in (x, w, b, h)]
    dyc, dfc = dy.cpu().double(), df.cpu().double()

    def loss(v):
        o, f, _ = ops.short_conv(*v, cu=cu, n=4)
        return float((o * dyc).sum() + (f * dfc).sum())

    g = torch.Generator().manual_seed(1)
    for i, name in enumerate(("dx", "dweight", "dbias", "dstate")):
        u, e = torch.randn(args[i].shape, generator=g, dtype=torch.float64), 1e-5
        hi, lo = ([v + s * e * u if k == i else v for k, v in enumerate(args)] for s in (1, -1))
        diff = (loss(hi) - loss(lo)) / (2 * e)
        mine = got[i].cpu().double()
        allow = 2.0 ** -8 * float((mine * u).norm()) * 4 if i == 0 else 1e-5 * float((mine * u).abs().sum())
        assert abs(float((mine * u).sum()) - diff) <= allow + 1e-7 * abs(diff), name


def test_conv_gradient_without_tokens():
    r = make(13)
    w, df = r(24, 4, dtype=F32), r(2, 3, 24, dtype=F32)
    dx, dw, db, dh = K.short_conv_backward(
        torch.empty(0, 24, dtype=BF16, device="cuda"), w, torch.empty(0, 24, device="cuda"),
        bias=w[:, 0].contiguous(), cu_seqlens=cu_of([0, 0]).cuda(), d_final_state=df)
    assert not dw.any() and not db.any() and torch.equal(dh, df)


@pytest.mark.parametrize("T,D,off,d32", [(14400, 2050, 0, True), (7180, 3841, 0, False),
                                         (13766, 2112, 1, False), (9001, 385, 0, True)])
def test_conv_gradient_one_channel_per_thread_over_waves(T, D, off, d32):
    """Widths and offsets that leave one channel per thread, at sizes of several waves
    of blocks, on a stream whose scratch is no larger than this call asks for."""
    r = make(T + D)
    x = r(T, D + off)[:, off:]
    w, b = r(D, 4, dtype=F32, scale=0.5), r(D, dtype=F32)
    dy = r(T, D + off, dtype=F32 if d32 else BF16)[:, off:]
    cu = cu_of([T - 5, 0, 5])
    K.check_device_error()
    assert K.kda_workspace_release() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = K.short_conv_backward(x, w, dy, bias=b, cu_seqlens=cu.cuda())
        again = K.short_conv_backward(x, w, dy, bias=b, cu_seqlens=cu.cuda())
        K.check_device_error()
    side.synchronize()
    ch = [0, 1, 31, 32, D // 2, D - 2, D - 1]
    ref = ops.short_conv_backward(x[:, ch], w[ch], dy[:, ch], b[ch], cu=cu, n=3)
    for g, g2, name in zip(got, again, ("dx", "dweight", "dbias", "dstate")):
        g, g2 = (g[ch], g2[ch]) if name in ("dweight", "dbias") else (g[..., ch], g2[..., ch])
        close(g, *ref[name], name)
        assert torch.equal(g, g2), "not the same bits again"


@pytest.mark.parametrize("D", [32, 7])
def test_conv_gradient_of_silu_at_large_z(D):
    """s (1 + z (1 - s)) tends to 1: an error of s itself must not be multiplied by z. The
    filter is one tap of 1, so z = x; a bf16 dx may be off by 2^-8 of it, the fp32 sums by
    2^-17 of their terms."""
    large = [15.0, 30.0, 1000.0, 1e5, 1e7, 1e10, 1e20, 1e30]
    x = make(D)(2 * len(large), D)
    x[:, ::3] = torch.tensor(large * 2, device="cuda").to(BF16)[:, None]
    w = torch.zeros(D, 2, device="cuda")
    w[:, 1] = 1
    z = x.cpu().double()
    s = torch.sigmoid(z)
    dz = s * (1 + z * torch.sigmoid(-z))
    for dtype in (F32, BF16):
        dx, dw, db, _ = K.short_conv_backward(x, w, torch.ones_like(x, dtype=dtype), torch.zeros(D, device="cuda"))
        close(dx, dz, s * (1 + z.abs() * torch.sigmoid(-z)), "dx")
        close(dw[:, 1], (dz * z).sum(0), (dz * z).abs().sum(0), "dweight")
        close(db, dz.sum(0), dz.abs().sum(0) + 1, "dbias")


FAR = [-43.0, -44.0, -50.0, -60.0, -87.0, -95.0, -130.0, -1e10, -1e30, 30.0, 1e30]


@pytest.mark.parametrize("D", [32, 7])
def test_conv_silu_far_from_zero(D):
    """z / (1 + e^-z) and its gradient to the ends of the range, ordinary channels beside.
    The filter is one tap of 1, so z = x. A bf16 result may be off by its rounding (2^-8 of
    it is allowed, and fp32's smallest normal number), an fp32 sum by 2^-17 of its terms."""
    T = 2 * len(FAR)
    x = make(D)(T, D)
    x[:, ::3] = torch.tensor(FAR * 2, device="cuda").to(BF16)[:, None]
    w = torch.zeros(D, 2, device="cuda")
    w[:, 1] = 1
    z = x.cpu().double()
    s = torch.sigmoid(z)

    def near(got, ref, tag, rel=2.0 ** -8):
        got = got.cpu().double()
        assert torch.isfinite(got).all(), tag
        assert ((got - ref).abs() <= rel * ref.abs() + 2.0 ** -126).all(), tag

    near(K.short_conv(x, w)[0], z * s, "prompt")
    near(K.short_conv_step(x, w)[0], z * s, "step")
    for dtype in (F32, BF16):
        dy = torch.ones(T, D, device="cuda", dtype=dtype)
        dx, dw, _, _ = K.short_conv_backward(x, w, dy)
        dz = s * (1 + z * (1 - s))
        near(dx, dz, "dx")
        size = (dz * z).abs().sum(0) + (dz.abs() * (1 + z.abs()) * z.abs() * 2.0 ** -24).sum(0)
        assert ((dw[:, 1].cpu().double() - (dz * z).sum(0)).abs() <= 2.0 ** -17 * size).all(), "dweight"


# ---------------------------------------------------------------- the scan

def ssm_case(lens, H, P, G, N, state, seed=0, fused=True, dt_scale=0.5, step=(1e-3, 0.1)):
    r = make(seed + H + P + N)
    T = sum(lens)
    if fused:
        xbc = r(T, H * P + 2 * G * N + 8)
        x = xbc[:, :H * P].view(T, H, P)
        b = xbc[:, H * P:H * P + G * N].view(T, G, N)
        c = xbc[:, H * P + G * N:H * P + 2 * G * N].view(T, G, N)
        dt = r(T, H + 3, dtype=F32, scale=dt_scale)[:, 3:]
    else:
        x, b, c, dt = r(T, H, P), r(T, G, N), r(T, G, N), r(T, H, dtype=F32, scale=dt_scale)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(step[1] / step[0])) * step[0]
    bias = s + torch.log(-torch.expm1(-s))
    a = -(1 + 15 * torch.rand(H, generator=g, device="cuda"))
    d = r(H, dtype=F32)
    s0 = r(len(lens), H, N, P, dtype=F32) if state else None
    return x, dt, a, b, c, d, bias, s0


SSM = [
    ([1], 1, 64, 1, 128, False),
    ([1, 0, 2, 63, 64, 65], 3, 64, 1, 128, True),
    ([0, 0, 200, 0], 4, 64, 2, 64, True),
    ([130, 17], 6, 128, 3, 128, True),
    ([333], 2, 128, 1, 64, False),
    ([1500, 40], 2, 64, 2, 128, True),
    ([129] * 5, 5, 64, 5, 128, False),
]


@pytest.mark.parametrize("lens,H,P,G,N,state", SSM)
def test_ssm(lens, H, P, G, N, state):
    x, dt, a, b, c, d, bias, s0 = ssm_case(lens, H, P, G, N, state)
    cu = cu_of(lens)
    out = torch.full((sum(lens), H, P), float("nan"), dtype=BF16, device="cuda")
    fin = torch.full((len(lens), H, N, P), float("nan"), device="cuda")
    o, f = K.ssm_prefill(x, dt, a, b, c, d, bias, initial_state=s0, cu_seqlens=cu.cuda(),
                         dt_softplus=True, out=out, final_state=fin)
    K.check_device_error()
    ro, rf, so, sf = ops.ssm(x, dt, a, b, c, d, bias, s0, cu=cu, n=len(lens), softplus=True)
    close(o, ro, so, "out")
    close(f, rf, sf, "state")
    if state:   # in place, the same bits
        s1 = s0.clone()
        o2, f2 = K.ssm_prefill(x, dt, a, b, c, d, bias, initial_state=s1, cu_seqlens=cu.cuda(),
                               dt_softplus=True, final_state=s1)
        assert torch.equal(o2, o) and torch.equal(s1, f)


def test_ssm_fixed_batch_plain_dt():
    x, dt, a, b, c, d, _, s0 = ssm_case([77] * 3, 4, 64, 1, 128, False, fused=False)
    dt = dt.abs() * 0.2
    y, f = K.ssm_prefill(x.view(3, 77, 4, 64), dt.view(3, 77, 4), a, b.view(3, 77, 1, 128),
                         c.view(3, 77, 1, 128))
    ro, rf, so, sf = ops.ssm(x, dt, a, b, c, n=3)
    close(y.reshape(231, 4, 64), ro, so, "out")
    close(f, rf, sf, "state")


@pytest.mark.parametrize("kind", ["strong", "weak", "idle"])
def test_ssm_extreme_decays(kind):
    """Decays that forget everything at once, that forget nothing over the whole
    sequence, and tokens with delta = 0, which leave the state as it is."""
    x, dt, a, b, c, d, _, s0 = ssm_case([700], 3, 64, 1, 128, True, fused=False)
    dt = dt.abs()
    if kind == "strong":
        a, dt = a * 300, dt + 0.5
        dt[::7] = 1e-4
    elif kind == "weak":
        a, dt = a * 1e-6, dt * 0.1
    else:
        dt = torch.where(torch.rand(dt.shape, device="cuda") < 0.9, torch.zeros_like(dt), dt)
        dt[130:470] = 0
    y, f = K.ssm_prefill(x, dt, a, b, c, d, initial_state=s0)
    ro, rf, so, sf = ops.ssm(x, dt, a, b, c, d, state=s0)
    close(y, ro, so, "out")
    close(f, rf, sf, "state")


def test_ssm_long_sequence_and_its_parts():
    """One head over 20000 tokens (cut over the SMs) against the reference on
    its first tokens and against itself in two calls."""
    x, dt, a, b, c, d, bias, s0 = ssm_case([20000], 2, 64, 1, 128, True)
    args = (a, b, c, d, bias)
    y, f = K.ssm_prefill(x, dt, *args, initial_state=s0, dt_softplus=True)
    ro, _, so, _ = ops.ssm(x[:2500], dt[:2500], a, b[:2500], c[:2500], d, bias, s0, softplus=True)
    close(y[:2500], ro, so, "out")
    cut = 11117
    y1, f1 = K.ssm_prefill(x[:cut], dt[:cut], a, b[:cut], c[:cut], d, bias, initial_state=s0,
                           dt_softplus=True)
    y2, f2 = K.ssm_prefill(x[cut:], dt[cut:], a, b[cut:], c[cut:], d, bias, initial_state=f1,
                           dt_softplus=True)
    both = torch.cat([y1, y2]).double()
    assert float((both - y.double()).norm() / y.double().norm()) < 2.0 ** -8
    assert float((f2.double() - f.double()).norm() / f.double().norm()) < 2.0 ** -18


@pytest.mark.parametrize("lens,H,P,G", [([384, 363, 783, 1, 6660], 64, 64, 1), ([20000], 16, 128, 2)])
def test_ssm_same_bits_from_cold_caches(lens, H, P, G):
    """Many heads whose sequences are cut, with initial states that come from HBM: some
    warps then wait long and others do not, which must not show."""
    x, dt, a, b, c, d, bias, s0 = ssm_case(lens, H, P, G, 128, True)
    cu = cu_of(lens)
    cold = torch.empty(320 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(6):
        cold.fill_(i)
        o, f = K.ssm_prefill(x, dt, a, b, c, d, bias, initial_state=s0, cu_seqlens=cu.cuda(),
                             dt_softplus=True)
        if first is None:
            first = o, f
        assert torch.equal(o, first[0]) and torch.equal(f, first[1])
    K.check_device_error()
    n, hs = (len(lens), [5, H - 2]) if P == 64 else (1, [1])
    t = sum(lens) if P == 64 else 4000
    g = [h // (H // G) for h in hs]
    ro, rf, so, sf = ops.ssm(x[:t, hs], dt[:t, hs], a[hs], b[:t, g], c[:t, g], d[hs], bias[hs], s0[:, hs],
                             cu=cu if P == 64 else [0, t], n=n, softplus=True)
    close(o[:t, hs], ro, so, "out")
    if P == 64:
        close(f[:, hs], rf, sf, "state")


def test_ssm_bad_cu_seqlens_is_reported_and_skips():
    x, dt, a, b, c, d, bias, _ = ssm_case([30], 2, 64, 1, 128, False)
    out = torch.zeros(30, 2, 64, dtype=BF16, device="cuda")
    fin = torch.zeros(2, 2, 128, 64, device="cuda")
    cu = torch.tensor([0, 31, 30], dtype=torch.int32, device="cuda")
    K.ssm_prefill(x, dt, a, b, c, d, bias, cu_seqlens=cu, out=out, final_state=fin)
    with pytest.raises(K.KdaError, match="CU_SEQLENS"):
        K.check_device_error()
    assert not out.any() and not fin.any()


def test_ssm_no_tokens_hands_the_state_on():
    x, dt, a, b, c, d, bias, s0 = ssm_case([0, 0], 2, 64, 1, 128, True)
    y, f = K.ssm_prefill(x, dt, a, b, c, d, bias, initial_state=s0, cu_seqlens=cu_of([0, 0]).cuda())
    assert torch.equal(f, s0)
    y, f = K.ssm_prefill(x, dt, a, b, c, d, bias, cu_seqlens=cu_of([0, 0]).cuda())
    K.check_device_error()
    assert not f.any()


@pytest.mark.parametrize("S,H,P,G,N,state", [(1, 1, 64, 1, 128, False), (37, 6, 64, 3, 128, True),
                                             (5, 4, 128, 1, 64, True), (9, 2, 128, 2, 128, True),
                                             (3, 5, 64, 1, 64, True)])
def test_ssm_step(S, H, P, G, N, state):
    x, dt, a, b, c, d, bias, s0 = ssm_case([1] * S, H, P, G, N, state)
    o, f = K.ssm_step(x, dt, a, b, c, s0, d, bias, dt_softplus=True)
    ro, rf, so, sf = ops.ssm(x, dt, a, b, c, d, bias, s0, cu=range(S + 1), n=S, softplus=True)
    close(o, ro, so, "out")
    close(f, rf, sf, "state")
    if state:
        s1 = s0.clone()
        o2, _ = K.ssm_step(x, dt, a, b, c, s1, d, bias, dt_softplus=True, in_place=True)
        assert torch.equal(o2, o) and torch.equal(s1, f)


@pytest.mark.parametrize("lens,H,P,G,N", [([300, 7], 3, 64, 1, 128), ([1100], 2, 128, 2, 64)])
def test_ssm_softplus_far_from_zero(lens, H, P, G, N):
    """Tokens masked with the lowest value of the type or -infinity (delta = 0: the state
    stays as it is), and steps far on either side of zero."""
    x, dt, a, b, c, d, bias, s0 = ssm_case(lens, H, P, G, N, True)
    T = sum(lens)
    low = [torch.finfo(F32).min, -math.inf, -2.5e38, -1e30, -130.0, -88.0, -40.0, 20.0, 100.0]
    for i, v in enumerate(low):
        dt[i::11] = v
    dt[T // 2:T // 2 + 40] = torch.finfo(F32).min
    cu = cu_of(lens)
    o, f = K.ssm_prefill(x, dt, a, b, c, d, bias, initial_state=s0, cu_seqlens=cu.cuda(),
                         dt_softplus=True)
    K.check_device_error()
    ro, rf, so, sf = ops.ssm(x, dt, a, b, c, d, bias, s0, cu=cu, n=len(lens), softplus=True)
    close(o, ro, so, "out")
    close(f, rf, sf, "state")
    # one token each, from the same values (and the largest, where x is 0)
    S = 12
    s0 = make(5)(S, H, N, P, dtype=F32)
    dt[11], x[11] = torch.finfo(F32).max, 0
    args = [t[:S] for t in (x, dt, b, c)]
    o, f = K.ssm_step(args[0], args[1], a, args[2], args[3], s0, d, bias, dt_softplus=True)
    ro, rf, so, sf = ops.ssm(args[0], args[1], a, args[2], args[3], d, bias, s0, cu=range(S + 1),
                             n=S, softplus=True)
    close(o, ro, so, "step out")
    close(f, rf, sf, "step state")


def test_ssm_nan_steps_stay_nan():
    x, dt, a, b, c, d, bias, _ = ssm_case([200], 2, 64, 1, 128, False)
    dt[150, 1] = math.nan
    o, f = K.ssm_prefill(x, dt, a, b, c, d, bias, dt_softplus=True)
    assert torch.isfinite(o[:, 0].float()).all() and torch.isfinite(f[0, 0]).all()
    assert torch.isfinite(o[:150].float()).all()
    assert o[150:, 1].float().isnan().all() and f[0, 1].isnan().all()
    o, f = K.ssm_step(x[149:151], dt[149:151], a, b[149:151], c[149:151], None, d, bias, dt_softplus=True)
    assert torch.isfinite(o[0].float()).all() and f[1, 1].isnan().all()


@pytest.mark.parametrize("huge", [1e9, 1e15, 1e30])
def test_ssm_steps_that_forget_everything_keep_later_decays_exact(huge):
    """A huge delta on a token with x = 0 empties the state; the sums of the tokens behind
    it in the same chunk must not drown in it."""
    x, dt, a, b, c, d, _, s0 = ssm_case([700], 3, 64, 1, 128, True, fused=False)
    dt = dt.abs()
    at = [0, 5, 60, 127, 128, 300, 301, 511, 650]
    dt[at], x[at] = huge, 0
    y, f = K.ssm_prefill(x, dt, a, b, c, d, initial_state=s0)
    ro, rf, so, sf = ops.ssm(x, dt, a, b, c, d, state=s0)
    close(y, ro, so, "out")
    close(f, rf, sf, "state")


@pytest.mark.parametrize("lens,H,P,G,N", [([200], 2, 64, 1, 128), ([1500, 40, 0, 300], 3, 64, 1, 64),
                                          ([900, 128], 2, 128, 2, 128), ([20000], 2, 64, 1, 128)])
def test_ssm_non_finite_x_stays_in_its_channel_and_behind_its_token(lens, H, P, G, N):
    """An infinity or NaN in x at token s: y is not finite from s to the sequence's end, nor
    is that column of the state, and every other value has the bits it has without it."""
    x, dt, a, b, c, d, bias, s0 = ssm_case(lens, H, P, G, N, True)
    cu, T = cu_of(lens), sum(lens)
    kw = dict(initial_state=s0, cu_seqlens=cu.cuda(), dt_softplus=True)
    o, f = K.ssm_prefill(x, dt, a, b, c, d, bias, **kw)
    x2, want, state = x.clone(), torch.ones(T, H, P, dtype=torch.bool), torch.ones(f.shape, dtype=torch.bool)
    spots = [(0, 0, 0, math.inf), (31, 0, 1, math.nan), (32, 1, P - 1, -math.inf), (100, 1, 17, math.nan),
             (127, 1, 40, math.inf), (150, 0, 1, math.nan), (170, 1, 40, math.nan), (T - 1, 0, 33, math.nan),
             (T - 20, 0, 34, math.inf), (T - 129, 1, 35, math.nan)]
    for t, h, p, v in spots:
        x2[t, h, p] = v
        seq = int(torch.searchsorted(cu.long()[1:], t, right=True))
        want[t:int(cu[seq + 1]), h, p] = False
        state[seq, h, :, p] = False
    o2, f2 = K.ssm_prefill(x2, dt, a, b, c, d, bias, **kw)
    K.check_device_error()
    assert torch.equal(torch.isfinite(o2.float()).cpu(), want)
    assert torch.equal(torch.isfinite(f2).cpu(), state)
    assert torch.equal(o2.cpu()[want], o.cpu()[want]) and torch.equal(f2.cpu()[state], f.cpu()[state])


@pytest.mark.parametrize("lens,chunk", [([300], 0), ([5000, 40], 2), ([5000, 40], 3)])
def test_ssm_wait_runs_out_then_clean_call(lens, chunk):
    """Tiles that never come (a test hook): the waits run out, the call says so and ends
    by itself, and the next one is right. Whole sequences, and ones that are cut (then
    the launch for the states gives up as well)."""
    x, dt, a, b, c, d, bias, s0 = ssm_case(lens, 20, 64, 1, 128, True)
    cu = cu_of(lens).cuda()
    kw = dict(initial_state=s0, cu_seqlens=cu, dt_softplus=True)
    ref = K.ssm_prefill(x, dt, a, b, c, d, bias, **kw)
    K.check_device_error()
    assert K.kda_test_stall_scan(-2) != 0
    assert K.kda_test_stall_scan(chunk) == 0
    try:
        K.ssm_prefill(x, dt, a, b, c, d, bias, **kw)
        with pytest.raises(K.KdaError, match="TIMEOUT"):
            K.check_device_error()
    finally:
        assert K.kda_test_stall_scan(-1) == 0
    K.check_device_error()
    got = K.ssm_prefill(x, dt, a, b, c, d, bias, **kw)
    K.check_device_error()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


# --------------------------------------------------------- paged attention

def cache_case(lens, Hq, Hkv, D, page, seed=0, poison=True, spare=3, one=True):
    r = make(seed + Hq + D + page)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    if one:
        both = r(pages, 2, page, Hkv, D)
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = r(pages, page, Hkv, D), r(pages, page, Hkv, D)
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    used = torch.zeros(pages, page, dtype=torch.bool)
    for i, n in enumerate(lens):
        table[i, :need[i]] = order[at:at + need[i]]
        for t in range(0, n, page):
            used[table[i, t // page].item(), :min(page, n - t)] = True
        at += need[i]
    if poison:   # rows no sequence holds
        k[~used.cuda()] = float("nan")
        v[~used.cuda()] = float("inf")
    q = r(len(lens), Hq, D)
    return q, k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def attention_close(out, lse, q, k, v, table, lens, scale=None):
    ro, rl, size, reach = ops.paged_attention(q, k, v, table, lens, scale)
    # weights p carry the error of their score, at most 2^-18 of sum |q||k|
    ro_tol = size * (1 + 2.0 ** -6 * reach[..., None])
    close(out, ro, ro_tol, "out")
    lse = lse.cpu().double()
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    err = (lse - rl)[~empty].abs() - 2.0 ** -18 * (1 + reach + rl.abs())[~empty]
    assert err.numel() == 0 or float(err.max()) <= 0, "lse"


PAGED = [
    # lens, Hq, Hkv, D, page, one cache
    ([1], 1, 1, 128, 16, True),
    ([0, 1, 15, 16, 17, 1000], 8, 2, 128, 16, True),
    ([63, 64, 65, 128, 129], 4, 4, 64, 64, False),
    ([700], 32, 8, 128, 1, True),
    ([100, 3, 0, 0, 517], 12, 4, 128, 17, True),
    ([2049, 5], 16, 1, 128, 100, False),
    ([300, 777], 20, 1, 64, 32, True),
    ([90], 64, 1, 128, 128, True),
    ([1200] * 3, 80, 2, 128, 64, True),
    ([17] * 40, 6, 2, 64, 8, True),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,one", PAGED)
def test_paged(lens, Hq, Hkv, D, page, one):
    q, k, v, table, n = cache_case(lens, Hq, Hkv, D, page, one=one)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((len(lens), Hq), float("nan"), device="cuda")
    o, l = K.paged_decode(q, k, v, table, n, out=out, lse=lse)
    K.check_device_error()
    attention_close(o, l, q, k, v, table, lens)
    o2, l2 = K.paged_decode(q, k, v, table, n)
    assert torch.equal(o, o2) and torch.equal(l, l2), "not the same bits again"
    torch.cuda.synchronize()


def test_paged_long_and_ragged():
    lens = [40000, 1, 0, 9000, 123]
    q, k, v, table, n = cache_case(lens, 16, 4, 128, 32)
    o, l = K.paged_decode(q, k, v, table, n)
    K.check_device_error()
    attention_close(o, l, q, k, v, table, lens)


@pytest.mark.parametrize("scale", [1.0, 4.0, -0.5, 0.0])
def test_paged_scores_far_apart(scale):
    """Scores of hundreds: the running maximum moves and most weights vanish."""
    lens = [5, 400, 3000]
    q, k, v, table, n = cache_case(lens, 8, 2, 128, 16, seed=2)
    o, l = K.paged_decode(q, k, v, table, n, scale=scale)
    attention_close(o, l, q, k, v, table, lens, scale)


def test_paged_bad_tables_are_reported():
    lens = [50, 20, 40]
    q, k, v, table, n = cache_case(lens, 8, 2, 128, 16, poison=False)
    o, l = K.paged_decode(q, k, v, table, n)
    for bad_table, bad_len in ((k.shape[0], None), (-5, None), (None, -1), (None, 10 ** 6)):
        t2, n2 = table.clone(), n.clone()
        if bad_table is not None:
            t2[1, 1] = bad_table
        else:
            n2[1] = bad_len
        o2, l2 = K.paged_decode(q, k, v, t2, n2)
        with pytest.raises(K.KdaError, match="PAGE_TABLE"):
            K.check_device_error()
        for i in (0, 2):
            assert torch.equal(o2[i], o[i]) and torch.equal(l2[i], l[i])
    K.paged_decode(q, k, v, table, n)
    K.check_device_error()


def test_paged_offsets_past_32_bits():
    """Pages that lie more than 2^32 bytes into the cache."""
    page, Hkv, D, pages = 64, 8, 128, 40000          # 2 * 5.2 GB
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 11 GB")
    both = torch.empty(pages, 2, page, Hkv, D, dtype=BF16, device="cuda")
    table = torch.tensor([[39999, 0, 39998, 20000]], dtype=torch.int32)
    r = make(5)
    for i in table[0].tolist():
        both[i] = r(2, page, Hkv, D)
    k, v = both[:, 0], both[:, 1]
    q, n = r(1, 16, D), torch.tensor([230], dtype=torch.int32, device="cuda")
    o, l = K.paged_decode(q, k, v, table.cuda(), n)
    attention_close(o, l, q, k, v, table, [230])


def test_sizes_of_zero_are_refused():
    x, dt, a, b, c, d, bias, _ = ssm_case([4], 2, 64, 1, 128, False, fused=False)
    with pytest.raises(ValueError):
        K.ssm_prefill(x, dt, a, b[:, :0], c[:, :0])
    with pytest.raises(ValueError):
        K.ssm_step(x, dt, a, b[:, :0], c[:, :0])
    q, k, v, table, n = cache_case([5], 4, 2, 64, 16)
    with pytest.raises(K.KdaError, match="UNSUPPORTED_DIM"):
        K.paged_decode(q[..., :0].contiguous(), k[..., :0].contiguous(), v[..., :0].contiguous(), table, n)


# ------------------------------------------------- streams, graphs, threads

def test_side_stream_and_graph():
    """The operators on a stream of their own, and captured into a graph that is
    replayed on new inputs."""
    x, dt, a, b, c, d, bias, s0 = ssm_case([900, 60], 4, 64, 2, 128, True)
    cu = cu_of([900, 60]).cuda()
    w = make(1)(x.shape[1] * 64, 4, dtype=F32)
    q, k, v, table, n = cache_case([3000, 7], 8, 2, 128, 16)
    flat = x.reshape(960, 256).contiguous()
    dy = torch.randn(960, 256, device="cuda")

    def go():
        y, h = K.short_conv(flat, w, cu_seqlens=cu)
        s, f = K.ssm_prefill(y.view(960, 4, 64), dt, a, b, c, d, bias, initial_state=s0,
                             cu_seqlens=cu, dt_softplus=True)
        o, l = K.paged_decode(q, k, v, table, n)
        g = K.short_conv_backward(flat, w, dy, cu_seqlens=cu, d_initial_state=False)
        return [y, h, s, f, o, l, g[0], g[1]]

    ref = go()
    K.check_device_error()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = go()                       # sizes the stream's workspace too
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = go()
    for r, t in zip(ref, got):
        assert torch.equal(r, t)
    flat.mul_(0.5)
    q.mul_(0.5)
    ref = go()
    graph.replay()
    torch.cuda.synchronize()
    for r, t in zip(ref, held):
        assert torch.equal(r, t)


def test_first_use_inside_a_capture():
    """An operator that needs no workspace may be captured as its first call of all: its
    kernels are set up on first use, which no KDA call does for it."""
    code = """
import torch
import prefill_kda_chunk_gb300 as K
g = torch.Generator(device="cuda").manual_seed(0)
def r(*s, dtype=torch.bfloat16):
    return torch.randn(*s, generator=g, device="cuda").to(dtype)
q, k, v = r(64, 2, 128), r(64, 2, 128), r(64, 2, 128)
K.chunk_prefill(q, k, v, -r(64, 2, 128, dtype=torch.float32).abs(), r(64, 2, dtype=torch.float32).sigmoid())
x, w, h = r(40, 256), r(256, 4, dtype=torch.float32), r(40, 3, 256)
a, dt = -r(4, dtype=torch.float32).abs(), r(40, 4, dtype=torch.float32)
b, c, s = r(40, 1, 128), r(40, 1, 128), r(40, 4, 128, 64, dtype=torch.float32)
def go():
    y, f = K.short_conv(x, w)
    z, e = K.short_conv_step(x, w, h)
    o, t = K.ssm_step(z.view(40, 4, 64), dt, a, b, c, s, dt_softplus=True)
    return [y, f, z, e, o, t]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = go()
graph.replay()
torch.cuda.synchronize()
K.check_device_error()
assert all(torch.equal(p, q) for p, q in zip(held, go()))
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


def test_two_threads_on_streams_of_their_own():
    """Calls from two threads, each on its own stream, at work at the same time: every
    call gives the bits that it gives alone."""
    import threading

    x, dt, a, b, c, d, bias, s0 = ssm_case([2500, 60], 4, 64, 2, 128, True)
    cu = cu_of([2500, 60]).cuda()
    w = make(1)(256, 4, dtype=F32)
    q, k, v, table, n = cache_case([30000, 7, 900], 8, 2, 128, 16)
    flat = [x.reshape(2560, 256).contiguous(), x.reshape(2560, 256) * 0.5]
    dy = torch.randn(2560, 256, device="cuda")

    def go(i):
        y, h = K.short_conv(flat[i], w, cu_seqlens=cu)
        s, f = K.ssm_prefill(y.view(2560, 4, 64), dt, a, b, c, d, bias, initial_state=s0,
                             cu_seqlens=cu, dt_softplus=True)
        o, l = K.paged_decode(q[i:i + 2].contiguous(), k, v, table[i:i + 2].contiguous(),
                              n[i:i + 2].contiguous())
        g = K.short_conv_backward(flat[i], w, dy, cu_seqlens=cu, d_initial_state=False)
        return [y, h, s, f, o, l, g[0], g[1]]

    ref = [go(i) for i in (0, 1)]
    K.check_device_error()
    failed, start = [], threading.Barrier(2)

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()) as _:
                start.wait()
                for _ in range(20):
                    got = go(i)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(r, t) for r, t in zip(ref[i], got)):
                    failed.append(i)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    K.check_device_error()
    assert not failed
