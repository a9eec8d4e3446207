// C ABI of the operators around the KDA layers (declared in include/kda.h):
// short causal convolution, selective state space scan and paged decode
// attention. Argument validation here; the kernels in kda_conv.cu, kda_ssm.cu
// and kda_paged.cu.

#include <cuda_runtime.h>

#include <atomic>
#include <climits>

#include "kda.h"
#include "kda_device.cuh"
#include "kda_internal.h"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;

std::atomic<int> g_stall_scan{INT_MAX};   // kda_test_stall_scan

// A block of rows: `row` bytes each, `step` bytes apart.
struct Rows {
    const void *p;
    int64_t rows, row, step;
};

bool misaligned(const void *p, uintptr_t a) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

Rows flat(const void *p, int64_t bytes) { return {p, 1, bytes, bytes}; }

// Whether two blocks share a byte. Two slices of one fused buffer (equal
// steps) overlap as ranges without sharing any: their rows are compared modulo
// the step.
bool share(const Rows &a, const Rows &b) {
    if (a.p == nullptr || b.p == nullptr || a.rows <= 0 || b.rows <= 0 || a.row <= 0 || b.row <= 0)
        return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t ea = pa + (a.rows - 1) * a.step + a.row, eb = pb + (b.rows - 1) * b.step + b.row;
    if (pa >= eb || pb >= ea) return false;
    if (a.step == b.step && a.rows > 1 && b.rows > 1) {
        const int64_t step = a.step;
        const int64_t off = pb >= pa ? static_cast<int64_t>((pb - pa) % step)
                                     : (step - static_cast<int64_t>((pa - pb) % step)) % step;
        return off < a.row || off + b.row > step;   // b's rows start `off` bytes after a's
    }
    return true;
}

bool any_shared(const Rows *outs, int n_out, const Rows *ins, int n_in) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (share(outs[o], ins[i])) return true;
        for (int i = o + 1; i < n_out; ++i)
            if (share(outs[o], outs[i])) return true;
    }
    return false;
}

// Token count of a batch, as for the prefill: N = B sequences of T tokens, or
// one packed row of T tokens cut by cu_seqlens.
kda_status batch_tokens(int64_t B, int64_t T, int64_t N, bool packed, int64_t *tokens) {
    if (B < 1 || T < 0 || N < 1 || N > (int64_t(1) << 30)) return KDA_ERR_BAD_SHAPE;
    if (packed ? B != 1 : N != B) return KDA_ERR_BAD_SHAPE;
    if (T > kMaxElems || B > kMaxElems / (T > 0 ? T : 1)) return KDA_ERR_BAD_SHAPE;
    *tokens = B * T;
    // cu_seqlens holds 32-bit positions, and tiles are counted in 32 bits
    if (*tokens >= (int64_t(1) << 31)) return KDA_ERR_BAD_SHAPE;
    return KDA_OK;
}

bool rows_fit(int64_t rows, int64_t stride, int64_t width) {
    return stride >= width && stride <= kMaxElems && rows <= kMaxElems / stride;
}

}  // namespace

extern "C" {

kda_status kda_short_conv(const void *x, const float *weight, const float *bias,
                          const void *initial_state, const int32_t *cu_seqlens, int64_t B,
                          int64_t T, int64_t D, int64_t W, int64_t N, int64_t x_stride, int flags,
                          void *out, int64_t out_stride, void *final_state, void *stream) {
    if ((flags & ~KDA_CONV_SILU) != 0) return KDA_ERR_BAD_FLAGS;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED_DIM;
    int64_t tokens = 0;
    kda_status rc = batch_tokens(B, T, N, cu_seqlens != nullptr, &tokens);
    if (rc != KDA_OK) return rc;
    if (D < 1 || D > (int64_t(1) << 24) || !rows_fit(tokens, x_stride, D) ||
        !rows_fit(tokens, out_stride, D) || N > kMaxElems / (W * D))
        return KDA_ERR_BAD_SHAPE;
    if ((tokens > 0 && (!x || !out)) || !weight) return KDA_ERR_NULL_ARG;
    if (misaligned(x, 2) || misaligned(out, 2) || misaligned(initial_state, 2) ||
        misaligned(final_state, 2) || misaligned(weight, 4) || misaligned(bias, 4) ||
        misaligned(cu_seqlens, 4))
        return KDA_ERR_MISALIGNED;
    const int64_t nh = N * (W - 1) * D * 2;
    const Rows ins[] = {{x, tokens, 2 * D, 2 * x_stride}, flat(weight, 4 * D * W),
                        flat(bias, 4 * D), flat(initial_state, nh),
                        flat(cu_seqlens, 4 * (N + 1))};
    const Rows outs[] = {{out, tokens, 2 * D, 2 * out_stride}, flat(final_state, nh)};
    if (any_shared(outs, 2, ins, 5)) return KDA_ERR_ALIAS;

    const void *ptrs[] = {x, weight, bias, initial_state, cu_seqlens, out, final_state};
    kda::CallContext ctx;
    rc = static_cast<kda_status>(kda::begin_call(kda::kConv, ptrs, 7, stream, 0, 0, &ctx));
    if (rc != KDA_OK) return rc;
    kda::ConvParams p{};
    p.x = x; p.weight = weight; p.bias = bias; p.hist_in = initial_state; p.cu = cu_seqlens;
    p.tokens = tokens; p.seq_len = T; p.dim = D;
    p.x_stride = x_stride; p.out_stride = out_stride;
    p.n_seqs = static_cast<int32_t>(N); p.width = static_cast<int32_t>(W);
    p.silu = (flags & KDA_CONV_SILU) != 0;
    p.out = out; p.hist_out = final_state; p.err = ctx.err;
    return kda::launch_conv(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK
                                                                                 : KDA_ERR_CUDA;
}

kda_status kda_short_conv_step(const void *x, const float *weight, const float *bias,
                               const void *state_in, int64_t N, int64_t D, int64_t W,
                               int64_t x_stride, int flags, void *out, int64_t out_stride,
                               void *state_out, void *stream) {
    if ((flags & ~KDA_CONV_SILU) != 0) return KDA_ERR_BAD_FLAGS;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED_DIM;
    if (N < 0 || N >= (int64_t(1) << 31) || D < 1 || D > (int64_t(1) << 24) ||
        !rows_fit(N, x_stride, D) || !rows_fit(N, out_stride, D) || N > kMaxElems / (W * D))
        return KDA_ERR_BAD_SHAPE;
    if (N > 0 && (!x || !out || !weight || !state_out)) return KDA_ERR_NULL_ARG;
    if (misaligned(x, 2) || misaligned(out, 2) || misaligned(state_in, 2) ||
        misaligned(state_out, 2) || misaligned(weight, 4) || misaligned(bias, 4))
        return KDA_ERR_MISALIGNED;
    const int64_t nh = N * (W - 1) * D * 2;
    const Rows ins[] = {{x, N, 2 * D, 2 * x_stride}, flat(weight, 4 * D * W), flat(bias, 4 * D),
                        flat(state_in == state_out ? nullptr : state_in, nh)};
    const Rows outs[] = {{out, N, 2 * D, 2 * out_stride}, flat(state_out, nh)};
    if (any_shared(outs, 2, ins, 4)) return KDA_ERR_ALIAS;
    if (N == 0) return KDA_OK;   // an empty batch enqueues nothing

    const void *ptrs[] = {x, weight, bias, state_in, out, state_out};
    kda::CallContext ctx;
    const kda_status rc = static_cast<kda_status>(kda::begin_call(kda::kConv, ptrs, 6, stream, 0, 0, &ctx));
    if (rc != KDA_OK) return rc;
    kda::ConvParams p{};
    p.x = x; p.weight = weight; p.bias = bias; p.hist_in = state_in;
    p.tokens = N; p.seq_len = 1; p.dim = D;
    p.x_stride = x_stride; p.out_stride = out_stride;
    p.n_seqs = static_cast<int32_t>(N); p.width = static_cast<int32_t>(W);
    p.silu = (flags & KDA_CONV_SILU) != 0;
    p.out = out; p.hist_out = state_out; p.err = ctx.err;
    return kda::launch_conv_step(p, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_short_conv_backward(const void *x, const float *weight, const float *bias,
                                   const void *initial_state, const int32_t *cu_seqlens,
                                   int64_t B, int64_t T, int64_t D, int64_t W, int64_t N,
                                   int64_t x_stride, int flags, const void *d_out,
                                   int64_t dout_stride, const float *d_final_state, void *dx,
                                   int64_t dx_stride, float *dweight, float *dbias,
                                   float *d_initial_state, void *stream) {
    if ((flags & ~(KDA_CONV_SILU | KDA_CONV_DOUT_FP32)) != 0) return KDA_ERR_BAD_FLAGS;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED_DIM;
    int64_t tokens = 0;
    kda_status rc = batch_tokens(B, T, N, cu_seqlens != nullptr, &tokens);
    if (rc != KDA_OK) return rc;
    if (D < 1 || D > (int64_t(1) << 24) || !rows_fit(tokens, x_stride, D) ||
        !rows_fit(tokens, dout_stride, D) || !rows_fit(tokens, dx_stride, D) ||
        N > kMaxElems / (W * D))
        return KDA_ERR_BAD_SHAPE;
    if ((tokens > 0 && (!x || !d_out || !dx)) || !weight || !dweight) return KDA_ERR_NULL_ARG;
    const int dsize = (flags & KDA_CONV_DOUT_FP32) != 0 ? 4 : 2;
    if (misaligned(x, 2) || misaligned(dx, 2) || misaligned(initial_state, 2) ||
        misaligned(d_out, dsize) || misaligned(d_final_state, 4) ||
        misaligned(d_initial_state, 4) || misaligned(weight, 4) || misaligned(bias, 4) ||
        misaligned(dweight, 4) || misaligned(dbias, 4) || misaligned(cu_seqlens, 4))
        return KDA_ERR_MISALIGNED;
    const int64_t nh = N * (W - 1) * D;
    const Rows ins[] = {{x, tokens, 2 * D, 2 * x_stride}, flat(weight, 4 * D * W),
                        flat(bias, 4 * D), flat(initial_state, 2 * nh),
                        flat(cu_seqlens, 4 * (N + 1)),
                        {d_out, tokens, dsize * D, dsize * dout_stride},
                        flat(d_final_state, 4 * nh)};
    const Rows outs[] = {{dx, tokens, 2 * D, 2 * dx_stride}, flat(dweight, 4 * D * W),
                         flat(dbias, 4 * D), flat(d_initial_state, 4 * nh)};
    if (any_shared(outs, 4, ins, 7)) return KDA_ERR_ALIAS;

    const void *ptrs[] = {x, weight, bias, initial_state, cu_seqlens, d_out, d_final_state, dx,
                          dweight, dbias, d_initial_state};
    kda::ConvParams p{};
    p.x = x; p.weight = weight; p.bias = bias; p.hist_in = initial_state; p.cu = cu_seqlens;
    p.tokens = tokens; p.seq_len = T; p.dim = D;
    p.x_stride = x_stride; p.out_stride = dx_stride; p.dout_stride = dout_stride;
    p.n_seqs = static_cast<int32_t>(N); p.width = static_cast<int32_t>(W);
    p.silu = (flags & KDA_CONV_SILU) != 0;
    p.dout32 = dsize == 4;
    p.out = dx; p.dout = d_out; p.dhist_out = d_final_state; p.dhist_in = d_initial_state;
    p.dweight = dweight; p.dbias = dbias;
    const kda::ConvBackwardPlan plan = kda::plan_conv_backward(p);
    kda::CallContext ctx;
    rc = static_cast<kda_status>(kda::begin_call(kda::kConv, ptrs, 11, stream, plan.scratch_bytes, 0, &ctx));
    if (rc != KDA_OK) return rc;
    p.partial = reinterpret_cast<float *>(ctx.ws);
    p.err = ctx.err;
    return kda::launch_conv_backward(p, plan, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_test_conv_backward_plan(const void *x, const void *d_out, const void *dx,
                                       int64_t tokens, int64_t D, int64_t W, int64_t x_stride,
                                       int64_t dout_stride, int64_t dx_stride, int flags,
                                       int64_t plan[5]) {
    if ((flags & ~(KDA_CONV_SILU | KDA_CONV_DOUT_FP32)) != 0) return KDA_ERR_BAD_FLAGS;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED_DIM;
    if (tokens < 0 || D < 1) return KDA_ERR_BAD_SHAPE;
    if (!plan) return KDA_ERR_NULL_ARG;
    kda::ConvParams p{};
    p.x = x; p.dout = d_out; p.out = const_cast<void *>(dx);
    p.tokens = tokens; p.dim = D; p.width = static_cast<int32_t>(W);
    p.x_stride = x_stride; p.out_stride = dx_stride; p.dout_stride = dout_stride;
    p.dout32 = (flags & KDA_CONV_DOUT_FP32) != 0;
    const kda::ConvBackwardPlan pl = kda::plan_conv_backward(p);
    plan[0] = pl.scratch_bytes; plan[1] = pl.channels; plan[2] = pl.cols;
    plan[3] = pl.run; plan[4] = pl.tiles;
    return KDA_OK;
}

// The checks that the two scan entry points share; `rows` tokens, `seqs` states.
static kda_status ssm_checks(const void *x, const float *dt, const float *a, const void *b,
                             const void *c, const float *d, const float *dt_bias,
                             const float *s_in, const int32_t *cu, int64_t rows, int64_t seqs,
                             int64_t H, int64_t P, int64_t G, int64_t n, int64_t x_stride,
                             int64_t dt_stride, int64_t b_stride, int64_t c_stride, int flags,
                             const void *out, const float *s_out) {
    if ((flags & ~KDA_SSM_DT_SOFTPLUS) != 0) return KDA_ERR_BAD_FLAGS;
    if ((P != 64 && P != 128) || (n != 64 && n != 128)) return KDA_ERR_UNSUPPORTED_DIM;
    if (H < 1 || H > 65535 || G < 1 || H % G != 0 || seqs > ((int64_t(1) << 31) - 1) / (2 * H) ||
        !rows_fit(rows, x_stride, H * P) || !rows_fit(rows, dt_stride, H) ||
        !rows_fit(rows, b_stride, G * n) || !rows_fit(rows, c_stride, G * n))
        return KDA_ERR_BAD_SHAPE;
    if (rows > 0 && (!x || !dt || !b || !c || !out)) return KDA_ERR_NULL_ARG;
    if (!a) return KDA_ERR_NULL_ARG;
    if (misaligned(x, 16) || misaligned(b, 16) || misaligned(c, 16) || misaligned(out, 16) ||
        misaligned(s_in, 16) || misaligned(s_out, 16) || misaligned(dt, 4) || misaligned(a, 4) ||
        misaligned(d, 4) || misaligned(dt_bias, 4) || misaligned(cu, 4) || x_stride % 8 != 0 ||
        b_stride % 8 != 0 || c_stride % 8 != 0)
        return KDA_ERR_MISALIGNED;
    const int64_t ns = seqs * H * n * P * 4;
    const Rows ins[] = {{x, rows, 2 * H * P, 2 * x_stride}, {dt, rows, 4 * H, 4 * dt_stride},
                        flat(a, 4 * H), {b, rows, 2 * G * n, 2 * b_stride},
                        {c, rows, 2 * G * n, 2 * c_stride}, flat(d, 4 * H), flat(dt_bias, 4 * H),
                        flat(s_in == s_out ? nullptr : s_in, ns), flat(cu, 4 * (seqs + 1))};
    const Rows outs[] = {flat(out, rows * H * P * 2), flat(s_out, ns)};
    return any_shared(outs, 2, ins, 9) ? KDA_ERR_ALIAS : KDA_OK;
}

static kda::SsmParams ssm_params(const void *x, const float *dt, const float *a, const void *b,
                                 const void *c, const float *d, const float *dt_bias,
                                 const float *s_in, const int32_t *cu, int64_t rows,
                                 int64_t seq_len, int64_t seqs, int64_t H, int64_t P, int64_t G,
                                 int64_t n, int64_t x_stride, int64_t dt_stride, int64_t b_stride,
                                 int64_t c_stride, int flags, void *out, float *s_out) {
    kda::SsmParams p{};
    p.x = x; p.dt = dt; p.a = a; p.b = b; p.c = c; p.d = d; p.dt_bias = dt_bias; p.s0 = s_in;
    p.cu = cu; p.tokens = rows; p.seq_len = seq_len;
    p.x_stride = x_stride; p.dt_stride = dt_stride; p.b_stride = b_stride; p.c_stride = c_stride;
    p.n_seqs = static_cast<int32_t>(seqs); p.heads = static_cast<int32_t>(H);
    p.groups = static_cast<int32_t>(G); p.p = static_cast<int32_t>(P);
    p.n = static_cast<int32_t>(n);
    p.softplus = (flags & KDA_SSM_DT_SOFTPLUS) != 0;
    p.out = out; p.s_final = s_out;
    p.stall = g_stall_scan.load();
    return p;
}

kda_status kda_ssm_prefill(const void *x, const float *dt, const float *a, const void *b,
                           const void *c, const float *d, const float *dt_bias,
                           const float *initial_state, const int32_t *cu_seqlens, int64_t B,
                           int64_t T, int64_t H, int64_t P, int64_t G, int64_t n, int64_t N,
                           int64_t x_stride, int64_t dt_stride, int64_t b_stride,
                           int64_t c_stride, int flags, void *out, float *final_state,
                           void *stream) {
    int64_t tokens = 0;
    kda_status rc = batch_tokens(B, T, N, cu_seqlens != nullptr, &tokens);
    if (rc != KDA_OK) return rc;
    rc = ssm_checks(x, dt, a, b, c, d, dt_bias, initial_state, cu_seqlens, tokens, N, H, P, G, n,
                    x_stride, dt_stride, b_stride, c_stride, flags, out, final_state);
    if (rc != KDA_OK) return rc;
    kda::SsmParams p = ssm_params(x, dt, a, b, c, d, dt_bias, initial_state, cu_seqlens, tokens, T,
                                  N, H, P, G, n, x_stride, dt_stride, b_stride, c_stride, flags,
                                  out, final_state);
    const void *ptrs[] = {x, dt, a, b, c, d, dt_bias, initial_state, cu_seqlens, out, final_state};
    kda::CallContext ctx;
    rc = static_cast<kda_status>(kda::begin_call(kda::kSsm, ptrs, 11, stream, kda::ssm_workspace(p), 0, &ctx));
    if (rc != KDA_OK) return rc;
    p.err = ctx.err;
    return kda::launch_ssm(p, ctx, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK
                                                                                     : KDA_ERR_CUDA;
}

kda_status kda_test_stall_scan(int chunk) {
    if (chunk < -1) return KDA_ERR_BAD_SHAPE;
    g_stall_scan.store(chunk < 0 ? INT_MAX : chunk);
    return KDA_OK;
}

kda_status kda_ssm_step(const void *x, const float *dt, const float *a, const void *b,
                        const void *c, const float *d, const float *dt_bias,
                        const float *state_in, int64_t N, int64_t H, int64_t P, int64_t G,
                        int64_t n, int64_t x_stride, int64_t dt_stride, int64_t b_stride,
                        int64_t c_stride, int flags, void *out, float *state_out, void *stream) {
    if (N < 0) return KDA_ERR_BAD_SHAPE;
    kda_status rc = ssm_checks(x, dt, a, b, c, d, dt_bias, state_in, nullptr, N, N, H, P, G, n,
                               x_stride, dt_stride, b_stride, c_stride, flags, out, state_out);
    if (rc != KDA_OK) return rc;
    if (N > 0 && !state_out) return KDA_ERR_NULL_ARG;
    if (N == 0) return KDA_OK;   // an empty batch enqueues nothing
    kda::SsmParams p = ssm_params(x, dt, a, b, c, d, dt_bias, state_in, nullptr, N, 1, N, H, P, G,
                                  n, x_stride, dt_stride, b_stride, c_stride, flags, out,
                                  state_out);
    const void *ptrs[] = {x, dt, a, b, c, d, dt_bias, state_in, out, state_out};
    kda::CallContext ctx;
    rc = static_cast<kda_status>(kda::begin_call(kda::kSsm, ptrs, 10, stream, 0, 0, &ctx));
    if (rc != KDA_OK) return rc;
    p.err = ctx.err;
    return kda::launch_ssm_step(p, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_paged_decode(const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *page_table, const int32_t *seq_lens, int64_t B,
                            int64_t Hq, int64_t Hkv, int64_t D, int64_t pages, int64_t page_size,
                            int64_t max_pages, int64_t k_page_stride, int64_t v_page_stride,
                            float scale, void *out, float *lse, void *stream) {
    if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED_DIM;
    const int64_t lim = int64_t(1) << 31;
    if (B < 0 || B > 65536 || Hkv < 1 || Hkv > 65535 || Hq < Hkv || Hq > 65535 || Hq % Hkv != 0 ||
        pages < 0 || pages >= lim || page_size < 1 || page_size >= lim || max_pages < 0 ||
        max_pages >= lim || max_pages * page_size >= lim ||
        page_size > kMaxElems / (Hkv * D) ||
        !rows_fit(pages, k_page_stride, page_size * Hkv * D) ||
        !rows_fit(pages, v_page_stride, page_size * Hkv * D))
        return KDA_ERR_BAD_SHAPE;
    if (B > 0 && (!q || !out || !seq_lens)) return KDA_ERR_NULL_ARG;
    if (B > 0 && max_pages > 0 && (!page_table || (pages > 0 && (!k_cache || !v_cache))))
        return KDA_ERR_NULL_ARG;
    if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
        misaligned(out, 16) || misaligned(page_table, 4) || misaligned(seq_lens, 4) ||
        misaligned(lse, 4) || k_page_stride % 8 != 0 || v_page_stride % 8 != 0)
        return KDA_ERR_MISALIGNED;
    const int64_t nq = B * Hq * D * 2, page = page_size * Hkv * D * 2;
    const Rows ins[] = {flat(q, nq), {k_cache, pages, page, 2 * k_page_stride},
                        {v_cache, pages, page, 2 * v_page_stride},
                        flat(page_table, B * max_pages * 4), flat(seq_lens, B * 4)};
    const Rows outs[] = {flat(out, nq), flat(lse, B * Hq * 4)};
    if (any_shared(outs, 2, ins, 5)) return KDA_ERR_ALIAS;
    if (B == 0) return KDA_OK;   // an empty batch enqueues nothing

    kda::PagedParams p{};
    p.q = q; p.k = k_cache; p.v = v_cache; p.table = page_table; p.lens = seq_lens;
    p.k_stride = k_page_stride; p.v_stride = v_page_stride;
    p.pages = pages; p.max_pages = max_pages;
    p.batch = static_cast<int32_t>(B); p.hq = static_cast<int32_t>(Hq);
    p.hkv = static_cast<int32_t>(Hkv); p.dim = static_cast<int32_t>(D);
    p.page_size = static_cast<int32_t>(page_size);
    p.scale = scale; p.out = out; p.lse = lse;
    const void *ptrs[] = {q, k_cache, v_cache, page_table, seq_lens, out, lse};
    kda::CallContext ctx;
    const kda_status rc = static_cast<kda_status>(
        kda::begin_call(kda::kPaged, ptrs, 7, stream, kda::paged_workspace(p), kda::paged_sync(p), &ctx));
    if (rc != KDA_OK) return rc;
    p.err = ctx.err;
    return kda::launch_paged(p, ctx, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
