// Selective state space scan with one decay per head (kda_ssm_prefill) and
// its single-token step (kda_ssm_step).
//
//   S_t = exp(a delta_t) S_{t-1} + delta_t b_t x_t^T,   y_t = S_t^T c_t + d x_t
//
// S is n x P per (sequence, head), fp32; b and c are shared by the heads of a
// group.

#include "kda_device.cuh"
#include "kda_internal.h"
#include "kda_seqs.cuh"

namespace kda {

namespace {

__device__ __forceinline__ float bf16_at(const void *p, int64_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ float delta_of(const SsmParams &p, int64_t t, int h) {
    float v = p.dt[t * p.dt_stride + h];
    if (p.dt_bias != nullptr) v += __ldg(p.dt_bias + h);
    // log(1 + e^v) without overflow, and exact for large negative v
    return p.softplus ? fmaxf(v, 0.f) + log1pf(__expf(-fabsf(v))) : v;
}

// One block per (sequence, head): thread (q, j) keeps S[j * kN / kParts ..][q].
template <int kN, int kP>
__global__ void __launch_bounds__(256) ssm_serial_kernel(SsmParams p) {
    constexpr int kParts = 256 / kP, kRows = kN / kParts;
    __shared__ float s_b[kN], s_c[kN], s_y[kParts][kP];
    const Seqs seqs{p.cu, p.seq_len, p.n_seqs};
    if (!check_cu(seqs, p.tokens, p.err)) return;
    const int n = blockIdx.x / p.heads, h = blockIdx.x % p.heads, g = h / (p.heads / p.groups);
    const int q = threadIdx.x % kP, j = threadIdx.x / kP;
    const int64_t a = seqs.start(n), b = seqs.start(n + 1);
    const int64_t st = (static_cast<int64_t>(n) * p.heads + h) * kN * kP + j * kRows * kP + q;
    float s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = p.s0 != nullptr ? p.s0[st + i * kP] : 0.f;
    const float av = __ldg(p.a + h), dv = p.d != nullptr ? __ldg(p.d + h) : 0.f;
    for (int64_t t = a; t < b; ++t) {
        __syncthreads();
        if (threadIdx.x < kN) {
            s_b[threadIdx.x] = bf16_at(p.b, t * p.b_stride + g * kN + threadIdx.x);
            s_c[threadIdx.x] = bf16_at(p.c, t * p.c_stride + g * kN + threadIdx.x);
        }
        const float delta = delta_of(p, t, h), decay = __expf(av * delta);
        const float x = bf16_at(p.x, t * p.x_stride + h * kP + q);
        __syncthreads();
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            s[i] = fmaf(s[i], decay, delta * x * s_b[j * kRows + i]);
            y = fmaf(s[i], s_c[j * kRows + i], y);
        }
        s_y[j][q] = y;
        __syncthreads();
        if (j == 0) {
            for (int k = 1; k < kParts; ++k) y += s_y[k][q];
            static_cast<__nv_bfloat16 *>(p.out)[(t * p.heads + h) * kP + q] =
                __float2bfloat16_rn(fmaf(dv, x, y));
        }
    }
    if (p.s_final != nullptr)
#pragma unroll
        for (int i = 0; i < kRows; ++i) p.s_final[st + i * kP] = s[i];
}

template <int kN, int kP>
cudaError_t launch_serial(const SsmParams &p, cudaStream_t stream) {
    ssm_serial_kernel<kN, kP><<<p.n_seqs * p.heads, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t configure_ssm() { return cudaSuccess; }

int64_t ssm_workspace(const SsmParams &) { return 0; }

cudaError_t launch_ssm(const SsmParams &p, const CallContext &, cudaStream_t stream) {
    if (p.n == 64) return p.p == 64 ? launch_serial<64, 64>(p, stream) : launch_serial<64, 128>(p, stream);
    return p.p == 64 ? launch_serial<128, 64>(p, stream) : launch_serial<128, 128>(p, stream);
}

cudaError_t launch_ssm_step(const SsmParams &p, cudaStream_t stream) {
    if (p.n == 64) return p.p == 64 ? launch_serial<64, 64>(p, stream) : launch_serial<64, 128>(p, stream);
    return p.p == 64 ? launch_serial<128, 64>(p, stream) : launch_serial<128, 128>(p, stream);
}

}  // namespace kda
