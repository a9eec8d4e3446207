// Attention of one new token per sequence over a paged key-value cache
// (kda_paged_decode): out = softmax(scale q K^T) V and its log-sum-exp, one
// pass over the cache with the running maximum and sum of the softmax.

#include <math_constants.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

// One block per (sequence, query head); a warp takes every fourth token.
template <int D>
__global__ void __launch_bounds__(128) paged_simple_kernel(PagedParams p) {
    constexpr int E = D / 32;
    __shared__ float s_m[4], s_l[4], s_o[4][D];
    const int b = blockIdx.x / p.hq, h = blockIdx.x % p.hq, kv = h / (p.hq / p.hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t len = __ldg(p.lens + b);
    if (len < 0 || len > p.max_pages * p.page_size) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrPage);
        len = 0;
    }
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (static_cast<int64_t>(b) * p.hq + h) * D;
    float qv[E], o[E], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = __bfloat162float(q[lane + 32 * e]) * p.scale;
        o[e] = 0.f;
    }
    for (int64_t t = warp; t < len; t += 4) {
        int64_t page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + t / p.page_size);
        if (page < 0 || page >= p.pages) {
            if (lane == 0) atomicOr(p.err, kErrPage);
            if (p.pages == 0) break;
            page = 0;
        }
        const int64_t in = ((t % p.page_size) * p.hkv + kv) * D;
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(p.k) + page * p.k_stride + in;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v) + page * p.v_stride + in;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(qv[e], __bfloat162float(k[lane + 32 * e]), s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float top = fmaxf(m, s);
        const float f = top == -CUDART_INF_F ? 0.f : expf(m - top);
        const float w = top == -CUDART_INF_F ? 0.f : expf(s - top);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * __bfloat162float(v[lane + 32 * e]);
        m = top;
    }
    s_m[warp] = m;
    s_l[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = o[e];
    __syncthreads();
    float top = -CUDART_INF_F, sum = 0.f;
    for (int w = 0; w < 4; ++w) top = fmaxf(top, s_m[w]);
    float f[4];
    for (int w = 0; w < 4; ++w) {
        f[w] = s_m[w] == -CUDART_INF_F ? 0.f : expf(s_m[w] - top);
        sum += s_l[w] * f[w];
    }
    const int64_t row = static_cast<int64_t>(b) * p.hq + h;
    for (int i = threadIdx.x; i < D; i += 128) {
        float r = 0.f;
        for (int w = 0; w < 4; ++w) r += s_o[w][i] * f[w];
        static_cast<__nv_bfloat16 *>(p.out)[row * D + i] = __float2bfloat16_rn(sum > 0.f ? r / sum : 0.f);
    }
    if (threadIdx.x == 0 && p.lse != nullptr) p.lse[row] = sum > 0.f ? logf(sum) + top : -CUDART_INF_F;
}

}  // namespace

cudaError_t configure_paged() { return cudaSuccess; }
int64_t paged_workspace(const PagedParams &) { return 0; }
int64_t paged_sync(const PagedParams &) { return 0; }

cudaError_t launch_paged(const PagedParams &p, const CallContext &, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.batch) * p.hq;
    if (p.dim == 64) paged_simple_kernel<64><<<grid, 128, 0, stream>>>(p);
    else paged_simple_kernel<128><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
