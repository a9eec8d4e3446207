// Decode attention over a paged cache of 8-bit numbers (kda_paged_decode_fp8).

#include <cuda_fp8.h>
#include <math_constants.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) paged8_kernel(Paged8Params p) {
    constexpr int kPer = D / 32;
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
    const Cache8 &c = p.c;
    const int b = blockIdx.x / p.hq, h = blockIdx.x % p.hq, kv = h / (p.hq / c.hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int len = c.lens[b];
    if (len < 0 || len > c.max_pages * c.page_size || (len > 0 && c.pages == 0)) {
        if (threadIdx.x == 0) atomicOr(c.err, kErrPage);
        len = 0;
    }
    float q[kPer], o[kPer] = {}, m = -CUDART_INF_F, l = 0.f;
    const int64_t row = static_cast<int64_t>(b) * p.hq + h;
    for (int e = 0; e < kPer; ++e)
        q[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[row * D + kPer * lane + e]);
    auto number = [](uint8_t x) { return __half2float(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)); };
    for (int t = warp; t < len; t += kWarps) {
        int page = c.table[b * c.max_pages + t / c.page_size];
        if (page < 0 || page >= c.pages) {
            if (lane == 0) atomicOr(c.err, kErrPage);
            page = 0;
        }
        const int64_t in = t % c.page_size;
        const uint8_t *k = c.k + page * c.k_page + in * c.k_token + kv * c.k_head + kPer * lane;
        const uint8_t *v = c.v + page * c.v_page + in * c.v_token + kv * c.v_head + kPer * lane;
        float s = 0.f;
        for (int e = 0; e < kPer; ++e) s = fmaf(q[e], number(k[e]), s);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= p.scale * c.ks[page * c.ks_page + kv];
        const float top = fmaxf(m, s), base = top == -CUDART_INF_F ? 0.f : top;
        const float f = expf(m - base), w = expf(s - base), vs = w * c.vs[page * c.vs_page + kv];
        m = top;
        l = l * f + w;
        for (int e = 0; e < kPer; ++e) o[e] = o[e] * f + vs * number(v[e]);
    }
    s_m[warp] = m;
    s_l[warp] = l;
    for (int e = 0; e < kPer; ++e) s_o[warp][kPer * lane + e] = o[e];
    __syncthreads();
    if (threadIdx.x >= D) return;
    float top = -CUDART_INF_F, sum = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    const float base = top == -CUDART_INF_F ? 0.f : top;
    for (int w = 0; w < kWarps; ++w) {
        const float f = expf(s_m[w] - base);
        sum += s_l[w] * f;
        acc += s_o[w][threadIdx.x] * f;
    }
    static_cast<__nv_bfloat16 *>(p.out)[row * D + threadIdx.x] =
        __float2bfloat16_rn(sum > 0.f ? acc / sum : sum == 0.f ? 0.f : sum);
    if (threadIdx.x == 0 && p.lse != nullptr) p.lse[row] = sum == 0.f ? -CUDART_INF_F : base + logf(sum);
}

}  // namespace

cudaError_t configure_paged8() { return cudaSuccess; }
int64_t paged8_workspace(const Paged8Params &) { return 0; }
int64_t paged8_sync(const Paged8Params &) { return 0; }

cudaError_t launch_paged8(const Paged8Params &p, const CallContext &, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.c.batch) * p.hq;
    auto kernel = p.c.dim == 64 ? paged8_kernel<64> : paged8_kernel<128>;
    kernel<<<grid, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
