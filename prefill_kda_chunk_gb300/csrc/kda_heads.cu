// Norms of query and key heads and the rotation by position in one pass
// (kda_qk_norm_rope), and its gradients. For a head x of D channels, weights w and the
// rotation R by the token's angles
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = R (x r w)
//   g = R^T dy,  dw = sum g x r,  dx = r (g w - x r mean(g w x r))
//
// A head is a row; D / 8 lanes share it, 16 bytes of it each, so that a row is one
// load, one store and a few shuffles. The angles are the same for all heads of a
// token: a block takes rows of a few tokens and forms their sines and cosines once,
// in shared memory.

#include <type_traits>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kHeadsThreads = 256;
constexpr int kHeadsTokens = 8;      // tokens of a block's angles
// rows of a lane group whose loads are on their way together
constexpr int kAhead = 4;

// cos and sin of position * f, where f turns by f / 2 pi a position. The turns are
// formed as two floats (f / 2 pi to 2^-48, the position in two parts that fp32 holds
// exactly, each product with its rounding error) and whole turns are dropped on the way.
__device__ __forceinline__ void angle(int pos, float f, float &c, float &s) {
    const float inv = 0.15915494f, inv_lo = 6.42063833e-9f;   // 1 / 2 pi
    const float hi = f * inv, lo = fmaf(f, inv, -hi) + f * inv_lo;
    const float p0 = static_cast<float>(pos & 4095), p1 = static_cast<float>(pos & ~4095);
    const float a = p0 * hi, b = p1 * hi;
    float t = (a - rintf(a)) + (b - rintf(b));
    t += fmaf(p0, hi, -a) + fmaf(p1, hi, -b) + (p0 + p1) * lo;
    t -= rintf(t);
    sincospif(2.f * t, &s, &c);
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// Eight channels of a row turned by the token's angles, or back (sign = -1).
// cs: the token's cosines, then its sines, rot / 2 each.
template <bool kPairs>
__device__ __forceinline__ void turn(float (&x)[8], const float *cs, int rot, int at, int lane, float sign) {
    const int half = rot / 2;
    if (kPairs) {
        if (8 * at >= rot) return;
        const float4 c = *reinterpret_cast<const float4 *>(cs + 4 * at);
        const float4 s = *reinterpret_cast<const float4 *>(cs + half + 4 * at);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1], t = sign * ss[i];
            x[2 * i] = fmaf(a, cc[i], -b * t);
            x[2 * i + 1] = fmaf(b, cc[i], a * t);
        }
    } else {
        const bool in = 8 * at < rot, low = 8 * at < half;
        const int from = !in ? lane : low ? lane + rot / 16 : lane - rot / 16;
        float other[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, x[i], from);
        if (!in) return;
        const int f = low ? 8 * at : 8 * at - half;
        const float sg = low ? -sign : sign;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 c = *reinterpret_cast<const float4 *>(cs + f + 4 * j);
            const float4 s = *reinterpret_cast<const float4 *>(cs + half + f + 4 * j);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[4 * j + i] = fmaf(x[4 * j + i], cc[i], other[4 * j + i] * (sg * ss[i]));
        }
    }
}

// The sines and cosines of tokens [t0, t0 + n).
__device__ __forceinline__ void fill_angles(const HeadsParams &p, float *cs, int64_t t0, int n) {
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < n * half; i += kHeadsThreads) {
        const int t = i / half, f = i % half;
        float c, s;
        angle(__ldg(p.pos + t0 + t), __ldg(p.freq + f), c, s);
        cs[t * p.rot + f] = c;
        cs[t * p.rot + half + f] = s;
    }
}

__device__ __forceinline__ void weights8(const float *w, int at, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = w != nullptr ? __ldg(w + 8 * at + i) : 1.f;
}

// Block b takes the rows (token, head) [b * rows, (b + 1) * rows), which lie in at most
// kHeadsTokens + 1 tokens.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kHeadsThreads) heads_kernel(HeadsParams p, int rows) {
    constexpr int kLanes = D / 8, kGroups = kHeadsThreads / kLanes;
    extern __shared__ __align__(16) float cs[];
    const int lane = threadIdx.x & 31, at = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int H = p.hq + p.hk;
    const int64_t total = p.tokens * H, row0 = static_cast<int64_t>(blockIdx.x) * rows;
    const int count = static_cast<int>(total - row0 < rows ? total - row0 : rows);
    const int64_t t0 = row0 / H;
    const int h0 = static_cast<int>(row0 - t0 * H);
    if (p.rot > 0) {
        fill_angles(p, cs, t0, (h0 + count - 1) / H + 1);
        __syncthreads();
    }
    float qw[8], kw[8];
    weights8(p.qw, at, qw);
    weights8(p.kw, at, kw);
    for (int base = 0; base < count; base += kGroups * kAhead) {
        uint4 in[kAhead];
        int tok[kAhead], head[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = base + i * kGroups + group, near = r < count ? r : count - 1;
            tok[i] = (h0 + near) / H;   // (lane groups past the end join in the shuffles)
            head[i] = r < count ? h0 + r - tok[i] * H : -1;
            in[i] = make_uint4(0, 0, 0, 0);
            if (head[i] >= 0) {
                const int64_t t = t0 + tok[i];
                const uint16_t *src = head[i] < p.hq
                    ? static_cast<const uint16_t *>(p.q) + t * p.q_stride + head[i] * D
                    : static_cast<const uint16_t *>(p.k) + t * p.k_stride + (head[i] - p.hq) * D;
                in[i] = *reinterpret_cast<const uint4 *>(src + 8 * at);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (base + i * kGroups >= count) break;   // (the same for the whole block)
            float x[8];
            unpack8(in[i], x);
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
            const float r = rsqrtf(row_sum<kLanes>(sum) * (1.f / D) + p.eps);
            const bool is_q = head[i] < p.hq;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= r * (is_q ? qw[e] : kw[e]);
            if (p.rot > 0) turn<kPairs>(x, cs + tok[i] * p.rot, p.rot, at, lane, 1.f);
            if (head[i] >= 0) {
                const int64_t t = t0 + tok[i];
                uint16_t *dst = is_q
                    ? static_cast<uint16_t *>(p.q_out) + t * p.qo_stride + head[i] * D
                    : static_cast<uint16_t *>(p.k_out) + t * p.ko_stride + (head[i] - p.hq) * D;
                *reinterpret_cast<uint4 *>(dst + 8 * at) = pack8(x);
            }
        }
    }
}

// Blocks of the gradient: each walks a run of rows, kHeadsTokens tokens' angles at a time,
// and leaves its part of the weights' gradients.
constexpr int kGradBlocks = 4 * kPlannedSms;

__device__ __forceinline__ void load8(const void *p, int64_t i, bool f32, float (&x)[8]) {
    if (f32) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = s[0], b = s[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i), x);
    }
}

template <int D, bool kPairs, bool kF32>
__global__ void __launch_bounds__(kHeadsThreads) heads_backward_kernel(HeadsParams p) {
    constexpr int kLanes = D / 8, kGroups = kHeadsThreads / kLanes;
    extern __shared__ __align__(16) float cs[];
    const int lane = threadIdx.x & 31, at = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int H = p.hq + p.hk;
    const int64_t total = p.tokens * H;
    const int64_t row0 = total * blockIdx.x / gridDim.x, row1 = total * (blockIdx.x + 1) / gridDim.x;
    float qw[8], kw[8], dqw[8], dkw[8];
    weights8(p.qw, at, qw);
    weights8(p.kw, at, kw);
#pragma unroll
    for (int e = 0; e < 8; ++e) dqw[e] = dkw[e] = 0.f;
    for (int64_t start = row0; start < row1;) {
        const int64_t t0 = start / H;
        const int h0 = static_cast<int>(start - t0 * H);
        int64_t end = (t0 + kHeadsTokens) * H;
        if (end > row1) end = row1;
        const int count = static_cast<int>(end - start);
        if (p.rot > 0) {
            __syncthreads();
            fill_angles(p, cs, t0, (h0 + count - 1) / H + 1);
            __syncthreads();
        }
        for (int base = 0; base < count; base += kGroups) {
            const int r = base + group, near = r < count ? r : count - 1;
            const int tok = (h0 + near) / H, head = r < count ? h0 + r - tok * H : -1;
            const bool is_q = head < p.hq;
            const int64_t t = t0 + tok;
            float x[8], g[8];
            if (head >= 0) {
                load8(is_q ? p.q : p.k,
                      (is_q ? t * p.q_stride + head * D : t * p.k_stride + (head - p.hq) * D) + 8 * at,
                      false, x);
                load8(is_q ? p.dq : p.dk,
                      (is_q ? t * p.dq_stride + head * D : t * p.dk_stride + (head - p.hq) * D) + 8 * at,
                      kF32, g);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = g[e] = 0.f;
            }
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
            const float rr = rsqrtf(row_sum<kLanes>(sum) * (1.f / D) + p.eps);
            if (p.rot > 0) turn<kPairs>(g, cs + tok * p.rot, p.rot, at, lane, -1.f);
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] *= rr;
                const float part = head >= 0 ? g[e] * x[e] : 0.f;
                if (is_q) dqw[e] += part;
                else dkw[e] += part;
                g[e] *= is_q ? qw[e] : kw[e];
                dot = fmaf(g[e], x[e], dot);
            }
            dot = row_sum<kLanes>(dot) * (1.f / D);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = rr * fmaf(-x[e], dot, g[e]);
            if (head >= 0) {
                uint16_t *dst = is_q
                    ? static_cast<uint16_t *>(p.q_out) + t * p.qo_stride + head * D
                    : static_cast<uint16_t *>(p.k_out) + t * p.ko_stride + (head - p.hq) * D;
                *reinterpret_cast<uint4 *>(dst + 8 * at) = pack8(x);
            }
        }
        start = end;
    }
    if (p.dqw == nullptr && p.dkw == nullptr) return;
    // the groups of a block, in order
    __shared__ float part[2][kGroups][D];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        part[0][group][8 * at + e] = dqw[e];
        part[1][group][8 * at + e] = dkw[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kHeadsThreads) {
        float s = 0.f;
        for (int j = 0; j < kGroups; ++j) s += part[i / D][j][i % D];
        p.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = s;
    }
}

// dweight[i] = the sum of the blocks' parts: a warp takes 32 channels, every eighth block.
__global__ void __launch_bounds__(256) heads_weights_kernel(HeadsParams p, int blocks) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    float s = 0.f;
    for (int b = warp; b < blocks; b += 8) s += p.partial[static_cast<int64_t>(b) * 2 * p.dim + i];
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0) return;
    for (int j = 1; j < 8; ++j) s += part[j][lane];
    float *dst = i < p.dim ? p.dqw : p.dkw;
    if (dst != nullptr) dst[i % p.dim] = s;
}

template <typename F>
cudaError_t with_dim(const HeadsParams &p, F &&go) {
    if (p.dim == 64) return go(std::integral_constant<int, 64>());
    if (p.dim == 128) return go(std::integral_constant<int, 128>());
    return go(std::integral_constant<int, 256>());
}

int angles_bytes(const HeadsParams &p) { return (kHeadsTokens + 1) * p.rot * 4; }

}  // namespace

cudaError_t configure_heads() { return cudaSuccess; }

cudaError_t launch_heads(const HeadsParams &p, cudaStream_t stream) {
    const int64_t H = p.hq + p.hk, total = p.tokens * H;
    return with_dim(p, [&](auto d) {
        constexpr int D = decltype(d)::value, kGroups = kHeadsThreads * 8 / D;
        int64_t rows = kGroups * 8;
        if (rows > H * kHeadsTokens) rows = H * kHeadsTokens;
        const unsigned grid = static_cast<unsigned>((total + rows - 1) / rows);
        auto kernel = p.pairs ? heads_kernel<D, true> : heads_kernel<D, false>;
        kernel<<<grid, kHeadsThreads, angles_bytes(p), stream>>>(p, static_cast<int>(rows));
        return cudaGetLastError();
    });
}

int64_t heads_workspace(const HeadsParams &p) {
    return p.dqw != nullptr || p.dkw != nullptr ? static_cast<int64_t>(kGradBlocks) * 2 * p.dim * 4 : 0;
}

cudaError_t launch_heads_backward(const HeadsParams &p, cudaStream_t stream) {
    const int64_t total = p.tokens * (p.hq + p.hk);
    return with_dim(p, [&](auto d) {
        constexpr int D = decltype(d)::value, kGroups = kHeadsThreads * 8 / D;
        const int64_t want = (total + kGroups - 1) / kGroups;
        const int grid = static_cast<int>(want < 1 ? 1 : want < kGradBlocks ? want : kGradBlocks);
        auto kernel = p.pairs ? (p.dout32 ? heads_backward_kernel<D, true, true> : heads_backward_kernel<D, true, false>)
                              : (p.dout32 ? heads_backward_kernel<D, false, true> : heads_backward_kernel<D, false, false>);
        kernel<<<grid, kHeadsThreads, angles_bytes(p), stream>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || (p.dqw == nullptr && p.dkw == nullptr)) return e;
        heads_weights_kernel<<<2 * D / 32, 256, 0, stream>>>(p, grid);
        return cudaGetLastError();
    });
}

}  // namespace kda
