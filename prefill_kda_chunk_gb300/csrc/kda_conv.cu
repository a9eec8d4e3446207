// Short causal convolution, one filter of W = 2..4 taps per channel, with its
// history, its single-token step and its gradient (kda_short_conv*).
//
//   z[t] = bias + sum_j w[j] x[t - (W-1) + j],  y = z / (1 + e^-z) or z
//
// Each element of x is read for one multiply-add per tap, so the operator is
// bound by HBM (4 B per element forward, 6 or 8 for the gradient). A thread owns VEC
// neighbouring channels and walks its tokens in order with the last W - 1 rows in
// registers: every row is read once, but for the W - 1 rows in front of each
// warp's run of tokens (which come out of L2). A warp covers 32 * VEC
// channels of one token (512 contiguous bytes at VEC = 8), and rows arrive through a
// ring in shared memory, 12 of each warp on their way at a time. Sequence ends only
// move the window, so a packed batch runs like one long sequence. All sums are fp32.
//
// Measured at T = D = 8192, W = 4: forward 52 us (5.2 TB/s, 76 % of copy bandwidth),
// gradient with fp32 d_out 98 us (5.5 TB/s, 80 %); one token for each of 256 sequences,
// D = 24576: 19 us (5.4 TB/s, 79 %).

#include "kda_device.cuh"
#include "kda_internal.h"
#include "kda_seqs.cuh"

#include <type_traits>

namespace kda {

namespace {

constexpr int kWarps = 8;

template <int VEC>
struct Raw;
template <>
struct Raw<8> { using T = uint4; };
template <>
struct Raw<4> { using T = uint2; };
template <>
struct Raw<1> { using T = uint16_t; };

__device__ __forceinline__ float bf16_bits(uint32_t b) { return __uint_as_float(b << 16); }

template <int VEC>
__device__ __forceinline__ void widen(const typename Raw<VEC>::T &r, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = bf16_bits(r);
    } else {
        const uint32_t *u = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            f[2 * i] = bf16_bits(u[i]);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
}

template <int VEC>
__device__ __forceinline__ typename Raw<VEC>::T narrow(const float (&f)[VEC]) {
    typename Raw<VEC>::T r;
    if constexpr (VEC == 1) {
        r = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
        uint32_t *u = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) u[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    }
    return r;
}

template <int VEC>
__device__ __forceinline__ typename Raw<VEC>::T load_row(const void *base, int64_t at) {
    return *reinterpret_cast<const typename Raw<VEC>::T *>(static_cast<const uint16_t *>(base) + at);
}

template <int VEC>
__device__ __forceinline__ void load_f32(const float *src, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = *src;
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            reinterpret_cast<float4 *>(f)[i] = reinterpret_cast<const float4 *>(src)[i];
    }
}

template <int VEC>
__device__ __forceinline__ void store_f32(float *dst, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        *dst = f[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            reinterpret_cast<float4 *>(dst)[i] = reinterpret_cast<const float4 *>(f)[i];
    }
}

// The arithmetic on a thread's channels goes two by two, in packed instructions: with
// single ones the forward issued in 74 % of all slots, this way in 63 % (53 us against 51,
// before the branch for z below kFar).
template <int VEC>
__device__ __forceinline__ void times(float (&a)[VEC], const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        a[0] *= x[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) mul2(a[i], a[i + 1], x[i], x[i + 1]);
    }
}

// 1 / (1 + e^-z) of two values with one reciprocal: r = 1 / (a b), 1 / a = r b. The
// exponential and the reciprocal share one unit of 16 results a clock and SM, which two
// of each per pair would keep as busy as HBM. e^-z is held at 2^63, so that the
// product stays finite and no channel can reach the other: right down to z = kFar.
// e0 and e1 are e^-z: the gradient takes 1 - s as e^-z s, since s is 1 but for its
// rounding at large z and z would multiply that. Returns a b.
__device__ __forceinline__ float sigmoid2(float z0, float z1, float &s0, float &s1, float &e0, float &e1) {
    mul2(z0, z1, -1.44269504f, -1.44269504f);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(fminf(z0, 63.f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(fminf(z1, 63.f)));
    float a = e0, b = e1, r;
    add2(a, b, 1.f, 1.f);
    const float ab = a * b;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ab));
    s0 = b;
    s1 = a;
    mul2(s0, s1, r, r);
    return ab;
}
// s and 1 - s (`rest`) of a thread's channels, right down to kFar; the products a b, none
// of them below 1, are added to `products`. Where they add up to kFarSum or more, a
// channel may be below kFar.
constexpr float kFar = -43.66f, kFarSum = 4.6e18f;   // (2^62)
template <int VEC>
__device__ __forceinline__ void sigmoids_near(const float (&z)[VEC], float (&s)[VEC], float (&rest)[VEC],
                                              float (&products)[2]) {
    if constexpr (VEC == 1) {
        float s1, e1;
        products[0] += sigmoid2(z[0], 0.f, s[0], s1, rest[0], e1);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float u = sigmoid2(z[i], z[i + 1], s[i], s[i + 1], rest[i], rest[i + 1]);
            const float v = sigmoid2(z[i + 2], z[i + 3], s[i + 2], s[i + 3], rest[i + 2], rest[i + 3]);
            add2(products[0], products[1], u, v);
        }
    }
    times<VEC>(rest, s);
}
// ... at any z: below kFar the sigmoid is e^z to fp32's precision (down to its
// subnormals), which only a thread with such a channel computes.
template <int VEC>
__device__ __forceinline__ void sigmoids(const float (&z)[VEC], float (&s)[VEC], float (&rest)[VEC]) {
    float products[2] = {0.f, 0.f};
    sigmoids_near<VEC>(z, s, rest, products);
    if (products[0] + products[1] >= kFarSum) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float t;
            asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(z[i] * 1.44269504f));
            if (z[i] < kFar) s[i] = t;
        }
    }
}
template <int VEC>
__device__ __forceinline__ void plus(float (&a)[VEC], const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        a[0] += x[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) add2(a[i], a[i + 1], x[i], x[i + 1]);
    }
}
template <int VEC>
__device__ __forceinline__ void plus(float (&a)[VEC], const float (&x)[VEC], const float (&y)[VEC]) {
    if constexpr (VEC == 1) {
        a[0] = fmaf(x[0], y[0], a[0]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) muladd2(a[i], a[i + 1], x[i], x[i + 1], y[i], y[i + 1]);
    }
}
template <int VEC>
__device__ __forceinline__ void copy(float (&a)[VEC], const float (&x)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) a[i] = x[i];
}
template <int VEC>
__device__ __forceinline__ void silu(float (&z)[VEC]) {
    float s[VEC], rest[VEC];
    sigmoids<VEC>(z, s, rest);
    times<VEC>(z, s);
}

// The filters of a block's 32 VEC channels, read once and kept tap by tap in shared
// memory: read from [D, W] by each thread, their scattered sectors cost more than
// the rows (T = D = 8192: 115 us against 84).
template <int W, int VEC>
struct Filters {
    float w[W + 1][32 * VEC];   // the taps, then the bias
    __device__ __forceinline__ void load(const ConvParams &p, int64_t d0) {
        for (int i = threadIdx.x; i < 32 * VEC * W; i += blockDim.x) {
            const int c = i / W;
            w[i % W][c] = d0 + c < p.dim ? __ldg(p.weight + d0 * W + i) : 0.f;
        }
        for (int c = threadIdx.x; c < 32 * VEC; c += blockDim.x)
            w[W][c] = p.bias != nullptr && d0 + c < p.dim ? __ldg(p.bias + d0 + c) : 0.f;
        __syncthreads();
    }
};

// Asynchronous copy of one thread's piece of a row to its own place in shared memory.
template <typename T>
__device__ __forceinline__ void copy_piece(T *dst, const void *src) {
    if constexpr (sizeof(T) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Waits for all groups of copies but the last N.
template <int N>
__device__ __forceinline__ void copies_but() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// The filter of a thread's channels.
template <int W, int VEC>
struct Filter {
    float w[W][VEC], b[VEC];
    __device__ __forceinline__ Filter(const Filters<W, VEC> &f, int lane) {
#pragma unroll
        for (int j = 0; j < W; ++j) load_f32<VEC>(f.w[j] + lane * VEC, w[j]);
        load_f32<VEC>(f.w[W] + lane * VEC, b);
    }
};

// The W - 1 rows in front of token t of a sequence that starts at token a.
template <int W, int VEC>
__device__ __forceinline__ void load_window(const ConvParams &p, int n, int64_t a, int64_t t,
                                            int64_t d, float (&win)[W - 1][VEC]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t r = t - (W - 1) + j;
        if (r >= a) {
            widen<VEC>(load_row<VEC>(p.x, r * p.x_stride + d), win[j]);
        } else if (p.hist_in != nullptr) {
            widen<VEC>(load_row<VEC>(p.hist_in,
                                     (static_cast<int64_t>(n) * (W - 1) + (W - 1) + (r - a)) * p.dim + d),
                       win[j]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) win[j][i] = 0.f;
        }
    }
}

// z of the next row, which then enters the window.
template <int W, int VEC>
__device__ __forceinline__ void step_window(const Filter<W, VEC> &f, float (&win)[W - 1][VEC],
                                            const float (&row)[VEC], float (&z)[VEC]) {
    copy<VEC>(z, f.b);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) plus<VEC>(z, f.w[j], win[j]);
    plus<VEC>(z, f.w[W - 1], row);
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) copy<VEC>(win[j], win[j + 1]);
    copy<VEC>(win[W - 2], row);
}

// Rows per warp: at most `most`, and such that the blocks fill whole waves of two per
// SM. The W - 1 rows read twice are 5 % at 64 (out of L2), and the gradient's W - 1
// tokens worked on twice are as many, so that it takes longer runs (T = D = 8192:
// runs of 64, 96 and 128 rows at most took 110, 103 and 99 us, the forward's 53, 53 and
// 55, before the arithmetic went two by two).
constexpr int kRun = 64, kBackRun = 128, kMinRun = 4, kSlots = 2 * kPlannedSms;
int64_t run_for(int64_t tokens, int64_t cols, int64_t most) {
    int64_t run = most;
    for (int64_t waves = 1;; ++waves) {
        const int64_t blocks = kSlots * waves / cols > 0 ? kSlots * waves / cols : 1;   // along the tokens
        run = (tokens + blocks * kWarps - 1) / (blocks * kWarps);
        if (run <= most) break;
        if (waves == 16) return most;   // (many waves: they need not be whole)
    }
    return run < kMinRun ? kMinRun : run;
}

constexpr int kGroup = 4, kDepth = 4;   // rows of a group, groups of the ring
constexpr int kForwardVec = 8, kBackwardVec = 4;   // channels per thread at most
template <int VEC>
constexpr int ring_bytes() {
    return VEC > 1 ? kDepth * kGroup * kWarps * 32 * 2 * VEC : 0;
}

template <int W, int VEC, bool SILU>
__global__ void __launch_bounds__(kWarps * 32, VEC == 4 ? 3 : 2)
conv_kernel(ConvParams p, int run, int64_t col_blocks) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) Filters<W, VEC> filters;
    using R = typename Raw<VEC>::T;
    R *ring = reinterpret_cast<R *>(smem) + threadIdx.x;
    const Seqs seqs{p.cu, p.seq_len, p.n_seqs};
    if (!check_cu(seqs, p.tokens, p.err)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x / col_blocks, d0 = (blockIdx.x % col_blocks) * 32 * VEC;
    filters.load(p, d0);
    const int64_t t0 = (tile * kWarps + warp) * run;
    const int64_t t1 = t0 + run < p.tokens ? t0 + run : p.tokens;
    if (t0 >= p.tokens && t0 > 0) return;
    const int64_t d = d0 + lane * VEC;
    int n = first_seq(seqs, t0);
    if (d >= p.dim) return;
    const Filter<W, VEC> f(filters, lane);
    for (; n < p.n_seqs; ++n) {
        const int64_t a = seqs.start(n), b = seqs.start(n + 1);
        if (a >= t1 && t1 < p.tokens) break;
        const int64_t lo = a > t0 ? a : t0, hi = b < t1 ? b : t1;
        float win[W - 1][VEC];
        load_window<W, VEC>(p, n, a, lo, d, win);
        const uint16_t *src = static_cast<const uint16_t *>(p.x) + lo * p.x_stride + d;
        uint16_t *dst = static_cast<uint16_t *>(p.out) + lo * p.out_stride + d;
        auto row_out = [&](const R &raw, uint16_t *to, float (&products)[2]) {
            float row[VEC], z[VEC];
            widen<VEC>(raw, row);
            step_window<W, VEC>(f, win, row, z);
            if (SILU) {
                float s[VEC], rest[VEC];
                if constexpr (VEC > 1) sigmoids_near<VEC>(z, s, rest, products);
                else sigmoids<VEC>(z, s, rest);
                times<VEC>(z, s);
            }
            *reinterpret_cast<R *>(to) = narrow<VEC>(z);
        };
        const int rows = static_cast<int>(hi - lo);
        if constexpr (VEC > 1) {
            // groups of kGroup rows pass through a ring in shared memory, kDepth - 1
            // of them in flight; a thread reads only what it copied itself
            auto fetch = [&](int r0) {
                R *to = ring + r0 / kGroup % kDepth * kGroup * kWarps * 32;
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    if (r0 + u < rows) copy_piece(to + u * kWarps * 32, src);
                    src += p.x_stride;
                }
                cp_async_commit();
            };
#pragma unroll
            for (int g = 0; g < kDepth - 1; ++g) fetch(g * kGroup);
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += kGroup) {
                fetch(r0 + (kDepth - 1) * kGroup);
                copies_but<kDepth - 1>();
                const R *from = ring + r0 / kGroup % kDepth * kGroup * kWarps * 32;
                float products[2] = {0.f, 0.f};
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    if (r0 + u < rows) row_out(from[u * kWarps * 32], dst, products);
                    dst += p.out_stride;
                }
                // a group with a channel below kFar is formed again, row by row out of L2
                // (a branch per group: with one per row the forward takes 53.4 us, this way 52.2)
                if (SILU && products[0] + products[1] >= kFarSum) {
#pragma unroll 1
                    for (int u = 0; u < kGroup && r0 + u < rows; ++u) {
                        float past[W - 1][VEC], row[VEC], z[VEC];
                        const int64_t t = lo + r0 + u;
                        load_window<W, VEC>(p, n, a, t, d, past);
                        widen<VEC>(load_row<VEC>(p.x, t * p.x_stride + d), row);
                        step_window<W, VEC>(f, past, row, z);
                        silu<VEC>(z);
                        *reinterpret_cast<R *>(static_cast<uint16_t *>(p.out) + t * p.out_stride + d) =
                            narrow<VEC>(z);
                    }
                }
            }
        } else {
#pragma unroll 4
            for (int r = 0; r < rows; ++r) {
                float products[2];
                row_out(*reinterpret_cast<const R *>(src), dst, products);
                src += p.x_stride;
                dst += p.out_stride;
            }
        }
        if (b <= t1 && p.hist_out != nullptr) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                *reinterpret_cast<typename Raw<VEC>::T *>(
                    static_cast<uint16_t *>(p.hist_out) +
                    (static_cast<int64_t>(n) * (W - 1) + j) * p.dim + d) = narrow<VEC>(win[j]);
        }
    }
}

// One token per sequence: a warp takes 32 VEC channels of kStepRows sequences, reads W
// rows of each and writes one row of out and the shifted history. Every address it
// writes was read by the same thread before, so the history may be updated in
// place.
constexpr int kStepRows = 4;
template <int W, int VEC, bool SILU>
__global__ void __launch_bounds__(kWarps * 32) conv_step_kernel(ConvParams p, int64_t col_blocks) {
    __shared__ __align__(16) Filters<W, VEC> filters;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t d0 = (blockIdx.x % col_blocks) * 32 * VEC, d = d0 + lane * VEC;
    const int64_t n0 = (blockIdx.x / col_blocks) * kWarps * kStepRows + warp;
    using R = typename Raw<VEC>::T;
    R raw[kStepRows][W];
    if (d < p.dim) {
#pragma unroll
        for (int u = 0; u < kStepRows; ++u) {
            const int64_t n = n0 + u * kWarps;
            if (n >= p.tokens) break;
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                raw[u][j] = p.hist_in != nullptr
                                ? load_row<VEC>(p.hist_in, (n * (W - 1) + j) * p.dim + d) : R{};
            raw[u][W - 1] = load_row<VEC>(p.x, n * p.x_stride + d);
        }
    }
    filters.load(p, d0);
    if (d >= p.dim) return;
    const Filter<W, VEC> f(filters, lane);
#pragma unroll
    for (int u = 0; u < kStepRows; ++u) {
        const int64_t n = n0 + u * kWarps;
        if (n >= p.tokens) break;
        float z[VEC];
        copy<VEC>(z, f.b);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float row[VEC];
            widen<VEC>(raw[u][j], row);
            plus<VEC>(z, f.w[j], row);
        }
        if (SILU) silu<VEC>(z);
        *reinterpret_cast<R *>(static_cast<uint16_t *>(p.out) + n * p.out_stride + d) = narrow<VEC>(z);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            *reinterpret_cast<R *>(static_cast<uint16_t *>(p.hist_out) + (n * (W - 1) + j) * p.dim + d) =
                raw[u][j + 1];
    }
}

// The gradient walks the same runs. At token t, dz_t completes dx of row
// t - (W-1); the W - 1 rows still open wait in `open` (open[i]: row
// t - (W-1) + 1 + i). A run goes on W - 1 tokens past its own to complete its
// last rows, and its weight sums take its own tokens only. The sums of the
// eight warps are joined in shared memory in warp order and written per tile;
// conv_reduce_kernel adds the tiles in order, so the result does not depend on
// timing.
constexpr int kBackGroup = 4, kBackDepth = 3;
template <int W, int VEC, bool D32>
constexpr int back_bytes() {
    const int ring = VEC > 1 ? kBackDepth * kBackGroup * kWarps * 32 * VEC * (2 + (D32 ? 4 : 2)) : 0;
    const int sums = kWarps * (W + 1) * VEC * 32 * 4;
    return ring > sums ? ring : sums;
}

template <int W, int VEC, bool SILU, bool D32>
__global__ void __launch_bounds__(kWarps * 32, 2)
conv_backward_kernel(ConvParams p, int run, int64_t col_blocks) {
    extern __shared__ __align__(16) uint8_t smem[];   // the ring, then the warps' sums
    using R = typename Raw<VEC>::T;
    using G1 = std::conditional_t<D32, float, uint16_t>;
    using G = std::conditional_t<D32, std::conditional_t<VEC == 1, float, float4>, R>;
    float(*sums)[(W + 1) * VEC * 32] = reinterpret_cast<float(*)[(W + 1) * VEC * 32]>(smem);
    constexpr int kPieces = kBackDepth * kBackGroup * kWarps * 32;
    G *dring = reinterpret_cast<G *>(smem) + threadIdx.x;
    R *ring = reinterpret_cast<R *>(smem + kPieces * sizeof(G)) + threadIdx.x;
    __shared__ __align__(16) Filters<W, VEC> filters;
    const Seqs seqs{p.cu, p.seq_len, p.n_seqs};
    if (!check_cu(seqs, p.tokens, p.err)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x / col_blocks;
    const int64_t t0 = (tile * kWarps + warp) * run;
    const int64_t t1 = t0 + run < p.tokens ? t0 + run : p.tokens;
    const int64_t d0 = (blockIdx.x % col_blocks) * 32 * VEC, d = d0 + lane * VEC;
    filters.load(p, d0);
    const bool live = d < p.dim && (t0 < p.tokens || t0 == 0);
    int n = first_seq(seqs, t0);
    float dw[W][VEC], db[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    if (live) {
        const Filter<W, VEC> f(filters, lane);
        for (; n < p.n_seqs; ++n) {
            const int64_t a = seqs.start(n), b = seqs.start(n + 1);
            if (a >= t1 && t1 < p.tokens) break;
            const int64_t lo = a > t0 ? a : t0, hi = b < t1 ? b : t1;
            const int64_t end = hi + W - 1 < b ? hi + W - 1 : b;
            float win[W - 1][VEC], open[W - 1][VEC];
            load_window<W, VEC>(p, n, a, lo, d, win);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) open[j][i] = 0.f;
            // row r of this sequence is complete
            auto emit = [&](int64_t r, const float (&v)[VEC]) {
                if (r >= lo) {
                    if (r < hi)
                        *reinterpret_cast<typename Raw<VEC>::T *>(static_cast<uint16_t *>(p.out) +
                                                                  r * p.out_stride + d) = narrow<VEC>(v);
                } else if (lo == a && p.dhist_in != nullptr) {
                    store_f32<VEC>(p.dhist_in +
                                       (static_cast<int64_t>(n) * (W - 1) + (W - 1) + (r - a)) * p.dim + d,
                                   v);
                }
            };
            const uint16_t *src = static_cast<const uint16_t *>(p.x) + lo * p.x_stride + d;
            int64_t at = lo * p.dout_stride + d;
            // token t: dz completes row t - (W - 1), which goes to `done`
            auto token = [&](const R &raw, const float (&g)[VEC], bool own, float (&done)[VEC]) {
                float row[VEC], z[VEC], dz[VEC];
                widen<VEC>(raw, row);
                copy<VEC>(z, f.b);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) plus<VEC>(z, f.w[j], win[j]);
                plus<VEC>(z, f.w[W - 1], row);
                copy<VEC>(dz, g);
                if (SILU) {   // s (1 + z (1 - s))
                    float sg[VEC], rest[VEC], ones[VEC];
                    sigmoids<VEC>(z, sg, rest);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) ones[i] = 1.f;
                    plus<VEC>(ones, z, rest);
                    times<VEC>(sg, ones);
                    times<VEC>(dz, sg);
                }
                copy<VEC>(done, open[0]);
                plus<VEC>(done, f.w[0], dz);
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) {
                    copy<VEC>(open[j], open[j + 1]);
                    plus<VEC>(open[j], f.w[j + 1], dz);
                }
                copy<VEC>(open[W - 2], dz);
                times<VEC>(open[W - 2], f.w[W - 1]);
                if (own) {
                    plus<VEC>(db, dz);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) plus<VEC>(dw[j], dz, win[j]);
                    plus<VEC>(dw[W - 1], dz, row);
                }
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) copy<VEC>(win[j], win[j + 1]);
                copy<VEC>(win[W - 2], row);
            };
            const int rows = static_cast<int>(end - lo), own = static_cast<int>(hi - lo);
            auto gradient = [&](const G &got, float (&g)[VEC]) {
                if constexpr (D32) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) g[i] = reinterpret_cast<const float *>(&got)[i];
                } else {
                    widen<VEC>(got, g);
                }
            };
            // row r of the run: the first W - 1 complete rows of the history or none
            auto one = [&](int r, const R &raw, const G &got) {
                float g[VEC], done[VEC];
                gradient(got, g);
                token(raw, g, r < own, done);
                emit(lo + r - (W - 1), done);
            };
            if constexpr (VEC > 1) {
                // through a ring as in the forward
                auto fetch = [&](int r0) {
                    const int to = r0 / kBackGroup % kBackDepth * kBackGroup * kWarps * 32;
#pragma unroll
                    for (int u = 0; u < kBackGroup; ++u) {
                        if (r0 + u < rows) {
                            copy_piece(ring + to + u * kWarps * 32, src);
                            copy_piece(dring + to + u * kWarps * 32, static_cast<const G1 *>(p.dout) + at);
                        }
                        src += p.x_stride;
                        at += p.dout_stride;
                    }
                    cp_async_commit();
                };
#pragma unroll
                for (int g = 0; g < kBackDepth - 1; ++g) fetch(g * kBackGroup);
                uint16_t *dst = static_cast<uint16_t *>(p.out) + (lo - (W - 1)) * p.out_stride + d;
#pragma unroll 1
                for (int r0 = 0; r0 < rows; r0 += kBackGroup) {
                    fetch(r0 + (kBackDepth - 1) * kBackGroup);
                    copies_but<kBackDepth - 1>();
                    const int from = r0 / kBackGroup % kBackDepth * kBackGroup * kWarps * 32;
                    if (r0 >= W - 1 && r0 + kBackGroup <= own) {
#pragma unroll
                        for (int u = 0; u < kBackGroup; ++u) {
                            float g[VEC], done[VEC];
                            gradient(dring[from + u * kWarps * 32], g);
                            token(ring[from + u * kWarps * 32], g, true, done);
                            *reinterpret_cast<R *>(dst + u * p.out_stride) = narrow<VEC>(done);
                        }
                    } else {
#pragma unroll 1
                        for (int u = 0; u < kBackGroup && r0 + u < rows; ++u)
                            one(r0 + u, ring[from + u * kWarps * 32], dring[from + u * kWarps * 32]);
                    }
                    dst += kBackGroup * p.out_stride;
                }
            } else {
#pragma unroll 2
                for (int r = 0; r < rows; ++r) {
                    one(r, *reinterpret_cast<const R *>(src), static_cast<const G1 *>(p.dout)[at]);
                    src += p.x_stride;
                    at += p.dout_stride;
                }
            }
            if (end == b) {   // the rows that final_state holds
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    if (p.dhist_out != nullptr) {
                        float g[VEC];
                        load_f32<VEC>(p.dhist_out + (static_cast<int64_t>(n) * (W - 1) + j) * p.dim + d, g);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) open[j][i] += g[i];
                    }
                    emit(b - (W - 1) + j, open[j]);
                }
            }
        }
    }
    __syncthreads();   // the ring is read
    float *mine = sums[warp];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) mine[j * 32 * VEC + lane * VEC + i] = dw[j][i];
        mine[W * 32 * VEC + lane * VEC + i] = db[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32 * VEC; i += kWarps * 32) {
        const int64_t c = d0 + i % (32 * VEC);
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[w][i];
        if (c < p.dim) p.partial[(tile * (W + 1) + i / (32 * VEC)) * p.dim + c] = s;
    }
}

// dweight and dbias: the tiles' sums, eight interleaved partial sums per
// channel, then those in order.
__global__ void __launch_bounds__(256) conv_reduce_kernel(ConvParams p, int64_t tiles) {
    __shared__ float part[8][32];
    const Seqs seqs{p.cu, p.seq_len, p.n_seqs};
    if (!check_cu(seqs, p.tokens, p.err)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const int j = blockIdx.y;
    float s = 0.f;
    if (d < p.dim)
        for (int64_t t = warp; t < tiles; t += 8) s += p.partial[(t * (p.width + 1) + j) * p.dim + d];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && d < p.dim) {
        float r = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) r += part[w][lane];
        if (j < p.width) p.dweight[d * p.width + j] = r;
        else if (p.dbias != nullptr) p.dbias[d] = r;
    }
}

bool aligned(const void *p, int64_t stride, int64_t bytes, int64_t elem) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * elem % bytes == 0);
}

// Channels per thread: 8 or 4 when every row of every array starts on a
// 16- or 8-byte boundary, else 1. The gradient keeps 4 W + 5 sums and rows per
// channel in registers and takes 4 at most (T = D = 8192: 8 take 291 us).
int conv_vec(const ConvParams &p, int most) {
    for (int v : {8, 4}) {
        const int64_t b = 2 * v;
        if (v <= most && p.dim % v == 0 && aligned(p.x, p.x_stride, b, 2) &&
            aligned(p.out, p.out_stride, b, 2) && aligned(p.hist_in, p.dim, b, 2) &&
            aligned(p.hist_out, p.dim, b, 2) &&
            aligned(p.dout, p.dout_stride, p.dout32 ? 16 : b, p.dout32 ? 4 : 2) &&
            aligned(p.dhist_in, p.dim, 16, 4) && aligned(p.dhist_out, p.dim, 16, 4))
            return v;
    }
    return 1;
}

template <int MOST, typename F>
cudaError_t with_shape(const ConvParams &p, F &&go) {
    auto silu = [&](auto w, auto v) {
        return p.silu ? go(w, v, std::true_type()) : go(w, v, std::false_type());
    };
    auto vec = [&](auto w) {
        const int v = conv_vec(p, MOST);
        if constexpr (MOST == 8)
            if (v == 8) return silu(w, std::integral_constant<int, 8>());
        return v == 4 ? silu(w, std::integral_constant<int, 4>())
                      : silu(w, std::integral_constant<int, 1>());
    };
    switch (p.width) {
        case 2: return vec(std::integral_constant<int, 2>());
        case 3: return vec(std::integral_constant<int, 3>());
        default: return vec(std::integral_constant<int, 4>());
    }
}

int64_t tiles_of(int64_t tokens, int64_t run) {
    const int64_t t = (tokens + run * kWarps - 1) / (run * kWarps);
    return t > 0 ? t : 1;   // no tokens: the histories are still handed on
}

}  // namespace

cudaError_t configure_conv() {
    auto raise = [](auto kernel, int bytes) {
        return bytes > 0 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
                         : cudaSuccess;
    };
    for (int width = 2; width <= 4; ++width)
        for (int vec : {1, 4, 8})
            for (bool silu : {false, true}) {
                ConvParams p{};   // (no arrays: the channels alone choose the form)
                p.width = width;
                p.dim = vec;
                p.silu = silu;
                cudaError_t e = with_shape<8>(p, [&](auto w, auto v, auto s) {
                    constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
                    return raise(conv_kernel<W, VEC, decltype(s)::value>, ring_bytes<VEC>());
                });
                if (e != cudaSuccess) return e;
                e = with_shape<kBackwardVec>(p, [&](auto w, auto v, auto s) {
                    constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
                    constexpr bool S = decltype(s)::value;
                    const cudaError_t r =
                        raise(conv_backward_kernel<W, VEC, S, true>, back_bytes<W, VEC, true>());
                    return r != cudaSuccess
                               ? r : raise(conv_backward_kernel<W, VEC, S, false>, back_bytes<W, VEC, false>());
                });
                if (e != cudaSuccess) return e;
            }
    return cudaSuccess;
}

cudaError_t launch_conv(const ConvParams &p, cudaStream_t stream) {
    if (p.tokens == 0 && p.hist_out == nullptr) return cudaSuccess;
    return with_shape<kForwardVec>(p, [&](auto w, auto v, auto s) {
        constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
        const int64_t cols = (p.dim + 32 * VEC - 1) / (32 * VEC), run = run_for(p.tokens, cols, kRun);
        conv_kernel<W, VEC, decltype(s)::value>
            <<<static_cast<unsigned>(tiles_of(p.tokens, run) * cols), kWarps * 32, ring_bytes<VEC>(), stream>>>(
                p, static_cast<int>(run), cols);
        return cudaGetLastError();
    });
}

cudaError_t launch_conv_step(const ConvParams &p, cudaStream_t stream) {
    return with_shape<8>(p, [&](auto w, auto v, auto s) {
        constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
        const int64_t cols = (p.dim + 32 * VEC - 1) / (32 * VEC);
        const int64_t rows = (p.tokens + kWarps * kStepRows - 1) / (kWarps * kStepRows);
        conv_step_kernel<W, VEC, decltype(s)::value>
            <<<static_cast<unsigned>(rows * cols), kWarps * 32, 0, stream>>>(p, cols);
        return cudaGetLastError();
    });
}

// How the gradient is launched. The scratch is sized from the same plan: the channels per
// block follow from the alignment, and with fewer of them a run can be longer or
// shorter (whole waves), so the tiles of one form say nothing about another's.
ConvBackwardPlan plan_conv_backward(const ConvParams &p) {
    ConvBackwardPlan pl;
    pl.channels = 32 * conv_vec(p, kBackwardVec);
    pl.cols = (p.dim + pl.channels - 1) / pl.channels;
    pl.run = run_for(p.tokens, pl.cols, kBackRun);
    pl.tiles = tiles_of(p.tokens, pl.run);
    pl.scratch_bytes = pl.tiles * (p.width + 1) * p.dim * 4;
    return pl;
}

cudaError_t launch_conv_backward(const ConvParams &p, const ConvBackwardPlan &pl, cudaStream_t stream) {
    const cudaError_t e = with_shape<kBackwardVec>(p, [&](auto w, auto v, auto s) {
        constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
        constexpr bool S = decltype(s)::value;
        if (pl.channels != 32 * VEC) return cudaErrorInvalidValue;   // (another call's plan)
        const unsigned grid = static_cast<unsigned>(pl.tiles * pl.cols);
        const int run = static_cast<int>(pl.run);
        if (p.dout32)
            conv_backward_kernel<W, VEC, S, true>
                <<<grid, kWarps * 32, back_bytes<W, VEC, true>(), stream>>>(p, run, pl.cols);
        else
            conv_backward_kernel<W, VEC, S, false>
                <<<grid, kWarps * 32, back_bytes<W, VEC, false>(), stream>>>(p, run, pl.cols);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((p.dim + 31) / 32), p.width + (p.dbias != nullptr));
    conv_reduce_kernel<<<grid, 256, 0, stream>>>(p, pl.tiles);
    return cudaGetLastError();
}

}  // namespace kda
