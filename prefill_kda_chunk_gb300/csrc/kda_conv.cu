// Short causal convolution, one filter of W = 2..4 taps per channel, with its
// history, its single-token step and its gradient (kda_short_conv*).
//
//   z[t] = bias + sum_j w[j] x[t - (W-1) + j],  y = z / (1 + e^-z) or z
//
// Each element of x is read for one multiply-add per tap, so the operator is
// bound by HBM (4 B per element forward). A thread owns VEC neighbouring
// channels and walks its tokens in order with the last W - 1 rows in
// registers: every row is read once, but for the W - 1 rows in front of each
// warp's run of tokens (which come out of L2). A warp covers 32 * VEC
// channels of one token (512 contiguous bytes at VEC = 8). Sequence ends only
// move the window, so a packed batch runs like one long sequence.

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

// 1 / (1 + e^-z) of two values with one reciprocal: r = 1 / (a b), 1 / a = r b. The
// exponential and the reciprocal share one unit of 16 results a clock and SM, which two
// of each per pair would keep as busy as HBM. e^-z is held at 2^63, so that the
// product stays finite and no channel can reach the other: below z = -43.7 the
// result is 2^-63 instead of something smaller.
__device__ __forceinline__ void sigmoid2(float z0, float z1, float &s0, float &s1) {
    float e0, e1, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(fminf(z0 * -1.44269504f, 63.f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(fminf(z1 * -1.44269504f, 63.f)));
    const float a = 1.f + e0, b = 1.f + e1;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
    s0 = r * b;
    s1 = r * a;
}
template <int VEC>
__device__ __forceinline__ void sigmoids(const float (&z)[VEC], float (&s)[VEC]) {
    if constexpr (VEC == 1) {
        float other;
        sigmoid2(z[0], 0.f, s[0], other);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) sigmoid2(z[i], z[i + 1], s[i], s[i + 1]);
    }
}
template <int VEC>
__device__ __forceinline__ void silu(float (&z)[VEC]) {
    float s[VEC];
    sigmoids<VEC>(z, s);
#pragma unroll
    for (int i = 0; i < VEC; ++i) z[i] *= s[i];
}

// The filters of a block's 32 VEC channels, read once and kept tap by tap in shared
// memory: read from [D, W] by each thread, their scattered sectors cost more than
// the rows (T = D = 8192: 115 us against 57).
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
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float s = f.b[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) s = fmaf(f.w[j][i], win[j][i], s);
        z[i] = fmaf(f.w[W - 1][i], row[i], s);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][i] = win[j + 1][i];
        win[W - 2][i] = row[i];
    }
}

// Rows per warp: enough that the W - 1 rows read twice are few (9 % at 32, out of L2),
// but fewer when the call would leave SMs without a block.
constexpr int kRun = 32, kMinRun = 4;
int64_t run_for(int64_t tokens, int64_t cols) {
    const int64_t blocks = (2 * 152 + cols - 1) / cols;   // along the tokens, two per SM
    int64_t run = (tokens + blocks * kWarps - 1) / (blocks * kWarps);
    run = (run + kMinRun - 1) / kMinRun * kMinRun;
    return run < kMinRun ? kMinRun : run > kRun ? kRun : run;
}

template <int W, int VEC, bool SILU>
__global__ void __launch_bounds__(kWarps * 32, 3)
conv_kernel(ConvParams p, int run, int64_t col_blocks) {
    __shared__ __align__(16) Filters<W, VEC> filters;
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
        using R = typename Raw<VEC>::T;
        const uint16_t *src = static_cast<const uint16_t *>(p.x) + lo * p.x_stride + d;
        uint16_t *dst = static_cast<uint16_t *>(p.out) + lo * p.out_stride + d;
        auto row_out = [&](const R &raw, uint16_t *to) {
            float row[VEC], z[VEC];
            widen<VEC>(raw, row);
            step_window<W, VEC>(f, win, row, z);
            if (SILU) silu<VEC>(z);
            *reinterpret_cast<R *>(to) = narrow<VEC>(z);
        };
        constexpr int U = 8;   // rows in flight
        int left = static_cast<int>(hi - lo);
#pragma unroll 1
        for (; left >= U; left -= U) {
            R raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u] = *reinterpret_cast<const R *>(src);
                src += p.x_stride;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                row_out(raw[u], dst);
                dst += p.out_stride;
            }
        }
#pragma unroll 1
        for (; left > 0; --left) {
            row_out(*reinterpret_cast<const R *>(src), dst);
            src += p.x_stride;
            dst += p.out_stride;
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
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[i] = f.b[i];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float row[VEC];
            widen<VEC>(raw[u][j], row);
#pragma unroll
            for (int i = 0; i < VEC; ++i) z[i] = fmaf(f.w[j][i], row[i], z[i]);
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
template <int W, int VEC, bool SILU, bool D32>
__global__ void __launch_bounds__(kWarps * 32, 2)
conv_backward_kernel(ConvParams p, int run, int64_t col_blocks) {
    __shared__ float sums[kWarps][(W + 1) * VEC * 32];
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
            using R = typename Raw<VEC>::T;
            const uint16_t *src = static_cast<const uint16_t *>(p.x) + lo * p.x_stride + d;
            int64_t at = lo * p.dout_stride + d;
            auto load = [&](R &raw, float (&g)[VEC]) {
                raw = *reinterpret_cast<const R *>(src);
                if constexpr (D32)
                    load_f32<VEC>(static_cast<const float *>(p.dout) + at, g);
                else
                    widen<VEC>(load_row<VEC>(p.dout, at), g);
                src += p.x_stride;
                at += p.dout_stride;
            };
            // token t: dz completes row t - (W - 1), which goes to `done`
            auto token = [&](const R &raw, const float (&g)[VEC], bool own, float (&done)[VEC]) {
                float row[VEC], z[VEC], sg[VEC];
                widen<VEC>(raw, row);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    z[i] = f.b[i];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) z[i] = fmaf(f.w[j][i], win[j][i], z[i]);
                    z[i] = fmaf(f.w[W - 1][i], row[i], z[i]);
                }
                if (SILU) sigmoids<VEC>(z, sg);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float dz = g[i];
                    if (SILU) dz *= sg[i] * (1.f + z[i] * (1.f - sg[i]));
                    done[i] = fmaf(f.w[0][i], dz, open[0][i]);
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) open[j][i] = fmaf(f.w[j + 1][i], dz, open[j + 1][i]);
                    open[W - 2][i] = f.w[W - 1][i] * dz;
                    if (own) {
                        db[i] += dz;
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(dz, win[j][i], dw[j][i]);
                        dw[W - 1][i] = fmaf(dz, row[i], dw[W - 1][i]);
                    }
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) win[j][i] = win[j + 1][i];
                    win[W - 2][i] = row[i];
                }
            };
            int64_t t = lo;
            // the first W - 1 tokens complete rows in front of this run: the history's
#pragma unroll 1
            for (; t < end && t < lo + W - 1; ++t) {
                R raw;
                float g[VEC], done[VEC];
                load(raw, g);
                token(raw, g, t < hi, done);
                emit(t - (W - 1), done);
            }
            constexpr int U = 4;   // rows in flight
            uint16_t *dst = static_cast<uint16_t *>(p.out) + (t - (W - 1)) * p.out_stride + d;
#pragma unroll 1
            for (; t + U <= hi; t += U) {
                R raw[U];
                float g[U][VEC];
#pragma unroll
                for (int u = 0; u < U; ++u) load(raw[u], g[u]);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float done[VEC];
                    token(raw[u], g[u], true, done);
                    *reinterpret_cast<R *>(dst) = narrow<VEC>(done);
                    dst += p.out_stride;
                }
            }
#pragma unroll 1
            for (; t < end; ++t) {
                R raw;
                float g[VEC], done[VEC];
                load(raw, g);
                token(raw, g, t < hi, done);
                emit(t - (W - 1), done);
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

cudaError_t launch_conv(const ConvParams &p, cudaStream_t stream) {
    if (p.tokens == 0 && p.hist_out == nullptr) return cudaSuccess;
    return with_shape<4>(p, [&](auto w, auto v, auto s) {
        constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
        const int64_t cols = (p.dim + 32 * VEC - 1) / (32 * VEC), run = run_for(p.tokens, cols);
        conv_kernel<W, VEC, decltype(s)::value>
            <<<static_cast<unsigned>(tiles_of(p.tokens, run) * cols), kWarps * 32, 0, stream>>>(
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

// Partial sums of the weights' gradients; with 4 channels per thread the runs are the
// shortest.
int64_t conv_backward_tiles(int64_t tokens, int64_t dim) {
    return tiles_of(tokens, run_for(tokens, (dim + 127) / 128));
}

cudaError_t launch_conv_backward(const ConvParams &p, cudaStream_t stream) {
    int64_t tiles = 0;
    const cudaError_t e = with_shape<4>(p, [&](auto w, auto v, auto s) {
        constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
        constexpr bool S = decltype(s)::value;
        const int64_t cols = (p.dim + 32 * VEC - 1) / (32 * VEC), run = run_for(p.tokens, cols);
        tiles = tiles_of(p.tokens, run);
        const unsigned grid = static_cast<unsigned>(tiles * cols);
        if (p.dout32)
            conv_backward_kernel<W, VEC, S, true>
                <<<grid, kWarps * 32, 0, stream>>>(p, static_cast<int>(run), cols);
        else
            conv_backward_kernel<W, VEC, S, false>
                <<<grid, kWarps * 32, 0, stream>>>(p, static_cast<int>(run), cols);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((p.dim + 31) / 32), p.width + (p.dbias != nullptr));
    conv_reduce_kernel<<<grid, 256, 0, stream>>>(p, tiles);
    return cudaGetLastError();
}

}  // namespace kda
