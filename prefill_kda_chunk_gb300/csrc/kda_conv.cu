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

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// The filter of a thread's channels.
template <int W, int VEC>
struct Filter {
    float w[W][VEC], b[VEC];
    __device__ __forceinline__ void load(const ConvParams &p, int64_t d) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = __ldg(p.weight + (d + i) * W + j);
            b[i] = p.bias != nullptr ? __ldg(p.bias + d + i) : 0.f;
        }
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

// Rows per warp: enough that the W - 1 rows read twice are few, but fewer when
// the call is too small to fill the SMs.
constexpr int kRun = 32;

template <int W, int VEC, bool SILU>
__global__ void __launch_bounds__(kWarps * 32)
conv_kernel(ConvParams p, int run, int64_t col_blocks) {
    const Seqs seqs{p.cu, p.seq_len, p.n_seqs};
    if (!check_cu(seqs, p.tokens, p.err)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x / col_blocks;
    const int64_t t0 = (tile * kWarps + warp) * run;
    const int64_t t1 = t0 + run < p.tokens ? t0 + run : p.tokens;
    if (t0 >= p.tokens && t0 > 0) return;
    const int64_t d = ((blockIdx.x % col_blocks) * 32 + lane) * VEC;
    int n = first_seq(seqs, t0);
    if (d >= p.dim) return;
    Filter<W, VEC> f;
    f.load(p, d);
    for (; n < p.n_seqs; ++n) {
        const int64_t a = seqs.start(n), b = seqs.start(n + 1);
        if (a >= t1 && t1 < p.tokens) break;
        const int64_t lo = a > t0 ? a : t0, hi = b < t1 ? b : t1;
        float win[W - 1][VEC];
        load_window<W, VEC>(p, n, a, lo, d, win);
        constexpr int U = 8;   // rows in flight
        for (int64_t t = lo; t < hi; t += U) {
            typename Raw<VEC>::T raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < hi) raw[u] = load_row<VEC>(p.x, (t + u) * p.x_stride + d);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= hi) break;
                float row[VEC], z[VEC];
                widen<VEC>(raw[u], row);
                step_window<W, VEC>(f, win, row, z);
                if (SILU) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) z[i] *= sigmoid(z[i]);
                }
                *reinterpret_cast<typename Raw<VEC>::T *>(static_cast<uint16_t *>(p.out) +
                                                          (t + u) * p.out_stride + d) = narrow<VEC>(z);
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

// One token per sequence: a thread owns VEC channels of one sequence, reads its
// W rows and writes one row of out and the shifted history. Every address it
// writes was read by the same thread before, so the history may be updated in
// place.
template <int W, int VEC, bool SILU>
__global__ void __launch_bounds__(256) conv_step_kernel(ConvParams p, int64_t cols) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.tokens * cols) return;
    const int64_t n = i / cols, d = (i % cols) * VEC;
    float win[W - 1][VEC], row[VEC], z[VEC];
    const auto raw = load_row<VEC>(p.x, n * p.x_stride + d);
    const int64_t h = n * (W - 1) * p.dim + d;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (p.hist_in != nullptr) {
            widen<VEC>(load_row<VEC>(p.hist_in, h + j * p.dim), win[j]);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) win[j][k] = 0.f;
        }
    }
    Filter<W, VEC> f;
    f.load(p, d);
    widen<VEC>(raw, row);
    step_window<W, VEC>(f, win, row, z);
    if (SILU) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) z[k] *= sigmoid(z[k]);
    }
    *reinterpret_cast<typename Raw<VEC>::T *>(static_cast<uint16_t *>(p.out) + n * p.out_stride + d) =
        narrow<VEC>(z);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        *reinterpret_cast<typename Raw<VEC>::T *>(static_cast<uint16_t *>(p.hist_out) + h + j * p.dim) =
            narrow<VEC>(win[j]);
}

// The gradient walks the same runs. At token t, dz_t completes dx of row
// t - (W-1); the W - 1 rows still open wait in `open` (open[i]: row
// t - (W-1) + 1 + i). A run goes on W - 1 tokens past its own to complete its
// last rows, and its weight sums take its own tokens only. The sums of the
// eight warps are joined in shared memory in warp order and written per tile;
// conv_reduce_kernel adds the tiles in order, so the result does not depend on
// timing.
template <int W, int VEC, bool SILU, bool D32>
__global__ void __launch_bounds__(kWarps * 32)
conv_backward_kernel(ConvParams p, int64_t col_blocks) {
    __shared__ float sums[kWarps][(W + 1) * VEC * 32];
    const Seqs seqs{p.cu, p.seq_len, p.n_seqs};
    if (!check_cu(seqs, p.tokens, p.err)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x / col_blocks;
    const int64_t t0 = (tile * kWarps + warp) * kRun;
    const int64_t t1 = t0 + kRun < p.tokens ? t0 + kRun : p.tokens;
    const int64_t d0 = (blockIdx.x % col_blocks) * 32 * VEC, d = d0 + lane * VEC;
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
        Filter<W, VEC> f;
        f.load(p, d);
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
            constexpr int U = 4;   // rows in flight
            for (int64_t t = lo; t < end; t += U) {
                typename Raw<VEC>::T raw[U];
                float g[U][VEC];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (t + u < end) {
                        raw[u] = load_row<VEC>(p.x, (t + u) * p.x_stride + d);
                        const int64_t at = (t + u) * p.dout_stride + d;
                        if constexpr (D32)
                            load_f32<VEC>(static_cast<const float *>(p.dout) + at, g[u]);
                        else
                            widen<VEC>(load_row<VEC>(p.dout, at), g[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (t + u >= end) break;
                    const bool own = t + u < hi;
                    float row[VEC], z[VEC], done[VEC];
                    widen<VEC>(raw[u], row);
                    float taps[W - 1][VEC];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) taps[j][i] = win[j][i];
                    step_window<W, VEC>(f, win, row, z);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        float dz = g[u][i];
                        if (SILU) {
                            const float s = sigmoid(z[i]);
                            dz *= s * (1.f + z[i] * (1.f - s));
                        }
                        done[i] = fmaf(f.w[0][i], dz, open[0][i]);
#pragma unroll
                        for (int j = 0; j + 1 < W - 1; ++j)
                            open[j][i] = fmaf(f.w[j + 1][i], dz, open[j + 1][i]);
                        open[W - 2][i] = f.w[W - 1][i] * dz;
                        if (own) {
                            db[i] += dz;
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(dz, taps[j][i], dw[j][i]);
                            dw[W - 1][i] = fmaf(dz, row[i], dw[W - 1][i]);
                        }
                    }
                    emit(t + u - (W - 1), done);
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
// 16- or 8-byte boundary, else 1.
int conv_vec(const ConvParams &p) {
    for (int v : {8, 4}) {
        const int64_t b = 2 * v;
        if (p.dim % v == 0 && aligned(p.x, p.x_stride, b, 2) && aligned(p.out, p.out_stride, b, 2) &&
            aligned(p.hist_in, p.dim, b, 2) && aligned(p.hist_out, p.dim, b, 2) &&
            aligned(p.dout, p.dout_stride, p.dout32 ? 16 : b, p.dout32 ? 4 : 2) &&
            aligned(p.dhist_in, p.dim, 16, 4) && aligned(p.dhist_out, p.dim, 16, 4))
            return v;
    }
    return 1;
}

template <typename F>
cudaError_t with_shape(const ConvParams &p, F &&go) {
    auto silu = [&](auto w, auto v) {
        return p.silu ? go(w, v, std::true_type()) : go(w, v, std::false_type());
    };
    auto vec = [&](auto w) {
        switch (conv_vec(p)) {
            case 8: return silu(w, std::integral_constant<int, 8>());
            case 4: return silu(w, std::integral_constant<int, 4>());
            default: return silu(w, std::integral_constant<int, 1>());
        }
    };
    switch (p.width) {
        case 2: return vec(std::integral_constant<int, 2>());
        case 3: return vec(std::integral_constant<int, 3>());
        default: return vec(std::integral_constant<int, 4>());
    }
}

}  // namespace

cudaError_t launch_conv(const ConvParams &p, cudaStream_t stream) {
    return with_shape(p, [&](auto w, auto v, auto s) {
        constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
        const int64_t cols = (p.dim + 32 * VEC - 1) / (32 * VEC);
        const int run = kRun;
        int64_t tiles = (p.tokens + run * kWarps - 1) / (run * kWarps);
        if (tiles == 0) tiles = 1;   // no tokens: the histories are still handed on
        if (p.tokens == 0 && p.hist_out == nullptr) return cudaSuccess;
        conv_kernel<W, VEC, decltype(s)::value>
            <<<static_cast<unsigned>(tiles * cols), kWarps * 32, 0, stream>>>(p, run, cols);
        return cudaGetLastError();
    });
}

cudaError_t launch_conv_step(const ConvParams &p, cudaStream_t stream) {
    return with_shape(p, [&](auto w, auto v, auto s) {
        constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
        const int64_t cols = (p.dim + VEC - 1) / VEC;
        conv_step_kernel<W, VEC, decltype(s)::value>
            <<<static_cast<unsigned>((p.tokens * cols + 255) / 256), 256, 0, stream>>>(p, cols);
        return cudaGetLastError();
    });
}

int64_t conv_backward_tiles(int64_t tokens) {
    const int64_t t = (tokens + kRun * kWarps - 1) / (kRun * kWarps);
    return t > 0 ? t : 1;
}

cudaError_t launch_conv_backward(const ConvParams &p, cudaStream_t stream) {
    const int64_t tiles = conv_backward_tiles(p.tokens);
    const cudaError_t e = with_shape(p, [&](auto w, auto v, auto s) {
        constexpr int W = decltype(w)::value, VEC = decltype(v)::value;
        constexpr bool S = decltype(s)::value;
        const int64_t cols = (p.dim + 32 * VEC - 1) / (32 * VEC);
        const unsigned grid = static_cast<unsigned>(tiles * cols);
        if (p.dout32)
            conv_backward_kernel<W, VEC, S, true><<<grid, kWarps * 32, 0, stream>>>(p, cols);
        else
            conv_backward_kernel<W, VEC, S, false><<<grid, kWarps * 32, 0, stream>>>(p, cols);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((p.dim + 31) / 32), p.width + (p.dbias != nullptr));
    conv_reduce_kernel<<<grid, 256, 0, stream>>>(p, tiles);
    return cudaGetLastError();
}

}  // namespace kda
