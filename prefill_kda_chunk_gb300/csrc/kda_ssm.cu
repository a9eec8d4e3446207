// Selective state space scan with one decay per head (kda_ssm_prefill) and
// its single-token step (kda_ssm_step).
//
//   S_t = exp(a delta_t) S_{t-1} + delta_t b_t x_t^T,   y_t = S_t^T c_t + d x_t
//
// S is n x P per (sequence, head), fp32; b and c are shared by the heads of a
// group.
//
// The prompt is taken in chunks of 128 tokens. With G the running sum of
// a delta log2(e) inside a chunk (G_t <= 0, token t included) and S the state
// that enters it,
//
//   y_t = 2^G_t (S^T c_t) + sum_{s <= t} (c_t . b_s) 2^(G_t - G_s) delta_s x_s + d x_t
//   S'  = 2^G_last S + sum_s b_s (2^(G_last - G_s) delta_s x_s)^T
//
// so a chunk of one head is four products, all on the 5th-generation tensor
// core with bf16 operands from shared memory (TMA, 128-byte swizzle) and fp32
// accumulators in tensor memory: C B^T (128 x 128 x n), M X with
// M = (C B^T) . decay, C S, and B^T (W X). b, c and x are bf16 as given, so
// what the products round is only what this kernel makes: M and S enter as two
// bf16 terms (16 bits of mantissa, well below the bf16 output's rounding), and
// the weighted rows W X as three (24 bits: the state is an fp32 result and
// keeps fp32's precision over any length).
//
// Every exponent is a difference of running sums kept as two floats, so it is
// as exact next to a token that forgets everything (G falls by thousands) as
// anywhere; between 32-token blocks it is split at the block's end into two
// factors <= 1, so only the diagonal blocks take an exponential per pair.
//
// Work split. The (head, 64 of P) units and chunks form one list, and CTA c
// of G (one per SM) takes an equal run of it, a run of chunks of one sequence
// after the other. Where a run starts in the middle of a sequence, its entry
// state comes from a launch before (kStates): there each CTA whose run ends in
// the middle of a sequence forms the state that its part of that sequence
// leaves (the state product only), and the CTAs behind add up what they need.

#include <cuda.h>

#include "kda_device.cuh"
#include "kda_internal.h"
#include "kda_seqs.cuh"
#include "kda_tcgen05.cuh"

#include <type_traits>

namespace kda {

namespace {

__device__ __forceinline__ float bf16_at(const void *p, int64_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ float delta_of(const SsmParams &p, int64_t t, int h) {
    float v = p.dt[t * p.dt_stride + h];
    if (p.dt_bias != nullptr) v += __ldg(p.dt_bias + h);
    // log(1 + e^v) without overflow, and exact for large negative v
    return p.softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
}

// ------------------------------------------------------------- one token

// One block per (sequence, head): thread (q, j) keeps S[j * kN / kParts ..][q].
template <int kN, int kP>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmParams p) {
    constexpr int kParts = 256 / kP, kRows = kN / kParts;
    __shared__ float s_b[kN], s_c[kN], s_y[kParts][kP];
    const int n = blockIdx.x / p.heads, h = blockIdx.x % p.heads, g = h / (p.heads / p.groups);
    const int q = threadIdx.x % kP, j = threadIdx.x / kP;
    const int64_t st = (static_cast<int64_t>(n) * p.heads + h) * kN * kP + j * kRows * kP + q;
    float s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = p.s0 != nullptr ? p.s0[st + i * kP] : 0.f;
    const float av = __ldg(p.a + h), dv = p.d != nullptr ? __ldg(p.d + h) : 0.f;
    if (threadIdx.x < kN) {
        s_b[threadIdx.x] = bf16_at(p.b, n * p.b_stride + g * kN + threadIdx.x);
        s_c[threadIdx.x] = bf16_at(p.c, n * p.c_stride + g * kN + threadIdx.x);
    }
    const float delta = delta_of(p, n, h), decay = expf(av * delta);
    const float x = bf16_at(p.x, n * p.x_stride + h * kP + q);
    __syncthreads();
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        s[i] = fmaf(s[i], decay, delta * x * s_b[j * kRows + i]);
        y = fmaf(s[i], s_c[j * kRows + i], y);
        p.s_final[st + i * kP] = s[i];
    }
    s_y[j][q] = y;
    __syncthreads();
    if (j == 0) {
        for (int k = 1; k < kParts; ++k) y += s_y[k][q];
        static_cast<__nv_bfloat16 *>(p.out)[(static_cast<int64_t>(n) * p.heads + h) * kP + q] =
            __float2bfloat16_rn(fmaf(dv, x, y));
    }
}

// --------------------------------------------------------------- a prompt

constexpr int kL = 128;              // tokens per chunk
constexpr int kPS = 64;              // channels of P per unit
constexpr int kSsmSms = 152;
constexpr int kCompute = 256;        // threads of the eight compute warps
constexpr int kThreads = kCompute + 64;   // and the control and scalar warps

// Shared memory, from a 1024-byte boundary. Tiles of 128-byte rows with the
// 16-byte granule index XOR-ed by the row's low three bits.
constexpr int kOffC = 0;                         // [n / 64][128 tokens][64]
constexpr int kOffB = 32768;                     // two buffers of the same
constexpr int kOffX = kOffB + 2 * 32768;         // two buffers of [128 tokens][64]
constexpr int kOffW = kOffX + 2 * 16384;         // three terms of the weighted rows
constexpr int kOffS = kOffW + 3 * 16384;         // two terms of the state, [n][64]
constexpr int kOffSc = kOffS + 2 * 16384;        // two buffers of Scalars
struct Scalars {
    float hi[kL], lo[kL];   // G_t as a sum of two floats, in units of log 2
    float dt[kL];           // delta_t; 0 past the sequence's end
    float to_block[kL];     // 2^(G at the end of t's 32-block - G_t) delta_t
    float to_end[kL];       // 2^(G_last - G_t) delta_t
    float from[kL];         // 2^G_t
    float end_hi[4], end_lo[4];   // G at the end of each 32-block
    float decay, pad[7];    // 2^G_last
};
constexpr int kOffBar = kOffSc + 2 * static_cast<int>(sizeof(Scalars));
enum {   // barriers, 8 bytes each
    kFullC, kFullBX, kScal = kFullBX + 2, kCB = kScal + 2, kCSDS, kMX, kMReady, kSReady, kWReady,
    kDone, kDrain, kBars
};
constexpr int kSmem = kOffBar + 8 * kBars + 1024;

// Tensor memory columns.
constexpr uint32_t kTmCB = 0, kTmM = 128, kTmY = 256, kTmCS = 320, kTmDS = 384, kTmCols = 512;

// ---- instruction and shared-memory descriptors (bf16, fp32 accumulate)
constexpr uint32_t kAMajor = 1u << 15, kBMajor = 1u << 16;   // operand contiguous along M / N
// 128-byte swizzled tiles, eight rows of 128 bytes per atom. Contiguous along
// K: sbo = step between 8-row groups. Contiguous along M or N: sbo = step
// between groups of 8 along K, lbo = step between blocks of 64 along M / N.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return tc::sdesc(saddr, lbo, sbo) | (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (a, b) as two bf16 terms: hi + lo
__device__ __forceinline__ uint32_t split2(float a, float b, uint32_t &lo) {
    const uint32_t h = pack_bf16(a, b);
    const float2 f = unpack_bf16(h);
    lo = pack_bf16(a - f.x, b - f.y);
    return h;
}

struct SsmMaps {
    CUtensorMap x, b, c;   // [tokens][channels], boxes of 128 tokens x 64 channels
};

struct SsmPlan {
    int slices;                // units per head
    int cps;                   // chunks per sequence (fixed lengths)
    int64_t units;             // heads * slices
    const int32_t *chunk_off;  // packed: first chunk of each sequence [N + 1]
    const int *call_flags;     // packed: set by the prologue
    int64_t gran;              // chunks that stay together; 0: all of a unit's
    float *slots;              // [G][32][256] states at the cuts
    float *saved;              // the same: initial states that a cut run starts from (in place)
    float *decay;              // [G]
    bool in_place;
};

// The list of (unit, chunk) and the run of it that a CTA takes.
struct List {
    int64_t nc, W, gran, G;
    __device__ __forceinline__ List(const SsmParams &p, const SsmPlan &pl) {
        nc = pl.chunk_off != nullptr ? __ldg(pl.chunk_off + p.n_seqs)
                                     : static_cast<int64_t>(pl.cps) * p.n_seqs;
        W = pl.units * nc;
        gran = pl.gran > 0 ? pl.gran : nc > 0 ? nc : 1;
        const int64_t m = W / gran;
        G = m < gridDim.x ? m : gridDim.x;
    }
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * (W / gran) / G * gran; }
};

// A place in the list.
struct Walk {
    int u, n, pos;      // unit, sequence, chunk of the sequence
    int64_t ch, tok;    // chunk of the unit; the sequence's first token
    int len;            // the sequence's tokens
    __device__ __forceinline__ void at_seq(const SsmParams &p, const SsmPlan &pl) {
        if (pl.chunk_off != nullptr) {
            tok = __ldg(p.cu + n);
            len = __ldg(p.cu + n + 1) - static_cast<int>(tok);
        } else {
            tok = p.seq_len * n;
            len = static_cast<int>(p.seq_len);
        }
    }
    __device__ __forceinline__ void go(const SsmParams &p, const SsmPlan &pl, int64_t nc, int64_t q) {
        u = static_cast<int>(q / nc);
        ch = q % nc;
        if (pl.chunk_off != nullptr) {
            int lo = 0, hi = p.n_seqs;   // last sequence with chunk_off <= ch
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(pl.chunk_off + mid) <= ch) lo = mid;
                else hi = mid;
            }
            n = lo;
            pos = static_cast<int>(ch - __ldg(pl.chunk_off + n));
        } else {
            n = static_cast<int>(ch / pl.cps);
            pos = static_cast<int>(ch % pl.cps);
        }
        at_seq(p, pl);
    }
    __device__ __forceinline__ void next(const SsmParams &p, const SsmPlan &pl, int64_t nc) {
        ++ch;
        ++pos;
        if (pos * kL < len) return;
        pos = 0;
        if (ch == nc) {
            ++u;
            ch = 0;
            n = -1;
        }
        do {   // (sequences without tokens have no chunk)
            ++n;
            if (n >= p.n_seqs) return;   // past the list's end
            at_seq(p, pl);
        } while (len == 0);
    }
    __device__ __forceinline__ bool last() const { return (pos + 1) * kL >= len; }
    __device__ __forceinline__ int valid() const { return min(kL, len - pos * kL); }
    __device__ __forceinline__ int64_t row() const { return tok + static_cast<int64_t>(pos) * kL; }
};

// The states of sequences without tokens are handed on.
template <int kN>
__device__ __forceinline__ void hand_on(const SsmParams &p, int thread, int threads) {
    if (p.s_final == nullptr) return;
    const Seqs seqs{p.cu, p.seq_len, p.n_seqs};
    const int64_t size = static_cast<int64_t>(p.heads) * kN * p.p / 4;
    for (int n = blockIdx.x; n < p.n_seqs; n += gridDim.x) {
        if (seqs.start(n + 1) != seqs.start(n)) continue;
        for (int64_t i = thread; i < size; i += threads) {
            const int64_t at = n * size + i;
            reinterpret_cast<float4 *>(p.s_final)[at] =
                p.s0 != nullptr ? reinterpret_cast<const float4 *>(p.s0)[at] : make_float4(0, 0, 0, 0);
        }
    }
}

template <int kN>
__global__ void __launch_bounds__(256) ssm_hand_on_kernel(SsmParams p) {
    const Seqs seqs{p.cu, p.seq_len, p.n_seqs};
    if (!check_cu(seqs, p.tokens, p.err)) return;
    hand_on<kN>(p, threadIdx.x, 256);
}

template <int kN, bool kStates>
__global__ void __launch_bounds__(kThreads, 1)
ssm_chunk_kernel(const __grid_constant__ SsmMaps maps, SsmParams p, SsmPlan pl) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    if (pl.call_flags != nullptr && (*pl.call_flags & kErrBadCu) != 0) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!kStates && tid < kCompute) hand_on<kN>(p, tid, kCompute);
    const List list(p, pl);
    const int c = blockIdx.x;
    if (c >= list.G) return;
    int64_t q0 = list.begin(c);
    const int64_t q1 = list.begin(c + 1);
    if (kStates) {   // only the part of the sequence that the end of the run cuts
        if (q1 >= list.W) return;
        Walk w;
        w.go(p, pl, list.nc, q1);
        if (w.pos == 0) return;
        if (q1 - w.pos > q0) q0 = q1 - w.pos;
    }
    const int count = static_cast<int>(q1 - q0);

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    const auto bar = [&](int i) { return sb + kOffBar + 8 * i; };
    Scalars *scal = reinterpret_cast<Scalars *>(smem + kOffSc);

    if (tid == 0) {
        s_abort = 0;
        for (int i : {static_cast<int>(kFullC), kFullBX + 0, kFullBX + 1, kScal + 0, kScal + 1,
                      static_cast<int>(kCB), static_cast<int>(kCSDS), static_cast<int>(kMX),
                      static_cast<int>(kDrain)})
            mbar_init(bar(i), 1);
        for (int i : {kMReady, kSReady, kWReady, kDone}) mbar_init(bar(i), kCompute);
        mbar_fence_init();
    }
    if (warp == 0) {
        tc::alloc(smem_u32(&s_tmem), kTmCols);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = s_tmem;

    // A bounded wait; once one has run out, all of them give up.
    auto wait = [&](int i, int phase) -> bool {
        if (s_abort == 0 && mbar_wait(bar(i), phase & 1)) return true;
        s_abort = 1;
        atomicOr(p.err, kErrTimeout);
        return false;
    };

    Walk w;
    w.go(p, pl, list.nc, q0);
    const int per_group = p.heads / p.groups;

    if (warp == 8) {
        // ------------------------------------------- control: copies and MMAs
        if (lane == 0) {
            Walk l = w;     // the next chunk whose b and x are copied
            int issued = 0, issued_c = 0, seen_c = 0, seen = 0;
            auto copy_bx = [&]() {
                const int h = l.u / pl.slices, s = issued & 1;
                const int row = static_cast<int>(l.row());
                mbar_arrive_expect_tx(bar(kFullBX + s), kL * 2 * (kN + kPS));
#pragma unroll
                for (int k = 0; k < kN / 64; ++k)
                    tma_2d(sb + kOffB + s * 32768 + k * 16384, &maps.b, (h / per_group) * kN + 64 * k, row,
                           bar(kFullBX + s));
                tma_2d(sb + kOffX + s * 16384, &maps.x, h * p.p + (l.u % pl.slices) * kPS, row,
                       bar(kFullBX + s));
                ++issued;
                l.next(p, pl, list.nc);
            };
            auto copy_c = [&](const Walk &v) {
                const int h = v.u / pl.slices, row = static_cast<int>(v.row());
                mbar_arrive_expect_tx(bar(kFullC), kL * 2 * kN);
#pragma unroll
                for (int k = 0; k < kN / 64; ++k)
                    tma_2d(sb + kOffC + k * 16384, &maps.c, (h / per_group) * kN + 64 * k, row, bar(kFullC));
                ++issued_c;
            };
            if (!kStates) copy_c(w);
            copy_bx();
            if (count > 1) copy_bx();
            for (int i = 0; i < count; ++i) {
                const uint32_t B = sb + kOffB + (i & 1) * 32768, X = sb + kOffX + (i & 1) * 16384;
                const uint32_t C = sb + kOffC, W = sb + kOffW, S = sb + kOffS;
                if (!wait(kFullBX + (i & 1), i >> 1)) break;
                ++seen;
                if (!kStates) {
                    if (!wait(kFullC, i)) break;
                    ++seen_c;
                    tc::fence_after();
                    // C B^T
#pragma unroll
                    for (int k = 0; k < kN / 16; ++k) {
                        const uint32_t o = (k >> 2) * 16384 + (k & 3) * 32;
                        mma_ss(tm + kTmCB, desc128(C + o, 16, 1024), desc128(B + o, 16, 1024),
                               tc::idesc(128, 128, 1), k > 0);
                    }
                    tc::commit(bar(kCB));
                }
                if (i > 0) {
                    // the outputs of the chunk before are read, its buffers free
                    if (!wait(kDone, i - 1)) break;
                    if (issued < count) copy_bx();
                }
                if (!wait(kWReady, i)) break;
                if (!kStates && !wait(kSReady, i)) break;
                tc::fence_after();
                if (!kStates) {
                    // C S, both terms of S
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < kN / 16; ++k)
                            mma_ss(tm + kTmCS, desc128(C + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024),
                                   desc128(S + t * 16384 + k * 2048, 16384, 1024),
                                   tc::idesc(128, kPS, 1) | kBMajor, t + k > 0);
                }
                // B^T (W X), the three terms of W X, the smallest first (for
                // n = 64 the upper 64 rows are formed from whatever lies there
                // and are not read)
#pragma unroll
                for (int t = 2; t >= 0; --t)
#pragma unroll
                    for (int k = 0; k < kL / 16; ++k)
                        mma_ss(tm + kTmDS, desc128(B + k * 2048, 16384, 1024),
                               desc128(W + t * 16384 + k * 2048, 16384, 1024),
                               tc::idesc(128, kPS, 1) | kAMajor | kBMajor, t < 2 || k > 0);
                tc::commit(bar(kCSDS));
                if (!kStates) {
                    if (!wait(kMReady, i)) break;
                    tc::fence_after();
                    // M X, both terms of M
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < kL / 16; ++k)
                            tc::mma_bf16_ts(tm + kTmY, tm + kTmM + t * 64 + k * 8,
                                            desc128(X + k * 2048, 16384, 1024),
                                            tc::idesc(128, kPS, 1) | kBMajor, t + k > 0);
                    tc::commit(bar(kMX));
                    if (i + 1 < count) {
                        if (!wait(kCSDS, i)) break;   // C is free
                        w.next(p, pl, list.nc);
                        copy_c(w);
                    }
                }
            }
            // what is still in flight after a wait that gave up: let it land
            for (; seen < issued; ++seen) mbar_wait(bar(kFullBX + (seen & 1)), (seen >> 1) & 1);
            for (; seen_c < issued_c; ++seen_c) mbar_wait(bar(kFullC), seen_c & 1);
            if (s_abort != 0) {
                tc::commit(bar(kDrain));
                mbar_wait(bar(kDrain), 0);
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        // --------------------------------- scalars: the decays of each chunk
        for (int i = 0; i < count; ++i) {
            if (i >= 2 && !wait(kDone, i - 2)) break;
            Scalars &s = scal[i & 1];
            const int h = w.u / pl.slices, valid = w.valid();
            const float a2 = __ldg(p.a + h) * 1.44269504088896341f;
            float dt[4];
            double g[4], sum = 0.0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * lane + j;
                dt[j] = t < valid ? delta_of(p, w.row() + t, h) : 0.f;
                sum += t < valid ? static_cast<double>(a2 * dt[j]) : 0.0;
                g[j] = sum;
            }
            double incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const double before = incl - sum;
            const double block = __shfl_sync(0xffffffffu, incl, lane | 7);
            const double end = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * lane + j;
                const double G = before + g[j];
                const float hi = static_cast<float>(G);
                s.hi[t] = hi;
                s.lo[t] = static_cast<float>(G - hi);
                s.dt[t] = dt[j];
                s.to_block[t] = exp2f(static_cast<float>(block - G)) * dt[j];
                s.to_end[t] = exp2f(static_cast<float>(end - G)) * dt[j];
                s.from[t] = exp2f(hi);
            }
            if ((lane & 7) == 7) {
                const float hi = static_cast<float>(block);
                s.end_hi[lane >> 3] = hi;
                s.end_lo[lane >> 3] = static_cast<float>(block - hi);
            }
            if (lane == 31) s.decay = exp2f(static_cast<float>(end));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kScal + (i & 1)));
            w.next(p, pl, list.nc);
        }
    } else {
        // ------------------------------------------------------------ compute
        // rows: token (M, Y) or state row (S) 32 q + lane; columns: the half hf
        const int q = warp & 3, hf = warp >> 2, r = 32 * q + lane;
        const uint32_t lanes = tm + (static_cast<uint32_t>(32 * q) << 16);
        const int srow = tid & (kL - 1), sh = tid >> 7;   // weighted rows: row and half
        float S[32];
        const bool has = r < kN;

        if (!kStates && hf == 0) {   // blocks above the diagonal stay zero
            const uint32_t z[16] = {};
            for (int b = q + 1; b < 4; ++b) {
                tc::st16(lanes + kTmM + 16 * b, z);
                tc::st16(lanes + kTmM + 64 + 16 * b, z);
            }
            tc::st_wait();
        }
        // this thread's 32 values in the state array
        auto state_at = [&](const Walk &v) {
            return ((static_cast<int64_t>(v.n) * p.heads + v.u / pl.slices) * kN + r) * p.p +
                   (v.u % pl.slices) * kPS + 32 * hf;
        };
        // ... and in the slots at the cuts
        const int64_t slot = static_cast<int64_t>(c) * 32 * kCompute + tid;
        // The state that enters chunk i of the run (its first, or a sequence's first).
        auto start_state = [&](const Walk &v, int i) {
#pragma unroll
            for (int j = 0; j < 32; ++j) S[j] = 0.f;
            if (v.pos > 0) {
                if (kStates) return;   // only what this part adds
                // what the runs in front left of this sequence, the nearest first
                const int64_t head = q0 - v.pos;
                float f = 1.f;
                for (int k = c - 1; k >= 0; --k) {
                    const float *src = pl.slots + static_cast<int64_t>(k) * 32 * kCompute + tid;
#pragma unroll
                    for (int j = 0; j < 32; ++j) S[j] = fmaf(src[j * kCompute], f, S[j]);
                    if (list.begin(k) <= head) break;
                    f *= pl.decay[k];
                }
                return;
            }
            if (p.s0 == nullptr) return;
            // in place, another CTA overwrites the initial state of a sequence
            // that the end of this run cuts: the first launch took a copy
            const bool cut = q0 + i + (v.len + kL - 1) / kL > q1;
            if (!kStates && pl.in_place && cut) {
#pragma unroll
                for (int j = 0; j < 32; ++j) S[j] = pl.saved[slot + j * kCompute];
                return;
            }
            if (has) {
                const float4 *src = reinterpret_cast<const float4 *>(p.s0 + state_at(v));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 f = src[j];
                    S[4 * j] = f.x; S[4 * j + 1] = f.y; S[4 * j + 2] = f.z; S[4 * j + 3] = f.w;
                }
            }
            if (kStates && pl.in_place) {
#pragma unroll
                for (int j = 0; j < 32; ++j) pl.saved[slot + j * kCompute] = S[j];
            }
        };
        // S as two bf16 terms for C S
        auto put_state = [&]() {
            if (!kStates && has) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint4 hi, lo;
                    hi.x = split2(S[8 * k], S[8 * k + 1], lo.x);
                    hi.y = split2(S[8 * k + 2], S[8 * k + 3], lo.y);
                    hi.z = split2(S[8 * k + 4], S[8 * k + 5], lo.z);
                    hi.w = split2(S[8 * k + 6], S[8 * k + 7], lo.w);
                    const int at = r * 128 + (((4 * hf + k) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4 *>(smem + kOffS + at) = hi;
                    *reinterpret_cast<uint4 *>(smem + kOffS + 16384 + at) = lo;
                }
            }
            fence_async();
            mbar_arrive(bar(kSReady));
        };
        // The weighted rows of chunk i as three bf16 terms. Rows past the end of
        // the sequence belong to another one: they are zeroed here, as no weight
        // of 0 makes an infinity or NaN vanish.
        auto put_rows = [&](int i, int valid) {
            uint8_t *X = smem + kOffX + (i & 1) * 16384, *W = smem + kOffW;
            const float wt = scal[i & 1].to_end[srow];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = srow * 128 + (((4 * sh + k) ^ (srow & 7)) << 4);
                uint4 x = *reinterpret_cast<const uint4 *>(X + at);
                if (srow >= valid) {
                    x = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(X + at) = x;
#pragma unroll
                    for (int m = 0; m < kN / 64; ++m)
                        *reinterpret_cast<uint4 *>(smem + kOffB + (i & 1) * 32768 + m * 16384 + at) = x;
                }
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t t0[4], t1[4], t2[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 v = unpack_bf16(xs[e]);
                    mul2(v.x, v.y, wt, wt);
                    t0[e] = pack_bf16(v.x, v.y);
                    const float2 f = unpack_bf16(t0[e]);
                    t1[e] = split2(v.x - f.x, v.y - f.y, t2[e]);
                }
                *reinterpret_cast<uint4 *>(W + at) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
                *reinterpret_cast<uint4 *>(W + 16384 + at) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                *reinterpret_cast<uint4 *>(W + 32768 + at) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
            }
            fence_async();
            mbar_arrive(bar(kWReady));
        };

        float run_decay = 1.f;   // over this part of the sequence
        start_state(w, 0);
        put_state();
        bool ok = wait(kScal, 0) && wait(kFullBX, 0);
        if (ok) put_rows(0, w.valid());
        for (int i = 0; ok && i < count; ++i) {
            const Scalars &s = scal[i & 1];
            const int valid = w.valid();
            if (!kStates) {
                // ---- M = (C B^T) . decay, two bf16 terms
                if (!(ok = wait(kCB, i))) break;
                tc::fence_after();
                const float hi_r = s.hi[r], lo_r = s.lo[r];
                for (int b = hf; b <= q; b += 2) {
                    uint32_t v[2][16];
                    tc::ld16(lanes + kTmCB + 32 * b, v[0]);
                    tc::ld16(lanes + kTmCB + 32 * b + 16, v[1]);
                    tc::ld_wait();
                    uint32_t hi[16], lo[16];
                    if (b < q) {
                        const float f = ex2((hi_r - s.end_hi[b]) + (lo_r - s.end_lo[b]));
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 e = *reinterpret_cast<const float4 *>(s.to_block + 32 * b + j);
                            float m0 = __uint_as_float(v[j >> 4][j & 15]);
                            float m1 = __uint_as_float(v[j >> 4][(j & 15) + 1]);
                            float m2 = __uint_as_float(v[j >> 4][(j & 15) + 2]);
                            float m3 = __uint_as_float(v[j >> 4][(j & 15) + 3]);
                            mul2(m0, m1, f, f);
                            mul2(m2, m3, f, f);
                            mul2(m0, m1, e.x, e.y);
                            mul2(m2, m3, e.z, e.w);
                            hi[j / 2] = split2(m0, m1, lo[j / 2]);
                            hi[j / 2 + 1] = split2(m2, m3, lo[j / 2 + 1]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const int t = 32 * b + j;
                            const float4 gh = *reinterpret_cast<const float4 *>(s.hi + t);
                            const float4 gl = *reinterpret_cast<const float4 *>(s.lo + t);
                            const float4 d = *reinterpret_cast<const float4 *>(s.dt + t);
                            const float ghs[4] = {gh.x, gh.y, gh.z, gh.w}, gls[4] = {gl.x, gl.y, gl.z, gl.w};
                            const float ds[4] = {d.x, d.y, d.z, d.w};
                            float m[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x = __uint_as_float(v[j >> 4][(j & 15) + e]);
                                m[e] = j + e <= lane
                                           ? x * (ex2((hi_r - ghs[e]) + (lo_r - gls[e])) * ds[e]) : 0.f;
                            }
                            hi[j / 2] = split2(m[0], m[1], lo[j / 2]);
                            hi[j / 2 + 1] = split2(m[2], m[3], lo[j / 2 + 1]);
                        }
                    }
                    tc::st16(lanes + kTmM + 16 * b, hi);
                    tc::st16(lanes + kTmM + 64 + 16 * b, lo);
                }
                tc::st_wait();
                tc::fence_before();
                mbar_arrive(bar(kMReady));
            }

            // ---- S = 2^G_last S + B^T (W X)
            if (!(ok = wait(kCSDS, i))) break;
            tc::fence_after();
            if (has) {
                uint32_t v[2][16];
                tc::ld16(lanes + kTmDS + 32 * hf, v[0]);
                tc::ld16(lanes + kTmDS + 32 * hf + 16, v[1]);
                tc::ld_wait();
                const float dec = s.decay;
#pragma unroll
                for (int j = 0; j < 32; ++j) S[j] = fmaf(S[j], dec, __uint_as_float(v[j >> 4][j & 15]));
            }
            tc::fence_before();
            run_decay *= s.decay;
            if (kStates) mbar_arrive(bar(kDone));
            const bool ends = w.last();
            if (!kStates && ends && p.s_final != nullptr && has) {
                float4 *dst = reinterpret_cast<float4 *>(p.s_final + state_at(w));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dst[j] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
            }
            const Walk now = w;
            if (i + 1 < count) {
                w.next(p, pl, list.nc);
                if (w.pos == 0) start_state(w, i + 1);
                put_state();
                if (!(ok = wait(kScal + ((i + 1) & 1), (i + 1) >> 1) &&
                           wait(kFullBX + ((i + 1) & 1), (i + 1) >> 1)))
                    break;
                put_rows(i + 1, w.valid());
            }

            if (!kStates) {
                // ---- y = 2^G (C S) + M X + d x
                if (!(ok = wait(kMX, i))) break;
                tc::fence_after();
                uint32_t y[2][16], cs[2][16];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    tc::ld16(lanes + kTmY + 32 * hf + 16 * k, y[k]);
                    tc::ld16(lanes + kTmCS + 32 * hf + 16 * k, cs[k]);
                }
                tc::ld_wait();
                tc::fence_before();
                const int h = now.u / pl.slices;
                const float from = s.from[r], dv = p.d != nullptr ? __ldg(p.d + h) : 0.f;
                uint4 o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(
                        smem + kOffX + (i & 1) * 16384 + r * 128 + (((4 * hf + k) ^ (r & 7)) << 4));
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                    uint32_t os[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 8 * k + 2 * e;
                        const float2 f = unpack_bf16(xs[e]);
                        os[e] = pack_bf16(
                            fmaf(dv, f.x, fmaf(from, __uint_as_float(cs[j >> 4][j & 15]),
                                               __uint_as_float(y[j >> 4][j & 15]))),
                            fmaf(dv, f.y, fmaf(from, __uint_as_float(cs[j >> 4][(j & 15) + 1]),
                                               __uint_as_float(y[j >> 4][(j & 15) + 1]))));
                    }
                    o[k] = make_uint4(os[0], os[1], os[2], os[3]);
                }
                mbar_arrive(bar(kDone));
                if (r < valid) {
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        static_cast<__nv_bfloat16 *>(p.out) + ((now.row() + r) * p.heads + h) * p.p +
                        (now.u % pl.slices) * kPS + 32 * hf);
#pragma unroll
                    for (int k = 0; k < 4; ++k) dst[k] = o[k];
                }
            }
        }
        if (kStates && ok) {
#pragma unroll
            for (int j = 0; j < 32; ++j) pl.slots[slot + j * kCompute] = has ? S[j] : 0.f;
            if (tid == 0) pl.decay[c] = run_decay;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after();
        tc::dealloc(tm, kTmCols);
    }
}

template <typename F>
cudaError_t with_n(const SsmParams &p, F &&go) {
    return p.n == 64 ? go(std::integral_constant<int, 64>()) : go(std::integral_constant<int, 128>());
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// [tokens][width] bf16, rows `stride` elements apart, boxes of 128 tokens x 64
// channels with 128-byte swizzling; rows past the end read as zero.
bool encode(CUtensorMap *m, const void *base, int64_t tokens, int64_t width, int64_t stride) {
    const EncodeFn enc = reinterpret_cast<EncodeFn>(tensor_map_encoder());
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {64, kL}, estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace: [chunk offsets (packed)][decays][states at the cuts][copies of
// initial states (in place)].
constexpr int64_t kSlotBytes = 32 * kCompute * 4;
int64_t offsets_bytes(const SsmParams &p) {
    return p.cu != nullptr ? align256((static_cast<int64_t>(p.n_seqs) + 1) * 4) : 0;
}

}  // namespace

cudaError_t configure_ssm() {
    for (auto kernel : {ssm_chunk_kernel<64, false>, ssm_chunk_kernel<64, true>,
                        ssm_chunk_kernel<128, false>, ssm_chunk_kernel<128, true>}) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int64_t ssm_workspace(const SsmParams &p) {
    return offsets_bytes(p) + 1024 + 2 * kSsmSms * kSlotBytes;
}

cudaError_t launch_ssm(const SsmParams &p, const CallContext &ctx, cudaStream_t stream) {
    if (p.tokens == 0) {
        if (p.s_final == nullptr) return cudaSuccess;
        return with_n(p, [&](auto n) {
            ssm_hand_on_kernel<decltype(n)::value>
                <<<p.n_seqs < 1024 ? p.n_seqs : 1024, 256, 0, stream>>>(p);
            return cudaGetLastError();
        });
    }
    SsmMaps maps;
    if (!encode(&maps.x, p.x, p.tokens, static_cast<int64_t>(p.heads) * p.p, p.x_stride) ||
        !encode(&maps.b, p.b, p.tokens, static_cast<int64_t>(p.groups) * p.n, p.b_stride) ||
        !encode(&maps.c, p.c, p.tokens, static_cast<int64_t>(p.groups) * p.n, p.c_stride))
        return cudaErrorInvalidValue;
    SsmPlan pl{};
    uint8_t *ws = ctx.ws;
    pl.slices = p.p / kPS;
    pl.units = static_cast<int64_t>(p.heads) * pl.slices;
    pl.cps = static_cast<int>((p.seq_len + kL - 1) / kL);
    pl.decay = reinterpret_cast<float *>(ws + offsets_bytes(p));
    pl.slots = reinterpret_cast<float *>(ws + offsets_bytes(p) + 1024);
    pl.saved = pl.slots + kSsmSms * kSlotBytes / 4;
    pl.in_place = p.s_final != nullptr && p.s_final == p.s0;
    if (p.cu != nullptr) {
        int32_t *off = reinterpret_cast<int32_t *>(ws);
        const cudaError_t e = launch_varlen_prologue(p.cu, p.n_seqs, p.tokens, off, ctx.call_flags, p.err,
                                                     stream, 7);
        if (e != cudaSuccess) return e;
        pl.chunk_off = off;
        pl.call_flags = ctx.call_flags;
    }
    // Whole sequences (or, packed, all of a unit's) stay in one run, and the
    // launch for the states at the cuts is saved, when they are short, or when
    // there are so many that the SMs are even without cuts.
    const int64_t nc = p.cu != nullptr ? (p.tokens + static_cast<int64_t>(kL - 1) * p.n_seqs) / kL
                                       : static_cast<int64_t>(pl.cps) * p.n_seqs;
    const bool whole = p.cu != nullptr ? p.tokens <= 4 * kL
                                       : pl.cps <= 4 || pl.units * p.n_seqs >= 8 * kSsmSms;
    pl.gran = !whole ? 1 : p.cu != nullptr ? 0 : pl.cps;
    const int64_t runs = pl.units * nc / (pl.gran > 0 ? pl.gran : nc);
    const unsigned grid = static_cast<unsigned>(runs < kSsmSms ? runs : kSsmSms);
    return with_n(p, [&](auto n) {
        constexpr int kN = decltype(n)::value;
        if (!whole) {
            ssm_chunk_kernel<kN, true><<<grid, kThreads, kSmem, stream>>>(maps, p, pl);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
        ssm_chunk_kernel<kN, false><<<grid, kThreads, kSmem, stream>>>(maps, p, pl);
        return cudaGetLastError();
    });
}

cudaError_t launch_ssm_step(const SsmParams &p, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.n_seqs) * p.heads;
    if (p.n == 64 && p.p == 64) ssm_step_kernel<64, 64><<<grid, 256, 0, stream>>>(p);
    else if (p.n == 64) ssm_step_kernel<64, 128><<<grid, 256, 0, stream>>>(p);
    else if (p.p == 64) ssm_step_kernel<128, 64><<<grid, 256, 0, stream>>>(p);
    else ssm_step_kernel<128, 128><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
