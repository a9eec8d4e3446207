// Attention of one new token per sequence over a paged cache of e4m3 numbers with a scale
// per page and head (kda_paged_decode_fp8). One pass over the cache:
//
//   s_j = scale ks_j (q . k_j),  out = sum_j 2^(s_j - M) vs_j v_j / sum_j 2^(s_j - M)
//
// (s in units of log 2). Every cached number is used once per query head that shares
// it, so the operator is bound by reading the cache: 2 D B per (token, key-value head).
//
// Both products are tcgen05 with 8-bit operands, which take the cache's tiles out of
// shared memory as they lie there, nothing converted. They are formed transposed, the
// tile of 128 tokens being the M side:
//   S^T (tokens x heads) = K (tokens x D) Q^T,   O^T (D x heads) = V^T (D x tokens) P^T.
// So the few heads of a group are the narrow side N, a thread owns a token, and the
// token's scales are one multiplication per score. What is not 8-bit enters as several
// e4m3 terms side by side along N, each of what the one before leaves, times 32 (at most
// 2^-5 of the one before is left): a query in two (bf16 has 8 bits of mantissa, e4m3 4:
// exact, down to 2^-22 of the row's largest channel), a weight times its value's scale
// in four (16 bits, far below out's own rounding, down to 2^-33 of the tile's largest).
// The terms' sums are added in fp32, finest first.
//
// A tile's weights are taken relative to the tile's own maximum, so nothing in front of
// the products depends on the tiles before; sums join in registers: sum_j 2^(s_j - M) in
// the threads of the tokens, the outputs in the threads of the channels. Values' scales go
// into the exponent (s_j + log2 vs_j): the weights of a tile then reach 1 whatever the
// scales are.
//
// Roles, one block per SM: 4 warps copy (cp.async, 16 bytes of a row each, so that any
// page size, stride and order of the pages will do), one warp issues the products, two
// groups of 4 warps take turns with the tiles' weights, 4 warps add up the outputs, one
// prepares the queries. Shares, pieces and the join of pieces: kda_pieces.cuh; a piece
// that is not a whole item leaves its sums in the workspace, and the last block to
// arrive joins them in the order of the blocks.

#include <cuda_fp8.h>
#include <math_constants.h>

#include "kda_device.cuh"
#include "kda_internal.h"
#include "kda_pieces.cuh"
#include "kda_tcgen05.cuh"

namespace kda {

namespace {

constexpr int kTile = 128;           // tokens
constexpr int kItemCost = 2;         // start and end of an item, in tiles
constexpr int kQTerms = 2, kPTerms = 4;
constexpr float kFiner = 32.f;       // from one term to the next
// Warps: two groups for the weights, one for the outputs (each of four: a warp reaches the
// 32 lanes of tensor memory of its number modulo 4), then the copies, MMAs and queries.
constexpr int kOutWarp = 8, kCopyWarp = 12, kMmaWarp = 16, kQueryWarp = 17;
constexpr int kThreads = 18 * 32;
constexpr int kCopyWarps = 4;
using Paged8Split = Split<kTile, kItemCost>;

// H = 8 or 16 query heads of one key-value head are an item.
template <int D, int H>
struct Shape {
    static constexpr int kTileBytes = kTile * D;
    static constexpr int kStages = D == 128 ? 6 : 10;
    // Tiles on their way behind the one that is announced. A tile is announced when the one
    // kAhead behind it has been asked for, and that one's place is free once the tile
    // kStages in front of it is done, for which the next one has to be there as well:
    // kAhead <= kStages - 2.
    static constexpr int kAhead = kStages - 3;
    static constexpr int kQRows = kQTerms * H, kPRows = kPTerms * H;
    // shared memory, from a 1024-byte boundary
    static constexpr int kOffV = kTileBytes;                        // V behind K in a stage
    static constexpr int kStage = 2 * kTileBytes;
    static constexpr int kOffQ = kStages * kStage;                  // two buffers
    static constexpr int kOffP = kOffQ + 2 * kQRows * D;            // two buffers
    static constexpr int kOffSc = kOffP + 2 * kPRows * kTile;       // ks and vs of a stage's tokens
    static constexpr int kOffMax = kOffSc + kStages * 2 * kTile * 4;    // [group][2][warp][2 H]
    static constexpr int kOffStat = kOffMax + 2 * 2 * 4 * 2 * H * 4;    // [2][H]: the tile's maximum
    static constexpr int kOffMul = kOffStat + 2 * H * 4;            // [2][H]: what a score is multiplied by
    static constexpr int kOffSum = kOffMul + 2 * H * 4;             // [2][8 warps][H]
    static constexpr int kOffTop = kOffSum + 2 * 8 * H * 4;         // [2][group][H]
    static constexpr int kOffJoin = kOffTop + 2 * 2 * H * 4;        // [2][H]
    static constexpr int kOffBar = kOffJoin + 2 * H * 4;
    // tensor memory columns: S, then O, two buffers each
    static constexpr int kTmO = 2 * kQRows;
    static constexpr int kTmCols = 2 * (kQRows + kPRows) <= 128 ? 128 : 256;
    static constexpr int kSlot = H * (D + 3);                       // floats of one partial result
};

// Barriers, 8 bytes each.
template <int kStages>
struct Bars {
    enum {
        kFull, kEmpty = kFull + kStages, kQFull = kEmpty + kStages, kQEmpty = kQFull + 2, kSFull = kQEmpty + 2,
        kPFull = kSFull + 2, kOFull = kPFull + 2, kOEmpty = kOFull + 2, kMax = kOEmpty + 2, kLFull = kMax + 2,
        kLEmpty = kLFull + 2, kJoin = kLEmpty + 2, kDrain, kCount
    };
    static __device__ __forceinline__ int arrivals(int i) {
        if (i < kEmpty) return kCopyWarps;
        if (i < kQFull) return 1;
        if (i < kQEmpty) return 1;
        if (i < kSFull) return 9;       // the products of a piece, and the 8 warps that read kOffMul
        if (i < kPFull) return 1;
        if (i < kOFull) return 4;
        if (i < kOEmpty) return 1;
        if (i < kLFull) return 4;       // kOEmpty, kMax
        if (i < kLEmpty) return 8;
        return i < kDrain ? 4 : 1;      // kLEmpty, kJoin
    }
};

template <int D, int H>
constexpr int smem_bytes() {
    return Shape<D, H>::kOffBar + 8 * Bars<Shape<D, H>::kStages>::kCount;
}

// ---- descriptors: rows of D (K, V, Q) or 128 (P) bytes, 16-byte granules XOR-ed by the
// row within 1024 (512, for 64-byte rows) bytes. Contiguous along K (K, Q, P) the stride
// field is the step between groups of 8 rows; contiguous along M (V) the step between
// groups of 8 tokens: the same number.
template <int kRow>
__device__ __forceinline__ uint64_t desc(uint32_t saddr) {
    constexpr uint32_t hi = ((8u * kRow) >> 4) | (1u << 14) | ((kRow == 128 ? 2u : 4u) << 29);
    return (static_cast<uint64_t>(hi) << 32) | ((saddr >> 4) & 0x3FFF) | (1u << 16);
}
template <int kRow>
__device__ __forceinline__ int swizzled(int row, int granule) {
    return row * kRow + ((kRow == 128 ? granule ^ (row & 7) : granule ^ ((row >> 1) & 3)) << 4);
}

// e4m3 operands, fp32 accumulators.
__host__ __device__ constexpr uint32_t idesc8(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
constexpr uint32_t kAMajor = 1u << 15;   // A contiguous along M

// The whole warp calls these, an elected lane issues.
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(acc))
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The largest of a warp's values; NaN does not count.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float finite_base(float m) { return m == -CUDART_INF_F ? 0.f : m; }

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Two numbers of at most 256 as e4m3, the first in the low byte; what is left of them
// (at most 8, half a step) times kFiner.
__device__ __forceinline__ uint32_t take8(float &a, float &b) {
    const __nv_fp8x2_storage_t t = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(t, __NV_E4M3)));
    a = (a - f.x) * kFiner;
    b = (b - f.y) * kFiner;
    return t;
}

__host__ __device__ __forceinline__ Lengths lengths_of(const Cache8 &c) {
    return {c.lens, c.max_pages * c.page_size, c.batch, c.pages > 0};
}

template <int D, int H>
__global__ void __launch_bounds__(kThreads, 1) paged8_kernel(Paged8Params p, float *slots, int *arrived) {
    using S = Shape<D, H>;
    using B = Bars<S::kStages>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_last;
    const Cache8 &c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = p.hq / c.hkv, chunks = (group + H - 1) / H;
    const int items = c.hkv * chunks;   // work items of a sequence
    const Lengths lens = lengths_of(c);
    const Paged8Split::Share sh = Paged8Split::share<kThreads>(lens, items, c.err);

    // sequences without tokens
    for (int b = blockIdx.x; b < c.batch; b += gridDim.x) {
        bool ignore = false;
        if (lens.of(b, &ignore) != 0) continue;
        for (int i = tid; i < p.hq * D / 8; i += kThreads)
            reinterpret_cast<uint4 *>(p.out)[static_cast<int64_t>(b) * (p.hq * D / 8) + i] =
                make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr)
            for (int i = tid; i < p.hq; i += kThreads) p.lse[static_cast<int64_t>(b) * p.hq + i] = -CUDART_INF_F;
    }
    if (blockIdx.x >= sh.G) return;

    const uint32_t sb = smem_u32(smem);
    const auto bar = [&](int i) { return sb + S::kOffBar + 8 * i; };
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < B::kCount; ++i) mbar_init(bar(i), B::arrivals(i));
        mbar_fence_init();
    }
    if (warp == 0) {
        tc::alloc(smem_u32(&s_tmem), S::kTmCols);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = s_tmem;

    // A bounded wait, the same for a whole warp. Once one has run out, all stop.
    auto wait = [&](int i, int phase) -> bool {
        bool ok = mbar_try_wait(bar(i), phase & 1);
        if (!ok) {
            const unsigned long long t0 = globaltimer();
            for (;;) {
                for (int k = 0; k < 32 && !ok; ++k) ok = mbar_try_wait(bar(i), phase & 1);
                if (ok || *static_cast<volatile int *>(&s_abort) != 0) break;
                if (globaltimer() - t0 > kWaitLimitNs) {
                    *static_cast<volatile int *>(&s_abort) = 1;
                    atomicOr(c.err, kErrTimeout);
                    break;
                }
            }
        }
        return __all_sync(0xffffffffu, ok) != 0;
    };
    auto arrive = [&](int i) {   // one arrival per warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };

    Paged8Split::Pieces w = sh.pieces();
    if (warp >= kCopyWarp && warp < kMmaWarp) {
        // ------------------------------------------------------------- copies: 32 tokens each
        constexpr int G16 = D / 16, R = 32 / G16;   // granules of a row, rows per instruction
        const int first = 32 * (warp - kCopyWarp);
        bool more = w.next(lens, items);
        int tile = w.tile0, page = 0, n = 0, said = 0;
        auto page_of = [&] {   // (read a tile earlier)
            const int t = tile * kTile + first + lane;
            page = more && t < w.len ? __ldg(c.table + static_cast<int64_t>(w.b) * c.max_pages + t / c.page_size) : 0;
        };
        page_of();
        for (; more && n < p.stall; ++n) {
            const int s = n % S::kStages;
            if (n >= S::kStages && !wait(B::kEmpty + s, n / S::kStages - 1)) break;
            const int tok0 = tile * kTile + first, t = tok0 + lane, len = w.len, kv = w.item / chunks;
            int pg = page;
            if (++tile == w.tile1) {
                more = w.next(lens, items);
                tile = w.tile0;
            }
            page_of();
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(c.pages)) {
                if (t < len) atomicOr(c.err, kErrPage);
                pg = 0;
            }
            const int64_t in = t % c.page_size;
            const uint8_t *ka = c.k + pg * c.k_page + in * c.k_token + kv * c.k_head;
            const uint8_t *va = c.v + pg * c.v_page + in * c.v_token + kv * c.v_head;
            const uint32_t at = sb + s * S::kStage, sc = sb + S::kOffSc + (s * 2 * kTile + first + lane) * 4;
            const int g = lane % G16;
#pragma unroll
            for (int i = 0; i < 32 / R; ++i) {
                const int row = i * R + lane / G16;
                const uint64_t kr = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(ka), row);
                const uint64_t vr = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(va), row);
                const uint32_t dst = at + swizzled<D>(first + row, g);
                // rows past the end are zeros: whatever the page holds there stays unread
                const uint32_t bytes = tok0 + row < len ? 16 : 0;
                cp_async16(dst, reinterpret_cast<const uint8_t *>(kr) + 16 * g, bytes);
                cp_async16(dst + S::kOffV, reinterpret_cast<const uint8_t *>(vr) + 16 * g, bytes);
            }
            const uint32_t four = t < len ? 4 : 0;
            cp_async4(sc, c.ks + pg * c.ks_page + kv, four);
            cp_async4(sc + 4 * kTile, c.vs + pg * c.vs_page + kv, four);
            cp_async_commit();
            if (n >= S::kAhead) {
                cp_async_wait<S::kAhead>();
                fence_async();
                arrive(B::kFull + said++ % S::kStages);
            }
        }
        cp_async_wait<0>();
        fence_async();
        for (; said < n; ++said) arrive(B::kFull + said % S::kStages);
    } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------------------- the products
        constexpr uint32_t kIdS = idesc8(kTile, S::kQRows), kIdO = idesc8(D, S::kPRows) | kAMajor;
        int n = 0, pc = 0;
        bool ok = true;
        auto out = [&](int m) {   // O^T of tile m
            if (!wait(B::kPFull + (m & 1), m >> 1)) return false;
            tc::fence_after();
            const uint64_t v = desc<D>(sb + m % S::kStages * S::kStage + S::kOffV);
            const uint64_t q = desc<128>(sb + S::kOffP + (m & 1) * S::kPRows * kTile);
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)   // 32 tokens
                mma8(tm + S::kTmO + (m & 1) * S::kPRows, v + k * (32 * D >> 4), q + k * (32 >> 4), kIdO, k > 0);
            mma_commit(bar(B::kOFull + (m & 1)));
            mma_commit(bar(B::kEmpty + m % S::kStages));
            return true;
        };
        for (; ok && w.next(lens, items); ++pc) {
            ok = wait(B::kQFull + (pc & 1), pc >> 1);
            for (int tile = w.tile0; ok && tile < w.tile1; ++tile, ++n) {
                // (S's buffer is free: the weights of tile n - 2 are there, see `out`)
                if (!(ok = wait(B::kFull + n % S::kStages, n / S::kStages))) break;
                tc::fence_after();
                const uint64_t k8 = desc<D>(sb + n % S::kStages * S::kStage);
                const uint64_t q = desc<D>(sb + S::kOffQ + (pc & 1) * S::kQRows * D);
#pragma unroll
                for (int k = 0; k < D / 32; ++k)   // 32 channels
                    mma8(tm + (n & 1) * S::kQRows, k8 + k * (32 >> 4), q + k * (32 >> 4), kIdS, k > 0);
                mma_commit(bar(B::kSFull + (n & 1)));
                if (tile + 1 == w.tile1) mma_commit(bar(B::kQEmpty + (pc & 1)));
                if (n > 0) ok = out(n - 1);
            }
        }
        if (ok && n > 0) out(n - 1);
        // nothing is under way when tensor memory is given back
        mma_commit(bar(B::kDrain));
        for (int k = 0; k < 1000000 && !mbar_try_wait(bar(B::kDrain), 0); ++k) {
        }
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------------------------ the queries
        constexpr int kPer = D / 32;   // channels of a lane
        for (int pc = 0; w.next(lens, items); ++pc) {
            if (pc >= 2 && !wait(B::kQEmpty + (pc & 1), (pc >> 1) - 1)) break;
            const int kv = w.item / chunks, head0 = kv * group + w.item % chunks * H;
            const int heads = min(H, group - w.item % chunks * H);
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) +
                                     (static_cast<int64_t>(w.b) * p.hq + head0) * D + kPer * lane;
            uint32_t x[H][kPer / 2];
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < kPer / 2; ++e)
                    x[h][e] = h < heads ? __ldg(reinterpret_cast<const uint32_t *>(q + h * D) + e) : 0u;
            uint8_t *dst = smem + S::kOffQ + (pc & 1) * S::kQRows * D;
            float mul = 0.f;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < kPer / 2; ++e) top = max(top, max(x[h][e] & 0x7fffu, (x[h][e] >> 16) & 0x7fffu));
                top = __reduce_max_sync(0xffffffffu, top);
                // 2^-k brings the row's largest channel below 2^8; an infinity or NaN makes its
                // scores NaN
                const int k = max(static_cast<int>(top >> 7) - 127 - 7, -126);
                const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
                const float up = top >= 0x7f80u ? CUDART_NAN_F : __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
                if (lane == h) mul = p.scale * 1.44269504088896341f * up;
#pragma unroll
                for (int e = 0; e < kPer / 2; ++e) {
                    float a = __uint_as_float(x[h][e] << 16) * down, b = __uint_as_float(x[h][e] & 0xffff0000u) * down;
#pragma unroll
                    for (int t = 0; t < kQTerms; ++t) {
                        const int row = t * H + h, byte = kPer * lane + 2 * e;
                        *reinterpret_cast<uint16_t *>(dst + swizzled<D>(row, byte >> 4) + (byte & 15)) =
                            static_cast<uint16_t>(take8(a, b));
                    }
                }
            }
            if (lane < H) reinterpret_cast<float *>(smem + S::kOffMul)[(pc & 1) * H + lane] = mul;
            fence_async();
            arrive(B::kQFull + (pc & 1));
        }
    } else if (warp < kOutWarp) {
        // --------------------------------------------------- the weights; a thread has a token
        const int g = warp >> 2, q = warp & 3, t = 32 * q + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        float *maxima = reinterpret_cast<float *>(smem + S::kOffMax) + g * 2 * 4 * 2 * H;
        int n = 0, taken = 0;
        bool ok = true;
        for (int pc = 0; ok && w.next(lens, items); ++pc) {
            if (!(ok = wait(B::kQFull + (pc & 1), pc >> 1))) break;
            float mul[H], l[H], top = -CUDART_INF_F;   // top: lane h has head h's
#pragma unroll
            for (int h = 0; h < H; ++h) {
                mul[h] = reinterpret_cast<const float *>(smem + S::kOffMul)[(pc & 1) * H + h];
                l[h] = 0.f;
            }
            arrive(B::kQEmpty + (pc & 1));
            for (int tile = w.tile0; tile < w.tile1; ++tile, ++n) {
                if ((n & 1) != g) continue;
                const int s = n % S::kStages, b = n & 1;
                if (!(ok = wait(B::kFull + s, n / S::kStages)) || !(ok = wait(B::kSFull + b, n >> 1))) break;
                tc::fence_after();
                const float *sc = reinterpret_cast<const float *>(smem + S::kOffSc) + s * 2 * kTile + t;
                const float ks = sc[0], lv = __log2f(sc[kTile]);
                uint32_t raw[S::kQRows / 16][16];
#pragma unroll
                for (int i = 0; i < S::kQRows / 16; ++i) tc::ld16(tm + lanes + b * S::kQRows + 16 * i, raw[i]);
                tc::ld_wait();
                const bool live = tile * kTile + t < w.len;
                float x[H];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float hi = __uint_as_float(raw[h / 16][h % 16]);
                    const float lo = __uint_as_float(raw[(H + h) / 16][(H + h) % 16]);
                    x[h] = live ? fmaf(lo, 1.f / kFiner, hi) * (mul[h] * ks) : -CUDART_INF_F;
                }
                // maxima over the tile's tokens: lane h those of s, lane H + h those of s + log2 vs
                float mine = -CUDART_INF_F;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float a = warp_max(x[h]), v = warp_max(x[h] + lv);
                    if (lane == h) mine = a;
                    if (lane == H + h) mine = v;
                }
                float *m = maxima + (taken & 1) * 4 * 2 * H;
                if (lane < 2 * H) m[q * 2 * H + lane] = mine;
                arrive(B::kMax + g);
                if (!(ok = wait(B::kMax + g, taken))) break;
                ++taken;
                if (n >= 2 && !(ok = wait(B::kOEmpty + b, (n >> 1) - 1))) break;
                float base = 0.f, f = 0.f;
                if (lane < 2 * H) {
                    const float all = fmaxf(fmaxf(m[lane], m[2 * H + lane]), fmaxf(m[4 * H + lane], m[6 * H + lane]));
                    if (lane < H) {
                        const float now = fmaxf(top, all);
                        base = finite_base(now);
                        f = ex2(top - base);
                        top = now;
                    } else {
                        base = finite_base(all);
                        if (q == 0) reinterpret_cast<float *>(smem + S::kOffStat)[b * H + lane - H] = all;
                    }
                }
                uint8_t *dst = smem + S::kOffP + b * S::kPRows * kTile;
#pragma unroll
                for (int h = 0; h < H; h += 2) {
                    float wt[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float xb = __shfl_sync(0xffffffffu, base, h + j);
                        const float fb = __shfl_sync(0xffffffffu, f, h + j);
                        const float yb = __shfl_sync(0xffffffffu, base, H + h + j);
                        l[h + j] = fmaf(l[h + j], fb, ex2(x[h + j] - xb));
                        wt[j] = ex2(x[h + j] + lv - yb) * 256.f;   // e4m3 reaches 448
                    }
#pragma unroll
                    for (int k = 0; k < kPTerms; ++k) {
                        const uint32_t two = take8(wt[0], wt[1]);
                        dst[swizzled<128>(k * H + h, t >> 4) + (t & 15)] = static_cast<uint8_t>(two);
                        dst[swizzled<128>(k * H + h + 1, t >> 4) + (t & 15)] = static_cast<uint8_t>(two >> 8);
                    }
                }
                fence_async();
                tc::fence_before();
                arrive(B::kPFull + b);
            }
            if (!ok) break;
            // the piece's sums
            if (pc >= 2 && !(ok = wait(B::kLEmpty + (pc & 1), (pc >> 1) - 1))) break;
            float mine = 0.f;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float v = l[h];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
                if (lane == h) mine = v;
            }
            if (lane < H) {
                reinterpret_cast<float *>(smem + S::kOffSum)[((pc & 1) * 8 + warp) * H + lane] = mine;
                if (q == 0) reinterpret_cast<float *>(smem + S::kOffTop)[((pc & 1) * 2 + g) * H + lane] = top;
            }
            arrive(B::kLFull + (pc & 1));
        }
    } else {
        // ------------------------------------------------- the outputs; a thread has a channel
        const int q = warp & 3, t = 32 * q + lane;
        // (64 channels: rows 16 q .. of O^T lie in a quarter's first 16 lanes)
        const int d = D == 128 ? t : 16 * q + lane;
        const bool has = D == 128 || lane < 16;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        const int64_t U = sh.U, G = sh.G;
        const int me = blockIdx.x;
        float *join = reinterpret_cast<float *>(smem + S::kOffJoin);
        int n = 0, joined = 0;
        bool ok = true;
        auto together = [&]() -> bool {   // the four warps
            arrive(B::kJoin);
            return wait(B::kJoin, joined++);
        };
        for (int pc = 0; w.next(lens, items); ++pc) {
            const int kv = w.item / chunks, head0 = kv * group + w.item % chunks * H;
            const int heads = min(H, group - w.item % chunks * H);
            float acc[H], top = -CUDART_INF_F;   // top: lane h has head h's
#pragma unroll
            for (int h = 0; h < H; ++h) acc[h] = 0.f;
            for (int tile = w.tile0; ok && tile < w.tile1; ++tile, ++n) {
                const int b = n & 1;
                if (!(ok = wait(B::kOFull + b, n >> 1))) break;
                tc::fence_after();
                uint32_t raw[S::kPRows / 16][16];
#pragma unroll
                for (int i = 0; i < S::kPRows / 16; ++i)
                    tc::ld16(tm + lanes + S::kTmO + b * S::kPRows + 16 * i, raw[i]);
                float f = 0.f, gain = 0.f;
                if (lane < H) {
                    const float all = reinterpret_cast<const float *>(smem + S::kOffStat)[b * H + lane];
                    const float now = fmaxf(top, all), base = finite_base(now);
                    f = ex2(top - base);
                    gain = ex2(all - base) * (1.f / 256);
                    top = now;
                }
                tc::ld_wait();
                tc::fence_before();
                arrive(B::kOEmpty + b);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float o = __uint_as_float(raw[(3 * H + h) / 16][(3 * H + h) % 16]);
#pragma unroll
                    for (int k = kPTerms - 2; k >= 0; --k)
                        o = fmaf(o, 1.f / kFiner, __uint_as_float(raw[(k * H + h) / 16][(k * H + h) % 16]));
                    acc[h] = fmaf(acc[h], __shfl_sync(0xffffffffu, f, h), o * __shfl_sync(0xffffffffu, gain, h));
                }
            }
            // ---- the piece's end: lane h has the sum and maximum of head h
            const bool whole = w.tile0 == 0 && w.tile1 == w.tiles;
            // of a block's partial pieces only its first can belong to an item that
            // started in front of its share, and only its last to another one
            float *slot = slots + static_cast<int64_t>(2 * me + (sh.u0 <= w.item_at)) * S::kSlot;
            if (ok) ok = wait(B::kLFull + (pc & 1), pc >> 1);
            if (ok) {
                float sum = 0.f, most = -CUDART_INF_F;
                if (lane < H) {
                    const float *ls = reinterpret_cast<const float *>(smem + S::kOffSum) + (pc & 1) * 8 * H + lane;
                    const float *ms = reinterpret_cast<const float *>(smem + S::kOffTop) + (pc & 1) * 2 * H + lane;
                    most = fmaxf(ms[0], ms[H]);
                    const float base = finite_base(most);
                    sum = (ls[0] + ls[H] + ls[2 * H] + ls[3 * H]) * ex2(ms[0] - base) +
                          (ls[4 * H] + ls[5 * H] + ls[6 * H] + ls[7 * H]) * ex2(ms[H] - base);
                }
                arrive(B::kLEmpty + (pc & 1));
                const int64_t row = static_cast<int64_t>(w.b) * p.hq + head0;
                if (whole) {
                    const float mine = sum > 0.f ? ex2(finite_base(top) - finite_base(most)) / sum : sum == 0.f ? 0.f : sum;
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const float by = __shfl_sync(0xffffffffu, mine, h);
                        if (h < heads && has)
                            static_cast<__nv_bfloat16 *>(p.out)[(row + h) * D + d] =
                                __float2bfloat16_rn(by == 0.f ? 0.f : acc[h] * by);
                    }
                    if (q == 0 && lane < heads && p.lse != nullptr)
                        p.lse[row + lane] = sum == 0.f ? -CUDART_INF_F
                                                       : finite_base(most) * 0.69314718055994531f + logf(sum);
                } else {
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        if (has) slot[h * D + d] = acc[h];
                    if (q == 0 && lane < H) {
                        slot[H * D + lane] = top;
                        slot[H * (D + 1) + lane] = most;
                        slot[H * (D + 2) + lane] = sum;
                    }
                }
            }
            if (whole) continue;
            // ---- the last block of this item to arrive joins the pieces. (The arrival is made
            // even if a wait has run out: the counters stay right.)
            const int c0 = Paged8Split::owner(w.item_at + kItemCost, U, G),
                      c1 = Paged8Split::owner(w.item_at + kItemCost + w.tiles - 1, U, G);
            if (ok) ok = together();   // (the slot is written)
            if (q == 0 && lane == 0) {
                int *ctr = arrived + static_cast<int64_t>(w.b) * items + w.item;
                const int before = add_acq_rel(ctr, 1);
                s_last = before == c1 - c0;
                if (s_last) *ctr = 0;   // for the next call
            }
            if (ok) ok = together();
            if (!ok || !*static_cast<volatile int *>(&s_last)) continue;
            const int last = c0 * U / G <= w.item_at;
            auto piece = [&](int k) { return slots + static_cast<int64_t>(2 * k + (k == c0 ? last : 0)) * S::kSlot; };
            for (int h = q; h < H; h += 4) {   // a warp per head: its maximum and sum
                float most = -CUDART_INF_F, sum = 0.f;
                for (int k = c0 + lane; k <= c1; k += 32) {
                    const float mk = __ldcg(piece(k) + H * (D + 1) + h), lk = __ldcg(piece(k) + H * (D + 2) + h);
                    const float now = fmaxf(most, mk), base = finite_base(now);
                    sum = fmaf(sum, ex2(most - base), lk * ex2(mk - base));
                    most = now;
                }
                float all = most;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
                const float base = finite_base(all);
                sum *= ex2(most - base);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) {
                    join[h] = base;
                    join[H + h] = sum;
                    if (h < heads && p.lse != nullptr)
                        p.lse[static_cast<int64_t>(w.b) * p.hq + head0 + h] =
                            sum == 0.f ? -CUDART_INF_F : base * 0.69314718055994531f + logf(sum);
                }
            }
            if (!(ok = together())) continue;
#pragma unroll
            for (int h = 0; h < H; ++h) acc[h] = 0.f;
            for (int k = c0; k <= c1; ++k) {
                const float *src = piece(k);
                const float by = lane < H ? ex2(finite_base(__ldcg(src + H * D + lane)) - join[lane]) : 0.f;
#pragma unroll
                for (int h = 0; h < H; ++h)
                    acc[h] = fmaf(has ? __ldcg(src + h * D + d) : 0.f, __shfl_sync(0xffffffffu, by, h), acc[h]);
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float sum = join[H + h];
                if (h < heads && has)
                    static_cast<__nv_bfloat16 *>(p.out)[(static_cast<int64_t>(w.b) * p.hq + head0 + h) * D + d] =
                        __float2bfloat16_rn(sum > 0.f ? acc[h] / sum : sum == 0.f ? 0.f : sum);
            }
            // (the next piece's join comes after barriers of its own: `join` is read by then)
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::dealloc(tm, S::kTmCols);
}

constexpr int heads_of(int group) { return group <= 8 ? 8 : 16; }

template <typename F>
auto with_shape(const Paged8Params &p, F &&go) {
    const bool few = heads_of(p.hq / p.c.hkv) == 8;
    if (p.c.dim == 64)
        return few ? go(Shape<64, 8>(), paged8_kernel<64, 8>, smem_bytes<64, 8>())
                   : go(Shape<64, 16>(), paged8_kernel<64, 16>, smem_bytes<64, 16>());
    return few ? go(Shape<128, 8>(), paged8_kernel<128, 8>, smem_bytes<128, 8>())
               : go(Shape<128, 16>(), paged8_kernel<128, 16>, smem_bytes<128, 16>());
}

int64_t chunks_of(const Paged8Params &p) {
    const int group = p.hq / p.c.hkv, h = heads_of(group);
    return (group + h - 1) / h;
}

static_assert(smem_bytes<128, 16>() <= 232448 - 1024, "what a block can have");

}  // namespace

cudaError_t configure_paged8() {
    for (int dim : {64, 128})
        for (int group : {1, 16}) {
            Paged8Params p{};
            p.c.dim = dim;
            p.c.hkv = 1;
            p.hq = group;
            const cudaError_t e = with_shape(p, [](auto, auto kernel, int bytes) {
                return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            });
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

// Two partial results per block.
int64_t paged8_workspace(const Paged8Params &p) {
    return with_shape(p, [](auto s, auto, int) {
        return static_cast<int64_t>(kPlannedSms) * 2 * decltype(s)::kSlot * 4;
    });
}

// One arrival counter per (sequence, work item).
int64_t paged8_sync(const Paged8Params &p) {
    return static_cast<int64_t>(p.c.batch) * p.c.hkv * chunks_of(p) * 4;
}

cudaError_t launch_paged8(const Paged8Params &p, const CallContext &ctx, cudaStream_t stream) {
    // units the lengths may come to; empty sequences need a block as well
    const int64_t units = static_cast<int64_t>(p.c.batch) * p.c.hkv * chunks_of(p) *
                          Paged8Split::units_of(p.c.max_pages * p.c.page_size);
    const unsigned grid = static_cast<unsigned>(units < 1 ? 1 : units < kPlannedSms ? units : kPlannedSms);
    return with_shape(p, [&](auto, auto kernel, int bytes) {
        kernel<<<grid, kThreads, bytes, stream>>>(p, reinterpret_cast<float *>(ctx.ws), ctx.sync);
        return cudaGetLastError();
    });
}

}  // namespace kda
