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
// in four (2^-18.7 of it is left at most, 2^-21 in the mean: fp32's own errors in the
// weight are of that size; down to 2^-33 of the tile's largest). The terms' sums are
// added in fp32, finest first.
//
// A tile's weights are taken relative to the tile's own maximum, so nothing in front of
// the products depends on the tiles before; sums join in registers: sum_j 2^(s_j - M) in
// the threads of the tokens, the outputs in the threads of the channels. Values' scales go
// into the exponent (s_j + log2 vs_j): the weights of a tile then reach 1 whatever the
// scales are.
//
// Roles, one block per SM: two or four warps copy (by the tensor memory accelerator, or, where
// the pages do not allow it, 16 bytes a time with cp.async: any page size, stride and order of
// the pages will do), one warp issues each product, two groups of four warps take turns with
// the tiles' weights, four warps add up the outputs, one prepares the queries and says what
// the block's next piece is. Shares, pieces and their join: kda_pieces.cuh; a piece that is not
// a whole item leaves its sums in the workspace, and the last block to arrive joins them in
// the order of the blocks (where they are many, groups of them first).
//
// Measured (copy bandwidth: 1340 clocks for a tile of D = 128): 2 sequences of 131072 tokens, 32
// heads over 8 of 128: 92 to 94 us (5.8 TB/s, 84 to 86 % of copy bandwidth); 64 sequences of 1 to
// 16384 tokens, 64 heads over 8: 51 us (66 %); 256 of 1000, 32 heads over 8: 97 us (80 %); one of
// 700: 11 us, a chain of latencies. What a tile
// takes the weights' warps, some 1250 clocks with 8 heads, bounds D = 64 (8 x 32768 tokens: 74
// us, 54 %), and 1600 with 16 heads those (8 x 65536, 2 key-value heads: 66 us, 60 %).

#include <cuda.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "kda_device.cuh"
#include "kda_internal.h"
#include "kda_pieces.cuh"
#include "kda_tcgen05.cuh"

namespace kda {

namespace {

constexpr int kTile = 128;           // tokens
constexpr int kItemCost = 3;         // start and end of an item, in tiles (64 ragged sequences: 64 us with 1, 54 with 2, 50 with 3 or 4)
constexpr int kQTerms = 2, kPTerms = 4;
constexpr float kFiner = 32.f;       // from one term to the next
constexpr unsigned long long kLandNs = 100000000;   // within which copies and products end
// Warps: groups of four for the weights, then one for the outputs (a warp reaches the 32 lanes
// of tensor memory of its number modulo 4), then one for each of the two products, one for
// the queries, and those for the copies. With 16 heads the second product's warp does the
// queries too: by tensor copies these are 16 warps, and a thread can have 128 registers. Where
// threads copy they are 18, of 96 registers, which the weights' loop overflows by some 100 bytes
// (64 channels, 16 heads, 3 x 78520 tokens, pages of 17: 73 us, a quarter of copy bandwidth).
constexpr int groups_of(int) { return 2; }
constexpr int copy_warps(int heads, bool tma) { return tma && heads > 8 ? 2 : 4; }
constexpr int threads_of(int heads, bool tma) { return 32 * (4 * groups_of(heads) + (heads > 8 ? 6 : 7) + copy_warps(heads, tma)); }
using Paged8Split = Split<kTile, kItemCost>;
constexpr int kJoined = 8, kFlat = 16;   // pieces of a group; pieces that are joined without groups

// A piece of the block's share, as the queries' warp hands it to the other roles beside the
// queries themselves (with each going through the share by itself 256 sequences of 1000
// tokens took 119 us, this way 112).
struct alignas(16) Piece {
    int tile0, tile1, len, tiles;   // tile1 = 0 behind the last one
    int64_t row, item_at;           // of out; first unit
    int b, item, heads, pad;
};

// H = 8 or 16 query heads of one key-value head are an item.
template <int D, int H>
struct Shape {
    static constexpr int kHeads = H, kGroups = groups_of(H);
    static constexpr int kOutWarp = 4 * kGroups, kMmaWarpS = kOutWarp + 4, kMmaWarpO = kMmaWarpS + 1,
                         kQueryWarp = H > 8 ? kMmaWarpO : kMmaWarpO + 1, kCopyWarp = kQueryWarp + 1;
    static constexpr int kTileBytes = kTile * D;
    // Places for tiles of K and of V: a tile's keys are done with when S is formed, its values
    // only with O.
    // (Even numbers where two warps take turns: a place is then one warp's.)
    static constexpr int kKeys = D == 128 ? (H == 8 ? 6 : 5) : 10, kValues = D == 128 ? 6 : 12;
    // Buffers of S, of P and O, of queries and pieces.
    static constexpr int kSBufs = 4, kPBufs = H == 8 ? 4 : 3, kQBufs = H == 8 ? 4 : 3;
    static constexpr int kQRows = kQTerms * H, kPRows = kPTerms * H;
    // shared memory, from a 1024-byte boundary
    static constexpr int kOffV = kKeys * kTileBytes;
    static constexpr int kOffQ = kOffV + kValues * kTileBytes;
    static constexpr int kOffP = kOffQ + kQBufs * kQRows * D;
    static constexpr int kOffSc = kOffP + kPBufs * kPRows * kTile;  // ks and vs of a tile's tokens, by V's place
    static constexpr int kOffMax = kOffSc + kValues * 2 * kTile * 4;    // [group][2][warp][2 H]
    static constexpr int kOffStat = kOffMax + kGroups * 2 * 4 * 2 * H * 4;    // [kPBufs][H]: the tile's maximum
    static constexpr int kOffMul = kOffStat + kPBufs * H * 4;       // [kQBufs][H]: what a score is multiplied by
    static constexpr int kOffPiece = kOffMul + kQBufs * H * 4;      // [kQBufs]
    static constexpr int kOffSum = kOffPiece + kQBufs * static_cast<int>(sizeof(Piece));   // [2][weights' warps][H]
    static constexpr int kOffTop = kOffSum + 2 * 4 * kGroups * H * 4;         // [2][group][H]
    static constexpr int kOffJoin = kOffTop + 2 * kGroups * H * 4;        // [3][H]
    static constexpr int kOffCast = kOffJoin + 3 * H * 4;           // [weights' and outputs' warps][3][H]
    static constexpr int kOffBar = kOffCast + (4 * kGroups + 4) * 3 * H * 4;
    // tensor memory columns: S, then O
    static constexpr int kTmO = kSBufs * kQRows;
    static constexpr int kTmCols = kTmO + kPBufs * kPRows <= 256 ? 256 : 512;
    static constexpr int kSlot = H * (D + 3);                       // floats of one partial result
};

// Barriers, 8 bytes each, and the arrivals that complete a phase of each.
template <typename S, bool kTma>
struct Bars {
    static constexpr int kCopyWarps = copy_warps(S::kHeads, kTma);
    enum {
        kKFull, kVFull = kKFull + S::kKeys, kKEmpty = kVFull + S::kValues, kVEmpty = kKEmpty + S::kKeys,
        kQFull = kVEmpty + S::kValues, kQEmpty = kQFull + S::kQBufs, kSFull = kQEmpty + S::kQBufs,
        kSEmpty = kSFull + S::kSBufs, kPFull = kSEmpty + S::kSBufs, kOFull = kPFull + S::kPBufs, kOEmpty = kOFull + S::kPBufs,
        kLFull = kOEmpty + S::kPBufs, kLEmpty = kLFull + 2, kDrain = kLEmpty + 2, kCount = kDrain + 2
    };
    static __device__ __forceinline__ int arrivals(int i) {
        if (i < kVFull) return kTma ? 1 : 32 * kCopyWarps;
        if (i < kKEmpty) return kTma ? 1 : 33 * kCopyWarps;
        if (i < kQEmpty) return 1;      // kKEmpty, kVEmpty, kQFull
        // kQEmpty: the products of a piece, and the warps that have read what it is
        if (i < kSFull) return 1 + 4 * S::kGroups + 4 + (S::kQueryWarp != S::kMmaWarpO);
        if (i < kSEmpty) return 1;
        if (i < kOFull) return 4;       // kSEmpty, kPFull
        if (i < kOEmpty) return 1;
        if (i < kLFull) return 4;
        if (i < kLEmpty) return 4 * S::kGroups;
        return i < kDrain ? 4 : 1;
    }
};

template <int D, int H>
constexpr int smem_bytes() {
    return Shape<D, H>::kOffBar + 8 * Bars<Shape<D, H>, true>::kCount;
}

// ---- descriptors: rows of 128, 64 or 32 bytes (K, V, Q: D; P: its terms and heads, a token
// after the other), 16-byte granules XOR-ed by the row within each 8 rows. Contiguous
// along K (K, Q) the stride field is the step between groups of 8 rows; contiguous along M
// or N (V, P) the step between groups of 8 tokens: the same number.
template <int kRow>
__device__ __forceinline__ uint64_t desc(uint32_t saddr) {
    constexpr uint32_t hi = ((8u * kRow) >> 4) | (1u << 14) | ((kRow == 128 ? 2u : kRow == 64 ? 4u : 6u) << 29);
    return (static_cast<uint64_t>(hi) << 32) | ((saddr >> 4) & 0x3FFF) | (1u << 16);
}
template <int kRow>
__device__ __forceinline__ int swizzled(int row, int granule) {
    const int x = kRow == 128 ? row & 7 : kRow == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
    return row * kRow + ((granule ^ x) << 4);
}

// e4m3 operands, fp32 accumulators.
__host__ __device__ constexpr uint32_t idesc8(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
constexpr uint32_t kAMajor = 1u << 15, kBMajor = 1u << 16;   // contiguous along M / N

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

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int token, int head, int page,
                                       uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(token), "r"(head), "r"(page), "r"(bar)
        : "memory");
}
// An arrival once this thread's copies so far have landed.
__device__ __forceinline__ void arrive_landed(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// Sums over a warp's lanes of H values each: lanes 32 / H h .. get that of value h. Of two
// lanes each keeps half of the values and hands over the other half.
template <int H>
__device__ __forceinline__ float lane_sums(float (&v)[H], int lane) {
    int m = 16;
#pragma unroll
    for (int n = H / 2; n > 0; n >>= 1, m >>= 1) {
        const bool upper = (lane & m) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + n], m);
            v[i] = (upper ? v[i + n] : v[i]) + got;
        }
    }
    for (; m > 0; m >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
    return v[0];
}

// The four warps of a role.
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;\n" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(int id, bool x) {
    int any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.s32 p, %2, 0;\n bar.red.or.pred q, %1, 128, p;\n selp.s32 %0, 1, 0, q;\n}\n"
        : "=r"(any) : "r"(id), "r"(static_cast<int>(x)) : "memory");
    return any != 0;
}

// Two numbers of at most 256 as e4m3, the first in the low byte. Half a step, 8 at most, is
// left of them.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 from_e4m3(uint32_t t) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(t), __NV_E4M3));
}
// ... and what the first term leaves, times kFiner.
__device__ __forceinline__ uint32_t take8(float &a, float &b) {
    const uint32_t t = to_e4m3(a, b);
    const float2 f = __half22float2(from_e4m3(t));
    add2(a, b, -f.x, -f.y);
    mul2(a, b, kFiner, kFiner);
    return t;
}
// Four terms: behind the second, half precision's 11 bits hold what is left, and the two
// others 9 to 10 of those. (In half precision from behind the first term on a weight kept 16
// bits; out then rounded otherwise than the 64-bit result ten times as often. 8 sequences of 32768
// tokens, 64 channels: 73.6 us for 74.5, 16 heads: 64.3 for 65.9, others within 1 %.)
__device__ __forceinline__ void split4(float a, float b, uint32_t (&t)[kPTerms]) {
    static_assert(kPTerms == 4, "");
    t[0] = take8(a, b);
    t[1] = take8(a, b);
    const __half2 r = __floats2half2_rn(a, b);
    t[2] = __nv_cvt_halfraw2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3);
    t[3] = __nv_cvt_halfraw2_to_fp8x2(__hmul2(__hsub2(r, from_e4m3(t[2])), __float2half2_rn(kFiner)), __NV_SATFINITE, __NV_E4M3);
}

__host__ __device__ __forceinline__ Lengths lengths_of(const Cache8 &c) {
    return {c.lens, c.max_pages * c.page_size, c.batch, c.pages > 0};
}

// Where a role is in a ring of N places: which one, and which time around.
template <int N>
struct Place {
    int at = 0, turn = 0;
    __device__ __forceinline__ void step() {
        if (++at == N) {
            at = 0;
            ++turn;
        }
    }
};

struct Paged8Maps {
    CUtensorMap k, v;   // (channel, token, head, page), boxes of 2^shift tokens
    int shift;
};

// An arrival at a counter of n: the last one finds it complete, and sets it back for the next call.
__device__ __forceinline__ bool last_of(int *counter, int n) {
    const bool last = add_acq_rel(counter, 1) == n - 1;
    if (last) *counter = 0;
    return last;
}

// An item's pieces, in the blocks c0 .. c1, are joined by the last of them to arrive; more than kFlat
// in groups of kJoined first, and then the groups (8 ragged sequences up to 43116 tokens, one
// key-value head: 24 us, all at once 48). By the outputs' warps, at a piece's end, and not inlined:
// the roles' loops run slower with more code between them (256 sequences of 1000 tokens:
// inlined 110 us, this way 95; 16 heads, 8 x 65536, 72 and 68).
template <int D, int H>
__device__ __noinline__ void join_pieces(float *slots, int *arrived, int *item_counter, int c0, int c1, int slot0,
                                         __nv_bfloat16 *out, float *lse, int heads, float *join, int *s_last) {
    using S = Shape<D, H>;
    constexpr int kOutSync = 1 + S::kGroups;
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5 & 3, t = 32 * q + lane;
    const int d = D == 128 ? t : 16 * q + lane;
    const bool has = D == 128 || lane < 16;
    auto slot_at = [&](int k) { return k == c0 ? slot0 : 2 * k; };
    float acc[H];
    int lo = c0, step = 1, n = c1 - c0 + 1;
    bool whole_item = n <= kFlat;
    if (!whole_item) {
        lo = c0 + (static_cast<int>(blockIdx.x) - c0) / kJoined * kJoined;
        n = min(kJoined, c1 + 1 - lo);
    }
#pragma unroll 1
    for (;;) {
        group_sync(kOutSync);   // (the slot is written)
        if (q == 0 && lane == 0)
            *s_last = last_of(whole_item ? item_counter : arrived + slot_at(lo), n);
        group_sync(kOutSync);
        if (!*static_cast<volatile int *>(s_last)) return;
        auto part = [&](int m) { return slots + static_cast<int64_t>(slot_at(lo + m * step)) * S::kSlot; };
        // The pieces' maxima and sums: a warp takes a quarter of the heads, so many pieces at
        // a time as it has lanes for.
        {
            constexpr int kHs = H / 4, kPieces = 32 / kHs;
            const int h = q * kHs + lane % kHs;
            float most = -CUDART_INF_F, sum = 0.f;
#pragma unroll 1
            for (int k = lane / kHs; k < n; k += kPieces) {
                const float mk = __ldcg(part(k) + H * (D + 1) + h), lk = __ldcg(part(k) + H * (D + 2) + h);
                const float now = fmaxf(most, mk), base = finite_base(now);
                sum = fmaf(sum, ex2(most - base), lk * ex2(mk - base));
                most = now;
            }
            float all = most;
#pragma unroll
            for (int o = 16; o >= kHs; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
            const float base = finite_base(all);
            sum *= ex2(most - base);
#pragma unroll
            for (int o = 16; o >= kHs; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane < kHs) {
                join[h] = base;
                join[H + h] = sum;
                join[2 * H + h] = all;
                if (whole_item && h < heads && lse != nullptr)
                    lse[h] =
                        sum == 0.f ? -CUDART_INF_F : base * 0.69314718055994531f + logf(sum);
            }
        }
        group_sync(kOutSync);
#pragma unroll
        for (int h = 0; h < H; ++h) acc[h] = 0.f;
        // 32 numbers on their way at a time
        constexpr int kBatch = 32 / H;
#pragma unroll 1
        for (int k0 = 0; k0 < n; k0 += kBatch) {
            float by[kBatch], v[kBatch][H];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const bool is = k0 + i < n;
                const float *src = part(is ? k0 + i : 0);
                by[i] = is && lane < H ? __ldcg(src + H * D + lane) : -CUDART_INF_F;
#pragma unroll
                for (int h = 0; h < H; ++h) v[i][h] = is && has ? __ldcg(src + h * D + d) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                by[i] = lane < H ? ex2(by[i] - join[lane]) : 0.f;
#pragma unroll
                for (int h = 0; h < H; ++h) acc[h] = fmaf(v[i][h], __shfl_sync(0xffffffffu, by[i], h), acc[h]);
            }
        }
        if (whole_item) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float sum = join[H + h];
                if (h < heads && has)
                    out[h * D + d] =
                        __float2bfloat16_rn(sum > 0.f ? acc[h] / sum : sum == 0.f ? 0.f : sum);
            }
            break;
        }
        // the group, in the place of its first piece
        group_sync(kOutSync);   // (which is read)
        float *to = slots + static_cast<int64_t>(slot_at(lo)) * S::kSlot;
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (has) to[h * D + d] = acc[h];
        if (q == 0 && lane < H) {
            to[H * D + lane] = join[2 * H + lane];
            to[H * (D + 1) + lane] = join[2 * H + lane];
            to[H * (D + 2) + lane] = join[H + lane];
        }
        lo = c0;
        step = kJoined;
        n = (c1 - c0) / kJoined + 1;
        whole_item = true;
    }
}

template <int D, int H, bool kTma>
__global__ void __launch_bounds__(threads_of(H, kTma), 1)
paged8_kernel(const __grid_constant__ Paged8Maps maps, Paged8Params p, float *slots, int *arrived) {
    using S = Shape<D, H>;
    using B = Bars<S, kTma>;
    constexpr int kThreads = threads_of(H, kTma);
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_last;
    __shared__ unsigned long long s_moved;   // when the block last got on
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
        s_moved = globaltimer();
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

    // A bounded wait: it runs out when the first product has taken no tile for kWaitLimitNs (a
    // piece may take longer than that, and the queries of a later one wait for its end; one clock
    // for all waits: short code, as the roles' loops together are more than the instruction
    // caches hold. With a clock and a count of tiles in each wait 256 sequences of 1000 tokens
    // took 112 us for 95). Once one has run out none waits any more: all roles go through the piece
    // they are at to its end, whatever they find there, some 13 us a tile (four polls of each wait;
    // with a look at s_abort every 256 polls, minutes for the longest pieces. Loops that end there
    // took 16 heads, 8 x 65536, from 66 to 70 us, 256 x 1000 from 97 to 100).
    auto wait = [&](int i, int phase) {
        for (unsigned spins = 1; !mbar_try_wait(bar(i), phase & 1); ++spins) {
            if (spins % 4 != 0) continue;
            if (*static_cast<volatile int *>(&s_abort) != 0) break;
            // (signed: s_moved may be set between the two readings)
            if (static_cast<long long>(globaltimer() - *static_cast<volatile unsigned long long *>(&s_moved)) >
                static_cast<long long>(kWaitLimitNs)) {
                *static_cast<volatile int *>(&s_abort) = 1;
                atomicOr(c.err, kErrTimeout);
            }
        }
        __syncwarp();
    };
    auto arrive = [&](int i) {   // one arrival per warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };

    // Nothing that a warp has issued is under way when tensor memory is given back.
    auto drain = [&](int i) {
        mma_commit(bar(B::kDrain + i));
        mbar_wait(bar(B::kDrain + i), 0, kLandNs);
    };

    Paged8Split::Pieces w = sh.pieces();
    auto stopped = [&] { return *static_cast<volatile int *>(&s_abort) != 0; };
    // What piece pc is, where w is (or, if there are no more, the end), and its queries as two
    // terms each.
    auto queries = [&](int pc, bool more) {
        constexpr int kLanes = D / 8, kRows = 32 / kLanes;
        const int at = lane % kLanes, sub = lane / kLanes;
        const int buf = pc % S::kQBufs;
        if (pc >= S::kQBufs) wait(B::kQEmpty + buf, pc / S::kQBufs - 1);
        if (stopped()) return;   // (others may still be reading)
        Piece *piece = reinterpret_cast<Piece *>(smem + S::kOffPiece) + buf;
        if (!more) {
            if (lane == 0) piece->tile1 = 0;
            arrive(B::kQFull + buf);
            return;
        }
        const int kv = w.item / chunks, head0 = kv * group + w.item % chunks * H;
        const int heads = min(H, group - w.item % chunks * H);
        if (lane == 0)
            *piece = {w.tile0, w.tile1, w.len, w.tiles, static_cast<int64_t>(w.b) * p.hq + head0, w.item_at,
                      w.b, w.item, heads, 0};
        // D / 8 lanes take a head, 16 bytes each (a warp taking head after head, unrolled: 256
        // sequences of 1000 tokens 101 us for 95, 200 of 11 tokens 34 for 29)
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) +
                                 (static_cast<int64_t>(w.b) * p.hq + head0 + sub) * D + 8 * at;
        uint4 x[H / kRows];
#pragma unroll
        for (int i = 0; i < H / kRows; ++i)
            x[i] = i * kRows + sub < heads ? __ldg(reinterpret_cast<const uint4 *>(q + i * kRows * D)) : make_uint4(0, 0, 0, 0);
        uint8_t *dst = smem + S::kOffQ + buf * S::kQRows * D + 8 * (at & 1);
        // (rolled: shorter code. 16 heads, 8 x 65536: by two 64 us, by one 68; 8 heads, 256 x 1000: 101
        // and 95)
        constexpr int kUnroll = H > 8 ? 2 : 1;
#pragma unroll kUnroll
        for (int row = sub; row < H; row += kRows) {
            uint32_t u[4] = {x[0].x, x[0].y, x[0].z, x[0].w}, top = 0;
#pragma unroll
            for (int i = 0; i + 1 < H / kRows; ++i) x[i] = x[i + 1];
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __vmaxu2(top, u[e] & 0x7fff7fffu);
#pragma unroll
            for (int m = kLanes / 2; m > 0; m >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, m));
            top = max(top & 0xffffu, top >> 16);
            // 2^-k brings the row's largest channel below 2^8; an infinity or NaN makes its
            // scores NaN
            const int k = max(static_cast<int>(top >> 7) - 127 - 7, -126);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
            const float up = top >= 0x7f80u ? CUDART_NAN_F : __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
            if (at == 0) reinterpret_cast<float *>(smem + S::kOffMul)[buf * H + row] = p.scale * 1.44269504088896341f * up;
            uint32_t terms[kQTerms][2] = {};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a = __uint_as_float(u[e] << 16) * down, b = __uint_as_float(u[e] & 0xffff0000u) * down;
#pragma unroll
                for (int t = 0; t < kQTerms; ++t) terms[t][e / 2] |= take8(a, b) << (e % 2 * 16);
            }
#pragma unroll
            for (int t = 0; t < kQTerms; ++t)
                *reinterpret_cast<uint2 *>(dst + swizzled<D>(t * H + row, at >> 1)) = make_uint2(terms[t][0], terms[t][1]);
        }
        fence_async();
        arrive(B::kQFull + buf);
    };
    // The piece pc; none, too, once a wait has run out.
    auto piece_at = [&](int pc) -> const Piece & {
        wait(B::kQFull + pc % S::kQBufs, pc / S::kQBufs);
        return reinterpret_cast<const Piece *>(smem + S::kOffPiece)[pc % S::kQBufs];
    };
    if (warp >= S::kCopyWarp) {
        // ----------------------------------------------------------------------------- copies
        // What a lane copies of a tile: 32 tokens of a warp, one each; or (kTma) boxes of tokens
        // of one page, K's in one warp and V's in the next, the tiles in turns where there are
        // two such pairs (a box takes a warp 80 clocks). Pages are read kDeep tiles of the warp's
        // ahead, their scales kScale: farther where a warp has every tile (2 x 131072 tokens, pages
        // of 17: 116 us, with 2 and 1 145, with 6 and 3 127; pages of one, 65536: 70, 105 and 98; by
        // tensor copies, pages of 32: 91.6 with 3 and 1, 93.4 with 2 and 1).
        const int cw = warp - S::kCopyWarp, turns = kTma ? B::kCopyWarps / 2 : 1, turn = kTma ? cw / 2 : 0;
        const bool of_v = cw & 1;
        const int offset = kTma ? (lane & 15) << maps.shift : 32 * cw + lane;
        struct Spot {
            int tok0, len, kv, page, in;   // len: 0 behind the last tile
            float ks, vs;
        };
        bool more = w.next(lens, items);
        int tile = w.tile0;
        auto step = [&](int by) {
            for (int i = 0; i < by && more; ++i)
                if (++tile == w.tile1) {
                    more = w.next(lens, items);
                    tile = w.tile0;
                }
        };
        step(turn);
        auto look = [&]() -> Spot {
            Spot a{0, 0, 0, 0, 0, 0.f, 0.f};
            if (!more) return a;
            a.tok0 = tile * kTile;
            a.len = w.len;
            a.kv = w.item / chunks;
            const uint32_t t = static_cast<uint32_t>(a.tok0) + offset, at = p.page_of(t);
            a.in = static_cast<int>(t - at * c.page_size);
            if (offset < a.len - a.tok0 && offset < kTile) a.page = __ldg(c.table + static_cast<int64_t>(w.b) * c.max_pages + at);
            step(turns);
            return a;
        };
        auto scales = [&](Spot &a) {
            if (offset >= a.len - a.tok0 || offset >= kTile) return;
            if (static_cast<unsigned>(a.page) >= static_cast<unsigned>(c.pages)) {
                atomicOr(c.err, kErrPage);
                a.page = 0;
            }
            if (!kTma || (of_v && lane >= 16)) a.ks = __ldg(c.ks + a.page * c.ks_page + a.kv);
            if (!kTma || (of_v && lane < 16)) a.vs = __ldg(c.vs + a.page * c.vs_page + a.kv);
        };
        constexpr int kDeep = kTma ? 3 : 4, kScale = kTma ? 1 : 2;
        Spot spots[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) spots[i] = look();
#pragma unroll
        for (int i = 0; i < kScale; ++i) scales(spots[i]);
        Place<S::kKeys> kp;
        Place<S::kValues> vp;
        auto place_on = [&](int by) {
            for (int i = 0; i < by; ++i) {
                kp.step();
                vp.step();
            }
        };
        place_on(turn);
        int n = turn;
        for (; spots[0].len > 0 && n < p.stall; n += turns, place_on(turns)) {
            const Spot far = look();
            scales(spots[kScale]);
            const Spot &now = spots[0];
            const int ks = kp.at, vs = vp.at;
            if ((!kTma || !of_v) && kp.turn > 0) wait(B::kKEmpty + ks, kp.turn - 1);
            if ((!kTma || of_v) && vp.turn > 0) wait(B::kVEmpty + vs, vp.turn - 1);
            if (stopped()) break;   // (its places may be in use)
            const uint32_t to_k = sb + ks * S::kTileBytes, to_v = sb + S::kOffV + vs * S::kTileBytes;
            float *sc = reinterpret_cast<float *>(smem + S::kOffSc) + vs * 2 * kTile;
            const int left = now.len - now.tok0;
            if (kTma) {
                const uint32_t full = bar(of_v ? B::kVFull + vs : B::kKFull + ks);
                if (of_v && offset < kTile) sc[(lane < 16 ? kTile : 0) + (lane & 15)] = lane < 16 ? now.vs : now.ks;
                __syncwarp();
                if (lane == 0) {
                    const int rows = 1 << maps.shift, most = left < kTile ? left : kTile;
                    mbar_arrive_expect_tx(full, static_cast<uint32_t>(((most + rows - 1) >> maps.shift << maps.shift) * D));
                }
                __syncwarp();
                // rows past the end come with the box: those of V are zeroed with the weights
                if (lane < 16 && offset < left && offset < kTile)
                    tma_4d((of_v ? to_v : to_k) + offset * D, of_v ? &maps.v : &maps.k, now.in, now.kv, now.page, full);
                __syncwarp();
            } else {
                constexpr int G16 = D / 16, R = 32 / G16;   // granules of a row, rows per instruction
                const int g = lane % G16, first = offset - lane;
                // rows past the end are zeros: whatever the page holds there stays unread
                auto copy = [&](const uint8_t *from, uint32_t to) {
#pragma unroll
                    for (int i = 0; i < 32 / R; ++i) {
                        const int row = i * R + lane / G16;
                        const uint64_t src = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(from), row);
                        cp_async16(to + swizzled<D>(first + row, g), reinterpret_cast<const uint8_t *>(src) + 16 * g,
                                   first + row < left ? 16 : 0);
                    }
                };
                copy(c.k + now.page * c.k_page + now.in * c.k_token + now.kv * c.k_head, to_k);
                arrive_landed(bar(B::kKFull + ks));
                copy(c.v + now.page * c.v_page + now.in * c.v_token + now.kv * c.v_head, to_v);
                arrive_landed(bar(B::kVFull + vs));
                sc[offset] = now.ks;
                sc[kTile + offset] = now.vs;
                arrive(B::kVFull + vs);
            }
#pragma unroll
            for (int i = 0; i + 1 < kDeep; ++i) spots[i] = spots[i + 1];
            spots[kDeep - 1] = far;
        }
        // the last copies land before the block ends, whatever the others do
        cp_async_wait_all();
        if (kTma) {
            const int places = of_v ? S::kValues : S::kKeys, first = of_v ? B::kVFull : B::kKFull;
            for (int j = turn; j < n; j += turns)
                if (j + places >= n) mbar_wait(bar(first + j % places), j / places & 1, kLandNs);
        }
    } else if (warp == S::kMmaWarpS) {
        // ------------------------------------------------------------------------- S^T = K Q^T
        constexpr uint32_t kId = idesc8(kTile, S::kQRows);
        Place<S::kSBufs> sp;
        Place<S::kKeys> kp;
        for (int pc = 0;; ++pc) {
            const Piece &piece = piece_at(pc);
            const int tile0 = piece.tile0, tile1 = piece.tile1;
            if (tile1 == 0 || stopped()) break;
            const uint64_t q = desc<D>(sb + S::kOffQ + pc % S::kQBufs * S::kQRows * D);
            for (int tile = tile0; tile < tile1; ++tile, sp.step(), kp.step()) {
                if (sp.turn > 0) wait(B::kSEmpty + sp.at, sp.turn - 1);
                wait(B::kKFull + kp.at, kp.turn);
                if (kp.at == 0) *static_cast<volatile unsigned long long *>(&s_moved) = globaltimer();
                fence_async();   // (the threads' copies were ordinary writes)
                tc::fence_after();
                const uint64_t k8 = desc<D>(sb + kp.at * S::kTileBytes);
#pragma unroll
                for (int k = 0; k < D / 32; ++k)   // 32 channels
                    mma8(tm + sp.at * S::kQRows, k8 + k * (32 >> 4), q + k * (32 >> 4), kId, k > 0);
                mma_commit(bar(B::kSFull + sp.at));
                mma_commit(bar(B::kKEmpty + kp.at));
                if (tile + 1 == tile1) mma_commit(bar(B::kQEmpty + pc % S::kQBufs));
            }
        }
        drain(0);
    } else if (warp == S::kMmaWarpO) {
        // ------------------------------------------------------------------------ O^T = V^T P^T
        constexpr uint32_t kId = idesc8(D, S::kPRows) | kAMajor | kBMajor;
        constexpr bool kQueries = S::kQueryWarp == S::kMmaWarpO;
        if (kQueries) queries(0, w.next(lens, items));
        Place<S::kPBufs> pp;
        Place<S::kValues> vp;
        for (int pc = 0;; ++pc) {
            const Piece &piece = piece_at(pc);
            const int count = piece.tile1 == 0 ? 0 : piece.tile1 - piece.tile0;
            if (count == 0 || stopped()) break;
            if (kQueries) queries(pc + 1, w.next(lens, items));   // (a piece ahead)
            else arrive(B::kQEmpty + pc % S::kQBufs);
            for (int i = 0; i < count; ++i, pp.step(), vp.step()) {
                const int b = pp.at;
                // (the weights are there: O's buffer is free)
                wait(B::kVFull + vp.at, vp.turn);
                wait(B::kPFull + b, pp.turn);
                fence_async();
                tc::fence_after();
                const uint64_t v = desc<D>(sb + S::kOffV + vp.at * S::kTileBytes);
                const uint64_t q = desc<S::kPRows>(sb + S::kOffP + b * S::kPRows * kTile);
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k)   // 32 tokens
                    mma8(tm + S::kTmO + b * S::kPRows, v + k * (32 * D >> 4), q + k * (32 * S::kPRows >> 4), kId, k > 0);
                mma_commit(bar(B::kOFull + b));
                mma_commit(bar(B::kVEmpty + vp.at));
            }
        }
        drain(1);
    } else if (S::kQueryWarp != S::kMmaWarpO && warp == S::kQueryWarp) {
        bool more = true;
        for (int pc = 0; more; ++pc) {
            more = w.next(lens, items);
            queries(pc, more);
        }
    } else if (warp < S::kOutWarp) {
        // --------------------------------------------------- the weights; a thread has a token
        const int g = warp >> 2, q = warp & 3, t = 32 * q + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        float *maxima = reinterpret_cast<float *>(smem + S::kOffMax) + g * 2 * 4 * 2 * H;
        float *cast = reinterpret_cast<float *>(smem + S::kOffCast) + warp * 3 * H;
        int n = 0;
        Place<S::kValues> vp;
        Place<S::kPBufs> pp;
        for (int pc = 0;; ++pc) {
            const Piece &piece = piece_at(pc);
            const int tile0 = piece.tile0, tile1 = piece.tile1, len = piece.len;
            if (group_any(1 + g, tile1 == 0 || stopped())) break;
            float mul[H], l[H], top = -CUDART_INF_F;   // top: lane h has head h's
#pragma unroll
            for (int h = 0; h < H; ++h) {
                mul[h] = reinterpret_cast<const float *>(smem + S::kOffMul)[pc % S::kQBufs * H + h];
                l[h] = 0.f;
            }
            arrive(B::kQEmpty + pc % S::kQBufs);
            for (int tile = tile0; tile < tile1; ++tile, ++n, vp.step(), pp.step()) {
                if (n % S::kGroups != g) continue;
                const int vs = vp.at, b = pp.at, sbuf = n % S::kSBufs;
                wait(B::kVFull + vs, vp.turn);
                wait(B::kSFull + sbuf, n / S::kSBufs);
                tc::fence_after();
                const float *sc = reinterpret_cast<const float *>(smem + S::kOffSc) + vs * 2 * kTile + (kTma ? t >> maps.shift : t);
                const float ks = sc[0];
                uint32_t raw[S::kQRows / 16][16];
#pragma unroll
                for (int i = 0; i < S::kQRows / 16; ++i) tc::ld16(tm + lanes + sbuf * S::kQRows + 16 * i, raw[i]);
                tc::ld_wait();
                tc::fence_before();
                arrive(B::kSEmpty + sbuf);
                const bool live = t < len - tile * kTile;
                const float lv = live ? __log2f(sc[kTile]) : 0.f;
                if (kTma && !live) {   // no weight of 0 makes an infinity or NaN vanish
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        *reinterpret_cast<uint4 *>(smem + S::kOffV + vs * S::kTileBytes + t * D + 16 * i) =
                            make_uint4(0, 0, 0, 0);
                }
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
                float *m = maxima + (n / S::kGroups & 1) * 4 * 2 * H;
                if (lane < 2 * H) m[q * 2 * H + lane] = mine;
                group_sync(1 + g);
                if (pp.turn > 0) wait(B::kOEmpty + b, pp.turn - 1);
                if (lane < 2 * H) {
                    const float all = fmaxf(fmaxf(m[lane], m[2 * H + lane]), fmaxf(m[4 * H + lane], m[6 * H + lane]));
                    if (lane < H) {
                        const float now = fmaxf(top, all), base = finite_base(now);
                        cast[lane] = base;
                        cast[H + lane] = ex2(top - base);
                        top = now;
                    } else {
                        cast[H + lane] = finite_base(all) - 8.f;   // weights up to 2^8: e4m3 reaches 448
                        if (q == 0) reinterpret_cast<float *>(smem + S::kOffStat)[b * H + lane - H] = all;
                    }
                }
                __syncwarp();
                uint32_t terms[kPTerms][H / 4];   // the token's row of P
#pragma unroll
                for (int h = 0; h < H; h += 4) {
                    const float4 xb = *reinterpret_cast<const float4 *>(cast + h);
                    const float4 fb = *reinterpret_cast<const float4 *>(cast + H + h);
                    const float4 yb = *reinterpret_cast<const float4 *>(cast + 2 * H + h);
                    const float xs[4] = {xb.x, xb.y, xb.z, xb.w}, fs[4] = {fb.x, fb.y, fb.z, fb.w},
                                ys[4] = {yb.x, yb.y, yb.z, yb.w};
                    float wt[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        l[h + j] = fmaf(l[h + j], fs[j], ex2(x[h + j] - xs[j]));
                        wt[j] = ex2(x[h + j] + lv - ys[j]);
                    }
                    uint32_t lo[kPTerms], hi[kPTerms];
                    split4(wt[0], wt[1], lo);
                    split4(wt[2], wt[3], hi);
#pragma unroll
                    for (int k = 0; k < kPTerms; ++k) terms[k][h / 4] = lo[k] | (hi[k] << 16);
                }
                uint8_t *dst = smem + S::kOffP + b * S::kPRows * kTile;
#pragma unroll
                for (int i = 0; i < S::kPRows / 16; ++i) {
                    const uint32_t *from = &terms[0][0] + 4 * i;
                    *reinterpret_cast<uint4 *>(dst + swizzled<S::kPRows>(t, i)) = make_uint4(from[0], from[1], from[2], from[3]);
                }
                fence_async();
                arrive(B::kPFull + b);
            }
            // the piece's sums
            if (pc >= 2) wait(B::kLEmpty + (pc & 1), (pc >> 1) - 1);
            const float sum = lane_sums(l, lane);
            const int h = lane * H / 32;
            if (lane * H % 32 == 0)
                reinterpret_cast<float *>(smem + S::kOffSum)[((pc & 1) * 4 * S::kGroups + warp) * H + h] = sum;
            if (lane < H && q == 0) reinterpret_cast<float *>(smem + S::kOffTop)[((pc & 1) * S::kGroups + g) * H + lane] = top;
            arrive(B::kLFull + (pc & 1));
        }
    } else {
        // ------------------------------------------------- the outputs; a thread has a channel
        const int q = warp & 3, t = 32 * q + lane;
        // (64 channels: rows 16 q .. of O^T lie in a quarter's first 16 lanes)
        const int d = D == 128 ? t : 16 * q + lane;
        const bool has = D == 128 || lane < 16;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        constexpr int kOutSync = 1 + S::kGroups;
        const int64_t U = sh.U, G = sh.G;
        const int me = blockIdx.x;
        float *join = reinterpret_cast<float *>(smem + S::kOffJoin);
        Place<S::kPBufs> pp;
        auto item_counter = [&](const Piece &piece) { return arrived + 2 * kPlannedSms + static_cast<int64_t>(piece.b) * items + piece.item; };
        auto owners = [&](const Piece &piece, int &c0, int &c1) {
            c0 = Paged8Split::owner(piece.item_at + kItemCost, U, G);
            c1 = Paged8Split::owner(piece.item_at + kItemCost + piece.tiles - 1, U, G);
        };
        // Which of the slots (and group counters) of block k, two of each, an item's piece has.
        auto slot_of = [&](const Piece &piece, int k, int c0) { return 2 * k + (k == c0 && c0 * U / G <= piece.item_at); };
        int pc = 0;
        float *cast = reinterpret_cast<float *>(smem + S::kOffCast) + warp * 3 * H;
        for (;; ++pc) {
            const Piece piece = piece_at(pc);
            if (group_any(kOutSync, piece.tile1 == 0 || stopped())) break;
            arrive(B::kQEmpty + pc % S::kQBufs);
            const int heads = piece.heads;
            float acc[H], top = -CUDART_INF_F;   // top: lane h has head h's
#pragma unroll
            for (int h = 0; h < H; ++h) acc[h] = 0.f;
            for (int tile = piece.tile0; tile < piece.tile1; ++tile, pp.step()) {
                const int b = pp.at;
                wait(B::kOFull + b, pp.turn);
                tc::fence_after();
                uint32_t raw[S::kPRows / 16][16];
#pragma unroll
                for (int i = 0; i < S::kPRows / 16; ++i)
                    tc::ld16(tm + lanes + S::kTmO + b * S::kPRows + 16 * i, raw[i]);
                if (lane < H) {
                    const float all = reinterpret_cast<const float *>(smem + S::kOffStat)[b * H + lane];
                    const float now = fmaxf(top, all), base = finite_base(now);
                    cast[lane] = ex2(top - base);
                    cast[H + lane] = ex2(all - base) * (1.f / 256);
                    top = now;
                }
                tc::ld_wait();
                tc::fence_before();
                arrive(B::kOEmpty + b);
#pragma unroll
                for (int h = 0; h < H; h += 4) {
                    const float4 fb = *reinterpret_cast<const float4 *>(cast + h);
                    const float4 gb = *reinterpret_cast<const float4 *>(cast + H + h);
                    const float fs[4] = {fb.x, fb.y, fb.z, fb.w}, gains[4] = {gb.x, gb.y, gb.z, gb.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = h + j;
                        float o = __uint_as_float(raw[(3 * H + i) / 16][(3 * H + i) % 16]);
#pragma unroll
                        for (int k = kPTerms - 2; k >= 0; --k)
                            o = fmaf(o, 1.f / kFiner, __uint_as_float(raw[(k * H + i) / 16][(k * H + i) % 16]));
                        acc[i] = fmaf(acc[i], fs[j], o * gains[j]);
                    }
                }
                __syncwarp();   // (`cast` is read)
            }
            // ---- the piece's end: lane h has the sum and maximum of head h
            const bool whole = piece.tile0 == 0 && piece.tile1 == piece.tiles;
            // of a block's partial pieces only its first can belong to an item that
            // started in front of its share, and only its last to another one
            float *slot = slots + static_cast<int64_t>(2 * me + (sh.u0 <= piece.item_at)) * S::kSlot;
            wait(B::kLFull + (pc & 1), pc >> 1);
            {
                float sum = 0.f, most = -CUDART_INF_F;
                if (lane < H) {
                    const float *ls = reinterpret_cast<const float *>(smem + S::kOffSum) + (pc & 1) * 4 * S::kGroups * H + lane;
                    const float *ms = reinterpret_cast<const float *>(smem + S::kOffTop) + (pc & 1) * S::kGroups * H + lane;
#pragma unroll
                    for (int g = 0; g < S::kGroups; ++g) most = fmaxf(most, ms[g * H]);
                    const float base = finite_base(most);
#pragma unroll
                    for (int g = 0; g < S::kGroups; ++g)
                        sum = fmaf((ls[4 * g * H] + ls[(4 * g + 1) * H]) + (ls[(4 * g + 2) * H] + ls[(4 * g + 3) * H]),
                                   ex2(ms[g * H] - base), sum);
                }
                arrive(B::kLEmpty + (pc & 1));
                const int64_t row = piece.row;
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
            int c0, c1;
            owners(piece, c0, c1);
            join_pieces<D, H>(slots, arrived, item_counter(piece), c0, c1, slot_of(piece, c0, c0), static_cast<__nv_bfloat16 *>(p.out) + piece.row * D,
                              p.lse != nullptr ? p.lse + piece.row : nullptr, heads, join, &s_last);
            // (the next piece's join comes after barriers of its own: `join` is read by then)
        }
        // Where a wait has run out, the arrivals for the pieces that are left, so that the counters
        // are right for the next call.
        if (q == 0 && lane == 0 && stopped())
            for (int i = 0; w.next(lens, items); ++i) {
                if (i < pc || (w.tile0 == 0 && w.tile1 == w.tiles)) continue;
                Piece piece{};
                piece.item_at = w.item_at;
                piece.tiles = w.tiles;
                piece.b = w.b;
                piece.item = w.item;
                int c0, c1;
                owners(piece, c0, c1);
                const int n = c1 - c0 + 1, lo = c0 + (me - c0) / kJoined * kJoined;
                if (n <= kFlat) last_of(item_counter(piece), n);
                else if (last_of(arrived + slot_of(piece, lo, c0), min(kJoined, c1 + 1 - lo)))
                    last_of(item_counter(piece), (n - 1) / kJoined + 1);
            }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::dealloc(tm, S::kTmCols);
}

constexpr int heads_of(int group) { return group <= 8 ? 8 : 16; }

// Pages of a multiple of 8 tokens are copied by the tensor memory accelerator, in boxes of
// the largest power of two that divides them; others by threads, 16 bytes a time (2 x 131072
// tokens, pages of 32: 92 us and 115; 64 ragged sequences, pages of 64: 50 and 68).
int box_rows(const Cache8 &c) {
    const int two = c.page_size & -c.page_size;
    return two < 8 ? 0 : two < kTile ? two : kTile;
}

template <typename F>
auto with_shape(const Paged8Params &p, F &&go) {
    const bool few = heads_of(p.hq / p.c.hkv) == 8, tma = box_rows(p.c) > 0;
    auto pick = [&](auto s, auto bytes, auto with, auto without) { return go(s, tma ? with : without, bytes, threads_of(decltype(s)::kHeads, tma)); };
    if (p.c.dim == 64)
        return few ? pick(Shape<64, 8>(), smem_bytes<64, 8>(), paged8_kernel<64, 8, true>, paged8_kernel<64, 8, false>)
                   : pick(Shape<64, 16>(), smem_bytes<64, 16>(), paged8_kernel<64, 16, true>, paged8_kernel<64, 16, false>);
    return few ? pick(Shape<128, 8>(), smem_bytes<128, 8>(), paged8_kernel<128, 8, true>, paged8_kernel<128, 8, false>)
               : pick(Shape<128, 16>(), smem_bytes<128, 16>(), paged8_kernel<128, 16, true>, paged8_kernel<128, 16, false>);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode(CUtensorMap *m, const Cache8 &c, const uint8_t *base, int64_t page, int64_t token, int64_t head) {
    const EncodeFn enc = reinterpret_cast<EncodeFn>(tensor_map_encoder());
    if (enc == nullptr) return false;
    // an axis of one row has no step of its own
    const int64_t row = c.dim;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.hkv), static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.page_size > 1 ? token : row),
                                   static_cast<cuuint64_t>(c.hkv > 1 ? head : row),
                                   static_cast<cuuint64_t>(c.pages > 1 ? page : row)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(c.dim), static_cast<cuuint32_t>(box_rows(c)), 1, 1},
                     estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, c.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t chunks_of(const Paged8Params &p) {
    const int group = p.hq / p.c.hkv, h = heads_of(group);
    return (group + h - 1) / h;
}

static_assert(smem_bytes<128, 16>() <= 232448 - 1024, "what a block can have");

}  // namespace

cudaError_t configure_paged8() {
    for (int dim : {64, 128})
        for (int group : {1, 16})
            for (int page : {1, 16}) {
                Paged8Params p{};
                p.c.dim = dim;
                p.c.page_size = page;
                p.c.hkv = 1;
                p.hq = group;
                const cudaError_t e = with_shape(p, [](auto, auto kernel, int bytes, int) {
                    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
                });
                if (e != cudaSuccess) return e;
            }
    return cudaSuccess;
}

// Two partial results per block.
int64_t paged8_workspace(const Paged8Params &p) {
    return with_shape(p, [](auto s, auto, int, int) {
        return static_cast<int64_t>(kPlannedSms) * 2 * decltype(s)::kSlot * 4;
    });
}

// Arrival counters: two per block for groups of pieces, then one per (sequence, work item).
int64_t paged8_sync(const Paged8Params &p) {
    return (2 * kPlannedSms + static_cast<int64_t>(p.c.batch) * p.c.hkv * chunks_of(p)) * 4;
}

cudaError_t launch_paged8(const Paged8Params &p, const CallContext &ctx, cudaStream_t stream) {
    // Units the lengths may come to; empty sequences need a block as well. An item of n units is not
    // cut into more than some 2 sqrt(n) pieces, as a unit takes a block four times as long as a
    // piece takes the join, or, where that makes groups of pieces, into 4 sqrt(n). (Cut as finely
    // as it goes, joined at once: two sequences of up to 12893 tokens, one key-value head, 24 us
    // for 16; one of 131072 36 for 21; 8192 tokens, 8 heads, 16 for 15.)
    const int64_t items = static_cast<int64_t>(p.c.batch) * p.c.hkv * chunks_of(p),
                  units = Paged8Split::units_of(p.c.max_pages * p.c.page_size);
    auto root = [](int64_t x) {
        int64_t r = 1;
        while (r < kPlannedSms && (r + 1) * (r + 1) <= x) ++r;
        return r;
    };
    int64_t pieces = root(4 * units);
    if (pieces > kFlat) pieces = root(16 * units);
    if (pieces > units) pieces = units;
    const unsigned grid = static_cast<unsigned>(items * pieces < 1 ? 1 : items * pieces < kPlannedSms ? items * pieces : kPlannedSms);
    Paged8Maps maps{};
    while (2 << maps.shift <= box_rows(p.c)) ++maps.shift;
    if (box_rows(p.c) > 0 && p.c.pages > 0 &&
        (!encode(&maps.k, p.c, p.c.k, p.c.k_page, p.c.k_token, p.c.k_head) ||
         !encode(&maps.v, p.c, p.c.v, p.c.v_page, p.c.v_token, p.c.v_head)))
        return cudaErrorInvalidValue;
    return with_shape(p, [&](auto, auto kernel, int bytes, int threads) {
        kernel<<<grid, threads, bytes, stream>>>(maps, p, reinterpret_cast<float *>(ctx.ws), ctx.sync);
        return cudaGetLastError();
    });
}

}  // namespace kda
