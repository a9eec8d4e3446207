// Attention of one new token per sequence over a paged key-value cache
// (kda_paged_decode): out = softmax(scale q K^T) V and its log-sum-exp, one
// pass over the cache with the running maximum and sum of the softmax.
//
// Every key and value is used once per query head that shares it, so the
// operator is bound by reading the cache: 4 D B per (token, key-value head).
//
// Split. The cache is cut into tiles of 64 tokens of one work item (sequence,
// key-value head, up to 16 of its query heads). An item costs its tiles and
// kItemCost more for its start and end; these units are numbered sequence by
// sequence, and CTA c of G takes the units [c U / G, (c + 1) U / G): all CTAs
// have the same work, be the lengths ragged, few or one. A CTA's tiles of one
// item are a piece. A piece that is the whole item writes the result; the
// others leave their maximum, sum and unnormalised output in the workspace,
// and the last CTA to arrive joins them in CTA order (which one that is does
// not change the result).
//
// Inside a CTA each of 4 warps works for itself on strips of 16 tokens with a
// ring of kStages strips in shared memory, so nothing waits on a block barrier
// but the join at the end of a piece. Its copies run ahead across the ends of pieces:
// while one is joined, the next one's keys are on their way (64 sequences of 1 to 16384
// tokens: 80 to 102 us, and 94 to 117 with a start from nothing at each piece).
// The products are formed transposed,
// S^T = K Q^T (16 tokens x 8 heads per MMA) and O^T = V^T P^T: a group of 8 or
// fewer query heads then fills the N = 8 side of one MMA instead of half of
// an M = 16 side. P goes from accumulators to operand with an 8 x 8 register
// transpose. It enters the product as two bf16 terms (16 bits of mantissa
// together): the tensor pipe is far from busy here, and one term alone would
// add an error as large as the output's own rounding.
//
// Measured: 2 sequences of 131072 tokens, 32 heads over 8 of 128: 163 us (6.6 TB/s,
// 97 % of copy bandwidth); 64 sequences of 1 to 16384 tokens, 64 heads over 8: 73 to 94 us
// (81 to 86 %, by the lengths drawn); one of 700 tokens: 12 us, a chain of latencies.

#include <math_constants.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kPagedWarps = 4;
constexpr int kStrip = 16;                      // tokens per warp step
constexpr int kTile = kPagedWarps * kStrip;     // tokens per tile of the split
// Start and end of an item, in tiles: the join, and steps that wait for the first keys
// (those 64 sequences: 100 to 129 us with 1, 78 to 99 with 2, 73 to 94 with 3 or 4).
constexpr int kItemCost = 4;
constexpr int kStages = 3;                      // strips in flight per warp
constexpr int kPagedCtasPerSm = 2;
constexpr int kMaxCtas = kPlannedSms * kPagedCtasPerSm;

// Heads of one work item: 8 NT query heads of one key-value head. Two sets of 8 share
// one reading of the keys and values; larger groups read them again, out of L2, as
// four sets would not fit in registers (8 sequences of 32768 tokens, 2 key-value heads of
// 128, groups of 16 and 32: with one set 88 and 160 us, with two 59 and 92).
struct Plan {
    int nt;       // 1 or 2
    int chunks;   // items per key-value head
};

__host__ __device__ inline Plan plan_heads(int group) {
    const int nt = group <= 8 ? 1 : 2;
    return {nt, (group + 8 * nt - 1) / (8 * nt)};
}

template <int D, int NT>
struct Shape {
    static constexpr int kRow = 2 * D;                       // bytes of a row in shared memory
    static constexpr int kStage = 2 * kStrip * kRow;         // K and V of a strip
    static constexpr int kWarpBytes = kStages * kStage;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kOut = D + 4;                       // padded floats of an output row
    static constexpr int kSmem = kPagedWarps * kWarpBytes;
    static constexpr int kSlot = kHeads * (D + 2);           // floats of one partial result
    static_assert(8 * kOut * 4 <= kStage, "outputs go through a slot of the ring");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Tokens of sequence b, or 0 where the length cannot be right.
__device__ __forceinline__ int length_of(const PagedParams &p, int b, bool *bad) {
    const int len = __ldg(p.lens + b);
    if (len < 0 || len > p.max_pages * p.page_size || (len > 0 && p.pages == 0)) {
        *bad = true;
        return 0;
    }
    return len;
}

// Units of an item of a sequence of this length.
__host__ __device__ __forceinline__ int64_t units_of(int64_t len) {
    return len > 0 ? (len + kTile - 1) / kTile + kItemCost : 0;
}

// Owner of unit u when G CTAs split U units evenly.
__device__ __forceinline__ int owner(int64_t u, int64_t U, int64_t G) {
    return static_cast<int>(((u + 1) * G - 1) / U);
}

// Adds to a counter, after this block's writes before the barrier in front of it and before
// its reads behind the next one.
__device__ __forceinline__ int add_acq_rel(int *p, int v) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;\n" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// A CTA's way through its share [u, u1) of the units, piece by piece.
struct Pieces {
    int64_t u, u1, seq_at;   // next unit; end of the share; first unit of sequence b
    int b;
    // the piece: its item, and the tiles of it
    int len, tiles, item, tile0, tile1;
    int64_t item_at;

    __device__ __forceinline__ bool next(const PagedParams &p, int items) {
        while (u < u1) {
            bool ignore = false;
            len = length_of(p, b, &ignore);
            const int64_t units = units_of(len);
            if (u >= seq_at + units * items) {
                seq_at += units * items;
                ++b;
                continue;
            }
            tiles = static_cast<int>(units) - kItemCost;
            item = static_cast<int>((u - seq_at) / units);
            item_at = seq_at + item * units;
            const int64_t tile_at = item_at + kItemCost;
            // the tiles among the units [u, min(u1, end of the item))
            tile0 = static_cast<int>(u > tile_at ? u - tile_at : 0);
            tile1 = static_cast<int>(u1 - tile_at < tiles ? u1 - tile_at : tiles);
            u = item_at + units;
            if (tile0 < tile1) return true;
        }
        return false;
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(kPagedWarps * 32, kPagedCtasPerSm)
paged_kernel(PagedParams p, float *slots, int *arrived) {
    using S = Shape<D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sum[kPagedWarps], s_off;
    __shared__ int s_first, s_last;
    __shared__ float s_m[kPagedWarps][8], s_l[kPagedWarps][8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = p.hq / p.hkv, chunks = (group + S::kHeads - 1) / S::kHeads;
    const int items = p.hkv * chunks;   // work items of a sequence

    // ---- the split: units before each thread's run of sequences, by a block scan
    const int per = (p.batch + kPagedWarps * 32 - 1) / (kPagedWarps * 32);
    bool bad = false;
    int64_t mine = 0;
    for (int i = 0, b = tid * per; i < per && b < p.batch; ++i, ++b)
        mine += units_of(length_of(p, b, &bad)) * items;
    if (bad && blockIdx.x == 0) atomicOr(p.err, kErrPage);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, U = 0;
#pragma unroll
    for (int w = 0; w < kPagedWarps; ++w) {
        if (w < warp) before += s_sum[w];
        U += s_sum[w];
    }
    const int64_t G = U < gridDim.x ? U : gridDim.x;

    // sequences without tokens
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        bool ignore = false;
        if (length_of(p, b, &ignore) != 0) continue;
        for (int i = tid; i < p.hq * D / 8; i += kPagedWarps * 32)
            reinterpret_cast<uint4 *>(p.out)[static_cast<int64_t>(b) * (p.hq * D / 8) + i] =
                make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr)
            for (int i = tid; i < p.hq; i += kPagedWarps * 32)
                p.lse[static_cast<int64_t>(b) * p.hq + i] = -CUDART_INF_F;
    }
    const int c = blockIdx.x;
    if (c >= G) return;
    const int64_t u0 = c * U / G, u1 = (c + 1) * U / G;
    if (u0 >= before && u0 < before + mine) {   // one thread of the block
        int64_t at = before;
        int b = tid * per;
        for (;; ++b) {
            bool ignore = false;
            const int64_t n = units_of(length_of(p, b, &ignore)) * items;
            if (u0 < at + n) break;
            at += n;
        }
        s_first = b;
        s_off = at;
    }
    __syncthreads();

    uint8_t *ring = smem + warp * S::kWarpBytes;
    const uint32_t ring_u = smem_u32(ring);
    const float to_log2 = p.scale * 1.44269504088896341f;
    const int q4 = lane & 3, r8 = lane >> 2;

    // ---- copies: they run kStages - 1 strips ahead, across the ends of pieces. The
    // page of this lane's token (lanes 16..31 repeat 0..15) is read a strip earlier.
    Pieces ahead{u0, u1, s_off, s_first};
    bool more = ahead.next(p, items);
    int tile = ahead.tile0, page = 0;
    auto page_of = [&] {
        const int t = tile * kTile + warp * kStrip + (lane & 15);
        page = more && t < ahead.len
                   ? __ldg(p.table + static_cast<int64_t>(ahead.b) * p.max_pages + t / p.page_size)
                   : 0;
    };
    int loaded = 0;   // strips
    auto load = [&] {
        if (more) {
            const int tok0 = tile * kTile + warp * kStrip, t = tok0 + (lane & 15), len = ahead.len;
            const int kv = ahead.item / chunks;
            int pg = page;
            if (++tile == ahead.tile1) {
                more = ahead.next(p, items);
                tile = ahead.tile0;
            }
            page_of();
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.pages)) {
                if (t < len) atomicOr(p.err, kErrPage);
                pg = 0;
            }
            const int64_t in = (static_cast<int64_t>(t % p.page_size) * p.hkv + kv) * D;
            const int64_t ka = pg * p.k_stride + in, va = pg * p.v_stride + in;
            const uint32_t dst = ring_u + loaded % kStages * S::kStage;
            constexpr int G16 = D / 8;             // 16-byte granules of a row
            constexpr int R = 32 / G16;            // rows per instruction
            const int g = lane % G16;
#pragma unroll
            for (int i = 0; i < kStrip / R; ++i) {
                const int row = i * R + lane / G16;
                const int64_t kr = __shfl_sync(0xffffffffu, ka, row);
                const int64_t vr = __shfl_sync(0xffffffffu, va, row);
                const uint32_t at = dst + row * S::kRow + ((g ^ (row & 7)) << 4);
                // rows past the end are zeros: whatever the page holds there stays unread
                const uint32_t n = tok0 + row < len ? 16 : 0;
                cp_async16(at, static_cast<const uint16_t *>(p.k) + kr + g * 8, n);
                cp_async16(at + kStrip * S::kRow, static_cast<const uint16_t *>(p.v) + vr + g * 8, n);
            }
            ++loaded;
        }
        cp_async_commit();
    };
    page_of();
#pragma unroll 1
    for (int s = 0; s < kStages - 1; ++s) load();

    Pieces w{u0, u1, s_off, s_first};
    int taken = 0;   // strips
    while (w.next(p, items)) {
        const int kv = w.item / chunks, head0 = kv * group + w.item % chunks * S::kHeads;
        const int heads = min(S::kHeads, group - w.item % chunks * S::kHeads);
        // ---- Q^T fragments: k = channel, n = head
        uint32_t qf[D / 16][NT][2];
        {
            const uint32_t *q = reinterpret_cast<const uint32_t *>(p.q) +
                                (static_cast<int64_t>(w.b) * p.hq + head0) * (D / 2);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int h = t * 8 + r8;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qf[k][t][0] = h < heads ? __ldg(q + h * (D / 2) + k * 8 + q4) : 0u;
                    qf[k][t][1] = h < heads ? __ldg(q + h * (D / 2) + k * 8 + 4 + q4) : 0u;
                }
            }
        }

        float o[D / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -CUDART_INF_F;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][t][e] = 0.f;
        }
        for (int step = w.tile0; step < w.tile1; ++step, ++taken) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            load();   // into the slot that the last step freed
            const int left = w.len - step * kTile - warp * kStrip;   // tokens of this strip, if < 16
            if (left <= 0) continue;
            const uint32_t ks = ring_u + taken % kStages * S::kStage, vs = ks + kStrip * S::kRow;

            // ---- S^T = K Q^T, two sums per tile to shorten the chain
            float st[NT][2][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[t][0][e] = st[t][1][e] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int row = lane & 15, g = 2 * k + (lane >> 4);
                uint32_t a[4];
                ldsm_x4(ks + row * S::kRow + ((g ^ (row & 7)) << 4), a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(st[t][k & 1], a, qf[k][t][0], qf[k][t][1]);
            }
            uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = (st[t][0][e] + st[t][1][e]) * to_log2;
                    if (r8 + (e >> 1) * 8 >= left) v[e] = -CUDART_INF_F;
                }
                float f[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {   // the lane's two heads
                    float x = fmaxf(v[j], v[j + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    const float top = fmaxf(m[t][j], x);
                    const float base = top == -CUDART_INF_F ? 0.f : top;
                    f[j] = ex2(m[t][j] - base);
                    m[t][j] = top;
                    v[j] = ex2(v[j] - base);
                    v[j + 2] = ex2(v[j + 2] - base);
                    l[t][j] = fmaf(l[t][j], f[j], v[j] + v[j + 2]);
                }
                if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        mul2(o[i][t][0], o[i][t][1], f[0], f[1]);
                        mul2(o[i][t][2], o[i][t][3], f[0], f[1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t w = pack_bf16(v[2 * j], v[2 * j + 1]);
                    const float2 b2 = unpack_bf16(w);
                    hi[t][j] = transpose8(w);
                    lo[t][j] = transpose8(pack_bf16(v[2 * j] - b2.x, v[2 * j + 1] - b2.y));
                }
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const int row = (lane & 7) + ((lane >> 4) << 3), g = 2 * i + ((lane >> 3) & 1);
                uint32_t a[4];
                ldsm_x4_t(vs + row * S::kRow + ((g ^ (row & 7)) << 4), a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mma16816(o[i][t], a, hi[t][0], hi[t][1]);
                    mma16816(o[i][t], a, lo[t][0], lo[t][1]);
                }
            }
            __syncwarp();   // the slot is free once every lane has read it
        }

        // ---- join the warps: 8 heads at a time, each warp's output through the slot of
        // its ring that the last step freed
        const bool whole = w.tile0 == 0 && w.tile1 == w.tiles;
        // of a CTA's partial pieces only its first can belong to an item that
        // started in front of its share, and only its last to another one
        float *slot = slots + static_cast<int64_t>(2 * c + (u0 <= w.item_at)) * S::kSlot;
        const int freed = (taken - 1) % kStages * S::kStage;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], d);
                const int h = 2 * q4 + j;
                if (r8 == 0) {
                    s_m[warp][h] = m[t][j];
                    s_l[warp][h] = l[t][j];
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    float *row = reinterpret_cast<float *>(ring + freed) + h * S::kOut + 16 * i + r8;
                    row[0] = o[i][t][j];
                    row[8] = o[i][t][j + 2];
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = tid; i < 8 * D; i += kPagedWarps * 32) {
                const int h = i / D, d = i % D;
                float top = -CUDART_INF_F;
#pragma unroll
                for (int v = 0; v < kPagedWarps; ++v) top = fmaxf(top, s_m[v][h]);
                const float base = top == -CUDART_INF_F ? 0.f : top;
                float acc = 0.f, sum = 0.f;
#pragma unroll
                for (int v = 0; v < kPagedWarps; ++v) {
                    const float f = ex2(s_m[v][h] - base);
                    acc = fmaf(reinterpret_cast<const float *>(smem + v * S::kWarpBytes + freed)[h * S::kOut + d],
                               f, acc);
                    sum = fmaf(s_l[v][h], f, sum);
                }
                if (8 * t + h >= heads) continue;
                if (whole) {
                    const int64_t row = static_cast<int64_t>(w.b) * p.hq + head0 + 8 * t + h;
                    static_cast<__nv_bfloat16 *>(p.out)[row * D + d] =
                        __float2bfloat16_rn(sum > 0.f ? acc / sum : sum == 0.f ? 0.f : sum);
                    if (d == 0 && p.lse != nullptr)
                        p.lse[row] = sum == 0.f ? -CUDART_INF_F : base * 0.69314718055994531f + logf(sum);
                } else {
                    slot[(8 * t + h) * D + d] = acc;
                    if (d == 0) {
                        slot[S::kHeads * D + 8 * t + h] = top;
                        slot[S::kHeads * (D + 1) + 8 * t + h] = sum;
                    }
                }
            }
            if (t + 1 < NT) __syncthreads();
        }
        if (!whole) {
            // ---- the last CTA of this (sequence, item) to arrive joins the pieces
            const int c0 = owner(w.item_at + kItemCost, U, G),
                      c1 = owner(w.item_at + kItemCost + w.tiles - 1, U, G);
            __syncthreads();   // (the slot is written)
            if (tid == 0) {
                int *ctr = arrived + static_cast<int64_t>(w.b) * items + w.item;
                const int n = add_acq_rel(ctr, 1) + 1;
                s_last = n == c1 - c0 + 1;
                if (s_last) *ctr = 0;   // for the next call
            }
            __syncthreads();
            if (s_last) {
                // A group of threads per head: each takes every so many-th piece's maximum
                // and sum, then VD channels of all pieces, several on their way at a time.
                // (A warp per head, piece after piece: 64 ragged sequences 76 to 97 us, this way
                // 73 to 94; 8 x 32768 tokens with groups of 16: 71 and 59.)
                constexpr int H = S::kHeads, kPer = kPagedWarps * 32 / H, VD = D / kPer;
                const int last = c0 * U / G <= w.item_at;
                const float *first = slots + static_cast<int64_t>(2 * c0 + last) * S::kSlot;
                auto piece = [&](int k) {
                    return k == c0 ? first : slots + static_cast<int64_t>(2 * k) * S::kSlot;
                };
                const int h = tid / kPer, j = tid % kPer;
                float top = -CUDART_INF_F, sum = 0.f;
                #pragma unroll 1
                for (int k = c0 + j; k <= c1 && h < heads; k += kPer) {
                    const float mk = __ldcg(piece(k) + H * D + h), lk = __ldcg(piece(k) + H * (D + 1) + h);
                    const float t = fmaxf(top, mk), base = t == -CUDART_INF_F ? 0.f : t;
                    sum = fmaf(sum, ex2(top - base), lk * ex2(mk - base));
                    top = t;
                }
                const float own = top;
#pragma unroll
                for (int d = 1; d < kPer; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float base = top == -CUDART_INF_F ? 0.f : top;
                sum *= ex2(own - base);
#pragma unroll
                for (int d = 1; d < kPer; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                float acc[VD];
#pragma unroll
                for (int e = 0; e < VD; ++e) acc[e] = 0.f;
#pragma unroll 4
                for (int k = c0; k <= c1 && h < heads; ++k) {
                    const float *src = piece(k);
                    const float f = ex2(__ldcg(src + H * D + h) - base);
#pragma unroll
                    for (int e = 0; e < VD; e += 4) {
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(src + h * D + j * VD + e));
                        acc[e] = fmaf(x.x, f, acc[e]);
                        acc[e + 1] = fmaf(x.y, f, acc[e + 1]);
                        acc[e + 2] = fmaf(x.z, f, acc[e + 2]);
                        acc[e + 3] = fmaf(x.w, f, acc[e + 3]);
                    }
                }
                if (h < heads) {
                    const int64_t row = static_cast<int64_t>(w.b) * p.hq + head0 + h;
                    uint32_t *out = static_cast<uint32_t *>(p.out) + (row * D + j * VD) / 2;
#pragma unroll
                    for (int e = 0; e < VD; e += 4) {
                        float y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[i] = sum > 0.f ? acc[e + i] / sum : sum == 0.f ? 0.f : sum;
                        *reinterpret_cast<uint2 *>(out + e / 2) =
                            make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                    }
                    if (j == 0 && p.lse != nullptr)
                        p.lse[row] = sum == 0.f ? -CUDART_INF_F : base * 0.69314718055994531f + logf(sum);
                }
            }
        }
        __syncthreads();   // the rings and the joined statistics are free again
    }
}

template <typename F>
auto with_shape(const PagedParams &p, F &&go) {
    const int nt = plan_heads(p.hq / p.hkv).nt;
    if (p.dim == 64)
        return nt == 1 ? go(Shape<64, 1>(), paged_kernel<64, 1>)
                       : go(Shape<64, 2>(), paged_kernel<64, 2>);
    return nt == 1 ? go(Shape<128, 1>(), paged_kernel<128, 1>)
                   : go(Shape<128, 2>(), paged_kernel<128, 2>);
}

}  // namespace

cudaError_t configure_paged() {
    for (int dim : {64, 128})
        for (int group : {1, 16}) {
            PagedParams p{};
            p.dim = dim;
            p.hq = group;
            p.hkv = 1;
            const cudaError_t e = with_shape(p, [](auto s, auto kernel) {
                return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            decltype(s)::kSmem);
            });
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

// Two partial results per CTA.
int64_t paged_workspace(const PagedParams &p) {
    return with_shape(p, [](auto s, auto) {
        return static_cast<int64_t>(kMaxCtas) * 2 * decltype(s)::kSlot * 4;
    });
}

// One arrival counter per (sequence, work item).
int64_t paged_sync(const PagedParams &p) {
    return static_cast<int64_t>(p.batch) * p.hkv * plan_heads(p.hq / p.hkv).chunks * 4;
}

cudaError_t launch_paged(const PagedParams &p, const CallContext &ctx, cudaStream_t stream) {
    // units the lengths may come to; empty sequences need a CTA as well
    const int64_t most = p.max_pages * p.page_size;
    const int64_t units = static_cast<int64_t>(p.batch) * p.hkv *
                          plan_heads(p.hq / p.hkv).chunks * units_of(most);
    const unsigned grid =
        static_cast<unsigned>(units < 1 ? 1 : units < kMaxCtas ? units : kMaxCtas);
    return with_shape(p, [&](auto s, auto kernel) {
        kernel<<<grid, kPagedWarps * 32, decltype(s)::kSmem, stream>>>(
            p, reinterpret_cast<float *>(ctx.ws), ctx.sync);
        return cudaGetLastError();
    });
}

}  // namespace kda
