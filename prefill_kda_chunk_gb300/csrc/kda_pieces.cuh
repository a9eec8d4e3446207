// How the decode attention kernels share a batch of caches of any lengths out to their
// blocks. A cache is cut into tiles of kTile tokens of one work item (sequence,
// key-value head, a set of its query heads). An item costs its tiles and kCost more for
// its start and end; these units are numbered sequence by sequence, and block c of G
// takes the units [c U / G, (c + 1) U / G): all blocks have the same work, be the
// lengths ragged, few or one. A block's tiles of one item are a piece.
#pragma once

#include <stdint.h>

#include "kda_device.cuh"

namespace kda {

struct Lengths {
    const int32_t *lens;
    int64_t most;     // tokens that a row of the page table can hold
    int32_t batch;
    bool pages;       // whether there are any
    // Tokens of sequence b, or 0 where the length cannot be right.
    __device__ __forceinline__ int of(int b, bool *bad) const {
        const int len = __ldg(lens + b);
        if (len < 0 || len > most || (len > 0 && !pages)) {
            *bad = true;
            return 0;
        }
        return len;
    }
};

// Adds to a counter, after this block's writes before the barrier in front of it and before
// its reads behind the next one.
__device__ __forceinline__ int add_acq_rel(int *p, int v) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;\n" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

template <int kTile, int kCost>
struct Split {
    // Units of an item of a sequence of this length.
    static __host__ __device__ __forceinline__ int64_t units_of(int64_t len) {
        return len > 0 ? (len + kTile - 1) / kTile + kCost : 0;
    }
    // Owner of unit u when G blocks split U units evenly.
    static __device__ __forceinline__ int owner(int64_t u, int64_t U, int64_t G) {
        return static_cast<int>(((u + 1) * G - 1) / U);
    }

    // A block's way through its share [u, u1) of the units, piece by piece.
    struct Pieces {
        int64_t u, u1;      // next unit; end of the share
        int64_t at;         // first unit of item `coming` of sequence `seq`
        int seq, coming, length;
        // the piece: its item, and the tiles of it
        int b, item, len, tiles, tile0, tile1;
        int64_t item_at;

        __device__ __forceinline__ bool next(const Lengths &s, int items) {
            while (u < u1) {
                const int64_t units = units_of(length);
                if (units == 0 || coming == items) {
                    bool ignore = false;
                    length = s.of(++seq, &ignore);
                    coming = 0;
                    continue;
                }
                b = seq;
                item = coming++;
                len = length;
                tiles = static_cast<int>(units) - kCost;
                item_at = at;
                const int64_t tile_at = item_at + kCost;
                // the tiles among the units [u, min(u1, end of the item))
                tile0 = static_cast<int>(u > tile_at ? u - tile_at : 0);
                tile1 = static_cast<int>(u1 - tile_at < tiles ? u1 - tile_at : tiles);
                u = at = item_at + units;
                if (tile0 < tile1) return true;
            }
            return false;
        }
    };

    // The batch's units and this block's share of them. All kThreads threads call it;
    // a wrong length is recorded by block 0. Blocks from G on have no share.
    struct Share {
        int64_t U, G, u0, u1, at;   // at, b, item: the item that the share starts in
        int b, item, len;
        __device__ __forceinline__ Pieces pieces() const { return {u0, u1, at, b, item, len}; }
    };
    template <int kThreads>
    static __device__ __forceinline__ Share share(const Lengths &s, int items, int *err) {
        constexpr int kWarps = kThreads / 32;
        __shared__ int64_t s_sum[kWarps], s_off;
        __shared__ int s_first;
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        // units before each thread's run of sequences, by a block scan
        const int per = (s.batch + kThreads - 1) / kThreads;
        bool bad = false;
        int64_t mine = 0;
        for (int i = 0, b = tid * per; i < per && b < s.batch; ++i, ++b)
            mine += units_of(s.of(b, &bad)) * items;
        if (bad && blockIdx.x == 0) atomicOr(err, kErrPage);
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
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += s_sum[w];
            U += s_sum[w];
        }
        Share r;
        r.U = U;
        r.G = U < gridDim.x ? U : gridDim.x;
        const int c = blockIdx.x;
        r.u0 = r.u1 = r.at = 0;
        r.b = r.item = r.len = 0;
        if (c >= r.G) return r;   // (the whole block)
        r.u0 = c * U / r.G;
        r.u1 = (c + 1) * U / r.G;
        if (r.u0 >= before && r.u0 < before + mine) {   // one thread of the block
            int64_t at = before;
            int b = tid * per;
            for (;; ++b) {
                bool ignore = false;
                const int64_t n = units_of(s.of(b, &ignore)) * items;
                if (r.u0 < at + n) break;
                at += n;
            }
            s_first = b;
            s_off = at;
        }
        __syncthreads();
        bool ignore = false;
        r.b = s_first;
        r.len = s.of(r.b, &ignore);
        const int64_t units = units_of(r.len);
        r.item = static_cast<int>((r.u0 - s_off) / units);
        r.at = s_off + r.item * units;
        return r;
    }
};

}  // namespace kda
