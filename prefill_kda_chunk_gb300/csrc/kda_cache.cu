// Page tables, positions and slots of a batch's next tokens (kda_page_plan), and new
// keys and values into a paged cache of 8-bit numbers (kda_paged_append_fp8).

#include <cuda_fp8.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

// ------------------------------------------------------------------ the plan
//
// Three prefix sums over the batch: pages given back, pages needed, new tokens. With them
// every entry is known by itself: the k-th needed page is the k-th from the top of the
// stack. The sums of up to 4096 slots are in a block's shared memory. Where no output is its
// input, a grid does all in one launch, each block with sums of its own; a call in place
// (a page given back may lie in a row of the table that the same call fills again, so that no
// entry is written before all are pushed) takes one block if there are few rows, else, like
// larger batches, a launch that sums and pushes and one that fills. Bound by launches and
// chains of loads: 256 slots with a token each, 256 pages wide, 6.7 us (in two launches 10.1); 64
// prompts of 65536 tokens together 7.7 us (11.0).

constexpr int kPlanThreads = 1024;
// Rows that one block writes in place (16 slots of 64 tokens: 5.0 us, in two launches about 5.5; of
// 256: 7.4 and 5.5).
constexpr int64_t kPlanAlone = 2048;
// Slots whose sums a block of plan_kernel holds in shared memory, and one of plan_fill_kernel,
// which has to load them first.
constexpr int kPlanHeld = 4096, kFillHeld = 1024;

// The sums: the top of the stack with what was given back, the pages that were there before, the
// rows, and the pages needed (-1: nothing is planned); then per slot its first row, the tokens held after the
// release, the number of the first page it needs, and that of the first it gives back.
struct PlanTotals {
    int64_t top, before, rows, need;
};
struct PlanMeta {   // in the workspace, from one launch to the next
    int64_t *m;
    __device__ __forceinline__ PlanTotals &all() const { return *reinterpret_cast<PlanTotals *>(m); }
    __device__ __forceinline__ int32_t &held(int i) const { return reinterpret_cast<int32_t *>(m + 4)[3 * i]; }
    __device__ __forceinline__ int32_t &need(int i) const { return reinterpret_cast<int32_t *>(m + 4)[3 * i + 1]; }
    __device__ __forceinline__ int32_t &back(int i) const { return reinterpret_cast<int32_t *>(m + 4)[3 * i + 2]; }
};

// (of tokens that a row of the table can hold, less than 2^31)
__device__ __forceinline__ int64_t pages_of(int64_t tokens, int64_t page) {
    return (static_cast<uint32_t>(tokens) + static_cast<uint32_t>(page) - 1) / static_cast<uint32_t>(page);
}

struct Sums {
    int64_t back, need, rows;
    __device__ __forceinline__ Sums operator+(const Sums &o) const { return {back + o.back, need + o.need, rows + o.rows}; }
    __device__ __forceinline__ Sums up(int d) const {   // the lane d in front
        return {__shfl_up_sync(0xffffffffu, back, d), __shfl_up_sync(0xffffffffu, need, d),
                __shfl_up_sync(0xffffffffu, rows, d)};
    }
};

__device__ __forceinline__ Sums warp_scan(Sums v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums u = v.up(o);
        if (lane >= o) v = v + u;
    }
    return v;
}

// Exclusive sums over the block's threads; `all` receives the totals.
__device__ __forceinline__ Sums scan(const Sums &v, Sums (&warps)[kPlanThreads / 32], Sums &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Sums in = warp_scan(v);
    if (lane == 31) warps[warp] = in;
    __syncthreads();
    if (warp == 0) warps[lane] = warp_scan(warps[lane]);
    __syncthreads();
    all = warps[kPlanThreads / 32 - 1];
    const Sums before = warp > 0 ? warps[warp - 1] : Sums{0, 0, 0};
    return {before.back + in.back - v.back, before.need + in.need - v.need, before.rows + in.rows - v.rows};
}

// The last of n slots whose `first` is at most x.
template <typename F>
__device__ __forceinline__ int last_from(int n, int64_t x, F &&first) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first(mid) <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The sums as plan_fill reads them, of one block's shared memory or of the workspace.
struct NearSums {
    int32_t *f;   // [4][n]
    int n;
    __device__ __forceinline__ int32_t &first(int i) const { return f[i]; }
    __device__ __forceinline__ int32_t &held(int i) const { return f[n + i]; }
    __device__ __forceinline__ int32_t &need(int i) const { return f[2 * n + i]; }
    __device__ __forceinline__ int32_t &back(int i) const { return f[3 * n + i]; }
};
struct FarSums {
    PlanMeta m;
    const int32_t *cu;
    __device__ __forceinline__ int32_t first(int i) const { return cu[i]; }
    __device__ __forceinline__ int32_t held(int i) const { return m.held(i); }
    __device__ __forceinline__ int32_t need(int i) const { return m.need(i); }
    __device__ __forceinline__ int32_t back(int i) const { return m.back(i); }
};

// The r-th page that is given back.
template <typename S>
__device__ __forceinline__ int32_t given_back(const PlanParams &p, const S &s, int64_t r) {
    const int i = last_from(p.batch, r, [&](int k) { return s.back(k); });
    return p.table[i * p.width + (r - s.back(i))];
}

// Thread `at` of `n` that write the entries, positions and slots; kPushed: the pages given back
// are in free_out already.
template <bool kPushed, typename S>
__device__ __forceinline__ void plan_fill(const PlanParams &p, const PlanTotals &all, const S &s, int64_t at, int64_t n) {
    const bool ok = all.need >= 0;
    const int64_t top = all.top, before = all.before;
    auto stacked = [&](int64_t k) {
        return k < before ? p.free[k] : kPushed ? p.free_out[k] : given_back(p, s, k - before);
    };
    if (p.free_out != p.free)
        for (int64_t k = at; k < p.pool; k += n)
            if (!ok || k < before || k >= top) p.free_out[k] = p.free[k];
            else if (!kPushed) p.free_out[k] = given_back(p, s, k - before);
    auto entry = [&](int i, int64_t j, int64_t have) { return stacked(top - 1 - (s.need(i) + j - have)); };
    if (p.table_out != p.table) {   // 128 entries of a slot's row by a warp
        const int lane = static_cast<int>(at & 31);
        const uint32_t parts = static_cast<uint32_t>((p.width + 127) / 128);
        for (int64_t w = at >> 5; w < static_cast<int64_t>(p.batch) * parts; w += n >> 5) {
            const int i = static_cast<int>(static_cast<uint32_t>(w) / parts), part = static_cast<int>(static_cast<uint32_t>(w) % parts);
            const int64_t have = pages_of(s.held(i), p.page_size),
                          end = ok ? pages_of(static_cast<int64_t>(s.held(i)) + p.news[i], p.page_size) : have;
            const int64_t row = i * p.width, j0 = part * 128, j1 = j0 + 128 < p.width ? j0 + 128 : p.width;
#pragma unroll 4
            for (int64_t j = j0 + lane; j < j1; j += 32)
                p.table_out[row + j] = j >= have && j < end ? entry(i, j, have) : p.table[row + j];
        }
    } else {   // the new ones (a warp per slot: 1000 slots with a page each 31 us,
        // this way 7)
        for (int64_t k = at; k < all.need; k += n) {
            const int i = last_from(p.batch, k, [&](int o) { return s.need(o); });
            p.table_out[i * p.width + pages_of(s.held(i), p.page_size) + (k - s.need(i))] = stacked(top - 1 - k);
        }
    }
    for (int64_t r = at; r < p.tokens; r += n) {
        int32_t pos = 0;
        int64_t slot = -1;
        if (r < all.rows) {
            const int i = last_from(p.batch, r, [&](int k) { return s.first(k); });
            const int64_t had = s.held(i), have = pages_of(had, p.page_size);
            pos = static_cast<int32_t>(had + r - s.first(i));
            const uint32_t j = static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page_size);
            const int32_t page = j >= have ? entry(i, j, have) : p.table[i * p.width + j];
            slot = static_cast<int64_t>(page) * p.page_size + (pos - static_cast<int64_t>(j) * p.page_size);
        }
        p.pos[r] = pos;
        p.slots[r] = slot;
    }
}

// How a call's launches share the work: all of it in one launch, of one block or (nothing in
// place) of a grid, or sums and pushes in a launch of one block in front of plan_fill_kernel.
enum class PlanHow { kAlone, kGrid, kTwo };

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanParams p, PlanHow how) {
    __shared__ Sums s_warps[kPlanThreads / 32];
    __shared__ PlanTotals s_all;
    extern __shared__ int32_t s_sums[];   // up to kPlanHeld slots
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const PlanMeta m{p.meta};
    const NearSums held_here{s_sums, p.batch};
    const int tid = threadIdx.x, per = (p.batch + kPlanThreads - 1) / kPlanThreads;
    const int i0 = tid * per < p.batch ? tid * per : p.batch, i1 = i0 + per < p.batch ? i0 + per : p.batch;
    const int64_t most = p.width * p.page_size, count = *p.count;
    const bool near = p.batch <= kPlanHeld, writes = blockIdx.x == 0;
    auto gone = [&](int i) { return p.release != nullptr && p.release[i] != 0; };
    Sums mine{0, 0, 0}, all;
    int bad = count < 0 || count > p.pool;
    for (int i = i0; i < i1; ++i) {
        const int64_t len = p.lens[i], add = p.news[i], held = gone(i) ? 0 : len;
        if (len < 0 || len > most || add < 0 || held + add > most) {
            bad = 1;
            continue;
        }
        if (gone(i)) mine.back += pages_of(len, p.page_size);
        mine.need += pages_of(held + add, p.page_size) - pages_of(held, p.page_size);
        mine.rows += add;
    }
    bad = __syncthreads_or(bad);
    Sums at = scan(mine, s_warps, all);
    const int64_t top = count + all.back;
    if (all.rows > p.tokens || top > p.pool) bad = 1;
    const bool ok = !bad && all.need <= top;
    if (!ok && writes && tid == 0) atomicOr(p.err, bad ? kErrPage : kErrPool);
    for (int i = i0; i < i1; ++i) {   // (sums that fit 32 bits, if anything is planned)
        const int64_t len = p.lens[i], held = gone(i) ? 0 : len, add = ok ? p.news[i] : 0;
        const int32_t first = static_cast<int32_t>(ok ? at.rows : 0), had = static_cast<int32_t>(ok ? held : len),
                      need = static_cast<int32_t>(ok ? at.need : 0), back = static_cast<int32_t>(ok ? at.back : 0);
        if (near) {
            held_here.first(i) = first;
            held_here.held(i) = had;
            held_here.need(i) = need;
            held_here.back(i) = back;
        }
        if (how == PlanHow::kTwo) {
            m.held(i) = had;
            m.need(i) = need;
            m.back(i) = back;
        }
        if (writes) p.cu[i] = first;
        if (!ok) {
            if (writes && p.lens_out != p.lens) p.lens_out[i] = static_cast<int32_t>(len);
            continue;
        }
        if (writes) p.lens_out[i] = static_cast<int32_t>(held + add);
        at.rows += add;
        at.need += pages_of(held + add, p.page_size) - pages_of(held, p.page_size);
        if (gone(i)) at.back += pages_of(len, p.page_size);
    }
    if (tid == 0) {
        const PlanTotals totals{ok ? top : count, count, ok ? all.rows : 0, ok ? all.need : -1};
        s_all = totals;
        if (how == PlanHow::kTwo) m.all() = totals;
        if (writes) {
            p.cu[p.batch] = static_cast<int32_t>(totals.rows);
            *p.count_out = static_cast<int32_t>(ok ? top - all.need : count);
        }
    }
    __syncthreads();
    if (how == PlanHow::kGrid) {
        plan_fill<false>(p, s_all, held_here, static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid,
                         static_cast<int64_t>(gridDim.x) * kPlanThreads);
        return;
    }
    if (ok)   // the pages given back (a slot's place in the order is below its row's width)
#pragma unroll 4
        for (int64_t r = tid; r < all.back; r += kPlanThreads)
            p.free_out[count + r] = near ? given_back(p, held_here, r) : given_back(p, FarSums{m, p.cu}, r);
    if (how == PlanHow::kAlone) {
        __syncthreads();
        plan_fill<true>(p, s_all, held_here, tid, kPlanThreads);
    }
}

__global__ void __launch_bounds__(256) plan_fill_kernel(PlanParams p) {
    __shared__ int32_t s_sums[3 * kFillHeld];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const FarSums far{PlanMeta{p.meta}, p.cu};
    const PlanTotals all = far.m.all();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, n = static_cast<int64_t>(gridDim.x) * 256;
    if (p.batch > kFillHeld) {
        plan_fill<true>(p, all, far, at, n);
        return;
    }
    const NearSums near{s_sums, p.batch};   // (but for `back`)
    for (int i = threadIdx.x; i < p.batch; i += 256) {
        near.first(i) = far.first(i);
        near.held(i) = far.held(i);
        near.need(i) = far.need(i);
    }
    __syncthreads();
    plan_fill<true>(p, all, near, at, n);
}

// ----------------------------------------------------------- into the cache
//
// A work item is the new rows of one page and some heads, keys or values. A group of warps
// takes it head by head: the largest value, the scale, the rows (and the page's other rows
// where the scale grew), with the next head's rows on their way into registers meanwhile.
// What leads to a page (cu_seqlens, length, table: a chain of loads) is then paid once for
// several heads. Slot i can touch n_i / page_size + 2 pages, so candidates are numbered with
// cu_seqlens[i] / page_size + 2 i in front of slot i, which a warp inverts with a 32-way
// search; no launch before this one is needed. Bound by reading k and v and writing the rows.
//
// Measured, 8 heads of 128: one prompt of 65536 tokens, pages of 32: 77 us (5.2 TB/s, 77 % of
// copy bandwidth; a page and head at a time 137 us, 61 % of the issue slots are taken); 16 ragged
// prompts of 8191 tokens: 14 us (52 %: launch, table and first rows are 6 us of it); a token for
// each of 256 slots: 4.7 us, a launch and a chain of loads.

__device__ __forceinline__ int64_t items_before(const AppendParams &p, int32_t cu, int i) {
    return cu / p.c.page_size + 2 * static_cast<int64_t>(i);
}
__device__ __forceinline__ int64_t items_before(const AppendParams &p, int i) {
    return items_before(p, __ldg(p.cu + i), i);
}

// Exponent of the least power of two that brings the bf16 number with these bits (not
// negative, finite) to 448 = 1.75 * 2^8 or below; from -126 on.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
    const int k = static_cast<int>(bits >> 7) - 127 - ((bits & 127) <= 96 ? 8 : 7);
    return k < -126 ? -126 : k;
}

constexpr uint32_t kOdd = 0x7f80;   // bf16 bits (without sign) of infinity; NaN above

// Two bf16 numbers' bits without sign; with kFine those of infinities and NaN as 0.
template <bool kFine>
__device__ __forceinline__ uint32_t magnitudes(uint32_t u) {
    u &= 0x7fff7fffu;
    if (kFine) {
        if ((u & 0xffff) >= kOdd) u &= 0xffff0000u;
        if (u >> 16 >= kOdd) u &= 0xffffu;
    }
    return u;
}
template <bool kFine>
__device__ __forceinline__ uint32_t largest(uint32_t top, const uint4 &u) {
    top = __vmaxu2(top, magnitudes<kFine>(u.x));
    top = __vmaxu2(top, magnitudes<kFine>(u.y));
    top = __vmaxu2(top, magnitudes<kFine>(u.z));
    return __vmaxu2(top, magnitudes<kFine>(u.w));
}

__device__ __forceinline__ uint32_t to_e4m3(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Eight numbers times inv. With infinities among them (odd) those become NaN: x 0 + x (the
// conversion would make them 448).
__device__ __forceinline__ uint2 quantise(const uint4 &u, float inv, bool odd) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
        if (odd) {
            a = fmaf(a, 0.f, a);
            b = fmaf(b, 0.f, b);
        }
        mul2(a, b, inv, inv);
        o[i] = to_e4m3(a, b);
    }
    return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

__device__ __forceinline__ uint32_t rescale4(uint32_t u, float f) {
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u >> (16 * i)), __NV_E4M3);
        const float2 x = __half22float2(__half2(h));
        o[i] = to_e4m3(x.x * f, x.y * f);
    }
    return o[0] | (o[1] << 16);
}

// cu_seqlens as a whole, by the first block of 256 threads.
__device__ __forceinline__ void check_cu(const AppendParams &p) {
    if (blockIdx.x != 0 || p.cu == nullptr) return;
    bool bad = false;
    for (int i = threadIdx.x; i <= p.c.batch; i += 256) {
        const int32_t a = i > 0 ? __ldg(p.cu + i - 1) : 0, b = __ldg(p.cu + i);
        bad |= b < a || b > p.tokens || (i == 0 && b != 0);
    }
    if (bad) atomicOr(p.c.err, kErrBadCu);
}

// W warps for each item of `per` heads; kKeep rows of a lane group in registers.
template <int D, int W, int kKeep>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p, int64_t items, int per) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kStep = kRows * W;
    __shared__ uint32_t s_top[3][8];
    const Cache8 &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
    check_cu(p);
    // ---- which rows (the warps of an item agree on everything)
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * 8 + warp) / W;
    if (item >= items) return;
    const int sets = (c.hkv + per - 1) / per, h0 = static_cast<int>(item % sets) * per, h1 = min(h0 + per, c.hkv);
    const bool is_v = (item / sets) & 1;
    const int64_t cand = item / (2 * sets);
    int i = static_cast<int>(cand);
    int64_t tok = cand, n = 1, which = 0, len;
    if (p.cu != nullptr) {
        int lo = 0, hi = c.batch;   // the last slot i with items_before(i) <= cand, in [lo, hi)
        while (hi - lo > 32) {
            const int step = (hi - lo + 31) / 32, k = lo + (lane + 1) * step;
            const int m = __popc(__ballot_sync(0xffffffffu, k < hi && items_before(p, k) <= cand));
            lo += m * step;
            hi = lo + step < hi ? lo + step : hi;
        }
        // 32 of them, with all there is to know, in one go
        const int k = lo + lane < hi ? lo + lane : hi - 1;
        int32_t a = __ldg(p.cu + k), b = __ldg(p.cu + k + 1), l = __ldg(c.lens + k);
        const int m = __popc(__ballot_sync(0xffffffffu, lo + lane < hi && items_before(p, a, k) <= cand));
        const int from = m > 0 ? m - 1 : 0;
        a = __shfl_sync(0xffffffffu, a, from);
        b = __shfl_sync(0xffffffffu, b, from);
        len = __shfl_sync(0xffffffffu, l, from);
        i = lo + from;
        if (a < 0 || b <= a || b > p.tokens) return;
        tok = a;
        n = b - a;
        which = cand - items_before(p, a, i);
        if (which < 0) return;
    } else {
        len = __ldg(c.lens + i);
    }
    const int64_t first = len - n;
    if (p.cu == nullptr && len == 0) return;
    if (first < 0 || len > c.max_pages * c.page_size) {
        if (lane == 0) atomicOr(c.err, kErrPage);
        return;
    }
    const int64_t j = first / c.page_size + which;
    const int64_t begin = which == 0 ? first : j * c.page_size;
    const int64_t end = (j + 1) * c.page_size < len ? (j + 1) * c.page_size : len;
    if (begin >= end) return;
    const int page = __ldg(c.table + i * c.max_pages + j);
    const int row = static_cast<int>(begin - j * c.page_size), rows = static_cast<int>(end - begin);
    tok += begin - first;
    const int at = lane % kLanes, sub = part * kRows + lane / kLanes;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const uint16_t *src = static_cast<const uint16_t *>(is_v ? p.v : p.k) + tok * stride + 8 * at;
    auto load = [&](int head, uint4 (&x)[kKeep]) {
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            const int r = sub + k * kStep;
            x[k] = make_uint4(0, 0, 0, 0);
            if (r < rows) x[k] = *reinterpret_cast<const uint4 *>(src + r * stride + head * D);
        }
    };
    uint4 now[kKeep], next[kKeep];
    load(h0, now);
    if (page < 0 || page >= c.pages) {
        if (lane == 0) atomicOr(c.err, kErrPage);
        return;
    }
    float *scales = is_v ? c.vs + page * c.vs_page : c.ks + page * c.ks_page;
    uint8_t *cells = (is_v ? c.v + page * c.v_page : c.k + page * c.k_page) + 8 * at;
    const int64_t step = is_v ? c.v_token : c.k_token, head_step = is_v ? c.v_head : c.k_head;
    // The largest over the warps of the item.
    auto settle = [&](uint32_t top, int turn) -> uint32_t {
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffff, top >> 16));
        if (W > 1) {   // (three places: one is written while the one before is read)
            if (lane == 0) s_top[turn % 3][warp] = top;
            asm volatile("bar.sync %0, %1;\n" ::"r"(1 + warp / W), "n"(32 * W) : "memory");
#pragma unroll
            for (int w = 0; w < W; ++w) top = max(top, s_top[turn % 3][warp - part + w]);
        }
        return top;
    };
    int turn = 0;
#pragma unroll 1
    for (int head = h0; head < h1; ++head) {
        const float old = row > 0 ? scales[head] : 0.f;
        if (head + 1 < h1) load(head + 1, next);
        const uint16_t *rest = src + head * D;   // rows behind those in registers: read twice
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kKeep; ++k) top = largest<false>(top, now[k]);
        for (int r = sub + kKeep * kStep; r < rows; r += kStep)
            top = largest<false>(top, *reinterpret_cast<const uint4 *>(rest + r * stride));
        top = settle(top, turn++);
        const bool odd = top >= kOdd;
        if (odd) {   // infinities and NaN do not count
            top = 0;
#pragma unroll
            for (int k = 0; k < kKeep; ++k) top = largest<true>(top, now[k]);
            for (int r = sub + kKeep * kStep; r < rows; r += kStep)
                top = largest<true>(top, *reinterpret_cast<const uint4 *>(rest + r * stride));
            top = settle(top, turn++);
        }
        float scale = __uint_as_float(static_cast<uint32_t>(scale_exponent(top) + 127) << 23);
        const bool grew = row > 0 && scale > old;
        if (row > 0 && !grew) scale = old;
        const float inv = 1.f / scale;
        uint8_t *dst = cells + head * head_step;
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            const int r = sub + k * kStep;
            if (r < rows) *reinterpret_cast<uint2 *>(dst + (row + r) * step) = quantise(now[k], inv, odd);
        }
        for (int r = sub + kKeep * kStep; r < rows; r += kStep)
            *reinterpret_cast<uint2 *>(dst + (row + r) * step) =
                quantise(*reinterpret_cast<const uint4 *>(rest + r * stride), inv, odd);
        if (grew) {   // the page's other rows, what they stand for as before
            const float f = old / scale;
#pragma unroll 4
            for (int r = sub; r < c.page_size; r += kStep) {
                if (r >= row && r < row + rows) continue;
                uint2 *q = reinterpret_cast<uint2 *>(dst + r * step);
                const uint2 u = *q;
                *q = make_uint2(rescale4(u.x, f), rescale4(u.y, f));
            }
        }
        // (every warp has read the old scale in front of the barrier)
        if (sub == 0 && at == 0 && (row == 0 || grew)) scales[head] = scale;
#pragma unroll
        for (int k = 0; k < kKeep; ++k) now[k] = next[k];
    }
}

// Pages of one token: every page starts anew, so that a row and head is all there is to a scale. A
// warp takes a token's keys and values, D / 8 lanes a head, four sets of heads on their way at a
// time. (As items of a page, one row in a warp: 32854 tokens, 8 heads of
// 64 167 us, this way 27.)
template <int D>
__global__ void __launch_bounds__(256) append_rows_kernel(AppendParams p) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kSets = 4;
    const Cache8 &c = p.c;
    const int lane = threadIdx.x & 31, at = lane % kLanes, sub = lane / kLanes;
    check_cu(p);
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (tok >= p.tokens) return;
    int64_t i = tok, a = tok, b = tok + 1;
    if (p.cu != nullptr) {
        int lo = 0, hi = c.batch;   // the last slot that starts at tok or in front of it, in [lo, hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, k = lo + lane * step;
            const int m = __popc(__ballot_sync(0xffffffffu, k < hi && __ldg(p.cu + k) <= tok));
            lo += (m > 0 ? m - 1 : 0) * step;
            hi = lo + step < hi ? lo + step : hi;
        }
        i = lo;
        a = __ldg(p.cu + i);
        b = __ldg(p.cu + i + 1);
        if (a < 0 || a > tok || b <= tok || b > p.tokens) return;
    }
    const int64_t len = __ldg(c.lens + i), j = len - b + tok;   // (a page of the slot's)
    if (p.cu == nullptr && len == 0) return;
    if (len < b - a || len > c.max_pages) {
        if (lane == 0) atomicOr(c.err, kErrPage);
        return;
    }
    const int page = __ldg(c.table + i * c.max_pages + j);
    if (page < 0 || page >= c.pages) {
        if (lane == 0) atomicOr(c.err, kErrPage);
        return;
    }
    for (int h0 = 0; h0 < 2 * c.hkv; h0 += kSets * kRows) {   // heads of the keys, then of the values
        uint4 x[kSets];
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            const int h = h0 + s * kRows + sub;
            const bool is_v = h >= c.hkv;
            const uint16_t *src = is_v ? static_cast<const uint16_t *>(p.v) + tok * p.v_stride + (h - c.hkv) * D
                                       : static_cast<const uint16_t *>(p.k) + tok * p.k_stride + h * D;
            x[s] = h < 2 * c.hkv ? *reinterpret_cast<const uint4 *>(src + 8 * at) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            const int h = h0 + s * kRows + sub;
            auto most = [&](uint32_t top) {
#pragma unroll
                for (int m = kLanes / 2; m > 0; m >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, m));
                return max(top & 0xffffu, top >> 16);
            };
            uint32_t top = most(largest<false>(0, x[s]));
            const bool odd = top >= kOdd;
            if (__any_sync(0xffffffffu, odd)) {   // infinities and NaN do not count
                const uint32_t fine = most(largest<true>(0, x[s]));
                if (odd) top = fine;
            }
            const float scale = __uint_as_float(static_cast<uint32_t>(scale_exponent(top) + 127) << 23);
            if (h >= 2 * c.hkv) continue;
            const bool is_v = h >= c.hkv;
            const int head = is_v ? h - c.hkv : h;
            uint8_t *dst = is_v ? c.v + page * c.v_page + head * c.v_head : c.k + page * c.k_page + head * c.k_head;
            *reinterpret_cast<uint2 *>(dst + 8 * at) = quantise(x[s], 1.f / scale, odd);
            if (at == 0) (is_v ? c.vs + page * c.vs_page : c.ks + page * c.ks_page)[head] = scale;
        }
    }
}

template <int D>
cudaError_t launch_append_dim(const AppendParams &p, cudaStream_t stream) {
    if (p.c.page_size == 1) {
        append_rows_kernel<D><<<static_cast<unsigned>((p.tokens + 7) / 8), 256, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const int64_t cand = p.cu == nullptr ? p.tokens : p.tokens / p.c.page_size + 2 * static_cast<int64_t>(p.c.batch);
    // Warps of an item: as many as keep a page's rows in registers, four or eight a lane. (One
    // warp, rows behind the first four read twice: pages of 32 tokens 108 us for 77, of 128 103
    // for 37; with eight warps and four rows 45.)
    const int rows = p.cu == nullptr ? 1 : p.c.page_size, group = 256 / D;
    int w = 1;
    while (w < 8 && rows > 4 * group * w) w *= 2;
    // Heads of an item: up to eight, as long as there are 24 warps for every SM. (One and eight
    // throughout: 65536 tokens 122 us and 77, 8191 tokens of 16 prompts 18 and 19, by the rule 14;
    // a token of 256 slots 4.8 and 6.0.)
    int per = 8;
    while (per > 1 && (per > p.c.hkv || cand * 2 * ((p.c.hkv + per - 1) / per) * w < 24 * kPlannedSms)) per /= 2;
    const int64_t items = cand * 2 * ((p.c.hkv + per - 1) / per);
    const unsigned grid = static_cast<unsigned>((items * w + 7) / 8);
    auto kernel = w == 1 ? append_kernel<D, 1, 4> : w == 2 ? append_kernel<D, 2, 4> : w == 4 ? append_kernel<D, 4, 4>
                  : rows <= 32 * group ? append_kernel<D, 8, 4> : append_kernel<D, 8, 8>;
    kernel<<<grid, 256, 0, stream>>>(p, items, per);
    return cudaGetLastError();
}

}  // namespace

namespace {

int64_t plan_cells(const PlanParams &p) {
    return p.tokens + (p.table_out != p.table ? p.batch * p.width : 0) + (p.free_out != p.free ? p.pool : 0);
}

PlanHow plan_how(const PlanParams &p) {
    const bool in_place = p.table_out == p.table || p.free_out == p.free || p.lens_out == p.lens || p.count_out == p.count;
    if (p.batch > kPlanHeld) return PlanHow::kTwo;
    return !in_place ? PlanHow::kGrid : plan_cells(p) <= kPlanAlone ? PlanHow::kAlone : PlanHow::kTwo;
}

}  // namespace

int64_t plan_workspace(const PlanParams &p) {
    return plan_how(p) == PlanHow::kTwo ? 32 + 12 * static_cast<int64_t>(p.batch) : 0;
}

cudaError_t configure_cache() {
    return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * kPlanHeld);
}

cudaError_t launch_plan(const PlanParams &p, cudaStream_t stream) {
    const PlanHow how = plan_how(p);
    const int64_t blocks = (plan_cells(p) + 255) / 256;
    auto grid = [&](int64_t most) { return static_cast<unsigned>(blocks < 1 ? 1 : blocks < most ? blocks : most); };
    const int held = p.batch <= kPlanHeld ? 16 * p.batch : 0;
    plan_kernel<<<how == PlanHow::kGrid ? grid(kPlannedSms) : 1, kPlanThreads, held, stream>>>(p, how);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || how != PlanHow::kTwo) return e;
    // (the second launch's blocks come up while the first one is at work)
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t next{};
    next.gridDim = dim3(grid(8 * kPlannedSms));
    next.blockDim = dim3(256);
    next.stream = stream;
    next.attrs = &overlap;
    next.numAttrs = 1;
    return cudaLaunchKernelEx(&next, plan_fill_kernel, p);
}

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream) {
    return p.c.dim == 64 ? launch_append_dim<64>(p, stream) : launch_append_dim<128>(p, stream);
}

}  // namespace kda
