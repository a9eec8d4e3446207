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
// stack. One block forms the sums and pushes the pages given back; the entries, positions
// and slots follow in the same block where they are few, and from a grid where they are
// many. (A page given back may lie in a row of the table that the same call fills again:
// no entry is written before all are pushed.) Bound by two launches and their chains of
// loads; 131072 entries copied out of place move in about a microsecond.

constexpr int kPlanThreads = 1024;
// Rows, and entries copied out of place, that the one block writes itself.
constexpr int64_t kPlanAlone = 8192;
// Slots whose offsets a block holds in shared memory.
constexpr int kPlanHeld = 1024;

// What the sums hand on: the top of the stack with what was given back, the pages that were
// there before, whether anything is planned, and the rows; then per slot the tokens held after
// the release, the number of the first page it needs, and that of the first it gives back.
struct PlanMeta {
    int64_t *m;
    __device__ __forceinline__ int64_t &top() const { return m[0]; }
    __device__ __forceinline__ int64_t &before() const { return m[1]; }
    __device__ __forceinline__ int64_t &ok() const { return m[2]; }
    __device__ __forceinline__ int64_t &rows() const { return m[3]; }
    __device__ __forceinline__ int64_t &held(int i) const { return m[4 + 3 * i]; }
    __device__ __forceinline__ int64_t &base(int i) const { return m[5 + 3 * i]; }
    __device__ __forceinline__ int64_t &back(int i) const { return m[6 + 3 * i]; }
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

__device__ __forceinline__ int32_t stacked(const PlanParams &p, int64_t before, int64_t k) {
    return k < before ? p.free[k] : p.free_out[k];   // (pushed ones are in the result only)
}

// Thread `at` of `n` that write the entries, positions and slots. held: kPlanHeld numbers of
// the block's.
__device__ void plan_fill(const PlanParams &p, int64_t at, int64_t n, int32_t *held) {
    const PlanMeta m{p.meta};
    const bool ok = m.ok() != 0, near = p.batch <= kPlanHeld;
    const int64_t top = m.top(), before = m.before(), rows = m.rows();
    if (near)
        for (int i = threadIdx.x; i < p.batch; i += blockDim.x) held[i] = p.cu[i];
    __syncthreads();
    if (p.free_out != p.free)
        for (int64_t k = at; k < p.pool; k += n)
            if (!ok || k < before || k >= top) p.free_out[k] = p.free[k];
    auto entry = [&](int i, int64_t j, int64_t have) {
        return stacked(p, before, top - 1 - (m.base(i) + j - have));
    };
    // a warp per slot: all of its row, or the new pages only
    const int lane = static_cast<int>(at & 31);
    const bool copy = p.table_out != p.table;
    if (ok || copy) {
        const uint32_t parts = copy ? static_cast<uint32_t>((p.width + 127) / 128) : 1;
        for (int64_t w = at >> 5; w < static_cast<int64_t>(p.batch) * parts; w += n >> 5) {
            const int i = static_cast<int>(static_cast<uint32_t>(w) / parts), part = static_cast<int>(static_cast<uint32_t>(w) % parts);
            const int64_t have = pages_of(m.held(i), p.page_size),
                          end = ok ? pages_of(m.held(i) + p.news[i], p.page_size) : have;
            const int64_t row = i * p.width, j0 = copy ? part * 128 : have,
                          j1 = copy ? (j0 + 128 < p.width ? j0 + 128 : p.width) : end;
#pragma unroll 4
            for (int64_t j = j0 + lane; j < j1; j += 32)
                p.table_out[row + j] = j >= have && j < end ? entry(i, j, have) : p.table[row + j];
        }
    }
    for (int64_t r = at; r < p.tokens; r += n) {
        int32_t pos = 0;
        int64_t slot = -1;
        if (r < rows) {
            const int i = near ? last_from(p.batch, r, [&](int k) { return held[k]; })
                               : last_from(p.batch, r, [&](int k) { return p.cu[k]; });
            const int64_t had = m.held(i), have = pages_of(had, p.page_size);
            pos = static_cast<int32_t>(had + r - p.cu[i]);
            const uint32_t j = static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page_size);
            const int32_t page = j >= have ? entry(i, j, have) : p.table[i * p.width + j];
            slot = static_cast<int64_t>(page) * p.page_size + (pos - static_cast<int64_t>(j) * p.page_size);
        }
        p.pos[r] = pos;
        p.slots[r] = slot;
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanParams p, bool alone) {
    __shared__ Sums s_warps[kPlanThreads / 32];
    __shared__ int32_t s_held[kPlanHeld];
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const PlanMeta m{p.meta};
    const int tid = threadIdx.x, per = (p.batch + kPlanThreads - 1) / kPlanThreads;
    const int i0 = tid * per < p.batch ? tid * per : p.batch, i1 = i0 + per < p.batch ? i0 + per : p.batch;
    const int64_t most = p.width * p.page_size, count = *p.count;
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
    const bool ok = !bad && all.need <= top, near = p.batch <= kPlanHeld;
    if (!ok && tid == 0) atomicOr(p.err, bad ? kErrPage : kErrPool);
    for (int i = i0; i < i1; ++i) {
        const int64_t len = p.lens[i], held = gone(i) ? 0 : len, add = ok ? p.news[i] : 0;
        m.held(i) = ok ? held : len;
        m.base(i) = at.need;
        m.back(i) = at.back;
        if (near) s_held[i] = static_cast<int32_t>(ok ? at.back : 0);
        p.cu[i] = static_cast<int32_t>(ok ? at.rows : 0);
        if (!ok) {
            if (p.lens_out != p.lens) p.lens_out[i] = p.lens[i];
            continue;
        }
        p.lens_out[i] = static_cast<int32_t>(held + add);
        at.rows += add;
        at.need += pages_of(held + add, p.page_size) - pages_of(held, p.page_size);
        if (gone(i)) at.back += pages_of(len, p.page_size);
    }
    if (tid == 0) {
        p.cu[p.batch] = static_cast<int32_t>(ok ? all.rows : 0);
        m.top() = ok ? top : count;
        m.before() = count;
        m.ok() = ok;
        m.rows() = ok ? all.rows : 0;
        *p.count_out = static_cast<int32_t>(ok ? top - all.need : count);
    }
    __syncthreads();
    if (ok)   // the pages given back (a slot's place in the order is below its row's width)
#pragma unroll 4
        for (int64_t r = tid; r < all.back; r += kPlanThreads) {
            const int i = near ? last_from(p.batch, r, [&](int k) { return s_held[k]; })
                               : last_from(p.batch, r, [&](int k) { return m.back(k); });
            p.free_out[count + r] = p.table[i * p.width + (r - (near ? s_held[i] : m.back(i)))];
        }
    if (alone) {
        __syncthreads();
        plan_fill(p, tid, kPlanThreads, s_held);
    }
}

__global__ void __launch_bounds__(256) plan_fill_kernel(PlanParams p) {
    __shared__ int32_t s_held[kPlanHeld];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    plan_fill(p, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, static_cast<int64_t>(gridDim.x) * 256, s_held);
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

// W warps for each item of `per` heads; kKeep rows of a lane group in registers.
template <int D, int W, int kKeep>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p, int64_t items, int per) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kStep = kRows * W;
    __shared__ uint32_t s_top[3][8];
    const Cache8 &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
    if (blockIdx.x == 0 && p.cu != nullptr) {   // the table as a whole, once
        bool bad = false;
        for (int i = threadIdx.x; i <= c.batch; i += 256) {
            const int32_t a = i > 0 ? __ldg(p.cu + i - 1) : 0, b = __ldg(p.cu + i);
            bad |= b < a || b > p.tokens || (i == 0 && b != 0);
        }
        if (bad) atomicOr(c.err, kErrBadCu);
    }
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

template <int D>
cudaError_t launch_append_dim(const AppendParams &p, cudaStream_t stream) {
    const int64_t cand = p.cu == nullptr ? p.tokens : p.tokens / p.c.page_size + 2 * static_cast<int64_t>(p.c.batch);
    // Warps of an item: as many as keep a page's rows in registers, four or eight a lane.
    const int rows = p.cu == nullptr ? 1 : p.c.page_size, group = 256 / D;
    int w = 1;
    while (w < 8 && rows > 4 * group * w) w *= 2;
    // Heads of an item: up to eight, as long as there are 32 warps for every SM.
    int per = 8;
    while (per > 1 && (per > p.c.hkv || cand * 2 * ((p.c.hkv + per - 1) / per) * w < 32 * kPlannedSms)) per /= 2;
    const int64_t items = cand * 2 * ((p.c.hkv + per - 1) / per);
    const unsigned grid = static_cast<unsigned>((items * w + 7) / 8);
    auto kernel = w == 1 ? append_kernel<D, 1, 4> : w == 2 ? append_kernel<D, 2, 4> : w == 4 ? append_kernel<D, 4, 4>
                  : rows <= 32 * group ? append_kernel<D, 8, 4> : append_kernel<D, 8, 8>;
    kernel<<<grid, 256, 0, stream>>>(p, items, per);
    return cudaGetLastError();
}

}  // namespace

int64_t plan_workspace(const PlanParams &p) { return 32 + 24 * static_cast<int64_t>(p.batch); }

cudaError_t configure_cache() { return cudaSuccess; }

cudaError_t launch_plan(const PlanParams &p, cudaStream_t stream) {
    int64_t cells = p.tokens;
    if (p.table_out != p.table) cells += p.batch * p.width;
    if (p.free_out != p.free) cells += p.pool;
    const bool alone = cells <= kPlanAlone;
    plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, alone);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || alone) return e;
    const int64_t blocks = (cells + 255) / 256, most = 8 * kPlannedSms;
    // (the second launch's blocks come up while the first one is at work)
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t next{};
    next.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most));
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
