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
// no entry is written before all are pushed.)

constexpr int kPlanThreads = 1024;
// Rows, and entries copied out of place, that the one block writes itself.
constexpr int64_t kPlanAlone = 8192;

// What the sums hand on: per slot the tokens held after the release and the number of
// the first page it needs; in front of them the top of the stack with what was given
// back, the pages that were there before, and whether anything is planned.
struct PlanMeta {
    int64_t *m;
    __device__ __forceinline__ int64_t &top() const { return m[0]; }
    __device__ __forceinline__ int64_t &before() const { return m[1]; }
    __device__ __forceinline__ int64_t &ok() const { return m[2]; }
    __device__ __forceinline__ int64_t &rows() const { return m[3]; }
    __device__ __forceinline__ int64_t &held(int i) const { return m[4 + 3 * i]; }
    __device__ __forceinline__ int64_t &base(int i) const { return m[5 + 3 * i]; }
    // pages given back (upper half), and those given back in front of them
    __device__ __forceinline__ int64_t &back(int i) const { return m[6 + 3 * i]; }
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int64_t page) { return (tokens + page - 1) / page; }

struct Sums {
    int64_t back, need, rows;
};

// Exclusive sums over the block's threads; `all` receives the totals.
__device__ __forceinline__ Sums scan(Sums v, Sums (&warps)[kPlanThreads / 32], Sums &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, in.back, o), b = __shfl_up_sync(0xffffffffu, in.need, o),
                      c = __shfl_up_sync(0xffffffffu, in.rows, o);
        if (lane >= o) {
            in.back += a;
            in.need += b;
            in.rows += c;
        }
    }
    if (lane == 31) warps[warp] = in;
    __syncthreads();
    Sums before{0, 0, 0};
    all = before;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const Sums s = warps[w];
        if (w < warp) {
            before.back += s.back;
            before.need += s.need;
            before.rows += s.rows;
        }
        all.back += s.back;
        all.need += s.need;
        all.rows += s.rows;
    }
    return {before.back + in.back - v.back, before.need + in.need - v.need, before.rows + in.rows - v.rows};
}

__device__ __forceinline__ int32_t stacked(const PlanParams &p, int64_t before, int64_t k) {
    return k < before ? p.free[k] : p.free_out[k];   // (pushed ones are in the result only)
}

// Thread `at` of `n` that write the entries, positions and slots.
__device__ void plan_fill(const PlanParams &p, int64_t at, int64_t n) {
    const PlanMeta m{p.meta};
    const bool ok = m.ok() != 0;
    const int64_t top = m.top(), before = m.before(), rows = m.rows();
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
        const int64_t parts = copy ? (p.width + 255) / 256 : 1;
        for (int64_t w = at >> 5; w < p.batch * parts; w += n >> 5) {
            const int i = static_cast<int>(w / parts);
            const int64_t have = pages_of(m.held(i), p.page_size),
                          end = ok ? pages_of(m.held(i) + p.news[i], p.page_size) : have;
            const int64_t row = i * p.width, j0 = copy ? w % parts * 256 : have,
                          j1 = copy ? (j0 + 256 < p.width ? j0 + 256 : p.width) : end;
            for (int64_t j = j0 + lane; j < j1; j += 32)
                p.table_out[row + j] = j >= have && j < end ? entry(i, j, have) : p.table[row + j];
        }
    }
    for (int64_t r = at; r < p.tokens; r += n) {
        int32_t pos = 0;
        int64_t slot = -1;
        if (r < rows) {
            int lo = 0, hi = p.batch - 1;   // the last slot that starts at or before r
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (p.cu[mid] <= r) lo = mid;
                else hi = mid - 1;
            }
            const int64_t held = m.held(lo), have = pages_of(held, p.page_size);
            pos = static_cast<int32_t>(held + r - p.cu[lo]);
            const int64_t j = pos / p.page_size;
            const int32_t page = j >= have ? entry(lo, j, have) : p.table[lo * p.width + j];
            slot = static_cast<int64_t>(page) * p.page_size + pos % p.page_size;
        }
        p.pos[r] = pos;
        p.slots[r] = slot;
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanParams p, bool alone) {
    __shared__ Sums s_warps[kPlanThreads / 32];
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
    const bool ok = !bad && all.need <= top;
    if (!ok && tid == 0) atomicOr(p.err, bad ? kErrPage : kErrPool);
    for (int i = i0; i < i1; ++i) {
        const int64_t len = p.lens[i], held = gone(i) ? 0 : len, add = ok ? p.news[i] : 0;
        m.held(i) = ok ? held : len;
        m.base(i) = at.need;
        p.cu[i] = static_cast<int32_t>(ok ? at.rows : 0);
        if (!ok) {
            if (p.lens_out != p.lens) p.lens_out[i] = p.lens[i];
            continue;
        }
        p.lens_out[i] = static_cast<int32_t>(held + add);
        at.rows += add;
        at.need += pages_of(held + add, p.page_size) - pages_of(held, p.page_size);
        const int64_t n = gone(i) ? pages_of(len, p.page_size) : 0;
        m.back(i) = (n << 32) | at.back;
        at.back += n;
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
    if (ok && p.release != nullptr) {   // a warp pushes the pages of one slot after the other
        const int lane = tid & 31;
        for (int i0 = tid & ~31; i0 < p.batch; i0 += kPlanThreads) {
            const int64_t mine = i0 + lane < p.batch ? m.back(i0 + lane) : 0;
            for (unsigned left = __ballot_sync(0xffffffffu, mine >> 32 != 0); left != 0; left &= left - 1) {
                const int src = __ffs(left) - 1;
                const int64_t v = __shfl_sync(0xffffffffu, mine, src), n = v >> 32, row = (i0 + src) * p.width;
                int32_t *dst = p.free_out + count + (v & 0xffffffff);
                for (int64_t j = lane; j < n; j += 32) dst[j] = p.table[row + j];   // (n <= the row's width)
            }
        }
    }
    if (alone) {
        __syncthreads();
        plan_fill(p, tid, kPlanThreads);
    }
}

__global__ void __launch_bounds__(256) plan_fill_kernel(PlanParams p) {
    plan_fill(p, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, static_cast<int64_t>(gridDim.x) * 256);
}

// ----------------------------------------------------------- into the cache
//
// A work item is the new rows of one page, one head, keys or values: a group of warps
// finds the largest value, settles the scale and writes the rows (and scales the page's
// older rows down where the scale grew). Slot i can touch n_i / page_size + 2 pages, so
// items are numbered with cu_seqlens[i] / page_size + 2 i in front of slot i, which a
// warp inverts with a 32-way search; no launch before this one is needed.

__device__ __forceinline__ int64_t items_before(const AppendParams &p, int i) {
    return static_cast<int64_t>(__ldg(p.cu + i)) / p.c.page_size + 2 * static_cast<int64_t>(i);
}

// Exponent of the least power of two that brings the bf16 number with these bits (not
// negative, finite) to 448 = 1.75 * 2^8 or below; from -126 on.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
    const int k = static_cast<int>(bits >> 7) - 127 - ((bits & 127) <= 96 ? 8 : 7);
    return k < -126 ? -126 : k;
}

// The larger of the two halves, as bf16 bits without sign; infinities and NaN as 0.
__device__ __forceinline__ uint32_t top_bits(uint32_t u) {
    uint32_t a = u & 0x7fff, b = (u >> 16) & 0x7fff;
    if (a >= 0x7f80) a = 0;
    if (b >= 0x7f80) b = 0;
    return a > b ? a : b;
}

__device__ __forceinline__ uint32_t to_e4m3(float a, float b) {
    // x 0 + x: an infinity becomes NaN (the conversion would make it 448)
    a = fmaf(a, 0.f, a);
    b = fmaf(b, 0.f, b);
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint2 quantise(const uint4 &u, float inv) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = to_e4m3(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
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

// W warps for each item.
template <int D, int W>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p, int64_t items) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kStep = kRows * W, kKeep = 8;
    __shared__ uint32_t s_top[8];
    const Cache8 &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * 8 + warp) / W;
    if (blockIdx.x == 0 && p.cu != nullptr) {   // the table as a whole, once
        bool bad = false;
        for (int i = threadIdx.x; i <= c.batch; i += 256) {
            const int32_t a = i > 0 ? __ldg(p.cu + i - 1) : 0, b = __ldg(p.cu + i);
            bad |= b < a || b > p.tokens || (i == 0 && b != 0);
        }
        if (bad) atomicOr(c.err, kErrBadCu);
    }
    // ---- which rows (warps of one item agree on everything up to the barriers below)
    bool live = item < items;
    const int head = static_cast<int>(item % c.hkv);
    const bool is_v = (item / c.hkv) & 1;
    const int64_t cand = item / (2 * c.hkv);
    int i = static_cast<int>(cand);
    int64_t tok = cand, n = 1, which = 0;
    if (p.cu != nullptr && live) {
        int lo = 0, hi = c.batch;   // the last slot i with items_before(i) <= cand, in [lo, hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, k = lo + (lane + 1) * step;
            const int m = __popc(__ballot_sync(0xffffffffu, k < hi && items_before(p, k) <= cand));
            lo += m * step;
            hi = lo + step < hi ? lo + step : hi;
        }
        i = lo;
        const int32_t a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1);
        live = a >= 0 && b >= a && b <= p.tokens;
        tok = a;
        n = live ? b - a : 0;
        which = cand - items_before(p, i);
        live = live && n > 0 && which >= 0;
    }
    int row = 0, rows = 0, page = 0;   // the first new row of the page, and how many
    if (live) {
        const int64_t len = __ldg(c.lens + i), first = len - n;
        if (p.cu == nullptr && len == 0) {
            live = false;
        } else if (first < 0 || len > c.max_pages * c.page_size) {
            if (lane == 0) atomicOr(c.err, kErrPage);
            live = false;
        } else {
            const int64_t j = first / c.page_size + which;
            const int64_t begin = which == 0 ? first : j * c.page_size;
            const int64_t end = (j + 1) * c.page_size < len ? (j + 1) * c.page_size : len;
            live = begin < end;
            if (live) {
                page = __ldg(c.table + i * c.max_pages + j);
                if (page < 0 || page >= c.pages) {
                    if (lane == 0) atomicOr(c.err, kErrPage);
                    live = false;
                }
                row = static_cast<int>(begin - j * c.page_size);
                rows = static_cast<int>(end - begin);
                tok += begin - first;
            }
        }
    }
    if (!live) rows = 0;
    const int at = lane % kLanes, sub = part * kRows + lane / kLanes;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const uint16_t *src = static_cast<const uint16_t *>(is_v ? p.v : p.k) + tok * stride + head * D + 8 * at;
    float *scale = is_v ? c.vs + page * c.vs_page + head : c.ks + page * c.ks_page + head;
    const float old = live && row > 0 ? *scale : 0.f;
    // ---- the largest value; the first rows stay in registers
    uint4 held[kKeep];
    uint32_t top = 0;
    auto look = [&](const uint4 &u) {
        const uint32_t a = max(top_bits(u.x), top_bits(u.y)), b = max(top_bits(u.z), top_bits(u.w));
        top = max(top, max(a, b));
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int r = sub + k * kStep;
        held[k] = make_uint4(0, 0, 0, 0);
        if (r < rows) held[k] = *reinterpret_cast<const uint4 *>(src + r * stride);
    }
#pragma unroll
    for (int k = 0; k < kKeep; ++k) look(held[k]);
    for (int r = sub + kKeep * kStep; r < rows; r += kStep)
        look(*reinterpret_cast<const uint4 *>(src + r * stride));
    top = __reduce_max_sync(0xffffffffu, top);
    if (W > 1) {
        if (lane == 0) s_top[warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) top = max(top, s_top[warp - part + w]);
    }
    if (!live) return;
    float now = __uint_as_float(static_cast<uint32_t>(scale_exponent(top) + 127) << 23);
    const bool grew = row > 0 && now > old;
    if (row > 0 && !grew) now = old;
    const float inv = 1.f / now;
    uint8_t *dst = is_v ? c.v + page * c.v_page + head * c.v_head : c.k + page * c.k_page + head * c.k_head;
    const int64_t step = is_v ? c.v_token : c.k_token;
    dst += 8 * at;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int r = sub + k * kStep;
        if (r < rows) *reinterpret_cast<uint2 *>(dst + (row + r) * step) = quantise(held[k], inv);
    }
    for (int r = sub + kKeep * kStep; r < rows; r += kStep)
        *reinterpret_cast<uint2 *>(dst + (row + r) * step) =
            quantise(*reinterpret_cast<const uint4 *>(src + r * stride), inv);
    if (grew) {
        const float f = old / now;
#pragma unroll 4
        for (int r = sub; r < row; r += kStep) {
            uint2 *q = reinterpret_cast<uint2 *>(dst + r * step);
            const uint2 u = *q;
            *q = make_uint2(rescale4(u.x, f), rescale4(u.y, f));
        }
    }
    if (sub == 0 && at == 0 && (row == 0 || grew)) *scale = now;
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
    plan_fill_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream) {
    const int64_t cand = p.cu == nullptr ? p.tokens : p.tokens / p.c.page_size + 2 * static_cast<int64_t>(p.c.batch);
    const int64_t items = cand * 2 * p.c.hkv;
    // Warps of an item: as many as keep the rows of a page in registers.
    const int rows = p.cu == nullptr ? 1 : p.c.page_size, hold = 8 * (p.c.dim == 64 ? 4 : 2);
    const int w = rows <= hold ? 1 : rows <= 4 * hold ? 4 : 8;
    const unsigned grid = static_cast<unsigned>((items * w + 7) / 8);
    auto kernel = p.c.dim == 64 ? (w == 1 ? append_kernel<64, 1> : w == 4 ? append_kernel<64, 4> : append_kernel<64, 8>)
                                : (w == 1 ? append_kernel<128, 1> : w == 4 ? append_kernel<128, 4> : append_kernel<128, 8>);
    kernel<<<grid, 256, 0, stream>>>(p, items);
    return cudaGetLastError();
}

}  // namespace kda
