// C ABI of the operators in front of and around an 8-bit paged cache (declared in
// include/kda.h): page plans, norms of queries and keys with the rotation, new tokens
// into the cache, decode attention over it. Argument validation here; the kernels in
// kda_cache.cu, kda_heads.cu and kda_paged8.cu.

#include <cuda_runtime.h>

#include <atomic>
#include <climits>

#include "kda.h"
#include "kda_checks.h"
#include "kda_device.cuh"
#include "kda_internal.h"

namespace {

using kda::any_shared;
using kda::flat;
using kda::kMaxElems;
using kda::misaligned;
using kda::Rows;
using kda::rows_fit;

constexpr int64_t k31 = int64_t(1) << 31;

std::atomic<int> g_stall_paged8{INT_MAX};   // kda_test_stall_paged_fp8
std::atomic<int> g_stall_heads{INT_MAX};    // kda_test_stall_qk_norm_rope

kda_status status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// ---- the cells of a cache: rows of `width` bytes on a grid of pages, tokens and heads
struct Cells {
    const void *p;
    int64_t width, n[3], step[3];   // pages, tokens, heads
};

// The axes of more than one row by their step, the smallest first; how many they are.
int by_step(const Cells &c, int (&order)[3]) {
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        if (c.n[i] <= 1) continue;
        int j = n++;
        for (; j > 0 && c.step[order[j - 1]] > c.step[i]; --j) order[j] = order[j - 1];
        order[j] = i;
    }
    return n;
}

// Each step past what the smaller ones span: no two rows overlap.
bool cells_fit(const Cells &c) {
    int order[3];
    const int n = by_step(c, order);
    int64_t span = c.width;
    for (int k = 0; k < n; ++k) {
        const int i = order[k];
        if (c.step[i] < span || c.step[i] > kMaxElems || c.n[i] > kMaxElems / c.step[i]) return false;
        span += (c.n[i] - 1) * c.step[i];
        if (span > kMaxElems) return false;
    }
    return true;
}

// As one range (cells_fit), none where the cache has no pages.
Rows range(const Cells &c) {
    int64_t span = c.width;
    for (int i = 0; i < 3; ++i) {
        if (c.n[i] == 0) return {nullptr, 0, 0, 0};
        span += (c.n[i] - 1) * c.step[i];
    }
    return flat(c.p, span);
}

// Whether two caches of the same shape share a byte. With the same steps they are the
// same pattern some offset apart: rows, heads or pages that lie beside one another are
// seen modulo the step of the axis that repeats them (and that the larger ones repeat).
bool cells_share(const Cells &a, const Cells &b) {
    if (!kda::share(range(a), range(b))) return false;
    int order[3];
    const int n = by_step(a, order);
    for (int k = 0; k < n; ++k)
        if (a.step[order[k]] != b.step[order[k]]) return true;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t apart = pa < pb ? pb - pa : pa - pb;
    int64_t span = a.width;   // of what repeats
    for (int k = 0; k < n; ++k) {
        const int64_t step = a.step[order[k]];
        bool repeats = true;
        for (int j = k + 1; j < n; ++j) repeats &= a.step[order[j]] % step == 0;
        const int64_t off = static_cast<int64_t>(apart % static_cast<uintptr_t>(step));
        if (repeats && off >= span && off + span <= step) return false;
        span += (a.n[order[k]] - 1) * step;
    }
    return true;
}

// Checks of a cache that the two entry points share.
kda_status cache_checks(const void *k, const void *v, const float *ks, const float *vs, int64_t B,
                        int64_t Hkv, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages,
                        int64_t ks_stride, int64_t vs_stride, Cells *kc, Cells *vc) {
    if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED_DIM;
    if (B < 0 || B > 65536 || Hkv < 1 || Hkv > 65535 || pages < 0 || pages >= k31 || page_size < 1 ||
        page_size >= k31 || max_pages < 0 || max_pages >= k31 || max_pages * page_size >= k31 ||
        !rows_fit(pages, ks_stride, Hkv) || !rows_fit(pages, vs_stride, Hkv))
        return KDA_ERR_BAD_SHAPE;
    for (Cells *c : {kc, vc}) {
        c->width = D;
        c->n[0] = pages;
        c->n[1] = page_size;
        c->n[2] = Hkv;
        for (int64_t s : c->step)
            if (s < 0) return KDA_ERR_BAD_SHAPE;
        if (!cells_fit(*c)) return KDA_ERR_BAD_SHAPE;
        for (int i = 0; i < 3; ++i)
            if (c->n[i] > 1 && c->step[i] % 16 != 0) return KDA_ERR_MISALIGNED;
    }
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(ks, 4) || misaligned(vs, 4))
        return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

kda::Cache8 cache_of(const Cells &k, const Cells &v, const float *ks, const float *vs,
                     const int32_t *table, const int32_t *lens, int64_t B, int64_t max_pages,
                     int64_t ks_stride, int64_t vs_stride) {
    kda::Cache8 c{};
    c.k = static_cast<uint8_t *>(const_cast<void *>(k.p));
    c.v = static_cast<uint8_t *>(const_cast<void *>(v.p));
    c.ks = const_cast<float *>(ks);
    c.vs = const_cast<float *>(vs);
    c.k_page = k.step[0]; c.k_token = k.step[1]; c.k_head = k.step[2];
    c.v_page = v.step[0]; c.v_token = v.step[1]; c.v_head = v.step[2];
    c.ks_page = ks_stride; c.vs_page = vs_stride;
    c.pages = k.n[0]; c.max_pages = max_pages;
    c.table = table; c.lens = lens;
    c.batch = static_cast<int32_t>(B); c.hkv = static_cast<int32_t>(k.n[2]);
    c.dim = static_cast<int32_t>(k.width); c.page_size = static_cast<int32_t>(k.n[1]);
    return c;
}

kda_status begin(kda::Operator op, const void *const *ptrs, int n, void *stream, int64_t ws,
                 int64_t sync, kda::CallContext *ctx) {
    return static_cast<kda_status>(kda::begin_call(op, ptrs, n, stream, ws, sync, ctx));
}

// Checks of the two entry points for heads; the outputs' blocks are the caller's.
kda_status heads_checks(const void *q, const void *k, const float *qw, const float *kw,
                        const float *freq, const int32_t *pos, int64_t T, int64_t Hq, int64_t Hk,
                        int64_t D, int64_t R, int64_t q_stride, int64_t k_stride, float eps) {
    if ((D != 64 && D != 128 && D != 256) || R < 0 || R > D || R % 16 != 0)
        return KDA_ERR_UNSUPPORTED_DIM;
    if (T < 0 || T >= k31 || Hq < 1 || Hk < 0 || Hq + Hk > 65535 || !(eps >= 0.f) ||
        !rows_fit(T, q_stride, Hq * D) || (Hk > 0 && !rows_fit(T, k_stride, Hk * D)))
        return KDA_ERR_BAD_SHAPE;
    if (T > 0 && (!q || (Hk > 0 && !k) || (R > 0 && (!freq || !pos)))) return KDA_ERR_NULL_ARG;
    if (misaligned(q, 16) || q_stride % 8 != 0 || (Hk > 0 && (misaligned(k, 16) || k_stride % 8 != 0)) ||
        misaligned(qw, 4) || misaligned(kw, 4) || misaligned(freq, 4) || misaligned(pos, 4))
        return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

kda::HeadsParams heads_params(const void *q, const void *k, const float *qw, const float *kw,
                              const float *freq, const int32_t *pos, int64_t T, int64_t Hq,
                              int64_t Hk, int64_t D, int64_t R, int64_t q_stride, int64_t k_stride,
                              float eps, int flags) {
    kda::HeadsParams p{};
    p.q = q; p.k = k; p.qw = qw; p.kw = kw; p.freq = freq; p.pos = pos;
    p.tokens = T; p.q_stride = q_stride; p.k_stride = k_stride;
    p.hq = static_cast<int32_t>(Hq); p.hk = static_cast<int32_t>(Hk);
    p.dim = static_cast<int32_t>(D); p.rot = static_cast<int32_t>(R);
    p.eps = eps;
    p.pairs = (flags & KDA_ROPE_INTERLEAVED) != 0;
    p.dout32 = (flags & KDA_ROPE_DOUT_FP32) != 0;
    p.stall = g_stall_heads.load();
    return p;
}

}  // namespace

extern "C" {

kda_status kda_page_plan(const int32_t *page_table, const int32_t *seq_lens,
                         const int32_t *new_lens, const uint8_t *release,
                         const int32_t *free_pages, const int32_t *free_count, int64_t B,
                         int64_t max_pages, int64_t pool, int64_t page_size, int64_t T,
                         int32_t *page_table_out, int32_t *seq_lens_out, int32_t *free_pages_out,
                         int32_t *free_count_out, int32_t *cu_seqlens, int32_t *positions,
                         int64_t *slots, void *stream) {
    if (B < 0 || B > 65536 || max_pages < 0 || max_pages >= k31 || pool < 0 || pool >= k31 ||
        page_size < 1 || page_size >= k31 || max_pages * page_size >= k31 || T < 0 || T >= k31)
        return KDA_ERR_BAD_SHAPE;
    if (!free_count || !free_count_out || !cu_seqlens || (T > 0 && (!positions || !slots)) ||
        (pool > 0 && (!free_pages || !free_pages_out)) || (B > 0 && (!seq_lens || !new_lens || !seq_lens_out)) ||
        (B * max_pages > 0 && (!page_table || !page_table_out)))
        return KDA_ERR_NULL_ARG;
    if (misaligned(page_table, 4) || misaligned(seq_lens, 4) || misaligned(new_lens, 4) ||
        misaligned(free_pages, 4) || misaligned(free_count, 4) || misaligned(page_table_out, 4) ||
        misaligned(seq_lens_out, 4) || misaligned(free_pages_out, 4) ||
        misaligned(free_count_out, 4) || misaligned(cu_seqlens, 4) || misaligned(positions, 4) ||
        misaligned(slots, 8))
        return KDA_ERR_MISALIGNED;
    const int64_t nt = 4 * B * max_pages;
    auto other = [](const void *in, const void *out, int64_t bytes) {
        return flat(in == out ? nullptr : in, bytes);
    };
    const Rows ins[] = {other(page_table, page_table_out, nt), other(seq_lens, seq_lens_out, 4 * B),
                        flat(new_lens, 4 * B), flat(release, B),
                        other(free_pages, free_pages_out, 4 * pool),
                        other(free_count, free_count_out, 4)};
    const Rows outs[] = {flat(page_table_out, nt), flat(seq_lens_out, 4 * B),
                         flat(free_pages_out, 4 * pool), flat(free_count_out, 4),
                         flat(cu_seqlens, 4 * (B + 1)), flat(positions, 4 * T), flat(slots, 8 * T)};
    if (any_shared(outs, 7, ins, 6)) return KDA_ERR_ALIAS;

    kda::PlanParams p{};
    p.table = page_table; p.lens = seq_lens; p.news = new_lens; p.free = free_pages;
    p.count = free_count; p.release = release;
    p.width = max_pages; p.pool = pool; p.page_size = page_size; p.tokens = T;
    p.batch = static_cast<int32_t>(B);
    p.table_out = page_table_out; p.lens_out = seq_lens_out; p.free_out = free_pages_out;
    p.count_out = free_count_out; p.cu = cu_seqlens; p.pos = positions; p.slots = slots;
    const void *ptrs[] = {page_table, seq_lens, new_lens, release, free_pages, free_count,
                          page_table_out, seq_lens_out, free_pages_out, free_count_out, cu_seqlens,
                          positions, slots};
    kda::CallContext ctx;
    const kda_status rc = begin(kda::kCache, ptrs, 13, stream, kda::plan_workspace(p), 0, &ctx);
    if (rc != KDA_OK) return rc;
    p.meta = reinterpret_cast<int64_t *>(ctx.ws);
    p.err = ctx.err;
    return status(kda::launch_plan(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_qk_norm_rope(const void *q, const void *k, const float *q_weight,
                            const float *k_weight, const float *inv_freq,
                            const int32_t *positions, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                            int64_t R, int64_t q_stride, int64_t k_stride, float eps, int flags,
                            void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                            void *stream) {
    if ((flags & ~KDA_ROPE_INTERLEAVED) != 0) return KDA_ERR_BAD_FLAGS;
    const kda_status bad = heads_checks(q, k, q_weight, k_weight, inv_freq, positions, T, Hq, Hk, D,
                                        R, q_stride, k_stride, eps);
    if (bad != KDA_OK) return bad;
    if (!rows_fit(T, q_out_stride, Hq * D) || (Hk > 0 && !rows_fit(T, k_out_stride, Hk * D)))
        return KDA_ERR_BAD_SHAPE;
    if (T > 0 && (!q_out || (Hk > 0 && !k_out))) return KDA_ERR_NULL_ARG;
    if (misaligned(q_out, 16) || q_out_stride % 8 != 0 ||
        (Hk > 0 && (misaligned(k_out, 16) || k_out_stride % 8 != 0)))
        return KDA_ERR_MISALIGNED;
    const Rows rq{q, T, 2 * Hq * D, 2 * q_stride}, rk{k, Hk > 0 ? T : 0, 2 * Hk * D, 2 * k_stride},
        none{nullptr, 0, 0, 0};
    const bool in_q = q_out == q && q_out_stride == q_stride,
               in_k = k_out == k && k_out_stride == k_stride;
    const Rows oq{q_out, T, 2 * Hq * D, 2 * q_out_stride},
        ok{k_out, Hk > 0 ? T : 0, 2 * Hk * D, 2 * k_out_stride};
    const Rows ins[] = {in_q ? none : rq, in_k ? none : rk, flat(q_weight, 4 * D),
                        flat(k_weight, 4 * D), flat(inv_freq, 2 * R), flat(positions, R > 0 ? 4 * T : 0)};
    const Rows outs[] = {oq, ok};
    if (any_shared(outs, 2, ins, 6)) return KDA_ERR_ALIAS;
    if (T == 0) return KDA_OK;   // an empty batch enqueues nothing

    kda::HeadsParams p = heads_params(q, k, q_weight, k_weight, inv_freq, positions, T, Hq, Hk, D, R,
                                      q_stride, k_stride, eps, flags);
    p.q_out = q_out; p.k_out = k_out; p.qo_stride = q_out_stride; p.ko_stride = k_out_stride;
    const void *ptrs[] = {q, Hk > 0 ? k : nullptr, q_weight, k_weight, R > 0 ? inv_freq : nullptr,
                          R > 0 ? positions : nullptr, q_out, Hk > 0 ? k_out : nullptr};
    kda::CallContext ctx;
    const kda_status rc = begin(kda::kHeads, ptrs, 8, stream, 0, 0, &ctx);
    if (rc != KDA_OK) return rc;
    p.err = ctx.err;
    return status(kda::launch_heads(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_qk_norm_rope_backward(
    const void *q, const void *k, const float *q_weight, const float *k_weight,
    const float *inv_freq, const int32_t *positions, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
    int64_t R, int64_t q_stride, int64_t k_stride, float eps, int flags, const void *dq_out,
    int64_t dq_out_stride, const void *dk_out, int64_t dk_out_stride, void *dq, int64_t dq_stride,
    void *dk, int64_t dk_stride, float *dq_weight, float *dk_weight, void *stream) {
    if ((flags & ~(KDA_ROPE_INTERLEAVED | KDA_ROPE_DOUT_FP32)) != 0) return KDA_ERR_BAD_FLAGS;
    const kda_status bad = heads_checks(q, k, q_weight, k_weight, inv_freq, positions, T, Hq, Hk, D,
                                        R, q_stride, k_stride, eps);
    if (bad != KDA_OK) return bad;
    if (!rows_fit(T, dq_out_stride, Hq * D) || !rows_fit(T, dq_stride, Hq * D) ||
        (Hk > 0 && (!rows_fit(T, dk_out_stride, Hk * D) || !rows_fit(T, dk_stride, Hk * D))))
        return KDA_ERR_BAD_SHAPE;
    if (T > 0 && (!dq_out || !dq || (Hk > 0 && (!dk_out || !dk)))) return KDA_ERR_NULL_ARG;
    const int64_t size = (flags & KDA_ROPE_DOUT_FP32) != 0 ? 4 : 2;
    if (misaligned(dq_out, 16) || dq_out_stride % (16 / size) != 0 || misaligned(dq, 16) || dq_stride % 8 != 0 ||
        (Hk > 0 && (misaligned(dk_out, 16) || dk_out_stride % (16 / size) != 0 || misaligned(dk, 16) ||
                    dk_stride % 8 != 0)) ||
        misaligned(dq_weight, 4) || misaligned(dk_weight, 4))
        return KDA_ERR_MISALIGNED;
    const int64_t tk = Hk > 0 ? T : 0;
    const Rows ins[] = {{q, T, 2 * Hq * D, 2 * q_stride}, {k, tk, 2 * Hk * D, 2 * k_stride},
                        flat(q_weight, 4 * D), flat(k_weight, 4 * D), flat(inv_freq, 2 * R),
                        flat(positions, R > 0 ? 4 * T : 0),
                        {dq_out, T, size * Hq * D, size * dq_out_stride},
                        {dk_out, tk, size * Hk * D, size * dk_out_stride}};
    const Rows outs[] = {{dq, T, 2 * Hq * D, 2 * dq_stride}, {dk, tk, 2 * Hk * D, 2 * dk_stride},
                         flat(dq_weight, 4 * D), flat(dk_weight, 4 * D)};
    if (any_shared(outs, 4, ins, 8)) return KDA_ERR_ALIAS;
    if (T == 0 && !dq_weight && !dk_weight) return KDA_OK;   // nothing to write

    kda::HeadsParams p = heads_params(q, k, q_weight, k_weight, inv_freq, positions, T, Hq, Hk, D, R,
                                      q_stride, k_stride, eps, flags);
    p.q_out = dq; p.k_out = dk; p.qo_stride = dq_stride; p.ko_stride = dk_stride;
    p.dq = dq_out; p.dk = dk_out; p.dq_stride = dq_out_stride; p.dk_stride = dk_out_stride;
    p.dqw = dq_weight; p.dkw = dk_weight;
    const bool hk = Hk > 0;
    const void *ptrs[] = {q, hk ? k : nullptr, q_weight, k_weight, R > 0 ? inv_freq : nullptr,
                          R > 0 ? positions : nullptr, dq_out, hk ? dk_out : nullptr, dq,
                          hk ? dk : nullptr, dq_weight, dk_weight};
    kda::CallContext ctx;
    const kda_status rc = begin(kda::kHeads, ptrs, 12, stream, kda::heads_workspace(p), 0, &ctx);
    if (rc != KDA_OK) return rc;
    p.partial = reinterpret_cast<float *>(ctx.ws);
    p.err = ctx.err;
    return status(kda::launch_heads_backward(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_paged_append_fp8(
    const void *k, const void *v, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
    const int32_t *page_table, const int32_t *seq_lens, const int32_t *cu_seqlens, int64_t T,
    int64_t B, int64_t Hkv, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages,
    int64_t k_stride, int64_t v_stride, int64_t k_page_stride, int64_t k_token_stride,
    int64_t k_head_stride, int64_t v_page_stride, int64_t v_token_stride, int64_t v_head_stride,
    int64_t k_scale_stride, int64_t v_scale_stride, void *stream) {
    Cells kc{k_cache, 0, {}, {k_page_stride, k_token_stride, k_head_stride}},
        vc{v_cache, 0, {}, {v_page_stride, v_token_stride, v_head_stride}};
    const kda_status bad = cache_checks(k_cache, v_cache, k_scale, v_scale, B, Hkv, D, pages,
                                        page_size, max_pages, k_scale_stride, v_scale_stride, &kc, &vc);
    if (bad != KDA_OK) return bad;
    if (T < 0 || T >= k31 || (T + 2 * B) * Hkv >= (int64_t(1) << 30) || (cu_seqlens == nullptr && T != B) ||
        !rows_fit(T, k_stride, Hkv * D) || !rows_fit(T, v_stride, Hkv * D))
        return KDA_ERR_BAD_SHAPE;
    const bool any = T > 0 && B > 0;
    if (any && (!k || !v || !seq_lens || (max_pages > 0 && !page_table) ||
                (pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale))))
        return KDA_ERR_NULL_ARG;
    if (misaligned(k, 16) || misaligned(v, 16) || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        misaligned(page_table, 4) || misaligned(seq_lens, 4) || misaligned(cu_seqlens, 4))
        return KDA_ERR_MISALIGNED;
    const Rows ins[] = {{k, T, 2 * Hkv * D, 2 * k_stride}, {v, T, 2 * Hkv * D, 2 * v_stride},
                        flat(page_table, 4 * B * max_pages), flat(seq_lens, 4 * B),
                        flat(cu_seqlens, 4 * (B + 1))};
    const Rows scales[] = {{k_scale, pages, 4 * Hkv, 4 * k_scale_stride},
                           {v_scale, pages, 4 * Hkv, 4 * v_scale_stride}};
    const Rows ck[] = {range(kc)}, cv[] = {range(vc)};
    if (any_shared(scales, 2, ins, 5) || any_shared(ck, 1, ins, 5) || any_shared(cv, 1, ins, 5) ||
        any_shared(ck, 1, scales, 2) || any_shared(cv, 1, scales, 2) || cells_share(kc, vc))
        return KDA_ERR_ALIAS;
    if (!any) return KDA_OK;   // an empty batch enqueues nothing

    kda::AppendParams p{};
    p.c = cache_of(kc, vc, k_scale, v_scale, page_table, seq_lens, B, max_pages, k_scale_stride,
                   v_scale_stride);
    p.k = k; p.v = v; p.cu = cu_seqlens; p.tokens = T; p.k_stride = k_stride; p.v_stride = v_stride;
    const void *ptrs[] = {k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_seqlens};
    kda::CallContext ctx;
    const kda_status rc = begin(kda::kCache, ptrs, 9, stream, 0, 0, &ctx);
    if (rc != KDA_OK) return rc;
    p.c.err = ctx.err;
    return status(kda::launch_append(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_test_stall_qk_norm_rope(int batch) {
    if (batch < -1) return KDA_ERR_BAD_SHAPE;
    g_stall_heads.store(batch < 0 ? INT_MAX : batch);
    return KDA_OK;
}

kda_status kda_test_stall_paged_fp8(int tile) {
    if (tile < -1) return KDA_ERR_BAD_SHAPE;
    g_stall_paged8.store(tile < 0 ? INT_MAX : tile);
    return KDA_OK;
}

kda_status kda_paged_decode_fp8(
    const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
    const float *v_scale, const int32_t *page_table, const int32_t *seq_lens, int64_t B,
    int64_t Hq, int64_t Hkv, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages,
    int64_t k_page_stride, int64_t k_token_stride, int64_t k_head_stride, int64_t v_page_stride,
    int64_t v_token_stride, int64_t v_head_stride, int64_t k_scale_stride, int64_t v_scale_stride,
    float scale, void *out, float *lse, void *stream) {
    Cells kc{k_cache, 0, {}, {k_page_stride, k_token_stride, k_head_stride}},
        vc{v_cache, 0, {}, {v_page_stride, v_token_stride, v_head_stride}};
    const kda_status bad = cache_checks(k_cache, v_cache, k_scale, v_scale, B, Hkv, D, pages,
                                        page_size, max_pages, k_scale_stride, v_scale_stride, &kc, &vc);
    if (bad != KDA_OK) return bad;
    if (Hq < Hkv || Hq > 65535 || Hq % Hkv != 0) return KDA_ERR_BAD_SHAPE;
    if (B > 0 && (!q || !out || !seq_lens)) return KDA_ERR_NULL_ARG;
    if (B > 0 && max_pages > 0 && (!page_table || (pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale))))
        return KDA_ERR_NULL_ARG;
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(page_table, 4) ||
        misaligned(seq_lens, 4) || misaligned(lse, 4))
        return KDA_ERR_MISALIGNED;
    const int64_t nq = B * Hq * D * 2;
    const Rows ins[] = {flat(q, nq), range(kc), range(vc),
                        {k_scale, pages, 4 * Hkv, 4 * k_scale_stride},
                        {v_scale, pages, 4 * Hkv, 4 * v_scale_stride},
                        flat(page_table, B * max_pages * 4), flat(seq_lens, B * 4)};
    const Rows outs[] = {flat(out, nq), flat(lse, B * Hq * 4)};
    if (any_shared(outs, 2, ins, 7)) return KDA_ERR_ALIAS;
    if (B == 0) return KDA_OK;   // an empty batch enqueues nothing

    kda::Paged8Params p{};
    p.c = cache_of(kc, vc, k_scale, v_scale, page_table, seq_lens, B, max_pages, k_scale_stride,
                   v_scale_stride);
    p.q = q; p.hq = static_cast<int32_t>(Hq); p.scale = scale; p.out = out; p.lse = lse;
    p.stall = g_stall_paged8.load();
    p.divide_by(static_cast<uint32_t>(page_size));
    const void *ptrs[] = {q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, out, lse};
    kda::CallContext ctx;
    const kda_status rc = begin(kda::kPaged8, ptrs, 9, stream, kda::paged8_workspace(p),
                                kda::paged8_sync(p), &ctx);
    if (rc != KDA_OK) return rc;
    p.c.err = ctx.err;
    return status(kda::launch_paged8(p, ctx, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
