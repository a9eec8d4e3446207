/*
 * kda.h -- C ABI of the GB300 (sm_103a) chunked prefill for Kimi Delta
 * Attention (KDA).
 *
 * The operation. KDA keeps one fixed-size recurrent state per (sequence,
 * head) in place of a growing key-value cache, and every token updates it
 * ("Kimi K3 開源基礎設施", section "FlashKDA"; "Kimi K3 的三個系統設計",
 * section "第一個設計"). The update is the gated delta rule with a decay per
 * key channel:
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(exp(g_t)) S_{t-1} + beta_t k_t v_t^T
 *     o_t = scale * S_t^T q_t
 *
 * with S a K x V fp32 matrix (row = key channel). Prefill computes it in
 * 16-token chunks with two kernels of different parallelism, a
 * token-parallel intra-chunk kernel and a recurrent inter-chunk kernel
 * ("Kimi K3 的三個系統設計", section "為什麼 FlashKDA 選擇 16-token chunks"),
 * over fixed-length or packed variable-length batches with K = V = 128
 * ("MoonEP / FlashKDA / AgentENV" release note, section "MoE通信とアテンション").
 *
 * Conventions for every entry point:
 *   - Pointers named as device pointers must be CUDA device memory (or
 *     managed memory) on the CURRENT device; the caller owns them. The
 *     library never frees them and holds none of them after the stream work
 *     the call enqueued has finished.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream). All work is enqueued on it; no entry point but
 *     kda_last_device_error() blocks the host.
 *   - Errors found from the arguments alone are returned before anything
 *     is enqueued and leave every output untouched.
 *   - Workspaces belong to the (device, stream) of the call. A graph keeps the
 *     ones that its calls were captured with, also when a later call on that
 *     stream needs larger ones; graphs captured on one stream share them with one
 *     another and with its later calls, so that replays and calls may follow one
 *     another in any order, but not run side by side.
 */
#ifndef KDA_GB300_H
#define KDA_GB300_H

#include <stdint.h>

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_NULL_ARG = -1,          /* a required pointer is NULL */
    KDA_ERR_BAD_SHAPE = -2,         /* B, T, H, N inconsistent or out of range */
    KDA_ERR_UNSUPPORTED_DIM = -3,   /* K or V is not 128 (or another size the entry point
                                       does not take: see there) */
    KDA_ERR_MISALIGNED = -4,        /* a pointer breaks the alignment rule below */
    KDA_ERR_BAD_CU_SEQLENS = -5,    /* (device) cu_seqlens not 0..T nondecreasing */
    KDA_ERR_CUDA = -6,              /* a CUDA runtime call failed */
    KDA_ERR_DEVICE_TIMEOUT = -7,    /* (device) a bounded wait inside a kernel ran out */
    KDA_ERR_NO_DEVICE_SUPPORT = -8, /* current device is not sm_103 */
    KDA_ERR_ALIAS = -9,             /* out or final_state overlaps an input */
    KDA_ERR_GATE_RANGE = -10,       /* (device) log decay rose by more than 80 inside a chunk */
    KDA_ERR_CAPTURE = -11,          /* workspace must grow while the stream is capturing */
    KDA_ERR_WRONG_DEVICE = -12,     /* a buffer or the stream belongs to another device */
    KDA_ERR_NOT_DEVICE_MEMORY = -13, /* a pointer is not CUDA device (or managed) memory */
    KDA_ERR_SCRATCH_LIMIT = -14,    /* kda_chunk_prefill_noalloc: the call needs more scratch
                                       than its fixed 64 MiB array holds */
    KDA_ERR_BAD_FLAGS = -15,        /* a flag bit the entry point does not know */
    KDA_ERR_BAD_PAGE_TABLE = -16,   /* (device) a sequence length or page index out of range */
    KDA_ERR_OUT_OF_PAGES = -17      /* (device) kda_page_plan: too few free pages */
} kda_status;

/*
 * Input preprocessing done inside the kernels (the `flags` argument of
 * kda_chunk_prefill_ex and kda_decode_step). The pages leave the production
 * of q, k and g to the model; these let a caller hand over raw projections and
 * skip a separate pass over them.
 *   KDA_PRE_NORM_QK      q and k are raw: the kernels use x / sqrt(sum x^2 + 1e-6)
 *                        over the 128 channels of each (token, head)
 *   KDA_PRE_GATE_LOGITS  g holds gate logits x: the per-token log decay is
 *                        logsigmoid(x) = -log(1 + exp(-x))
 */
enum { KDA_PRE_NORM_QK = 1, KDA_PRE_GATE_LOGITS = 2 };

/*
 * kda_chunk_prefill -- chunked KDA prefill over a batch of sequences.
 *
 * Layout (all row-major, tokens of all sequences packed back to back):
 *   q, k      device, bf16  [B*T, H, K]   (the method expects L2-normalised rows)
 *   v         device, bf16  [B*T, H, V]
 *   g         device, fp32  [B*T, H, K]   per-token log decay (<= 0), NOT cumulated
 *   beta      device, fp32  [B*T, H]      in (0, 1)
 *   initial_state device, fp32 [N, H, K, V] or NULL (= zero state);
 *             element [n,h,i,j] is S[key i][value j]
 *   cu_seqlens device, int32 [N+1] or NULL. NULL: N = B sequences of T tokens
 *             each. Non-NULL: B must be 1, sequence n holds tokens
 *             [cu[n], cu[n+1]); cu[0] = 0, cu[N] = T, nondecreasing (empty
 *             sequences allowed). Checked on the device: a violation makes
 *             the kernels skip all work and kda_last_device_error() report
 *             KDA_ERR_BAD_CU_SEQLENS.
 *   B, T, H, K, V, N  sizes; K = V = 128 only; H >= 1; T >= 0; N >= 1;
 *             B*T*H*128 < 2^40.
 *   scale     multiplies o (1/sqrt(K) is the usual choice).
 *   out       device, bf16 [B*T, H, V], written for every token.
 *             With zero tokens (B*T == 0) q, k, v, g, beta and out may be NULL.
 *   final_state device, fp32 [N, H, K, V] or NULL (= not written); may equal
 *             initial_state (updated in place).
 *   stream    cudaStream_t as void*.
 *
 * Alignment: q, k, v, g, out, initial_state, final_state 16-byte aligned;
 * beta and cu_seqlens 4-byte aligned.
 *
 * Gate range: g may be any finite log decay <= 0. Chunks whose per-channel
 * cumulative log decay stays in [-80, 80] use factored exponentials
 * exp(G_r) exp(-G_i); the others take an exact per-pair form (slower, same
 * results to rounding). Positive g is allowed as long as the cumulative log
 * decay does not rise by more than 80 between two points of a 16-token chunk
 * (counting the chunk start as 0); beyond that exp() leaves fp32's range and
 * the device flags KDA_ERR_GATE_RANGE (results then unspecified).
 *
 * Workspace: the library keeps one scratch buffer per (device, stream),
 * grown stream-ordered (cudaMallocAsync / cudaFreeAsync) when a call needs
 * more (17,412 B per chunk-head: its record and one list entry). A
 * fixed-length call on the 16-token path whose sequences have at least 64
 * chunks and with 4*N*H <= (SM count - 4) runs a segment-parallel scan with
 * P = 3*(SM count - 4) / (2*N*H) segments (at most 16, at least 16 chunks per
 * segment; or the P set by kda_set_scan_segments): every sequence is cut
 * into P segments whose affine state maps are built in parallel, a short
 * serial combine gives each segment's entry state, and all segments are
 * replayed side by side (same results to rounding; not with an in-place
 * state). It reserves (3P - 5) * N*H*64 KiB more. Concurrent calls on
 * different streams never share scratch. Growing is refused with KDA_ERR_CAPTURE
 * while the stream is being captured into a graph: make one call of the
 * largest size before capturing. kda_workspace_release() frees them.
 *
 * Returns KDA_OK once the work is enqueued, or a synchronous error. Errors
 * found on the device are reported by kda_last_device_error().
 */
KDA_API kda_status kda_chunk_prefill(const void *q, const void *k, const void *v, const float *g,
                             const float *beta, const float *initial_state,
                             const int32_t *cu_seqlens, int64_t B, int64_t T, int64_t H,
                             int64_t K, int64_t V, int64_t N, float scale, void *out,
                             float *final_state, void *stream);

/*
 * kda_chunk_prefill_ex -- kda_chunk_prefill with input preprocessing:
 * `flags` is a bitwise OR of KDA_PRE_* (0 = kda_chunk_prefill exactly). An
 * unknown bit returns KDA_ERR_BAD_FLAGS. Everything else, including the
 * gate range of the resulting log decays, is as for kda_chunk_prefill.
 */
KDA_API kda_status kda_chunk_prefill_ex(const void *q, const void *k, const void *v,
                                        const float *g, const float *beta,
                                        const float *initial_state, const int32_t *cu_seqlens,
                                        int64_t B, int64_t T, int64_t H, int64_t K, int64_t V,
                                        int64_t N, float scale, int flags, void *out,
                                        float *final_state, void *stream);

/*
 * kda_chunk_prefill_noalloc -- the same computation, arguments and results
 * as kda_chunk_prefill, for callers that cannot allocate device memory.
 * The pages have no counterpart to this entry point; it exists for users of
 * the library whose code may not call cudaMalloc/cudaMallocAsync (directly or
 * through this library): a host framework that owns all device allocations,
 * a serving loop that must not enter the driver's allocator on its hot path,
 * or a sandboxed plug-in. It allocates nothing. Its scratch is one
 * fixed-size device array inside the library (64 MiB, held on every GPU that
 * loads the library until the process exits). The call holds at once a
 * 256-byte flag block, the chunk-offset table of a packed batch ((N+1)*4 B),
 * every chunk record (17,408 B per 16-token chunk per head) and a 4-byte
 * list entry per chunk-head, each part rounded up to 256 B; a call that needs
 * more than 64 MiB (about 3850 chunk-heads) returns KDA_ERR_SCRATCH_LIMIT
 * before enqueuing anything. All calls share that array: calls whose GPU
 * work overlaps (e.g. on two streams) race and give wrong results. The first
 * call on a device does a one-time set-up with that device current (no
 * allocation); make it before any stream capture (a first call on a
 * capturing stream returns KDA_ERR_CAPTURE). Uncaptured calls check their
 * pointers and stream like kda_chunk_prefill (KDA_ERR_NOT_DEVICE_MEMORY,
 * KDA_ERR_WRONG_DEVICE). Device errors of this entry point are reported by
 * kda_last_device_error() like those of the others.
 */
KDA_API kda_status kda_chunk_prefill_noalloc(const void *q, const void *k, const void *v,
                                             const float *g, const float *beta,
                                             const float *initial_state,
                                             const int32_t *cu_seqlens, int64_t B, int64_t T,
                                             int64_t H, int64_t K, int64_t V, int64_t N,
                                             float scale, void *out, float *final_state,
                                             void *stream);

/*
 * kda_decode_step -- one new token for each of N sequences: the KDA state
 * update applied once per (sequence, head). The pages describe the state as
 * fixed-size and updated for every new token ("Kimi K3 的三個系統設計",
 * section 第一個設計); this is that step, batched:
 *
 *   S <- (I - beta k k^T) Diag(exp(g)) S + beta k v^T,   o = scale * S^T q
 *
 * with the post-update S, exactly the prefill recurrence at T = 1.
 *
 *   q, k, v      bf16 [N, H, 128], device, 16-byte aligned
 *   g            fp32 [N, H, 128] per-token log decay (any value; the
 *                exponentials are exact per channel, no range limit)
 *   beta         fp32 [N, H]
 *   state_in     fp32 [N, H, 128 (K), 128 (V)] or NULL (zero state)
 *   state_out    fp32 [N, H, 128, 128], written; may be state_in itself
 *                (in place) but may not overlap it otherwise
 *   N, H         sequences and heads (N * H < 2^31); K = V = 128 only
 *   flags        KDA_PRE_* bits (0: q, k, g used as given), as for
 *                kda_chunk_prefill_ex
 *   out          bf16 [N, H, 128], written; may not overlap any input or state
 *   stream       cudaStream_t (NULL = legacy default stream)
 *
 * Allocates nothing and reads no workspace: each (sequence, head) is one CTA
 * that reads its state once and writes it once. Returns KDA_OK once the work
 * is enqueued, or a synchronous error (the outputs are then untouched). It
 * has no device-side error conditions.
 */
KDA_API kda_status kda_decode_step(const void *q, const void *k, const void *v, const float *g,
                                   const float *beta, const float *state_in, float *state_out,
                                   int64_t N, int64_t H, int64_t K, int64_t V, float scale,
                                   int flags, void *out, void *stream);

/*
 * kda_chunk_prefill_backward -- gradients of kda_chunk_prefill (training).
 * The pages say that K3 trains with KDA ("Kimi K3 開源基礎設施"); this is the
 * reverse mode of the same map, for a loss L with dL/do = d_out and
 * dL/d(final_state) = d_final_state:
 *
 *   dq, dk, dg  fp32 [B*T, H, 128]  dL/dq, dL/dk, dL/dg (g = the log decay)
 *   dv          fp32 [B*T, H, 128]  dL/dv
 *   dbeta       fp32 [B*T, H]       dL/dbeta
 *   d_initial_state  fp32 [N, H, 128, 128] or NULL (not written):
 *               dL/d(initial_state) (the gradient of a zero state when
 *               initial_state is NULL)
 *
 * Inputs exactly as for kda_chunk_prefill (q, k, v bf16; g, beta fp32;
 * initial_state, cu_seqlens, B, T, H, K, V, N, scale), plus
 *   d_out          bf16 [B*T, H, 128], device
 *   d_final_state  fp32 [N, H, 128, 128] or NULL (= 0)
 * Outputs are device memory the caller owns, every element written; none may
 * overlap an input or another output. Alignment: 16 bytes for every array
 * but beta, dbeta and cu_seqlens (4 bytes). No input preprocessing: q, k
 * and g are used as given. Any finite g.
 *
 * Method: one CTA per (sequence, head) walks the sequence backwards token
 * by token, the state recomputed from checkpoints taken every 16 tokens.
 * Workspace (the call's stream's, as for the prefill): 64 KiB per 16-token
 * chunk per head plus 1 MiB per CTA of the persistent kernel, min(N * H,
 * 1024) of them. Errors as for the prefill
 * (bad cu_seqlens contents are flagged on the device, see
 * kda_last_device_error).
 */
KDA_API kda_status kda_chunk_prefill_backward(const void *q, const void *k, const void *v,
                                              const float *g, const float *beta,
                                              const float *initial_state,
                                              const int32_t *cu_seqlens, int64_t B, int64_t T,
                                              int64_t H, int64_t K, int64_t V, int64_t N,
                                              float scale, const void *d_out,
                                              const float *d_final_state, float *dq, float *dk,
                                              float *dv, float *dg, float *dbeta,
                                              float *d_initial_state, void *stream);

/*
 * kda_short_conv -- short causal convolution, one filter per channel, over a
 * batch of sequences: what stands in front of q, k and v of a KDA layer (and
 * of x, B and C of a state space layer). For token t of a sequence
 *
 *     z[t, d] = bias[d] + sum_{j < W} weight[d, j] * x[t - (W - 1) + j, d]
 *     out     = z, or z / (1 + exp(-z)) with KDA_CONV_SILU
 *
 * where rows before the sequence's first token come from its history (zeros
 * without initial_state). Sums in fp32, out rounded once to bf16.
 *
 *   x            device, bf16 [B*T, D], rows x_stride elements apart (so x may
 *                be a slice of a fused projection)
 *   weight       device, fp32 [D, W]; W = 2, 3 or 4 (others: KDA_ERR_UNSUPPORTED_DIM)
 *   bias         device, fp32 [D] or NULL
 *   initial_state device, bf16 [N, W-1, D] or NULL: the W-1 rows before each
 *                sequence, the newest last
 *   cu_seqlens, B, T, N  as for kda_chunk_prefill (contents checked on the
 *                device: a violation makes the kernels skip all work and
 *                kda_last_device_error() report KDA_ERR_BAD_CU_SEQLENS)
 *   out          device, bf16 [B*T, D], rows out_stride elements apart
 *   final_state  device, bf16 [N, W-1, D] or NULL: the last W-1 rows of
 *                (history, sequence); not initial_state itself
 *   1 <= D <= 2^24; x_stride, out_stride >= D; B*T < 2^31 and
 *   B*T*max(strides) < 2^40.
 *
 * Any D, strides and alignment to the element are taken; rows that start on
 * 16-byte boundaries (8-byte ones next) with D a multiple of 8 (4) run
 * fastest. No workspace.
 */
enum { KDA_CONV_SILU = 1, KDA_CONV_DOUT_FP32 = 2 };

KDA_API kda_status kda_short_conv(const void *x, const float *weight, const float *bias,
                                  const void *initial_state, const int32_t *cu_seqlens,
                                  int64_t B, int64_t T, int64_t D, int64_t W, int64_t N,
                                  int64_t x_stride, int flags, void *out, int64_t out_stride,
                                  void *final_state, void *stream);

/*
 * kda_short_conv_step -- one new token for each of N sequences: the
 * convolution at T = 1, the history shifted by one row.
 *   x, out       bf16 [N, D], rows x_stride / out_stride elements apart
 *   state_in     bf16 [N, W-1, D] or NULL (zeros)
 *   state_out    bf16 [N, W-1, D], written; may be state_in itself, but may not
 *                overlap it otherwise
 * weight, bias, D, W, flags (KDA_CONV_SILU) as for kda_short_conv. N = 0 is a
 * no-op.
 */
KDA_API kda_status kda_short_conv_step(const void *x, const float *weight, const float *bias,
                                       const void *state_in, int64_t N, int64_t D, int64_t W,
                                       int64_t x_stride, int flags, void *out,
                                       int64_t out_stride, void *state_out, void *stream);

/*
 * kda_short_conv_backward -- gradients of kda_short_conv for a loss L with
 * dL/d(out) = d_out and dL/d(final_state) = d_final_state:
 *
 *   dz = d_out, times s (1 + z (1 - s)) with s = 1 / (1 + exp(-z)) under KDA_CONV_SILU
 *   dx[t, d]      = sum_j weight[d, j] dz[t + (W - 1) - j, d]   (within the sequence)
 *   dweight[d, j] = sum_t dz[t, d] x[t - (W - 1) + j, d],   dbias[d] = sum_t dz[t, d]
 *
 * z is computed again from x. Rows of the history get d_initial_state by the
 * same sum; d_final_state is added to the rows that final_state holds.
 *   d_out        device [B*T, D], rows dout_stride elements apart: bf16, or fp32
 *                with KDA_CONV_DOUT_FP32 (the gradients of
 *                kda_chunk_prefill_backward are fp32)
 *   d_final_state fp32 [N, W-1, D] or NULL (zeros)
 *   dx           bf16 [B*T, D], rows dx_stride elements apart
 *   dweight      fp32 [D, W]; dbias fp32 [D] or NULL
 *   d_initial_state fp32 [N, W-1, D] or NULL (not written)
 * The sums over tokens are taken in fp32 in a fixed order (the same call gives
 * the same bits). Workspace (the stream's, as for the prefill): (W + 1) * D
 * floats for every 512 to 1024 tokens (for fewer, when the call is small).
 */
KDA_API kda_status kda_short_conv_backward(const void *x, const float *weight, const float *bias,
                                           const void *initial_state, const int32_t *cu_seqlens,
                                           int64_t B, int64_t T, int64_t D, int64_t W, int64_t N,
                                           int64_t x_stride, int flags, const void *d_out,
                                           int64_t dout_stride, const float *d_final_state,
                                           void *dx, int64_t dx_stride, float *dweight,
                                           float *dbias, float *d_initial_state, void *stream);

/*
 * kda_ssm_prefill -- selective state space scan with one decay per head over a
 * batch of sequences. With S an n x P fp32 matrix per (sequence, head) and
 * delta = dt, or softplus(dt + dt_bias) under KDA_SSM_DT_SOFTPLUS:
 *
 *     S_t = exp(a delta_t) S_{t-1} + delta_t b_t x_t^T
 *     y_t = S_t^T c_t + d x_t
 *
 *   x            device, bf16 [B*T, H, P], tokens x_stride elements apart
 *   dt           device, fp32 [B*T, H], tokens dt_stride elements apart
 *   a            device, fp32 [H]; a * delta is the log decay of a token and is
 *                expected to be <= 0 (a positive one is computed too, as long as
 *                the growth over any 128 tokens stays within fp32)
 *   b, c         device, bf16 [B*T, G, n], tokens b_stride / c_stride elements
 *                apart; head h uses group h / (H / G), H a multiple of G
 *   d            device, fp32 [H] or NULL (0)
 *   dt_bias      device, fp32 [H] or NULL (0); added whether or not softplus is taken
 *   initial_state device, fp32 [N, H, n, P] or NULL (zeros)
 *   cu_seqlens, B, T, N  as for kda_chunk_prefill
 *   out          device, bf16 [B*T, H, P] (contiguous)
 *   final_state  device, fp32 [N, H, n, P] or NULL (not written); may equal
 *                initial_state
 *   P = 64 or 128, n = 64 or 128 (others: KDA_ERR_UNSUPPORTED_DIM); H <= 65535,
 *   N*H < 2^30, B*T < 2^31.
 *
 * A log decay below -1024 log 2 counts as that (its exponential is 0 either way).
 * An infinity or NaN in x makes that channel of out NaN from its token to the
 * sequence's end, and that column of the state not finite; earlier tokens and
 * other channels are not touched.
 *
 * Alignment: x, b, c, out and the states 16 bytes, and x_stride, b_stride,
 * c_stride multiples of 8 elements; fp32 vectors and cu_seqlens 4 bytes.
 * States, decays and sums are held in fp32. The tensor core's operands are bf16: x, b
 * and c as they are, the state in S^T c and the decayed c . b in front of x as two
 * bf16 terms (16 bits of mantissa, below out's own rounding), and what enters the
 * state as three (24 bits). The outputs and states of a call are the
 * same bits every time. A packed batch of at most 512 tokens is not cut over the
 * SMs, so many short sequences in it take their turns, a chunk each (24 sequences
 * of 20 tokens: 115 us; of 22 tokens, which are cut: 25). Workspace (the stream's): 2,608 B of decays for every
 * 128 tokens of a sequence and head, 10 MB for the states where a sequence is
 * cut, and the chunk offsets of a packed batch.
 */
enum { KDA_SSM_DT_SOFTPLUS = 1 };

KDA_API kda_status kda_ssm_prefill(const void *x, const float *dt, const float *a, const void *b,
                                   const void *c, const float *d, const float *dt_bias,
                                   const float *initial_state, const int32_t *cu_seqlens,
                                   int64_t B, int64_t T, int64_t H, int64_t P, int64_t G,
                                   int64_t n, int64_t N, int64_t x_stride, int64_t dt_stride,
                                   int64_t b_stride, int64_t c_stride, int flags, void *out,
                                   float *final_state, void *stream);

/*
 * kda_ssm_step -- one new token for each of N sequences: the recurrence of
 * kda_ssm_prefill applied once per (sequence, head).
 *   x, dt, b, c, out  as there with one row per sequence
 *   state_in     fp32 [N, H, n, P] or NULL (zeros)
 *   state_out    fp32 [N, H, n, P], written; may be state_in itself (in place) but
 *                may not overlap it otherwise
 * Allocates nothing and uses no workspace; N = 0 is a no-op.
 */
KDA_API kda_status kda_ssm_step(const void *x, const float *dt, const float *a, const void *b,
                                const void *c, const float *d, const float *dt_bias,
                                const float *state_in, int64_t N, int64_t H, int64_t P, int64_t G,
                                int64_t n, int64_t x_stride, int64_t dt_stride, int64_t b_stride,
                                int64_t c_stride, int flags, void *out, float *state_out,
                                void *stream);

/*
 * kda_paged_decode -- attention of one new token per sequence over a paged
 * key-value cache (the full-attention layers of a hybrid model). For sequence
 * s, query head h and its key-value head h / (Hq / Hkv), over the cached
 * tokens j < seq_lens[s]:
 *
 *     out = sum_j softmax_j(scale q . k_j) v_j,   lse = log sum_j exp(scale q . k_j)
 *
 *   q            device, bf16 [B, Hq, D]
 *   k_cache, v_cache device, bf16 [pages, page_size, Hkv, D], pages k_page_stride
 *                / v_page_stride elements apart (both may be views of one cache);
 *                inside a page the layout is contiguous
 *   page_table   device, int32 [B, max_pages]: token j of sequence s lies in
 *                page page_table[s, j / page_size], row j % page_size. Entries
 *                past a sequence's last page are not read
 *   seq_lens     device, int32 [B], the new token's own key and value included;
 *                0 gives out = 0 and lse = -inf
 *   out          device, bf16 [B, Hq, D]
 *   lse          device, fp32 [B, Hq] or NULL (natural logarithm)
 *   D = 64 or 128 (others: KDA_ERR_UNSUPPORTED_DIM); Hq a multiple of Hkv;
 *   page_size >= 1; B <= 65536; Hq <= 65535; pages < 2^31;
 *   max_pages * page_size < 2^31.
 *
 * A length that is negative or beyond max_pages * page_size, or a page index
 * outside [0, pages), is reported by kda_last_device_error() as
 * KDA_ERR_BAD_PAGE_TABLE; such a length is taken as 0 and such a page as page 0
 * (nothing out of range is read), so the outputs of that sequence are then
 * meaningless and those of the others are right.
 *
 * Alignment: q, k_cache, v_cache, out 16 bytes, page strides multiples of 8
 * elements; int32 and fp32 arrays 4 bytes. Scores, softmax and sums in fp32; the
 * weights enter their product with v as two bf16 terms (16 bits of mantissa, below
 * out's own rounding; an infinity in v can therefore give NaN where the formula
 * gives an infinity). The sum over the cache is split over the SMs and joined in a fixed order (the
 * same call gives the same bits). Workspace: partial sums of the split.
 */
KDA_API kda_status kda_paged_decode(const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *page_table, const int32_t *seq_lens,
                                    int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t pages,
                                    int64_t page_size, int64_t max_pages, int64_t k_page_stride,
                                    int64_t v_page_stride, float scale, void *out, float *lse,
                                    void *stream);

/*
 * kda_page_plan -- page tables, positions and slots of a batch's next tokens, from
 * request lengths, on the GPU (what kda_paged_decode and the entry points below
 * read). Slot i of the batch holds seq_lens[i] tokens in the pages
 * page_table[i, 0 .. ceil(seq_lens[i] / page_size) - 1], and new_lens[i] tokens join
 * it; free_pages[0 .. free_count) is a stack of the pages that nobody holds.
 *
 *   1. Every slot with release[i] != 0 gives its pages back: they are pushed on the
 *      stack in the order of i, then of the page's place; the slot is then empty.
 *   2. Pages that the new tokens need are taken from the top of the stack, in the
 *      order of i, then of the page's place, and entered into the table.
 *   3. cu_seqlens[i] = new_lens[0] + .. + new_lens[i - 1]. Row r of slot i, in
 *      [cu_seqlens[i], cu_seqlens[i + 1]), is at position p = (tokens held) + r -
 *      cu_seqlens[i], in slot page_table[i, p / page_size] * page_size + p % page_size
 *      of the cache. Rows behind the last new token get position 0 and slot -1.
 *
 *   page_table   device, int32 [B, max_pages]
 *   seq_lens, new_lens device, int32 [B]
 *   release      device, uint8 [B] or NULL (none)
 *   free_pages   device, int32 [pool]; free_count device, int32 [1]
 *   page_table_out, seq_lens_out (tokens held after the call), free_pages_out,
 *   free_count_out: like their inputs; each may be its input itself (updated in
 *                place: only what changes is written), but may not overlap it otherwise
 *   cu_seqlens   device, int32 [B + 1]; positions device, int32 [T]; slots device,
 *                int64 [T]: T rows, at least as many as there are new tokens
 *   0 <= B <= 65536; page_size >= 1; max_pages * page_size < 2^31; T, pool < 2^31.
 *
 * Entries of the table and of the stack are moved, not looked at. A length that is
 * negative or past max_pages * page_size, more new tokens than T, or a free_count
 * outside [0, pool] (after the pages given back) is reported by kda_last_device_error()
 * as KDA_ERR_BAD_PAGE_TABLE, too few free pages as KDA_ERR_OUT_OF_PAGES; nothing is
 * planned then: tables, lengths and stack stay as they are, cu_seqlens is 0
 * throughout, and every row has position 0 and slot -1. Workspace: up to 12 B per slot.
 */
KDA_API kda_status kda_page_plan(const int32_t *page_table, const int32_t *seq_lens,
                                 const int32_t *new_lens, const uint8_t *release,
                                 const int32_t *free_pages, const int32_t *free_count, int64_t B,
                                 int64_t max_pages, int64_t pool, int64_t page_size, int64_t T,
                                 int32_t *page_table_out, int32_t *seq_lens_out,
                                 int32_t *free_pages_out, int32_t *free_count_out,
                                 int32_t *cu_seqlens, int32_t *positions, int64_t *slots,
                                 void *stream);

/*
 * kda_qk_norm_rope -- root-mean-square norm of every query and key head and the
 * rotation by its position, in one pass. For a head x of D channels
 *
 *     u = x / sqrt(mean(x^2) + eps) * weight
 *     (y_a, y_b) = (u_a cos t - u_b sin t, u_b cos t + u_a sin t),  t = position * inv_freq[i]
 *
 * over the pairs (a, b) = (i, i + R / 2), or (2 i, 2 i + 1) under KDA_ROPE_INTERLEAVED,
 * i < R / 2; channels from R on are u. Angles are reduced from the exact product of
 * the position and the fp32 frequency, so that far positions keep their precision
 * (to 2^-23 of a turn up to position 2^24).
 *
 *   q, k         device, bf16 [T, Hq, D], [T, Hk, D], tokens q_stride / k_stride elements
 *                apart (slices of a fused projection); Hk = 0: no keys (k, k_out NULL)
 *   q_weight, k_weight device, fp32 [D] or NULL (ones)
 *   inv_freq     device, fp32 [R / 2]; positions device, int32 [T] (any value); with
 *                R = 0 nothing is rotated and both may be NULL
 *   q_out, k_out device, bf16 like q and k, tokens q_out_stride / k_out_stride apart; each
 *                may be its input itself with the same stride (in place)
 *   D = 64, 128 or 256, R a multiple of 16 up to D (others: KDA_ERR_UNSUPPORTED_DIM);
 *   Hq >= 1; Hq + Hk <= 65535; eps >= 0; T < 2^31.
 *
 * Alignment: 16 bytes for q, k and the outputs, and strides multiples of 8 elements;
 * 4 bytes for the others. Norms, angles and products in fp32, results rounded once.
 */
enum { KDA_ROPE_INTERLEAVED = 1, KDA_ROPE_DOUT_FP32 = 2 };

KDA_API kda_status kda_qk_norm_rope(const void *q, const void *k, const float *q_weight,
                                    const float *k_weight, const float *inv_freq,
                                    const int32_t *positions, int64_t T, int64_t Hq, int64_t Hk,
                                    int64_t D, int64_t R, int64_t q_stride, int64_t k_stride,
                                    float eps, int flags, void *q_out, int64_t q_out_stride,
                                    void *k_out, int64_t k_out_stride, void *stream);

/*
 * kda_qk_norm_rope_backward -- gradients of kda_qk_norm_rope. With g = dL/dy turned
 * back by the angles and r = 1 / sqrt(mean(x^2) + eps):
 *
 *     dweight = sum over tokens and heads of g x r
 *     dx      = r (g weight - x r mean(g weight x r))
 *
 *   q, k, q_weight, k_weight, inv_freq, positions, sizes, eps: as given to the forward call
 *   dq_out, dk_out device [T, H, D], tokens dq_out_stride / dk_out_stride elements apart:
 *                bf16, or both fp32 with KDA_ROPE_DOUT_FP32
 *   dq, dk       device, bf16 like q and k, tokens dq_stride / dk_stride apart; not an input
 *   dq_weight, dk_weight device, fp32 [D] or NULL (not wanted)
 *
 * The weights' sums are taken in fp32 in a fixed order (the same call gives the same
 * bits). Workspace: 2 D floats for each of at most 304 blocks.
 */
KDA_API kda_status kda_qk_norm_rope_backward(
    const void *q, const void *k, const float *q_weight, const float *k_weight,
    const float *inv_freq, const int32_t *positions, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
    int64_t R, int64_t q_stride, int64_t k_stride, float eps, int flags, const void *dq_out,
    int64_t dq_out_stride, const void *dk_out, int64_t dk_out_stride, void *dq, int64_t dq_stride,
    void *dk, int64_t dk_stride, float *dq_weight, float *dk_weight, void *stream);

/*
 * kda_paged_append_fp8 -- new keys and values into a paged cache of 8-bit numbers
 * (e4m3), with one scale for each page and head: a cached number stands for itself
 * times its scale. Slot i's new tokens are rows [cu_seqlens[i], cu_seqlens[i + 1]) of k
 * and v, its last ones: they go to positions seq_lens[i] - (their number) .. seq_lens[i] - 1.
 *
 * The scale of a page and head, for keys and for values, is a power of two and only
 * grows: the least one (from 2^-126 on) that brings the largest new value to 448 or
 * below, or the one that the page has, if that is larger. A page whose row 0 is among
 * the new rows starts anew. When the scale grows, the other rows of the page are scaled
 * down to it, which is exact but for what leaves e4m3's range below. New
 * values are x / scale, rounded once to the nearest, ties to even; infinities and NaN
 * become NaN and do not count for the scale. (A scale that a caller has put into a page,
 * any positive number, is kept and used as its reciprocal.)
 *
 *   k, v         device, bf16 [T, Hkv, D], tokens k_stride / v_stride elements apart
 *   k_cache, v_cache device, e4m3 [pages, page_size, Hkv, D], channels contiguous; pages,
 *                tokens and heads the given strides (elements) apart, in any order, as
 *                long as no two rows overlap; both may lie in one buffer
 *   k_scale, v_scale device, fp32 [pages, Hkv], pages k_scale_stride / v_scale_stride apart;
 *                not inside the caches' buffers
 *   page_table, seq_lens, max_pages, pages as for kda_paged_decode, the new tokens included
 *                in seq_lens (as kda_page_plan leaves it)
 *   cu_seqlens   device, int32 [B + 1], rising from 0 to at most T, or NULL: T = B, a token
 *                for each slot (none where seq_lens is 0)
 *   D = 64 or 128 (others: KDA_ERR_UNSUPPORTED_DIM); B <= 65536; T < 2^31; (T + 2 B) * Hkv < 2^30.
 *
 * Pages that get new tokens must differ, those of one slot and those of different slots.
 * Rows of k and v behind the last slot are not read. A slot with a wrong cu_seqlens
 * (KDA_ERR_BAD_CU_SEQLENS), length or page index (KDA_ERR_BAD_PAGE_TABLE) is reported by
 * kda_last_device_error(); its tokens, or those of the bad page, are not written. Alignment:
 * 16 bytes for k, v and the caches, k_stride and v_stride multiples of 8 elements, the
 * caches' strides of 16. No workspace.
 */
KDA_API kda_status kda_paged_append_fp8(
    const void *k, const void *v, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
    const int32_t *page_table, const int32_t *seq_lens, const int32_t *cu_seqlens, int64_t T,
    int64_t B, int64_t Hkv, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages,
    int64_t k_stride, int64_t v_stride, int64_t k_page_stride, int64_t k_token_stride,
    int64_t k_head_stride, int64_t v_page_stride, int64_t v_token_stride, int64_t v_head_stride,
    int64_t k_scale_stride, int64_t v_scale_stride, void *stream);

/*
 * kda_paged_decode_fp8 -- kda_paged_decode over the cache of kda_paged_append_fp8:
 *
 *     s_j = scale k_scale[page of j] (q . k_j)
 *     out = sum_j softmax_j(s) v_scale[page of j] v_j,   lse = log sum_j exp(s_j)
 *
 *   k_cache, v_cache, their strides, k_scale, v_scale: as for kda_paged_append_fp8. Scales
 *                are any positive numbers (k_scale: any)
 *   q, page_table, seq_lens, out, lse, limits and errors as for kda_paged_decode; D, B,
 *   Hq, pages, max_pages, page_size likewise.
 *
 * Alignment: q, k_cache, v_cache, out 16 bytes, the caches' strides multiples of 16
 * elements; int32 and fp32 arrays 4 bytes. Scores, softmax and sums in fp32. The tensor
 * core takes the cache's numbers as they are; a query enters as two e4m3 terms (exact to
 * 2^-22 of its largest channel) and the weights, times the values' scales, as four (to
 * 2^-18.7 of each at most, 2^-21 in the mean; to 2^-33 of the largest among 128 tokens). The
 * sum over the cache is split over the SMs and joined in a fixed order (the same call gives
 * the same bits). Workspace: partial sums.
 */
KDA_API kda_status kda_paged_decode_fp8(
    const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
    const float *v_scale, const int32_t *page_table, const int32_t *seq_lens, int64_t B,
    int64_t Hq, int64_t Hkv, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages,
    int64_t k_page_stride, int64_t k_token_stride, int64_t k_head_stride, int64_t v_page_stride,
    int64_t v_token_stride, int64_t v_head_stride, int64_t k_scale_stride, int64_t v_scale_stride,
    float scale, void *out, float *lse, void *stream);

/* Static text for a status code (never NULL). */
KDA_API const char *kda_status_string(kda_status status);

/*
 * Synchronises `stream`, then returns and clears the first error a kernel
 * of this library recorded on the current device since the last call
 * (KDA_OK if none). Device errors are sticky per device, not per stream;
 * this reads both the library's error word and that of the fixed array of
 * kda_chunk_prefill_noalloc (if that entry point has run on the device).
 */
KDA_API kda_status kda_last_device_error(void *stream);

/*
 * Frees every cached workspace buffer of the current device after
 * synchronising the device. Safe to call at any time no call of this
 * library is in flight on the device; graphs that hold calls with a workspace
 * cannot be replayed after it.
 */
KDA_API kda_status kda_workspace_release(void);

/* Workspace bytes a call with these sizes needs (0 on bad sizes); the counters that some kernels
 * keep between calls, 40 H + 64 B for the launch in one, lie beside it. Host only. */
KDA_API int64_t kda_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N, int has_cu_seqlens);

/* The same for kda_chunk_prefill_backward with the gradient form set by
 * kda_set_backward_impl: chunked (default): 256 B of flags, the packed chunk
 * offsets, then per 16-token chunk per head 17,408 B of record, 4 B of list
 * entry (rounded up to 256 B in all), 1,280 B of (I + A)^-1 and 64 KiB of
 * bf16 states;
 * token-serial: 256 B of flags, the packed chunk offsets, 64 KiB per
 * 16-token chunk per head and 1 MiB for each of min(N * H, 1024) state
 * rings. Both entry points share the stream's buffer, grown to the larger. */
KDA_API int64_t kda_backward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N,
                                             int has_cu_seqlens);

/*
 * Measurement hook (per host thread). kda_stage_timing_begin(max_calls)
 * creates 3*max_calls timing events on the current device; each of the next
 * max_calls kda_chunk_prefill() calls of this thread records one before the
 * intra-chunk kernel, one between it and the recurrent kernel, and one after
 * the recurrent kernel, on the call's stream. kda_stage_timing_end()
 * waits for those events, writes the mean milliseconds per call of the
 * intra-chunk stage (prologue excluded; the intra-chunk kernel and the exact
 * form of the chunks outside the factored range) and of the recurrent stage, and the
 * number of calls timed, then frees the events. Host pointers; NULL outputs
 * are skipped. Errors: KDA_ERR_BAD_SHAPE for max_calls < 1, KDA_ERR_CUDA.
 */
KDA_API kda_status kda_stage_timing_begin(int max_calls);
KDA_API kda_status kda_stage_timing_end(double *intra_ms, double *recurrent_ms, int *calls);

/*
 * Selects the gradient form for later kda_chunk_prefill_backward calls
 * (process-wide, host only): 0 (default) = chunked: the forward's
 * intra-chunk kernels build the chunk records and each chunk's (I + A)^-1
 * (fp32), the forward chain runs again
 * keeping every chunk's entry state (bf16), a reverse chain over the chunks
 * keeps every chunk's dL/d(exit state) (bf16) and writes dL/d(initial
 * state), and a chunk-parallel kernel computes dq, dk, dv, dg and dbeta
 * (workspace: per chunk-head 17,408 B of record, 4 B of list entry, 1,280 B
 * of (I + A)^-1 and 64 KiB of states); 1 = the token-serial first form. Both compute the same
 * gradients to rounding. Other values: KDA_ERR_BAD_SHAPE.
 */
KDA_API kda_status kda_set_backward_impl(int impl);

/*
 * Test hook for the device-timeout report (process-wide, host only; not for
 * production use). For later calls on the 16-token path, the record producer
 * of every recurrent CTA issues no copy for chunk `chunk` of its sequence or
 * any later one, and both roles of that kernel give up a wait after `wait_ns`
 * nanoseconds (0: the default of 2 s). The consumers' wait for that chunk
 * then runs out: they record KDA_ERR_DEVICE_TIMEOUT in the device error word
 * and leave (outputs from that chunk on and the final state are then
 * unspecified). Every copy the producer did issue is waited for, so none is
 * in flight when a CTA exits. chunk = -1 turns the hook off (the default).
 * chunk < -1 or wait_ns < 0: KDA_ERR_BAD_SHAPE.
 */
KDA_API kda_status kda_test_stall_recurrent(int chunk, int64_t wait_ns);

/*
 * Test hook for kda_ssm_prefill (process-wide, host only): in later calls every
 * thread block copies the tiles of its first `chunk` chunks only, so that the waits
 * for the next one run out (after about a second each). The call then records
 * KDA_ERR_DEVICE_TIMEOUT and leaves, outputs and states unspecified; copies and
 * products under way are waited for. chunk = -1 turns the hook off (the default);
 * chunk < -1: KDA_ERR_BAD_SHAPE.
 */
KDA_API kda_status kda_test_stall_scan(int chunk);

/*
 * Test hook for kda_qk_norm_rope and its gradients, likewise (process-wide, host only): in
 * later calls a warp that has taken `batch` batches of heads asks for no more than the three
 * that are under way. Its wait for the next one runs out after two seconds and it stops there.
 * The call then records KDA_ERR_DEVICE_TIMEOUT, outputs unspecified. batch = -1 turns the hook
 * off (the default); batch < -1: KDA_ERR_BAD_SHAPE.
 */
KDA_API kda_status kda_test_stall_qk_norm_rope(int batch);

/*
 * Test hook for kda_paged_decode_fp8, likewise (process-wide, host only): in later calls
 * every thread block copies the first `tile` tiles of its share only, and the waits for
 * the next one run out (after about two seconds). The call then records
 * KDA_ERR_DEVICE_TIMEOUT and leaves, outputs unspecified. tile = -1 turns the hook off
 * (the default); tile < -1: KDA_ERR_BAD_SHAPE.
 */
KDA_API kda_status kda_test_stall_paged_fp8(int tile);

/*
 * Test hook: how kda_short_conv_backward would launch its kernel for arguments
 * of these sizes, strides and alignments (nothing is read from the pointers and no
 * GPU is needed). plan receives the bytes of scratch that the call asks for, the
 * channels of a block, the blocks along the channels, the tokens of a warp's run
 * and the tiles of eight runs; every tile writes (W + 1) * D floats of the scratch.
 */
KDA_API kda_status kda_test_conv_backward_plan(const void *x, const void *d_out, const void *dx,
                                               int64_t tokens, int64_t D, int64_t W,
                                               int64_t x_stride, int64_t dout_stride,
                                               int64_t dx_stride, int flags, int64_t plan[5]);

/*
 * Segments of the segment-parallel scan for later fixed-length calls on the
 * 16-token path (process-wide, host only): 0 (default) = chosen from the SM
 * count as described for kda_chunk_prefill, 1 = off (one chain per
 * sequence), P >= 2 = P segments (fewer when the sequence has fewer chunks
 * than P, or when that leaves a segment empty). Values outside [0, 4096]:
 * KDA_ERR_BAD_SHAPE. Takes effect for later calls (the workspace grows if
 * needed).
 */
KDA_API kda_status kda_set_scan_segments(int segments);

/*
 * Selects the chunk size and kernels for later calls (process-wide, host
 * only): 1 (default) = 16-token chunks, the intra-chunk kernel and then the
 * warp-level MMA recurrent kernel (state in registers, one CTA per
 * (sequence, head, 64 value channels)); 3 = 64-token chunks on the
 * 5th-generation tensor core, an intra-chunk kernel (tcgen05 Gram, W and U
 * products) and then a recurrent kernel (state in tensor memory, one CTA per
 * (sequence, head)); 4 = the 64-token kernels in one cooperative launch,
 * records passed through an L2-resident ring (3 when the heads leave fewer
 * than 16 SMs to the record builders). All compute the same result to
 * rounding. Other values: KDA_ERR_BAD_SHAPE.
 */
KDA_API kda_status kda_set_recurrent_impl(int impl);

/* Library build string: version and target architecture. Host only. */
KDA_API const char *kda_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_H */
