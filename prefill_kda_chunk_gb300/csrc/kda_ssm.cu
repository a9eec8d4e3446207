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
// core with bf16 operands (TMA, 128-byte swizzle) and fp32 accumulators in
// tensor memory: C B^T (128 x 128 x n), M X with M = (C B^T) . decay + d I, C S,
// and B^T (W X). b, c and x are bf16 as given, so what the products round is only
// what this kernel makes: M and S enter as two bf16 terms (16 bits of mantissa,
// well below the bf16 output's rounding), and the weighted rows W X as three (24
// bits: the state is an fp32 result and keeps fp32's precision over any length).
//
// Every exponent is a difference of running sums kept as two floats, a token's share of
// which is at least -1024 (its decay is then 0), so it is as exact next to a token
// that forgets everything as anywhere; between 32-token blocks it is split at the block's end into two
// factors <= 1, so only the diagonal blocks take an exponential per pair. These sums
// and factors come from a launch of their own (ssm_decays_kernel).
//
// Work split. The (head, 64 of P) units and chunks form one list, and CTA c
// of G (one per SM) takes an equal run of it, a run of chunks of one sequence
// after the other. Where a run starts in the middle of a sequence, its entry
// state comes from a launch before (kStates): there each CTA whose run ends in
// the middle of a sequence forms the state that its part of that sequence
// leaves (the state product only), and the CTAs behind add up what they need.
//
// Bound. Bytes do not bind (25 us at T 8192, 64 heads of 64, n 128): a chunk takes the
// tensor core 2700 clocks, most of it reading operands from shared memory at 128
// bytes a clock, and the warps 3000 issue slots of each quarter of the SM, most of
// them for M and for the terms of W X; with the waits between the roles it takes 5600.
// Measured at those sizes: decays 4 us, states 34, chunks 81, together 119.5 (1.4 TB/s,
// 21 % of copy bandwidth); 131072 tokens, 32 heads of 128: 1550 us.

#include <cuda.h>

#include "kda_device.cuh"
#include "kda_internal.h"
#include "kda_seqs.cuh"
#include "kda_tcgen05.cuh"

#include <cstddef>
#include <type_traits>

namespace kda {

namespace {

__device__ __forceinline__ float bf16_at(const void *p, int64_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v| <= 1, to a few units of the
// last place at every v (the state is linear in it). e^-|v|: the rounding error
// of |v| log2(e) is put back to first order. |v| is held at 128, where e is below
// fp32's range, so that the product stays finite up to the largest |v| and infinity
// (a token masked with the lowest value has delta = 0); a NaN passes. log(1 + e) = 2 atanh z with
// z = e / (2 + e) <= 1/3, whose series z (1 + z^2/3 + ... + z^16/17) ends at
// 3^-18/19 = 1.4e-10 and keeps the relative precision of small e.
__device__ __forceinline__ float softplus(float v) {
    const float x = fabsf(v) > 128.f ? -128.f : -fabsf(v), t = x * 1.44269504f;
    const float r = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;   // log2(e) - 1.44269504f
    const float e2 = ex2(t), e = fmaf(e2 * 0.69314718f, r, e2);
    const float z = __fdividef(e, 2.f + e), q = z * z;
    float s = 1.f / 17.f;
    s = fmaf(s, q, 1.f / 15.f);
    s = fmaf(s, q, 1.f / 13.f);
    s = fmaf(s, q, 1.f / 11.f);
    s = fmaf(s, q, 1.f / 9.f);
    s = fmaf(s, q, 1.f / 7.f);
    s = fmaf(s, q, 1.f / 5.f);
    s = fmaf(s, q, 1.f / 3.f);
    const float l = 2.f * fmaf(z * q, s, z);
    return v > 0.f ? v + l : l;
}
__device__ __forceinline__ float delta_of(float v, bool plus) { return plus ? softplus(v) : v; }
// A token's log decay, a delta log2(e), held at -1024: 2^-1024 is 0 in fp32, whatever
// growth within fp32's range stands beside it, and the running sums of a chunk stay so
// small (2^17) that two floats resolve the tokens behind the one that forgets all.
__device__ __forceinline__ float log_decay(float a2, float delta) {
    const float g = a2 * delta;
    return g < -1024.f ? -1024.f : g;
}

// ------------------------------------------------------------- one token

// One block per (sequence, head): thread (q, j) keeps S[j * kN / kParts ..][q]. Bound by
// reading and writing the state (256 sequences, 64 heads of 64, n 128: 156 us, 6.9
// TB/s, copy bandwidth).
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
    const float bias = p.dt_bias != nullptr ? __ldg(p.dt_bias + h) : 0.f;
    const float delta = delta_of(p.dt[n * p.dt_stride + h] + bias, p.softplus);
    const float decay = expf(av * delta);
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
// Warps: 0..7 form M and the outputs, 8..15 keep the state, then one for the
// MMAs of the state and C S, one each for C B^T and M X (in one warp, whichever came
// first held up the other) and one for the copies.
constexpr int kGroup = 8;
constexpr int kGroupThreads = 32 * kGroup;
constexpr int kCopyWarp = 2 * kGroup, kMmaWarpS = kCopyWarp + 1, kMmaWarpY = kCopyWarp + 2,
              kMmaWarpC = kCopyWarp + 3;
constexpr int kThreads = 32 * (kMmaWarpC + 1);
constexpr int kRing = 4;             // buffers for the decays of a chunk
constexpr int kCols = 32;            // columns of the state and of y per compute thread

// Shared memory, from a 1024-byte boundary. Tiles of 128-byte rows with the
// 16-byte granule index XOR-ed by the row's low three bits.
constexpr int kTileBytes = 16384;                // 128 rows
constexpr int kOffC = 0;                         // [n / 64][128 tokens][64]
constexpr int kOffS = kOffC + 2 * kTileBytes;    // two terms of the state, [n][64]
constexpr int kOffB = kOffS + 2 * kTileBytes;    // two buffers of [n / 64][128 tokens][64]
constexpr int kOffX = kOffB + 4 * kTileBytes;    // two buffers of [128 tokens][64]
constexpr int kOffW = kOffX + 2 * kTileBytes;    // three terms of the weighted rows
constexpr int kOffSc = kOffW + 3 * kTileBytes;   // kRing buffers of Scalars
// The decays of a chunk of one head, as a launch before leaves them in the workspace.
struct alignas(16) Decays {
    float hi[kL], lo[kL];   // -G_t as a sum of two floats, in units of log 2
    float dt[kL];           // delta_t; 0 past the sequence's end
    float to_block[kL];     // 2^(G at the end of t's 32-block - G_t) delta_t
    float end_hi[4], end_lo[4];   // G at the end of each 32-block
    // what the launch for the states needs starts here
    float to_end[kL];       // 2^(G_last - G_t) delta_t
    float decay, d, pad[2]; // 2^G_last; the head's d
};
constexpr int kDecaysBytes = static_cast<int>(sizeof(Decays));
constexpr int kDecaysTail = static_cast<int>(offsetof(Decays, to_end));
struct alignas(16) Scalars : Decays {
    // where the chunk is, so that the compute warps need not walk the list
    int valid;              // its tokens
    int unit, seq, pos;     // head and slice; sequence; chunk of the sequence
    int flags;              // kLast, kCut
    int xcol, gcol;         // its first column of x, and of b and c
    int64_t row;            // its first token
    // Infinities and NaN in x: the 32-row by 8-channel pieces that hold any (bit 8 * block
    // + granule), and in those the first row of each channel that does (kL: none).
    unsigned odd;
    uint8_t odd_from[4][kPS];
};
enum { kLast = 1, kCut = 2 };   // the sequence's last chunk; the run's end cuts the sequence
constexpr int kOffBar = kOffSc + kRing * static_cast<int>(sizeof(Scalars));
enum {   // barriers, 8 bytes each; pairs and the ring by the chunk's index
    // phases that one thread or a copy completes
    kFullC, kFullB, kFullX = kFullB + 2, kScal = kFullX + 2, kCB = kScal + kRing, kDS = kCB + 2,
    kCS = kDS + 2, kMX = kCS + 2, kDrain = kMX + 2, kDrain2, kDrain3,
    // phases that the warps of a group arrive at
    kMReady, kSReady = kMReady + 2, kXReady, kDone = kXReady + 2,
    // ... the state's, and in the launch for the states both (there one group can be a chunk
    // ahead of the other, hence two)
    kWReady = kDone + 2,
    // ... both (the launch for the states: the state's)
    kScFree = kWReady + 2, kBars = kScFree + kRing
};
constexpr int kOffMisc = kOffBar + 8 * kBars;    // tensor memory base, abort flag
constexpr int kSmem = kOffMisc + 8;
static_assert(kSmem <= 232448, "what a block can have");

// Tensor memory columns; the block takes all of them, so they start at 0. C B^T has
// two buffers of 128; M replaces it there: 16 columns (tokens s) become the 8 columns
// of its high terms and the 8 of its low terms. C moves here for C S: its tile in shared
// memory is free for the next chunk as soon as C B^T is formed, not only once the state
// that C meets is there. The launch for the states works on two chunks at a time.
constexpr uint32_t kTmCB = 0, kTmY = 256, kTmCS = 320, kTmC = 384, kTmDS = 448, kTmCols = 512;
__device__ __forceinline__ uint32_t tm_ds(bool states, int i) {
    return states ? 64u * (i & 1) : kTmDS;
}
// The weighted rows of chunk i; the launch for the states has two sets.
__device__ __forceinline__ int off_w(bool states, int i) {
    return states && (i & 1) != 0 ? kOffC : kOffW;
}

// ---- instruction and shared-memory descriptors (bf16, fp32 accumulate)
constexpr uint32_t kAMajor = 1u << 15, kBMajor = 1u << 16;   // operand contiguous along M / N
// 128-byte swizzled tiles, eight rows of 128 bytes per atom. Contiguous along
// K: the stride field is the step between 8-row groups. Contiguous along M or N:
// it is the step between groups of 8 along K, and the leading field the one
// between blocks of 64 along M / N. All tiles here have a stride of 1024 bytes,
// so that descriptors differ in their lower word only.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) {
    return ((saddr >> 4) & 0x3FFF) | (static_cast<uint32_t>(kTileBytes >> 4) << 16);
}

// Four MMAs, D (+)= A B, with both operands in shared memory, or A in tensor memory, and
// the commit of those before them. The operands of the second to fourth lie A1.. and
// B1.. behind the first's (those in tensor memory 8 columns apart). The whole warp
// calls them and the instructions elect a lane: descriptors then stay in uniform
// registers. (In a branch of one lane an MMA of N = 64 took 77 cycles in a loop and
// 52 unrolled, this way 48 and 40. One elected at a time, they took 120 and more
// beside the other warps' work: a dozen dependent instructions each; unrolled
// throughout, as much for fetching them.)
template <int A1, int A2, int A3, int B1, int B2, int B3>
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n .reg .pred p, t, e;\n .reg .b32 u, v;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n"
        " setp.eq.b32 t, 0, 0;\n elect.sync _|e, 0xffffffff;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n"
        " add.u32 u, %1, %6;\n add.u32 v, %2, %9;\n mov.b64 x, {u, %5};\n mov.b64 y, {v, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n"
        " add.u32 u, %1, %7;\n add.u32 v, %2, %10;\n mov.b64 x, {u, %5};\n mov.b64 y, {v, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n"
        " add.u32 u, %1, %8;\n add.u32 v, %2, %11;\n mov.b64 x, {u, %5};\n mov.b64 y, {v, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(static_cast<uint32_t>(acc)), "r"(kDescHi), "n"(A1), "n"(A2), "n"(A3),
        "n"(B1), "n"(B2), "n"(B3)
        : "memory");
}
template <int B1, int B2, int B3>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n .reg .pred p, t, e;\n .reg .b32 u, v;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n"
        " setp.eq.b32 t, 0, 0;\n elect.sync _|e, 0xffffffff;\n mov.b64 y, {%2, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n"
        " add.u32 u, %1, 8;\n add.u32 v, %2, %6;\n mov.b64 y, {v, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n"
        " add.u32 u, %1, 16;\n add.u32 v, %2, %7;\n mov.b64 y, {v, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n"
        " add.u32 u, %1, 24;\n add.u32 v, %2, %8;\n mov.b64 y, {v, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(static_cast<uint32_t>(acc)), "r"(kDescHi), "n"(B1), "n"(B2), "n"(B3)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_2d(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

// packed fp32 pairs: (a, b) = (a, b) * (x, y) + (u, v)
__device__ __forceinline__ void fma2(float &a, float &b, float x, float y, float u, float v) {
    asm("{\n .reg .b64 t, s, w;\n mov.b64 t, {%0, %1};\n mov.b64 s, {%2, %3};\n mov.b64 w, {%4, %5};\n"
        " fma.rn.f32x2 t, t, s, w;\n mov.b64 {%0, %1}, t;\n}\n"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y), "f"(u), "f"(v));
}

// Two bf16 values: acc stays +-0 as long as every x was finite, and becomes NaN otherwise.
__device__ __forceinline__ void look_for_odd(uint32_t &acc, uint32_t x) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
}

// (a, b) as two bf16 terms: hi + lo; (a, b) keeps what hi leaves
__device__ __forceinline__ uint32_t take2(float &a, float &b) {
    const uint32_t h = pack_bf16(a, b);
    float x = __uint_as_float(h << 16), y = __uint_as_float(h & 0xffff0000u);
    fma2(x, y, -1.f, -1.f, a, b);
    a = x;
    b = y;
    return h;
}
__device__ __forceinline__ uint32_t split2(float a, float b, uint32_t &lo) {
    const uint32_t h = take2(a, b);
    lo = pack_bf16(a, b);
    return h;
}

// Of the lanes l and l ^ m, the one without the bit m gives b for the other's a.
__device__ __forceinline__ void exchange(uint32_t &a, uint32_t &b, int m, int lane) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, (lane & m) != 0 ? a : b, m);
    if ((lane & m) != 0) a = got;
    else b = got;
}
__device__ __forceinline__ void exchange(uint4 &a, uint4 &b, int m, int lane) {
    exchange(a.x, b.x, m, lane);
    exchange(a.y, b.y, m, lane);
    exchange(a.z, b.z, m, lane);
    exchange(a.w, b.w, m, lane);
}

// hi + lo += x, with the rounding error of the sum kept in lo
struct Sum2 {
    float hi, lo;
    __device__ __forceinline__ void add(float xh, float xl) {
        const float s = hi + xh, b = s - hi;
        const float e = ((hi - (s - b)) + (xh - b)) + (lo + xl);
        hi = s + e;
        lo = e - (hi - s);
    }
};

// Waits for this thread's tensor memory loads and hands on the registers of one of
// them, so that no use (or copy) of them moves in front of the wait.
__device__ __forceinline__ void ld_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}

// A wait for a phase of an mbarrier, of 2^18 polls at most (about a second: one that
// finds nothing takes some 7800 clocks), in few instructions: this kernel waits in
// some twenty places, and with longer waits at each of them its loops did not fit
// the instruction cache (a chunk then took twice as long). No clock is read and no
// time to suspend given: a handshake of two warps that wait for one another takes
// 126 cycles this way, 234 with both.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
    uint32_t n;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 0;\n"
        "again%=: mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra done%=;\n"
        " add.u32 n, n, 1;\n setp.lt.u32 q, n, 262144;\n @q bra again%=;\n"
        "done%=: mov.u32 %0, n;\n}\n"
        : "=r"(n) : "r"(bar), "r"(parity) : "memory");
    return n < 262144;
}

struct SsmMaps {
    CUtensorMap x, b, c;   // [tokens][channels], boxes of 128 tokens x 64 channels
};

struct SsmPlan {
    int shift;                 // a head is 1 << shift units
    int cps;                   // chunks per sequence (fixed lengths)
    int64_t units;             // heads << shift
    const int32_t *chunk_off;  // packed: first chunk of each sequence [N + 1]
    const int *call_flags;     // packed: set by the prologue
    Decays *decays;            // [chunk of all sequences][heads]
    int64_t gran;              // chunks that stay together; 0: all of a unit's
    float *slots;              // [G][kCols][kGroupThreads] states at the cuts
    float *saved;              // the same: initial states that a cut run starts from (in place)
    float *decay;              // [G]
    bool in_place;
    int stall;                 // test hook: chunks of a run whose tiles are copied
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

// The launches of one call overlap: a launch may begin while the one in front of it still
// runs, sets itself up, and waits here until that one's writes are visible. Every
// CTA waits before it leaves, so that a launch is over only after all before it.
__device__ __forceinline__ void wait_for_launch() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// The decays of all chunks, a warp per chunk and head: running sums over each lane's four
// tokens, then over the lanes. A dependent chain of some 600 instructions: inside the
// chunk kernel, on a warp of its own, it took 3100 clocks per chunk, as long as that
// chunk's products, and a sixth of its instruction cache.
__global__ void __launch_bounds__(256) ssm_decays_kernel(SsmParams p, SsmPlan pl) {
    let_next_launch();
    if (pl.call_flags != nullptr && (*pl.call_flags & kErrBadCu) != 0) return;
    const List list(p, pl);
    const int lane = threadIdx.x & 31;
    const int64_t all = list.nc * p.heads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < all; i += gridDim.x * 8) {
        const int h = static_cast<int>(i % p.heads);
        Walk w;
        w.go(p, pl, list.nc, i / p.heads);   // (of the first unit: all have the same chunks)
        const int valid = w.valid();
        const float a2 = __ldg(p.a + h) * 1.44269504088896341f;
        const float bias = p.dt_bias != nullptr ? __ldg(p.dt_bias + h) : 0.f;
        const float *src = p.dt + (w.row() + 4 * lane) * p.dt_stride + h;
        float dt[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) dt[j] = 4 * lane + j < valid ? __ldg(src + j * p.dt_stride) : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) dt[j] = 4 * lane + j < valid ? delta_of(dt[j] + bias, p.softplus) : 0.f;
        Sum2 sum{0.f, 0.f}, g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum.add(log_decay(a2, dt[j]), 0.f);
            g[j] = sum;
        }
        Sum2 incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float vh = __shfl_up_sync(0xffffffffu, incl.hi, o);
            const float vl = __shfl_up_sync(0xffffffffu, incl.lo, o);
            if (lane >= o) incl.add(vh, vl);
        }
        float bh = __shfl_up_sync(0xffffffffu, incl.hi, 1), bl = __shfl_up_sync(0xffffffffu, incl.lo, 1);
        if (lane == 0) bh = bl = 0.f;
        const float kh = __shfl_sync(0xffffffffu, incl.hi, lane | 7);
        const float kl = __shfl_sync(0xffffffffu, incl.lo, lane | 7);
        const float eh = __shfl_sync(0xffffffffu, incl.hi, 31), el = __shfl_sync(0xffffffffu, incl.lo, 31);
        float v[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Sum2 G{bh, bl};
            G.add(g[j].hi, g[j].lo);
            v[0][j] = -G.hi;
            v[1][j] = -G.lo;
            v[2][j] = ex2((kh - G.hi) + (kl - G.lo)) * dt[j];
            v[3][j] = ex2((eh - G.hi) + (el - G.lo)) * dt[j];
        }
        Decays &s = pl.decays[i];
        *reinterpret_cast<float4 *>(s.hi + 4 * lane) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
        *reinterpret_cast<float4 *>(s.lo + 4 * lane) = make_float4(v[1][0], v[1][1], v[1][2], v[1][3]);
        *reinterpret_cast<float4 *>(s.dt + 4 * lane) = make_float4(dt[0], dt[1], dt[2], dt[3]);
        *reinterpret_cast<float4 *>(s.to_block + 4 * lane) = make_float4(v[2][0], v[2][1], v[2][2], v[2][3]);
        *reinterpret_cast<float4 *>(s.to_end + 4 * lane) = make_float4(v[3][0], v[3][1], v[3][2], v[3][3]);
        if ((lane & 7) == 7) {
            s.end_hi[lane >> 3] = kh;
            s.end_lo[lane >> 3] = kl;
        }
        // (carried over all the chunks of a sequence: the more exact exponential)
        if (lane == 31) {
            s.decay = exp2f(eh);
            s.d = p.d != nullptr ? __ldg(p.d + h) : 0.f;
        }
    }
}

template <int kN, bool kStates>
__global__ void __launch_bounds__(kThreads, 1)
ssm_chunk_kernel(const __grid_constant__ SsmMaps maps, SsmParams p, SsmPlan pl) {
    extern __shared__ __align__(1024) uint8_t smem[];
    volatile int &s_abort = *reinterpret_cast<volatile int *>(smem + kOffMisc + 4);
    if (pl.call_flags != nullptr && (*pl.call_flags & kErrBadCu) != 0) {
        wait_for_launch();
        return;
    }
    // (the shuffle tells the compiler that a warp's index is uniform: without it, it
    // guards every MMA's registers against lanes that differ, 32 instructions each)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (!kStates && tid < kGroupThreads) hand_on<kN>(p, tid, kGroupThreads);
    const List list(p, pl);
    const int c = blockIdx.x;
    int64_t q0 = c < list.G ? list.begin(c) : 0;
    const int64_t q1 = c < list.G ? list.begin(c + 1) : 0;
    if (kStates) {   // only the part of the sequence that the end of the run cuts
        Walk w;
        w.pos = 0;
        if (q1 < list.W && q1 > q0) w.go(p, pl, list.nc, q1);
        if (q1 - w.pos > q0) q0 = q1 - w.pos;
    }
    const int count = static_cast<int>(q1 - q0);
    if (count <= 0) {
        wait_for_launch();
        return;
    }

    const uint32_t sb = smem_u32(smem);
    const auto bar = [&](int i) { return sb + kOffBar + 8 * i; };
    Scalars *scal = reinterpret_cast<Scalars *>(smem + kOffSc);

    if (tid == 0) {
        s_abort = (sb & 1023) != 0;   // (the tiles' swizzle counts on it)
        for (int i = 0; i < kBars; ++i)
            mbar_init(bar(i), i < kMReady ? 1
                              : i >= kWReady && i < kScFree ? (kStates ? 2 * kGroup : kGroup)
                              : i >= kScFree ? (kStates ? kGroup : 2 * kGroup) : kGroup);
        mbar_fence_init();
    }
    if (warp == 0) {
        tc::alloc(sb + kOffMisc, kTmCols);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();

    if (kStates) let_next_launch();
    wait_for_launch();

    // A bounded wait; a role whose wait has run out stops, and says so.
    auto wait = [&](int i, int phase) -> bool { return wait_phase(bar(i), phase & 1); };
    auto arrive = [&](int i) {   // one arrival per warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };

    Walk w;
    w.go(p, pl, list.nc, q0);

    // k-steps of 16: 32 bytes along a row, or 16 rows of 128 bytes
    constexpr uint32_t kStepK = 32 >> 4, kStepMN = 2048 >> 4, kTile = kTileBytes >> 4;
    // after a wait that gave up: let the MMAs that this warp issued end
    auto drain = [&](int i) {
        __syncwarp();
        s_abort = 1;
        mma_commit(bar(i));
        wait_phase(bar(i), 0);
    };
    auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
    // The weighted rows of chunk i as three bf16 terms, in 32 tasks of 32
    // rows x 8 channels. Rows past the end of the sequence belong to
    // another one: they are zeroed here, as no weight of 0 makes an infinity or NaN
    // vanish. (With two groups each takes 16 of the tasks.)
    // Nor does one of M's zeros: an infinity or NaN of x would reach the tokens in front
    // of its own through M X. Such values become 0 in the tile that M X reads, while W X,
    // and with it the state, keep them, and take_out makes their channel NaN from their
    // token on. (Looking for them, an instruction per two values: T 8192, 64 heads 118.2
    // -> 119.5 us.)
    auto put_rows = [&](int i, int task0, int tasks) {
        uint8_t *X = smem + kOffX + (i & 1) * kTileBytes, *W = smem + off_w(kStates, i);
        Scalars &s = scal[i & (kRing - 1)];
        const int valid = s.valid;
        uint32_t odd = 0;
#pragma unroll 1
        for (int k0 = task0; k0 < task0 + tasks; k0 += 2) {
            uint4 xv[2];
            float wts[2];
            int ats[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {   // two tasks side by side
                const int k = k0 + m, row = (k >> 3) * 32 + lane, at = row * 128 + (((k ^ row) & 7) << 4);
                wts[m] = s.to_end[row];
                ats[m] = at;
                xv[m] = *reinterpret_cast<const uint4 *>(X + at);
                if (row >= valid) {
                    xv[m] = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(X + at) = xv[m];
#pragma unroll
                    for (int z = 0; z < kN / 64; ++z)
                        *reinterpret_cast<uint4 *>(smem + kOffB + (2 * (i & 1) + z) * kTileBytes + at) = xv[m];
                }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t xs[4] = {xv[m].x, xv[m].y, xv[m].z, xv[m].w};
                uint32_t t0[4], t1[4], t2[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!kStates) look_for_odd(odd, xs[e]);
                    float a = __uint_as_float(xs[e] << 16), b = __uint_as_float(xs[e] & 0xffff0000u);
                    mul2(a, b, wts[m], wts[m]);
                    t0[e] = take2(a, b);
                    t1[e] = split2(a, b, t2[e]);
                }
                *reinterpret_cast<uint4 *>(W + ats[m]) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
                *reinterpret_cast<uint4 *>(W + kTileBytes + ats[m]) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                *reinterpret_cast<uint4 *>(W + 2 * kTileBytes + ats[m]) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
            }
        }
        if (!kStates && __any_sync(0xffffffffu, (odd & 0x7fff7fffu) != 0)) {
#pragma unroll 1
            for (int k = task0; k < task0 + tasks; ++k) {
                const int row = (k >> 3) * 32 + lane;
                uint16_t *x = reinterpret_cast<uint16_t *>(X + row * 128 + (((k ^ row) & 7) << 4));
                bool any = false;
#pragma unroll 1
                for (int e = 0; e < 8; ++e) {
                    const bool is = (x[e] & 0x7f80) == 0x7f80;
                    const unsigned rows = __ballot_sync(0xffffffffu, is);
                    if (is) x[e] = 0;
                    if (lane == 0) s.odd_from[k >> 3][(k & 7) * 8 + e] = rows != 0 ? (k & ~7) * 4 + __ffs(rows) - 1 : kL;
                    any |= rows != 0;
                }
                if (lane == 0 && any) atomicOr(&s.odd, 1u << k);
            }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar(kWReady + (i & 1)));
            mbar_arrive(bar(kXReady + (i & 1)));
        }
    };
    auto landed = [&](int i) {
        // (b only where put_rows writes to it)
        return wait(kScal + (i & (kRing - 1)), i / kRing) && wait(kFullX + (i & 1), i >> 1) &&
               (scal[i & (kRing - 1)].valid == kL || wait(kFullB + (i & 1), i >> 1));
    };
    if (warp == kMmaWarpS) {
        // ------------------------------------------- MMAs: B^T (W X) and C S
        int j0 = 0;
#pragma unroll 1
        for (; j0 < count; ++j0) {
            const int i = __shfl_sync(0xffffffffu, j0, 0);   // (uniform, see above)
            // B^T (W X) (for n = 64 the upper 64 rows are formed from whatever lies
            // there and are not read)
            if (!all(wait(kFullB + (i & 1), i >> 1) && wait(kWReady + (i & 1), i >> 1))) break;
            tc::fence_after();
            const uint32_t B = desc_lo(sb + kOffB) + 2 * kTile * (i & 1);
            const uint32_t W = desc_lo(sb + off_w(kStates, i)), D = tm_ds(kStates, i);
#pragma unroll 1
            for (int k = 0; k < 6; ++k)   // the smallest term first
                mma4_ss<kStepMN, 2 * kStepMN, 3 * kStepMN, kStepMN, 2 * kStepMN, 3 * kStepMN>(
                    D, B + (k & 1) * 4 * kStepMN, W + (2 - (k >> 1)) * kTile + (k & 1) * 4 * kStepMN,
                    tc::idesc(128, kPS, 1) | kAMajor | kBMajor, k > 0);
            mma_commit(bar(kDS + (i & 1)));
            if (!kStates) {
                // C S, both terms of S, once that of the chunk before is read out
                if (!all(wait(kSReady, i) && (i < 1 || wait(kDone + ((i - 1) & 1), (i - 1) >> 1)))) break;
                tc::fence_after();
                const uint32_t S = desc_lo(sb + kOffS);
#pragma unroll 1
                for (int k = 0; k < 2; ++k)
#pragma unroll 1
                    for (int j = 0; j < kN / 64; ++j)
                        mma4_ts<kStepMN, 2 * kStepMN, 3 * kStepMN>(
                            kTmCS, kTmC + 32 * j, S + k * kTile + j * 4 * kStepMN,
                            tc::idesc(128, kPS, 1) | kBMajor, k + j > 0);
                mma_commit(bar(kCS + (i & 1)));
            }
        }
        if (j0 < count) drain(kDrain);
    } else if (warp == kMmaWarpC) {
        // ------------------------------------------------------ MMAs: C B^T
        int j0 = kStates ? count : 0;
#pragma unroll 1
        for (; j0 < count; ++j0) {
            const int i = __shfl_sync(0xffffffffu, j0, 0);   // (uniform, see above)
            // over M of two chunks before
            if (!all(wait(kFullB + (i & 1), i >> 1) && wait(kFullC, i) &&
                     (i < 2 || wait(kMX + (i & 1), (i >> 1) - 1))))
                break;
            tc::fence_after();
            const uint32_t B = desc_lo(sb + kOffB) + 2 * kTile * (i & 1), C = desc_lo(sb + kOffC);
            const uint32_t D = kTmCB + 128 * (i & 1);
#pragma unroll 1
            for (int k = 0; k < kN / 64; ++k)
                mma4_ss<kStepK, 2 * kStepK, 3 * kStepK, kStepK, 2 * kStepK, 3 * kStepK>(
                    D, C + k * kTile, B + k * kTile, tc::idesc(128, 128, 1), k > 0);
            mma_commit(bar(kCB + (i & 1)));
        }
        if (j0 < count) drain(kDrain2);
    } else if (warp == kMmaWarpY) {
        // -------------------------------------------------------- MMAs: M X
        int j0 = kStates ? count : 0;
#pragma unroll 1
        for (; j0 < count; ++j0) {
            const int i = __shfl_sync(0xffffffffu, j0, 0);   // (uniform, see above)
            // both terms of M along K, once the chunk before is read out
            if (!all(wait(kXReady + (i & 1), i >> 1) && wait(kMReady + (i & 1), i >> 1))) break;
            tc::fence_after();
            const uint32_t X = desc_lo(sb + kOffX) + kTile * (i & 1), A = kTmCB + 128 * (i & 1);
#pragma unroll 1
            for (int k = 0; k < 4; ++k)
                mma4_ts<0, kStepMN, kStepMN>(kTmY, A + 32 * k, X + 2 * k * kStepMN,
                                             tc::idesc(128, kPS, 1) | kBMajor, k > 0);
            mma_commit(bar(kMX + (i & 1)));
        }
        if (j0 < count) drain(kDrain3);
    } else if (warp == kCopyWarp) {
        // ---------------------------------------------------------- copies
        if (lane == 0) {
            // tiles of 64 channels of chunk i; b and c have kN / 64 of them
            auto copy = [&](int full, int off, const CUtensorMap &map, int col, int row, int n) {
                mbar_arrive_expect_tx(bar(full), kL * 128 * n);
#pragma unroll 1
                for (int k = 0; k < n; ++k) tma_2d(sb + off + k * kTileBytes, &map, col + 64 * k, row, bar(full));
            };
            // Where chunk j is, and its decays. Its tiles are fetched into L2: their
            // buffers are free for about half a chunk's time before they are needed,
            // less than a read from HBM takes.
            const int per_group = p.heads / p.groups;
            auto describe = [&](int j) -> bool {
                if (j >= kRing && !wait(kScFree + (j & (kRing - 1)), (j / kRing) - 1)) return false;
                if (j > 0) w.next(p, pl, list.nc);
                Scalars &s = scal[j & (kRing - 1)];
                const int h = w.u >> pl.shift, full = kScal + (j & (kRing - 1));
                s.valid = w.valid();
                s.unit = w.u;
                s.seq = w.n;
                s.pos = w.pos;
                s.flags = (w.last() ? kLast : 0) | (q0 + j + (w.len + kL - 1) / kL - w.pos > q1 ? kCut : 0);
                s.row = w.row();
                s.odd = 0;
                s.xcol = h * p.p + (w.u & pl.shift) * kPS;
                s.gcol = h / per_group * kN;
                constexpr int kFrom = kStates ? kDecaysTail : 0;
                mbar_arrive_expect_tx(bar(full), kDecaysBytes - kFrom);
                bulk_g2s(smem_u32(&s) + kFrom,
                         reinterpret_cast<const uint8_t *>(pl.decays + w.ch * p.heads + h) + kFrom,
                         kDecaysBytes - kFrom, bar(full));
                if (j > 0) {
                    const int row = static_cast<int>(s.row);
                    prefetch_2d(&maps.x, s.xcol, row);
#pragma unroll 1
                    for (int k = 0; k < kN; k += 64) {
                        prefetch_2d(&maps.b, s.gcol + k, row);
                        if (!kStates) prefetch_2d(&maps.c, s.gcol + k, row);
                    }
                }
                return true;
            };
            const int copied = min(count, pl.stall);
            int i = 0, sent_c = 0, described = describe(0) ? 1 : 0;
#pragma unroll 1
            for (; i < copied; ++i) {
                // what chunks i - 2 (b, x) and i - 1 (c) have left
                const Scalars &v = scal[i & (kRing - 1)];
                const int row = static_cast<int>(v.row), col = v.gcol, xcol = v.xcol, s = i & 1;
                if (kStates) {   // x is free as soon as its weighted rows are there
                    if (i > 1 && !wait(kWReady + s, (i >> 1) - 1)) break;
                    copy(kFullX + s, kOffX + s * kTileBytes, maps.x, xcol, row, 1);
                }
                if (i > 1 && (!wait(kDS + s, (i >> 1) - 1) || (!kStates && !wait(kCB + s, (i >> 1) - 1)))) break;
                copy(kFullB + s, kOffB + 2 * s * kTileBytes, maps.b, col, row, kN / 64);
                if (!kStates) {
                    if (i > 1 && !wait(kMX + s, (i >> 1) - 1)) break;
                    copy(kFullX + s, kOffX + s * kTileBytes, maps.x, xcol, row, 1);
                    if (i > 0 && (!wait(kSReady, i - 1) || !wait(kCB + (s ^ 1), (i - 1) >> 1))) break;
                    copy(kFullC, kOffC, maps.c, col, row, kN / 64);
                    sent_c = i + 1;
                }
                if (described < count) {
                    if (!describe(described)) {
                        ++i;   // (its copies are under way)
                        break;
                    }
                    ++described;
                }
            }
            // the last copies land before the block ends (after a wait that gave up
            // nobody else may have waited for them)
            for (int j = i > 2 ? i - 2 : 0; j < i; ++j) {
                wait_phase(bar(kFullB + (j & 1)), (j >> 1) & 1);
                wait_phase(bar(kFullX + (j & 1)), (j >> 1) & 1);
            }
            if (!kStates && sent_c > 0) wait_phase(bar(kFullC), (sent_c - 1) & 1);
            for (int j = described > kRing ? described - kRing : 0; j < described; ++j)
                wait_phase(bar(kScal + (j & (kRing - 1))), (j / kRing) & 1);
            if (i < count) {   // (of the chunk it gave up at, where it got so far)
                s_abort = 1;
                wait_phase(bar(kFullB + (i & 1)), (i >> 1) & 1);
                wait_phase(bar(kFullX + (i & 1)), (i >> 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp < kGroup) {
        // ------------------------------------------------- M and the output, row
        // 32 q + lane (the lanes of tensor memory that a warp reaches); columns of y:
        // the half hf
        const int q = warp & 3, hf = warp >> 2, r = 32 * q + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        // y = 2^G (C S) + M X of chunk i, ready to be stored, rounded to bf16 as out is
        uint4 ys[4];
        __nv_bfloat16 *dst = nullptr;
        int valid = 0;
        auto take_out = [&](int i) -> bool {
            const Scalars &s = scal[i & (kRing - 1)];
            const int h = s.unit >> pl.shift;
            const float from = ex2(-s.hi[r]);
            valid = s.valid;
            dst = static_cast<__nv_bfloat16 *>(p.out) +
                  ((s.row + (r & ~3)) * p.heads + h) * p.p + (s.unit & pl.shift) * kPS + kCols * hf +
                  8 * (lane & 3);
            if (!wait(kMX + (i & 1), i >> 1) || !wait(kCS + (i & 1), i >> 1)) return false;
            tc::fence_after();
            uint32_t y[2][16], cs[2][16];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                tc::ld16(lanes + kTmY + kCols * hf + 16 * k, y[k]);
                tc::ld16(lanes + kTmCS + kCols * hf + 16 * k, cs[k]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ld_wait16(y[k]);
                ld_wait16(cs[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t os[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 8 * (k & 1) + 2 * e;
                    float a = __uint_as_float(cs[k >> 1][j]), b = __uint_as_float(cs[k >> 1][j + 1]);
                    fma2(a, b, from, from, __uint_as_float(y[k >> 1][j]), __uint_as_float(y[k >> 1][j + 1]));
                    os[e] = pack_bf16(a, b);
                }
                ys[k] = make_uint4(os[0], os[1], os[2], os[3]);
            }
            // (written before the arrival that let M X start)
            const unsigned odd = *const_cast<const volatile unsigned *>(&s.odd);
            if (odd != 0) {
                uint32_t nan = 0;   // of this row's channels
#pragma unroll 1
                for (int ch = 0; ch < kCols; ++ch)
#pragma unroll 1
                    for (int b = 0; b < 4; ++b)
                        if ((odd >> (8 * b + ((kCols * hf + ch) >> 3)) & 1) != 0 &&
                            r >= s.odd_from[b][kCols * hf + ch])
                            nan |= 1u << ch;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        reinterpret_cast<uint32_t *>(&ys[k])[e] |=
                            (nan >> (8 * k + 2 * e) & 1 ? 0x7fffu : 0u) |
                            (nan >> (8 * k + 2 * e + 1) & 1 ? 0x7fff0000u : 0u);
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kDone + (i & 1)));
                mbar_arrive(bar(kScFree + (i & (kRing - 1))));
            }
            return true;
        };
        if (kStates) {   // half of the weighted rows
#pragma unroll 1
            for (int i = 0; i < count; ++i) {
                if (!landed(i) || (i > 1 && !wait(kDS + (i & 1), (i >> 1) - 1))) {
                    s_abort = 1;
                    break;
                }
                put_rows(i, 16 + 2 * warp, 2);
            }
        }
        int i = kStates ? count + 1 : 0;
#pragma unroll 1
        for (; i <= count; ++i) {
            // M of chunk i, then the output of the one before, whose products are done
            if (i < count) {
                const Scalars &s = scal[i & (kRing - 1)];
                // ---- M = (C B^T) . decay + d I, two bf16 terms
                if (!wait(kScal + (i & (kRing - 1)), i / kRing) || !wait(kCB + (i & 1), i >> 1)) break;
                tc::fence_after();
                const uint32_t at = lanes + kTmCB + 128 * (i & 1);
                const float hi_r = -s.hi[r], lo_r = -s.lo[r];
                const float dv = s.d;
                // 16 columns at a time, the half hf of each 32-token block (so that both warps
                // of these rows have as much of the diagonal), the next ones read before these
                // are worked on; blocks above the diagonal are zero.
                uint32_t ahead[16] = {};
                tc::ld16(at + 16 * hf, ahead);
                ld_wait16(ahead);
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    const int col = 32 * b + 16 * hf;
                    uint32_t v[16], hi[8], lo[8];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = ahead[j];
                    const bool more = b < q;
                    if (more) tc::ld16(at + col + 32, ahead);
                    if (b > q) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) hi[j] = lo[j] = 0u;
                    } else {
                        const float f = ex2((hi_r - s.end_hi[b]) + (lo_r - s.end_lo[b]));
                        if (b < q) {
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 e = *reinterpret_cast<const float4 *>(s.to_block + col + j);
                                float x[4] = {__uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                                              __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])};
                                mul2(x[0], x[1], f, f);
                                mul2(x[2], x[3], f, f);
                                mul2(x[0], x[1], e.x, e.y);
                                mul2(x[2], x[3], e.z, e.w);
                                hi[j / 2] = split2(x[0], x[1], lo[j / 2]);
                                hi[j / 2 + 1] = split2(x[2], x[3], lo[j / 2 + 1]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                float4 a = *reinterpret_cast<const float4 *>(s.hi + col + j);
                                float4 g = *reinterpret_cast<const float4 *>(s.lo + col + j);
                                const float4 d = *reinterpret_cast<const float4 *>(s.dt + col + j);
                                add2(a.x, a.y, hi_r, hi_r);
                                add2(a.z, a.w, hi_r, hi_r);
                                add2(g.x, g.y, lo_r, lo_r);
                                add2(g.z, g.w, lo_r, lo_r);
                                add2(a.x, a.y, g.x, g.y);
                                add2(a.z, a.w, g.z, g.w);
                                float x[4] = {ex2(a.x), ex2(a.y), ex2(a.z), ex2(a.w)};
                                mul2(x[0], x[1], d.x, d.y);
                                mul2(x[2], x[3], d.z, d.w);
                                mul2(x[0], x[1], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                                mul2(x[2], x[3], __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    x[e] = col + j + e > r ? 0.f : col + j + e == r ? x[e] + dv : x[e];
                                hi[j / 2] = split2(x[0], x[1], lo[j / 2]);
                                hi[j / 2 + 1] = split2(x[2], x[3], lo[j / 2 + 1]);
                            }
                        }
                    }
                    tc::st8(at + col, hi);
                    tc::st8(at + col + 8, lo);
                    if (more) ld_wait16(ahead);
                }
                tc::st_wait();
                tc::fence_before();
            }
            if (i > 0 && !take_out(i - 1)) break;
            arrive(kMReady + (i & 1));   // M is there and y's columns are free
            // stored behind the arrivals: an arrival waits for this warp's stores before it
            if (i > 0) {
                // four lanes exchange their 16-byte pieces, so that they write the 64
                // bytes of one row and not each its own
                exchange(ys[0], ys[1], 1, lane);
                exchange(ys[2], ys[3], 1, lane);
                exchange(ys[0], ys[2], 2, lane);
                exchange(ys[1], ys[3], 2, lane);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if ((r & ~3) + k < valid)
                        *reinterpret_cast<uint4 *>(dst + k * static_cast<int64_t>(p.heads) * p.p) = ys[k];
            }
        }
        if (i <= count) s_abort = 1;
    } else {
        // ---------------------------------------------------------- the state
        // row 32 q + lane of S; columns: the half hf
        const int q = warp & 3, hf = (warp >> 2) & 1, r = 32 * q + lane, gt = tid - kGroupThreads;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        float S[kCols];
        const bool has = 32 * q < kN;   // (of the warp's rows all or none)
        // this thread's values in the state array
        auto state_at = [&](const Scalars &v) {
            return ((static_cast<int64_t>(v.seq) * p.heads + (v.unit >> pl.shift)) * kN + r) * p.p +
                   (v.unit & pl.shift) * kPS + kCols * hf;
        };
        // ... and in the slots at the cuts
        const int64_t slot = static_cast<int64_t>(c) * kCols * kGroupThreads + gt;
        // The state that enters chunk i of the run (its first, or a sequence's first).
        auto start_state = [&](const Scalars &v) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) S[j] = 0.f;
            if (v.pos > 0) {
                if (kStates) return;   // only what this part adds
                // what the runs in front left of this sequence, the nearest first
                const int64_t head = q0 - v.pos;
                float f = 1.f;
                for (int k = c - 1; k >= 0; --k) {
                    const float *src = pl.slots + static_cast<int64_t>(k) * kCols * kGroupThreads + gt;
#pragma unroll
                    for (int j = 0; j < kCols; ++j) S[j] = fmaf(src[j * kGroupThreads], f, S[j]);
                    if (list.begin(k) <= head) break;
                    f *= pl.decay[k];
                }
                return;
            }
            if (p.s0 == nullptr) return;
            // in place, another CTA overwrites the initial state of a sequence
            // that the end of this run cuts: the first launch took a copy
            if (!kStates && pl.in_place && (v.flags & kCut) != 0) {
#pragma unroll
                for (int j = 0; j < kCols; ++j) S[j] = pl.saved[slot + j * kGroupThreads];
                return;
            }
            if (has) {
                const float4 *src = reinterpret_cast<const float4 *>(p.s0 + state_at(v));
#pragma unroll
                for (int j = 0; j < kCols / 4; ++j) {
                    const float4 f = src[j];
                    S[4 * j] = f.x; S[4 * j + 1] = f.y; S[4 * j + 2] = f.z; S[4 * j + 3] = f.w;
                }
            }
            if (kStates && pl.in_place) {
#pragma unroll
                for (int j = 0; j < kCols; ++j) pl.saved[slot + j * kGroupThreads] = S[j];
            }
        };
        // S as two bf16 terms, and C, for C S of chunk i
        auto put_state = [&](int i) -> bool {
            if (has) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint4 hi, lo;
                    hi.x = split2(S[8 * k], S[8 * k + 1], lo.x);
                    hi.y = split2(S[8 * k + 2], S[8 * k + 3], lo.y);
                    hi.z = split2(S[8 * k + 4], S[8 * k + 5], lo.z);
                    hi.w = split2(S[8 * k + 6], S[8 * k + 7], lo.w);
                    const int at = r * 128 + (((4 * hf + k) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4 *>(smem + kOffS + at) = hi;
                    *reinterpret_cast<uint4 *>(smem + kOffS + kTileBytes + at) = lo;
                }
            }
            fence_async();
            if (!wait(kFullC, i)) return false;
            constexpr int kHalf = kN / 16;   // 16-byte granules of half a row
            const uint8_t *C = smem + kOffC + r * 128 + (kHalf * hf >> 3) * kTileBytes;
#pragma unroll
            for (int k = 0; k < kHalf; k += 2) {
                const int g = (kHalf * hf & 7) + k;
                const uint4 x = *reinterpret_cast<const uint4 *>(C + ((g ^ (r & 7)) << 4));
                const uint4 y = *reinterpret_cast<const uint4 *>(C + (((g + 1) ^ (r & 7)) << 4));
                const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                tc::st8(lanes + kTmC + 4 * (kHalf * hf + k), v);
            }
            tc::st_wait();
            tc::fence_before();
            arrive(kSReady);
            return true;
        };

        float run_decay = 1.f;   // over this part of the sequence
        bool ok = true;
#pragma unroll 1
        for (int i = -1; i < count; ++i) {
            const Scalars &s = scal[i & (kRing - 1)], &next = scal[(i + 1) & (kRing - 1)];
            const bool more = i + 1 < count;
            if (kStates && more) {   // into the other set of weighted rows
                if (!(ok = landed(i + 1))) break;
                put_rows(i + 1, 2 * (warp - kGroup), 2);
                if (i < 0) start_state(next);
            }
            if (i >= 0) {
                // ---- S = 2^G_last S + B^T (W X)
                if (!(ok = wait(kDS + (i & 1), i >> 1))) break;
                const float dec = s.decay;
                if (has) {
                    tc::fence_after();
                    uint32_t v[2][16];
                    tc::ld16(lanes + tm_ds(kStates, i) + kCols * hf, v[0]);
                    tc::ld16(lanes + tm_ds(kStates, i) + kCols * hf + 16, v[1]);
                    ld_wait16(v[0]);
                    ld_wait16(v[1]);
#pragma unroll
                    for (int j = 0; j < kCols; j += 2)
                        fma2(S[j], S[j + 1], dec, dec, __uint_as_float(v[j >> 4][j & 15]),
                             __uint_as_float(v[j >> 4][(j & 15) + 1]));
                    tc::fence_before();
                }
                run_decay *= dec;
                if (!kStates && (s.flags & kLast) != 0 && p.s_final != nullptr && has) {
                    float4 *out = reinterpret_cast<float4 *>(p.s_final + state_at(s));
#pragma unroll
                    for (int j = 0; j < kCols / 4; ++j)
                        out[j] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
                }
                arrive(kScFree + (i & (kRing - 1)));
            }
            if (!kStates && more) {
                if (!(ok = landed(i + 1))) break;
                // Into the rows that this chunk's product has read. M is the more work the
                // later its rows, and its warps share an issue slot with these: the last
                // quarter takes none of the tasks, the first two most (T 131072, 32 heads
                // of 128, with even shares: 1573 us, this way 1552).
                put_rows(i + 1, 16 * hf + (q < 3 ? 6 * q : 0), q < 2 ? 6 : q == 2 ? 4 : 0);
                if (i < 0 || next.pos == 0) start_state(next);
                if (i >= 0 && !(ok = wait(kCS + (i & 1), i >> 1))) break;   // the terms of S are read
                if (!(ok = put_state(i + 1))) break;
            }
        }
        if (!ok) s_abort = 1;
        if (kStates && ok) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) pl.slots[slot + j * kGroupThreads] = has ? S[j] : 0.f;
            if (gt == 0) pl.decay[c] = run_decay;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (tid == 0 && s_abort != 0) atomicOr(p.err, kErrTimeout);
    if (warp == 0) {
        tc::fence_after();
        tc::dealloc(0, kTmCols);
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

// Workspace: [chunk offsets (packed)][decays of the runs][states at the cuts][copies of
// initial states (in place)][decays of the chunks].
constexpr int64_t kSlotBytes = static_cast<int64_t>(kCols) * kGroupThreads * 4;
int64_t offsets_bytes(const SsmParams &p) {
    return p.cu != nullptr ? align256((static_cast<int64_t>(p.n_seqs) + 1) * 4) : 0;
}

// At most this many chunks of a head.
int64_t most_chunks(const SsmParams &p) {
    return p.cu != nullptr ? (p.tokens + static_cast<int64_t>(kL - 1) * p.n_seqs) / kL
                           : (p.seq_len + kL - 1) / kL * p.n_seqs;
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
    return offsets_bytes(p) + 1024 + 2 * kPlannedSms * kSlotBytes + most_chunks(p) * p.heads * kDecaysBytes;
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
    pl.shift = p.p / kPS - 1;
    pl.units = static_cast<int64_t>(p.heads) << pl.shift;
    pl.cps = static_cast<int>((p.seq_len + kL - 1) / kL);
    pl.decay = reinterpret_cast<float *>(ws + offsets_bytes(p));
    pl.slots = reinterpret_cast<float *>(ws + offsets_bytes(p) + 1024);
    pl.saved = pl.slots + kPlannedSms * kSlotBytes / 4;
    pl.decays = reinterpret_cast<Decays *>(ws + offsets_bytes(p) + 1024 + 2 * kPlannedSms * kSlotBytes);
    pl.in_place = p.s_final != nullptr && p.s_final == p.s0;
    pl.stall = p.stall;
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
    // there are so many that the SMs are even without cuts (64 heads of 64: 512 tokens
    // 22 us whole and 25 cut, 20 x 1024 tokens 205 and 211; 8 heads: 1024 tokens 31 and 23).
    // These are fixed lengths. Of a packed batch the rule looks at the tokens only, which is
    // right for a few sequences and far off for many short ones: each is a chunk, and one
    // block per unit walks them all (8 heads: 4 x 128 tokens 29 us, 24 x 20 whole 115 and
    // 24 x 22 cut 25, 256 x 2 whole 1147 and 257 x 2 cut 85).
    const int64_t nc = most_chunks(p);
    const bool whole = p.cu != nullptr ? p.tokens <= 4 * kL
                                       : pl.cps <= 4 || pl.units * p.n_seqs >= 8 * kPlannedSms;
    pl.gran = !whole ? 1 : p.cu != nullptr ? 0 : pl.cps;
    const int64_t runs = pl.units * nc / (pl.gran > 0 ? pl.gran : nc);
    const unsigned grid = static_cast<unsigned>(runs < kPlannedSms ? runs : kPlannedSms);
    // a launch that may begin before the one in front of it is over
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t next{};
    next.gridDim = dim3(grid);
    next.blockDim = dim3(kThreads);
    next.dynamicSmemBytes = kSmem;
    next.stream = stream;
    next.attrs = &overlap;
    next.numAttrs = 1;
    const int64_t blocks = (nc * p.heads + 7) / 8;
    ssm_decays_kernel<<<static_cast<unsigned>(blocks < 8 * kPlannedSms ? blocks : 8 * kPlannedSms), 256, 0, stream>>>(p, pl);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return with_n(p, [&](auto n) {
        constexpr int kN = decltype(n)::value;
        if (!whole) {
            const cudaError_t e = cudaLaunchKernelEx(&next, ssm_chunk_kernel<kN, true>, maps, p, pl);
            if (e != cudaSuccess) return e;
        }
        return cudaLaunchKernelEx(&next, ssm_chunk_kernel<kN, false>, maps, p, pl);
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
