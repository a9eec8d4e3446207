// Norms of query and key heads and the rotation by position in one pass
// (kda_qk_norm_rope), and its gradients. For a head x of D channels, weights w and the
// rotation R by the token's angles
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = R (x r w)
//   g = R^T dy,  dw = sum g x r,  dx = r (g w - x r mean(g w x r))
//
// D / 8 lanes share a head, 16 bytes of it each, and keep the same channels from head to
// head: a warp takes some heads of one token with what a channel and its partner in the
// rotation are multiplied by (weight times cosine and sine) in registers. The sines and
// cosines of a token are formed once for them. Bound by reading and writing the heads.
// These come through a ring of bulk copies of each warp's own, a batch of heads (contiguous in
// a token) each, so that what is on its way takes no registers (with batches in registers the
// 8192 tokens below took 64 us, their gradient 94).
//
// Measured: 8192 tokens of 64 + 8 heads of 128: 52 us (5.8 TB/s, 86 % of copy bandwidth), the
// gradient 83 us (80 %, and 62 % of the issue slots taken); 5003 tokens of 16 + 2 heads of 64, gradient
// 17.0 us (40 %: start, end and the weights' sums are 6 us of it); one token 4.2 us, a launch and
// a chain of loads.

#include <type_traits>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kHeadsThreads = 256, kHeadsWarps = 8;
constexpr int kRing = 3;                      // batches of a warp
constexpr int kAhead = 4, kAheadGrad = 2;     // heads of a lane group in a batch
constexpr int kHeadsBlocks = 2, kGradBlocksPerSm = 2;   // of an SM
constexpr unsigned long long kLandNs = 100000000;       // within which a copy under way ends

// cos and sin of position * f, where f turns by f / 2 pi a position. The turns are
// formed as two floats (f / 2 pi to 2^-48, the position in two parts that fp32 holds
// exactly, each product with its rounding error) and whole turns are dropped on the way;
// what is left, half a turn at most, is exact to 2^-23 of a turn. (With the hardware's sine and
// cosine, off by 2^-21, one token took 4.0 us for 4.2, 8192 of 72 heads 51.5 for 51.9; a
// result rounded otherwise than the 64-bit one three times as often.)
__device__ __forceinline__ void angle(int pos, float f, float &c, float &s) {
    const float inv = 0.15915494f, inv_lo = 6.42063833e-9f;   // 1 / 2 pi
    const float hi = f * inv, lo = fmaf(f, inv, -hi) + f * inv_lo;
    const float p0 = static_cast<float>(pos & 4095), p1 = static_cast<float>(pos & ~4095);
    const float a = p0 * hi, b = p1 * hi;
    float t = (a - rintf(a)) + (b - rintf(b));
    t += fmaf(p0, hi, -a) + fmaf(p1, hi, -b) + (p0 + p1) * lo;
    sincospif(2.f * (t - rintf(t)), &s, &c);
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

// kN floats (4 or 8) from a 16-byte boundary
template <int kN>
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + i);
        x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
}

// A token's cosines, then its sines, by the warp that needs them.
__device__ __forceinline__ void fill_angles(const HeadsParams &p, float *cs, int pos) {
    const int half = p.rot / 2;
    __syncwarp();
    for (int f = threadIdx.x & 31; f < half; f += 32) {
        float c, s;
        angle(pos, __ldg(p.freq + f), c, s);
        cs[f] = c;
        cs[half + f] = s;
    }
    __syncwarp();
}

// Where the lane's channels stand in the rotation: (i, i + n) together, or (2i, 2i + 1).
template <bool kPairs>
struct Turn {
    bool in, low;   // rotated at all; the first of the pair
    int from;       // the lane that has the partners
    int partner;    // their first channel
    int f;          // first frequency
    __device__ __forceinline__ Turn(int rot, int at, int lane) {
        const int half = rot / 2;
        in = 8 * at < rot;
        low = 8 * at < half;
        from = kPairs || !in ? lane : low ? lane + rot / 16 : lane - rot / 16;
        partner = kPairs || !in ? 8 * at : low ? 8 * at + half : 8 * at - half;
        f = kPairs ? 4 * at : low ? 8 * at : 8 * at - half;
    }
    // Cosines, and sines with the sign that the partner enters with, of the lane's channels.
    __device__ __forceinline__ void angles(const float *cs, int rot, float (&c)[8], float (&s)[8]) const {
        constexpr int kN = kPairs ? 4 : 8;
        float cc[8], ss[8];
        const int i = in ? f : 0;
        load8<kN>(cs + i, cc);
        load8<kN>(cs + rot / 2 + i, ss);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int j = kPairs ? e / 2 : e;
            const bool first = kPairs ? e % 2 == 0 : low;
            c[e] = in ? cc[j] : 1.f;
            s[e] = in ? (first ? -ss[j] : ss[j]) : 0.f;
        }
    }
    // The partners of eight packed channels.
    __device__ __forceinline__ uint4 partners(const uint4 &u) const {
        if (kPairs)
            return make_uint4(__byte_perm(u.x, 0, 0x1032), __byte_perm(u.y, 0, 0x1032), __byte_perm(u.z, 0, 0x1032),
                              __byte_perm(u.w, 0, 0x1032));
        return make_uint4(__shfl_sync(0xffffffffu, u.x, from), __shfl_sync(0xffffffffu, u.y, from),
                          __shfl_sync(0xffffffffu, u.z, from), __shfl_sync(0xffffffffu, u.w, from));
    }
    __device__ __forceinline__ void partners(const float (&x)[8], float (&o)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = kPairs ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], from);
    }
};

// The weights of queries and keys in shared memory (ones where there are none).
template <int D>
__device__ __forceinline__ void fill_weights(const HeadsParams &p, float *w) {
    for (int i = threadIdx.x; i < D; i += kHeadsThreads) {
        w[i] = p.qw != nullptr ? __ldg(p.qw + i) : 1.f;
        w[D + i] = p.kw != nullptr ? __ldg(p.kw + i) : 1.f;
    }
}

// A warp's work in the forward kernel: the heads [q0, q1) of the queries and [k0, k1) of the keys of every token it
// comes to, in batches. Warp w of a block that takes 8 / parts tokens together has token
// w / parts of them, and one part of its heads.
struct Share {
    int q0, q1, k0, k1;
    int64_t token, step;   // (the first, and to the next)
    __device__ __forceinline__ Share(const HeadsParams &p, int parts) {
        const int w = threadIdx.x >> 5, part = w % parts, H = p.hq + p.hk, tokens = kHeadsWarps / parts;
        const int a = part * H / parts, b = (part + 1) * H / parts;
        q0 = min(a, p.hq);
        q1 = min(b, p.hq);
        k0 = max(a - p.hq, 0);
        k1 = max(b - p.hq, 0);
        token = static_cast<int64_t>(blockIdx.x) * tokens + w / parts;
        step = static_cast<int64_t>(gridDim.x) * tokens;
    }
};

// `step` heads, or what is left, from head h of the queries or keys of a token on.
struct Batch {
    int64_t token;
    bool keys;
    int h;
    __device__ __forceinline__ explicit Batch(const Share &mine)
        : token(mine.token), keys(mine.q0 >= mine.q1), h(keys ? mine.k0 : mine.q0) {}
    __device__ __forceinline__ int end(const Share &mine) const { return keys ? mine.k1 : mine.q1; }
    __device__ __forceinline__ void advance(const Share &mine, int step) {
        h += step;
        if (h < end(mine)) return;
        if (!keys && mine.k0 < mine.k1) {
            keys = true;
            h = mine.k0;
            return;
        }
        token += mine.step;
        keys = mine.q0 >= mine.q1;
        h = keys ? mine.k0 : mine.q0;
    }
};

// A wait for batch n has run out: what has been asked for from there on lands, within a limit.
// (Not inlined: in the loops it costs the gradient another 0.5 us.)
__device__ __noinline__ void gave_up(uint32_t bars, int n, int *err) {
    atomicOr(err, kErrTimeout);
    for (int i = n; i < n + kRing; ++i) mbar_wait(bars + 8 * (i % kRing), i / kRing & 1, kLandNs);
}

// A warp's ring: kRing places of kBytes, a barrier each.
template <int kBytes>
struct WarpRing {
    uint32_t base, bars;
    int n = 0;   // batches taken
    __device__ __forceinline__ WarpRing(uint8_t *places, uint64_t *barriers) {
        const int w = threadIdx.x >> 5;
        base = smem_u32(places) + w * kRing * kBytes;
        bars = smem_u32(barriers + w * kRing);
        if ((threadIdx.x & 31) == 0)
            for (int i = 0; i < kRing; ++i) mbar_init(bars + 8 * i, 1);
        mbar_fence_init();
        __syncwarp();
    }
    __device__ __forceinline__ uint32_t place(int i) const { return base + i % kRing * kBytes; }
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * (i % kRing); }
    // For the next batch; false where it has not come: the warp stops then, with its copies landed.
    __device__ __forceinline__ bool wait(int *err) const {
        if (__all_sync(0xffffffffu, mbar_wait(bar(n), n / kRing & 1))) return true;
        gave_up(bars, n, err);
        return false;
    }
};

__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

template <int D, bool kPairs>
__global__ void __launch_bounds__(kHeadsThreads, kHeadsBlocks) heads_kernel(HeadsParams p, int parts) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kStep = kRows * kAhead;
    extern __shared__ __align__(128) uint8_t places[];   // the warps' rings, then the angles
    __shared__ __align__(16) float weights[2 * D];
    __shared__ uint64_t barriers[kHeadsWarps * kRing];
    constexpr int kBytes = kStep * D * 2;
    float *table = reinterpret_cast<float *>(places + kHeadsWarps * kRing * kBytes) + (threadIdx.x >> 5) * p.rot;
    const int lane = threadIdx.x & 31, at = lane % kLanes, sub = lane / kLanes;
    const Turn<kPairs> turn(p.rot, at, lane);
    const Share mine(p, parts);
    WarpRing<kBytes> ring(places, barriers);
    auto ask = [&](const Batch &b, int i) {
        if (b.token >= p.tokens || lane != 0) return;
        const int rows = min(kStep, b.end(mine) - b.h);
        const uint16_t *src = (b.keys ? static_cast<const uint16_t *>(p.k) + b.token * p.k_stride
                                      : static_cast<const uint16_t *>(p.q) + b.token * p.q_stride) + b.h * D;
        mbar_arrive_expect_tx(ring.bar(i), rows * D * 2);
        bulk_g2s(ring.place(i), src, rows * D * 2, ring.bar(i));
    };
    Batch now(mine), ahead(mine);
    for (int i = 0; i < kRing; ++i) {
        ask(ahead, i);
        ahead.advance(mine, kStep);
    }
    fill_weights<D>(p, weights);
    __syncthreads();
    int pos = p.rot > 0 && mine.token < p.tokens ? __ldg(p.pos + mine.token) : 0;
    for (int64_t token = mine.token; token < p.tokens; token += mine.step) {
        if (p.rot > 0) {
            fill_angles(p, table, pos);
            if (token + mine.step < p.tokens) pos = __ldg(p.pos + token + mine.step);
        }
#pragma unroll 1
        for (int keys = 0; keys < 2; ++keys) {
            const int end = keys ? mine.k1 : mine.q1;
            if ((keys ? mine.k0 : mine.q0) >= end) continue;
            // y = (x a + partner b) r
            float a[8], b[8];
            load8<8>(weights + keys * D + 8 * at, a);
            if (p.rot > 0) {
                float w[8], c[8], s[8];
                turn.angles(table, p.rot, c, s);
                load8<8>(weights + keys * D + turn.partner, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = w[kPairs ? e ^ 1 : e];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mul2(a[e], a[e + 1], c[e], c[e + 1]);
                    mul2(b[e], b[e + 1], s[e], s[e + 1]);
                }
            }
            uint16_t *out = (keys ? static_cast<uint16_t *>(p.k_out) + token * p.ko_stride
                                  : static_cast<uint16_t *>(p.q_out) + token * p.qo_stride) + sub * D + 8 * at;
            while (now.token == token && now.keys == (keys != 0)) {
                if (!ring.wait(p.err)) return;
                const uint32_t from = ring.place(ring.n) + lane * 16;
#pragma unroll
                for (int i = 0; i < kAhead; i += 2) {   // two heads of a lane group side by side
                    if (now.h + i * kRows >= end) break;   // (the whole warp)
                    uint4 in[2];
                    float x[2][8], o[2][8], r[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) in[j] = lds16(from + (i + j) * 512);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float sq[2] = {0.f, 0.f};
                        unpack8(in[j], x[j]);
#pragma unroll
                        for (int e = 0; e < 8; e += 2) muladd2(sq[0], sq[1], x[j][e], x[j][e + 1], x[j][e], x[j][e + 1]);
                        r[j] = sq[0] + sq[1];
                    }
#pragma unroll
                    for (int m = kLanes / 2; m > 0; m >>= 1)
                        add2(r[0], r[1], __shfl_xor_sync(0xffffffffu, r[0], m), __shfl_xor_sync(0xffffffffu, r[1], m));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        r[j] = rsqrtf(r[j] * (1.f / D) + p.eps);
                        if (p.rot > 0) unpack8(turn.partners(in[j]), o[j]);
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            mul2(x[j][e], x[j][e + 1], a[e], a[e + 1]);
                            if (p.rot > 0) muladd2(x[j][e], x[j][e + 1], o[j][e], o[j][e + 1], b[e], b[e + 1]);
                            mul2(x[j][e], x[j][e + 1], r[j], r[j]);
                        }
                        // (what lies behind the last head is an earlier batch's)
                        const int head = now.h + (i + j) * kRows;
                        if (head + sub < end) *reinterpret_cast<uint4 *>(out + head * D) = pack8(x[j]);
                    }
                }
                __syncwarp();
                if (ring.n < p.stall) ask(ahead, ring.n);   // (the place just read)
                ++ring.n;
                now.advance(mine, kStep);
                ahead.advance(mine, kStep);
            }
        }
    }
}

// A warp's way through its share of the gradient's work: token after token the queries' heads, then the
// keys', cut into units of kUnit heads. All warps have as many units, one more or less; a
// token's heads may so be cut anywhere. A batch is up to kMost units of one token, of its
// queries or its keys. (Parts of tokens in turns, as the forward kernel takes them: 8192 tokens
// of 72 heads of 128 took 86 us, this way 81; 5003 of 18 heads 17.5 and 16.6. The forward kernel,
// nearer the memory's rate, gains from all warps reading one stretch of it: 51 us in turns, 57
// this way.)
template <int kUnit, int kMost>
struct Walk {
    int token, left;   // units left
    int h, heads;      // the batch: heads from h on
    bool keys;         // of the keys
    __device__ __forceinline__ static int units(int heads) { return (heads + kUnit - 1) / kUnit; }
    __device__ __forceinline__ explicit Walk(const HeadsParams &p) {
        const int nq = units(p.hq), n = nq + units(p.hk);
        const int64_t all = p.tokens * n, warps = static_cast<int64_t>(gridDim.x) * kHeadsWarps,
                      w = static_cast<int64_t>(blockIdx.x) * kHeadsWarps + (threadIdx.x >> 5);
        const int64_t u0 = w * all / warps, u1 = (w + 1) * all / warps;
        token = static_cast<int>(u0 / n);
        const int at = static_cast<int>(u0 - static_cast<int64_t>(token) * n);
        left = static_cast<int>(u1 - u0);
        keys = at >= nq;
        h = (keys ? at - nq : at) * kUnit;
        batch(p);
    }
    __device__ __forceinline__ void batch(const HeadsParams &p) {
        heads = min(min((keys ? p.hk : p.hq) - h, kMost * kUnit), left * kUnit);
    }
    __device__ __forceinline__ void advance(const HeadsParams &p) {
        left -= units(heads);
        h += heads;
        if (h >= (keys ? p.hk : p.hq)) {
            h = 0;
            if (keys || p.hk == 0) ++token;
            keys = !keys && p.hk > 0;
        }
        batch(p);
    }
};

// The gradient. With g = R^T dy, A = sum x^2, B = sum g w x over the channels:
//   dw += r g x,  dx = r w g - (r^3 B / D) x
// Blocks keep their parts of the weights' gradients in registers to the end.
constexpr int kGradBlocks = kGradBlocksPerSm * kPlannedSms;

template <int D, bool kPairs, bool kF32>
__global__ void __launch_bounds__(kHeadsThreads, kGradBlocksPerSm) heads_backward_kernel(HeadsParams p) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kStep = kRows * kAheadGrad, kSize = kF32 ? 4 : 2;
    using Walk = Walk<kRows, kAheadGrad>;
    extern __shared__ __align__(128) uint8_t places[];   // the warps' rings, then the angles
    __shared__ __align__(16) float weights[2 * D];
    __shared__ uint64_t barriers[kHeadsWarps * kRing];
    constexpr int kBytes = kStep * D * (2 + kSize), kOffY = kStep * D * 2;   // x, then dy
    float *table = reinterpret_cast<float *>(places + kHeadsWarps * kRing * kBytes) + (threadIdx.x >> 5) * p.rot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane % kLanes, sub = lane / kLanes;
    const Turn<kPairs> turn(p.rot, at, lane);
    WarpRing<kBytes> ring(places, barriers);
    // (the weights' sums are a second launch, which comes up while this one is at work)
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    auto ask = [&](const Walk &b, int i) {
        if (b.left == 0 || lane != 0) return;
        const int rows = b.heads;
        const bool keys = b.keys;
        const uint16_t *x = (keys ? static_cast<const uint16_t *>(p.k) + b.token * p.k_stride
                                  : static_cast<const uint16_t *>(p.q) + b.token * p.q_stride) + b.h * D;
        const uint8_t *y = static_cast<const uint8_t *>(keys ? p.dk : p.dq) +
                           (b.token * (keys ? p.dk_stride : p.dq_stride) + b.h * D) * kSize;
        mbar_arrive_expect_tx(ring.bar(i), rows * D * (2 + kSize));
        bulk_g2s(ring.place(i), x, rows * D * 2, ring.bar(i));
        bulk_g2s(ring.place(i) + kOffY, y, rows * D * kSize, ring.bar(i));
    };
    Walk now(p), ahead(now);
    for (int i = 0; i < kRing; ++i) {
        ask(ahead, i);
        ahead.advance(p);
    }
    fill_weights<D>(p, weights);
    __syncthreads();
    float dqw[8], dkw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dqw[e] = dkw[e] = 0.f;
    int pos = p.rot > 0 && now.left > 0 ? __ldg(p.pos + now.token) : 0;
    while (now.left > 0) {
        const int64_t token = now.token;
        float c[8], s[8];
        if (p.rot > 0) {
            fill_angles(p, table, pos);
            turn.angles(table, p.rot, c, s);
            if (token + 1 < p.tokens) pos = __ldg(p.pos + token + 1);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = -s[e];   // (back)
        }
        auto run = [&](bool keys, uint16_t *out, float (&dw)[8]) {
            const auto here = [&] { return now.left > 0 && now.token == token && now.keys == keys; };
            if (!here()) return;
            float w[8];
            load8<8>(weights + keys * D + 8 * at, w);
            out += sub * D + 8 * at;
            do {
                const int first = now.h, heads = now.heads;
                if (!ring.wait(p.err)) {
                    now.left = 0;
                    break;
                }
                const uint32_t from = ring.place(ring.n);
#pragma unroll
                for (int i = 0; i < kAheadGrad; ++i) {
                    if (i * kRows >= heads) break;   // (the whole warp)
                    const bool row = i * kRows + sub < heads;
                    float x[8], g[8], o[8];
                    // (what lies behind the last head is an earlier batch's)
                    uint4 u = lds16(from + i * 512 + lane * 16);
                    if (!row) u = make_uint4(0, 0, 0, 0);
                    unpack8(u, x);
                    if (kF32) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint4 v = lds16(from + kOffY + i * 1024 + lane * 32 + 16 * j);
                            g[4 * j] = __uint_as_float(v.x);
                            g[4 * j + 1] = __uint_as_float(v.y);
                            g[4 * j + 2] = __uint_as_float(v.z);
                            g[4 * j + 3] = __uint_as_float(v.w);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[e] = row ? g[e] : 0.f;
                        if (p.rot > 0) turn.partners(g, o);
                    } else {
                        u = lds16(from + kOffY + i * 512 + lane * 16);
                        if (!row) u = make_uint4(0, 0, 0, 0);
                        unpack8(u, g);
                        if (p.rot > 0) unpack8(turn.partners(u), o);
                    }
                    float A[2] = {0.f, 0.f}, B[2] = {0.f, 0.f}, t[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        if (p.rot > 0) {
                            mul2(g[e], g[e + 1], c[e], c[e + 1]);
                            muladd2(g[e], g[e + 1], o[e], o[e + 1], s[e], s[e + 1]);
                        }
                        t[e] = g[e];
                        t[e + 1] = g[e + 1];
                        mul2(t[e], t[e + 1], x[e], x[e + 1]);
                        muladd2(A[0], A[1], x[e], x[e + 1], x[e], x[e + 1]);
                        muladd2(B[0], B[1], t[e], t[e + 1], w[e], w[e + 1]);
                    }
                    float a = A[0] + A[1], b = B[0] + B[1];
#pragma unroll
                    for (int m = kLanes / 2; m > 0; m >>= 1)
                        add2(a, b, __shfl_xor_sync(0xffffffffu, a, m), __shfl_xor_sync(0xffffffffu, b, m));
                    const float r = row ? rsqrtf(a * (1.f / D) + p.eps) : 0.f;
                    const float k = -r * r * (r * b) * (1.f / D);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        muladd2(dw[e], dw[e + 1], t[e], t[e + 1], r, r);
                        mul2(g[e], g[e + 1], w[e], w[e + 1]);
                        mul2(g[e], g[e + 1], r, r);
                        muladd2(g[e], g[e + 1], x[e], x[e + 1], k, k);
                    }
                    if (row) *reinterpret_cast<uint4 *>(out + (first + i * kRows) * D) = pack8(g);
                }
                __syncwarp();
                if (ring.n < p.stall) ask(ahead, ring.n);   // (the place just read)
                ++ring.n;
                now.advance(p);
                ahead.advance(p);
            } while (here());
        };
        run(false, static_cast<uint16_t *>(p.q_out) + token * p.qo_stride, dqw);
        run(true, static_cast<uint16_t *>(p.k_out) + token * p.ko_stride, dkw);
    }
    if (p.dqw == nullptr && p.dkw == nullptr) return;
    // the lane groups of a block, in order
    __shared__ float part[2][kHeadsWarps * kRows][D];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        part[0][warp * kRows + sub][8 * at + e] = dqw[e];
        part[1][warp * kRows + sub][8 * at + e] = dkw[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kHeadsThreads) {
        float sum = 0.f;
        for (int j = 0; j < kHeadsWarps * kRows; ++j) sum += part[i / D][j][i % D];
        p.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = sum;
    }
}

// dweight[i] = the sum of the blocks' parts: a warp takes 32 channels, every eighth block.
__global__ void __launch_bounds__(256) heads_weights_kernel(HeadsParams p, int blocks) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    float s = 0.f;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
#pragma unroll 8
    for (int b = warp; b < blocks; b += 8) s += p.partial[static_cast<int64_t>(b) * 2 * p.dim + i];
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0) return;
    for (int j = 1; j < 8; ++j) s += part[j][lane];
    float *dst = i < p.dim ? p.dqw : p.dkw;
    if (dst != nullptr) dst[i % p.dim] = s;
}

template <typename F>
cudaError_t with_dim(const HeadsParams &p, F &&go) {
    if (p.dim == 64) return go(std::integral_constant<int, 64>());
    if (p.dim == 128) return go(std::integral_constant<int, 128>());
    return go(std::integral_constant<int, 256>());
}

// Parts that a token's heads are cut into, 1, 2, 4 or 8: those with the least time by this
// count. Warps take (token, part) after (token, part), as many rounds as that makes; one costs its
// lane groups' heads and four more for what is done for the token alone. (8192 tokens, 40 heads of
// 64: 17 us in one part, 21 in two; 72 heads of 128: 56 and 51.)
int parts_of(const HeadsParams &p) {
    const int64_t warps = static_cast<int64_t>(kHeadsBlocks) * kPlannedSms * kHeadsWarps;
    const int H = p.hq + p.hk, rows = 256 / p.dim;
    int best = 1;
    int64_t least = INT64_MAX;
    for (int parts = 1; parts <= kHeadsWarps && parts <= H; parts *= 2) {
        const int64_t cost = ((p.tokens * parts + warps - 1) / warps) * ((H + parts * rows - 1) / (parts * rows) + 4);
        if (cost < least) {
            least = cost;
            best = parts;
        }
    }
    return best;
}

// The rings of a block, `bytes` for each channel of a batch, and its warps' angles.
int heads_smem(const HeadsParams &p, int ahead, int bytes) {
    return kHeadsWarps * (kRing * 256 * ahead * bytes + p.rot * 4);
}

unsigned blocks_of(int64_t warps, int64_t most) {
    const int64_t blocks = (warps + kHeadsWarps - 1) / kHeadsWarps;
    return static_cast<unsigned>(blocks < 1 ? 1 : blocks < most ? blocks : most);
}

// A warp for each unit of a lane group's heads, as far as there are so many.
unsigned grad_grid(const HeadsParams &p) {
    const int unit = 256 / p.dim;
    return blocks_of(p.tokens * ((p.hq + unit - 1) / unit + (p.hk + unit - 1) / unit), kGradBlocks);
}

template <int D>
cudaError_t configure_heads_dim() {
    const auto more = [](auto kernel, int bytes) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    HeadsParams p{};
    p.rot = D;   // (the most that a block takes)
    const int forward = heads_smem(p, kAhead, 2), back = heads_smem(p, kAheadGrad, 6);
    cudaError_t e = more(heads_kernel<D, true>, forward);
    if (e == cudaSuccess) e = more(heads_kernel<D, false>, forward);
    if (e == cudaSuccess) e = more(heads_backward_kernel<D, true, true>, back);
    if (e == cudaSuccess) e = more(heads_backward_kernel<D, true, false>, back);
    if (e == cudaSuccess) e = more(heads_backward_kernel<D, false, true>, back);
    if (e == cudaSuccess) e = more(heads_backward_kernel<D, false, false>, back);
    return e;
}

}  // namespace

cudaError_t configure_heads() {
    cudaError_t e = configure_heads_dim<64>();
    if (e == cudaSuccess) e = configure_heads_dim<128>();
    return e == cudaSuccess ? configure_heads_dim<256>() : e;
}

cudaError_t launch_heads(const HeadsParams &p, cudaStream_t stream) {
    return with_dim(p, [&](auto d) {
        constexpr int D = decltype(d)::value;
        const int parts = parts_of(p);
        auto kernel = p.pairs ? heads_kernel<D, true> : heads_kernel<D, false>;
        kernel<<<blocks_of(p.tokens * parts, kHeadsBlocks * kPlannedSms), kHeadsThreads, heads_smem(p, kAhead, 2), stream>>>(p, parts);
        return cudaGetLastError();
    });
}

int64_t heads_workspace(const HeadsParams &p) {
    return p.dqw != nullptr || p.dkw != nullptr ? static_cast<int64_t>(kGradBlocks) * 2 * p.dim * 4 : 0;
}

cudaError_t launch_heads_backward(const HeadsParams &p, cudaStream_t stream) {
    return with_dim(p, [&](auto d) {
        constexpr int D = decltype(d)::value;
        const unsigned grid = grad_grid(p);
        auto kernel = p.pairs ? (p.dout32 ? heads_backward_kernel<D, true, true> : heads_backward_kernel<D, true, false>)
                              : (p.dout32 ? heads_backward_kernel<D, false, true> : heads_backward_kernel<D, false, false>);
        kernel<<<grid, kHeadsThreads, heads_smem(p, kAheadGrad, p.dout32 ? 6 : 4), stream>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || (p.dqw == nullptr && p.dkw == nullptr)) return e;
        cudaLaunchAttribute overlap;
        overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        overlap.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t sums{};
        sums.gridDim = dim3(2 * D / 32);
        sums.blockDim = dim3(256);
        sums.stream = stream;
        sums.attrs = &overlap;
        sums.numAttrs = 1;
        return cudaLaunchKernelEx(&sums, heads_weights_kernel, p, static_cast<int>(grid));
    });
}

}  // namespace kda
