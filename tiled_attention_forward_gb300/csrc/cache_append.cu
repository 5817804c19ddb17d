// cache_append.cu -- keys and values of new tokens into a paged cache (16-bit
// or 4-bit), with the position rotation of q and k applied on the way.
//
// Rotation of a row x at position p, over its first `rot` elements, for each
// pair (a, b) with angle index i = 0 .. rot/2 - 1:
//     a' = a cos[p][i] - b sin[p][i],   b' = b cos[p][i] + a sin[p][i]
// with (a, b) = (x[i], x[i + rot/2]), or (x[2i], x[2i+1]) when interleaved.
//
// 4-bit rows: each group of 32 consecutive elements keeps fp16 (scale, zero),
// zero = round16(min), scale = round16((max - min) / 15), and codes
// c = clamp(rint((x - zero) / scale), 0, 15) taken against the rounded scale
// and zero, so that rounding those two costs no accuracy beyond the range's
// ends; the row then stands for c * scale + zero.  fp16 for both types of
// tensor: 11 bits of zero matter more here than bf16's range, and |x| is
// clamped to 65504.
//
// Work split: one thread moves 16 bytes (8 elements) of a row, D/8 threads a
// row, so partner elements of a rotation pair and the 4 threads of a group
// meet by shuffles within a warp.  A block takes the query rows, or the key and
// value rows, of one or a few tokens; a thread starts the loads of two rows (of
// q, or a head's k and v) before the tokens' slots, positions and angles (which
// depend on one another) have come, and the angles go through shared memory once
// for all heads.  The kind of a row is known where it is compiled: selecting
// between k and v at run time, addresses included, took a third of all
// instructions (4-bit prompt 104 -> 91 us).
//
// Measured (GB300): 8191 tokens of 16 + 2 * 2 heads, D = 64, 16 bits (45 MB)
// 10.9 us, of which about 2.5 are the launch; 16000 tokens of 32 + 2 * 8 heads, D
// = 128, 74 us in 16 bits (5.8 TB/s) and 87 us into 4 bits (422 MB with the
// values held, 4.9 TB/s), bound by the latency of its loads and by issue slots
// (63 % busy, about 300 instructions for 16 bytes of a key or value row).  64
// tokens of 32 + 2 * 8 heads, D = 128, take 2.5 us; 17 of 16 + 2 * 16 heads, D =
// 64, into 4 bits 3.3.  (16000 tokens into 4 bits:) two rows ahead and five
// blocks an SM: four blocks took 89 us, six 91.
// Up to 16 rows a thread: 8 took 4 us more (blocks' starts), 32 three.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace fattn {

// Bit k set <=> a cache kernel found fattn_status k (INVALID_ARG: an index out of range).
__device__ uint32_t g_append_error_word;

namespace {

constexpr int kThreads = 256;
constexpr int kTurns = 16;      // rows that a thread takes, where there are enough
constexpr float kFp16Max = 65504.f;
constexpr float kTwo23 = 8388608.f;  // an integer added to it stands in the low bits

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// pack8 with fp16's ends for what is past them: the values that a 4-bit group
// stands for, of which the largest may be (its scale is rounded to nearest).
template <bool BF16>
__device__ __forceinline__ uint4 pack8_finite(const float (&x)[8]) {
    if (BF16) return pack8<BF16>(x);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// An 8 x 8 matrix of nibbles, one row per lane of a set of 8 lanes, transposed:
// lane n's nibble p becomes lane p's nibble n.  kLane[b]: the lane-id bit that
// stands for bit b of the set's index n.
template <int L0, int L1, int L2>
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t x, int lane) {
    constexpr uint32_t kMask[3] = {0x0f0f0f0fu, 0x00ff00ffu, 0x0000ffffu};
    constexpr int kLane[3] = {L0, L1, L2};
#pragma unroll
    for (int b = 0; b < 3; ++b) {
        const int sh = 4 << b;
        const uint32_t y = __shfl_xor_sync(0xffffffffu, x, kLane[b]);
        x = (lane & kLane[b]) ? ((x & ~kMask[b]) | ((y & ~kMask[b]) >> sh))
                              : ((x & kMask[b]) | ((y & kMask[b]) << sh));
    }
    return x;
}

// (d0, d1) = (a0, a1) * (b0, b1) [+ (c0, c1)]: two fp32 results an instruction.
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ float min3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Quantises this thread's 8 elements (4 threads hold a group): its codes as the
// floats 2^23 + code (whose low bits are the code), scale and zero.  A NaN takes
// no part in the range and gets code 0 (min and max drop it); values past the
// fp16 range get the codes of its ends.  The quotient is formed to the last bit
// (one Newton step on the residual, which fma gives exactly): 16-bit values
// stand on a grid, where quotients of exactly k + 1/2 are common, and a quotient
// off by one bit there would round to the other neighbour.
//
// `rotated`: x is off by up to 3 roundings of its pair's magnitude, which this
// group's range and that of the lane `partner`'s group bound (|a|, |b| <=
// sqrt(2) max(|a'|, |b'|)); else x is exact.  True where some rounding -- of the
// zero, the scale or a code -- is too close to its border for fp32 to tell the
// side: about one group in a thousand, which requantise() then settles.  (A
// code on the wrong side is off by a whole step, and a reader of the cache
// could not tell that from an error.)  Exact x needs this for the scale, and for
// a code where x - zero takes more than 24 bits (elements of very different
// size): of an exact difference the quotient is an exact tie or more than half
// a unit of its last place away from one.  16-bit values are often at a tie, so
// that is asked only of threads that have one.
__device__ __forceinline__ bool quantise(const float (&x)[8], bool rotated, int partner, float (&t)[8], __half& scale,
                                         __half& zero) {
    float lo = min3(x[0], x[1], x[2]), hi = max3(x[0], x[1], x[2]);
    lo = fminf(min3(lo, x[3], x[4]), min3(x[5], x[6], x[7]));
    hi = fmaxf(max3(hi, x[3], x[4]), max3(x[5], x[6], x[7]));
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    if (!(lo <= hi)) lo = hi = 0.f;  // nothing but NaN
    float most = fmaxf(-lo, hi);     // (before the clamp: pairs far past the range may turn into it)
    lo = fminf(fmaxf(lo, -kFp16Max), kFp16Max) + 0.f;  // (+ 0: never -0, whose bits differ from 0's below)
    hi = fminf(fmaxf(hi, -kFp16Max), kFp16Max);
    const float step = (hi - lo) * (1.f / 15.f);
    scale = __float2half_rn(step);
    zero = __float2half_rn(lo);
    most = fmaxf(most, __shfl_sync(0xffffffffu, most, partner));
    const float err = rotated ? 2.6e-7f * most : 0.f;  // 3 sqrt(2) 2^-24
    const float es = fmaf(0.14f, err, 2.4e-7f * step);  // 2 err / 15 and three roundings
    auto apart = [](float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
        return (w >> 16) != (w & 0xffffu);
    };
    bool near = apart(lo - err, lo + err) || apart(step - es, step + es);
    const float s = __half2float(scale), z = __half2float(zero);
    const float inv = s > 0.f ? __fdividef(1.f, s) : 0.f;
    const float top = 15.f * s;  // exact
    float worst = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float d0, d1, q0, q1, r0, r1;
        add2(d0, d1, x[e], x[e + 1], -z, -z);
        d0 = fminf(fmaxf(d0, 0.f), top);
        d1 = fminf(fmaxf(d1, 0.f), top);
        mul2(q0, q1, d0, d1, inv, inv);
        fma2(r0, r1, q0, q1, -s, -s, d0, d1);
        fma2(r0, r1, r0, r1, inv, inv, q0, q1);
        add2(t[e], t[e + 1], r0, r1, kTwo23, kTwo23);  // to the nearest, ties to even
        add2(q0, q1, t[e], t[e + 1], -kTwo23, -kTwo23);
        fma2(q0, q1, q0, q1, -1.f, -1.f, r0, r1);  // how far each quotient is from its code
        worst = max3(worst, fabsf(q0), fabsf(q1));
    }
    // The quotient's own error: 16 * 2 roundings, and that of x in steps.
    if (worst > 0.5f - fmaf(err, inv, 2.0e-6f)) {
        bool exact = !rotated;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = __fsub_rn(x[e], z);  // exact where both of its terms come back
            exact = exact && __fadd_rn(d, z) == x[e] && __fsub_rn(x[e], d) == z;
        }
        near = near || !exact;
    }
    return near;
}

// The same to twice fp32's precision: values are unevaluated sums h + l of two
// floats, products by fma and sums by the two-sum of Knuth (fp64 would take 10
// times as long on this part).  From the raw elements that a group's four lanes
// (from `base` on) hold, and their partners' that lanes `from` hold, with whether
// and by which angles they turn.  The whole warp calls it and takes one element a lane:
// with 8 a lane it was four times as many instructions, which a call for few
// tokens waits for (64 tokens 4.1 -> 3.3 us, 16000 91 -> 87), and whole warps
// never run this as often as to hide it.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ Two normal(float h, float l) {  // |h| >= |l|
    const float s = __fadd_rn(h, l);
    return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
template <bool BF16>
__device__ __forceinline__ float element(uint32_t w, bool high) {
    if (BF16) return __uint_as_float(high ? w & 0xffff0000u : w << 16);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(high ? w >> 16 : w)));
}
struct Exact {
    float t;           // 2^23 + code
    uint32_t params;   // zero << 16 | scale
};
template <bool BF16, int CHUNKS>
__device__ __noinline__ Exact requantise(uint4 raw, int from, int base, bool swap, bool turns, const float* angles,
                                         int at) {
    const int lane = threadIdx.x % 32, e = lane % 8, owner = base + lane / 8;
    auto pick = [&](int who) {
        const uint32_t a = __shfl_sync(0xffffffffu, raw.x, who), b = __shfl_sync(0xffffffffu, raw.y, who);
        const uint32_t c = __shfl_sync(0xffffffffu, raw.z, who), d = __shfl_sync(0xffffffffu, raw.w, who);
        return e < 4 ? (e < 2 ? a : b) : (e < 6 ? c : d);
    };
    const uint32_t wx = pick(owner), wy = pick(__shfl_sync(0xffffffffu, from, owner));
    turns = __shfl_sync(0xffffffffu, turns, owner);
    at = __shfl_sync(0xffffffffu, at, owner) + (e / 4) * 8 * CHUNKS + e % 4;
    Two x = {element<BF16>(wx, e & 1), 0.f};
    if (turns) {
        const float co = angles[at], si = angles[at + 4 * CHUNKS];
        const float y = element<BF16>(swap ? wx : wy, swap ? !(e & 1) : (e & 1));
        const float p = __fmul_rn(x.h, co), q = __fmul_rn(y, si);
        const Two w = two_sum(p, q);
        const float l = __fadd_rn(w.l, __fadd_rn(__fmaf_rn(x.h, co, -p), __fmaf_rn(y, si, -q)));
        x = fabsf(w.h) < INFINITY ? normal(w.h, l) : Two{w.h, 0.f};
    }
    auto less = [](const Two& a, const Two& b) { return a.h < b.h || (a.h == b.h && a.l < b.l); };
    Two lo = {INFINITY, 0.f}, hi = {-INFINITY, 0.f};
    if (x.h == x.h) lo = hi = x;
#pragma unroll 1
    for (int m = 1; m < 32; m <<= 1) {
        const Two a = {__shfl_xor_sync(0xffffffffu, lo.h, m), __shfl_xor_sync(0xffffffffu, lo.l, m)};
        const Two b = {__shfl_xor_sync(0xffffffffu, hi.h, m), __shfl_xor_sync(0xffffffffu, hi.l, m)};
        if (less(a, lo)) lo = a;
        if (less(hi, b)) hi = b;
    }
    if (lo.h > hi.h) lo = hi = {0.f, 0.f};
    auto clamp = [](Two& a) {
        if (a.h > kFp16Max) a = {kFp16Max, 0.f};
        if (a.h < -kFp16Max) a = {-kFp16Max, 0.f};
    };
    clamp(lo);
    clamp(hi);
    const Two d = two_sum(hi.h, -lo.h);
    const Two range = normal(d.h, __fadd_rn(d.l, __fsub_rn(hi.l, lo.l)));
    const float q0 = range.h / 15.f;
    const __half scale = __float2half_rn(__fadd_rn(q0, __fadd_rn(__fmaf_rn(-q0, 15.f, range.h), range.l) / 15.f));
    const __half zero = __float2half_rn(lo.h);
    const float s = __half2float(scale), z = __half2float(zero);
    const float inv = s > 0.f ? 1.f / s : 0.f, half = 0.5f * s;
    // k: the code that fp32 finds; then which side of k +- 1/2 the value is on.
    const Two w = two_sum(x.h, -z);
    const float low = __fadd_rn(w.l, x.l);
    float k = rintf(fminf(fmaxf(w.h * inv, 0.f), 15.f));
    const float rest = __fmaf_rn(-k, s, w.h);
    const float above = __fadd_rn(__fsub_rn(rest, half), low), below = __fadd_rn(__fadd_rn(rest, half), low);
    const bool odd = (static_cast<int>(k) & 1) != 0;
    if (k < 15.f && (above > 0.f || (above == 0.f && odd && s > 0.f)))
        k += 1.f;
    else if (k > 0.f && (below < 0.f || (below == 0.f && odd && s > 0.f)))
        k -= 1.f;
    const __half2 params = __halves2half2(scale, zero);
    return {kTwo23 + (s > 0.f ? k : 0.f), *reinterpret_cast<const uint32_t*>(&params)};
}

// Nibbles e = 0..7 from t[0..7] = 2^23 + code: a sum in 32-bit integers, from
// which the exponents' share is taken off.
__device__ __forceinline__ uint32_t pack_codes(float t0, float t1, float t2, float t3, float t4, float t5, float t6, float t7) {
    const float t[8] = {t0, t1, t2, t3, t4, t5, t6, t7};
    uint32_t w = __float_as_uint(t[7]);
#pragma unroll
    for (int e = 6; e >= 0; --e) w = w * 16u + __float_as_uint(t[e]);
    return w - 0x4b000000u * 0x11111111u;
}

enum Kind { kQuery, kKey, kValue, kKeyAndValue };  // the last: of a block, not of a row

// Where an item (a token's row of a head) is.
struct Item {
    int tl;  // token within the block
    int h;
};

// A block's shared memory, of which a launch takes what its tokens need.
template <int D>
struct Shared {
    static constexpr int kChunks = D / 8;
    static constexpr int kMaxTokens = D == 128 ? 16 : 64;  // (32 at D = 128: 2 % longer with two K/V heads)
    // Where the token's row of head 0 is in the cache: in rows (4 bits) or in
    // elements (16 bits).  -1: nothing of the token is written.
    int64_t place[kMaxTokens];
    // Each token's angles, as the thread of chunk c multiplies by them: cos of
    // its first 4 elements, signed sin of them, then of its other 4.
    float4 cs[kMaxTokens][4][kChunks];

    static size_t bytes(uint32_t tokens) { return sizeof(place) + tokens * sizeof(cs[0]); }
};

// One row's 8 elements: rotation, outputs, cache.  Whole warps call it, with
// lanes that are not `on` repeating some row.  `place`: the row's in the cache.
template <int D, bool BF16, bool KV4, Kind KIND>
__device__ __forceinline__ void append_row(const AppendArgs& a, const uint4& raw, uint32_t t, uint32_t h, bool on,
                                           int64_t place, const float* angles, int at) {
    constexpr int kChunks = D / 8;
    const int c = threadIdx.x % kChunks, lane = threadIdx.x % 32;
    uint4 rounded = raw;
    bool turns = false;
    int from = lane;  // the lane of this thread's partner elements
    float x[8];
    if ((KV4 && KIND != kQuery) || (KIND != kValue && a.rot > 0)) unpack8<BF16>(raw, x);
    // Rotation (q and k rows).  Halves: chunk c < rot/16 holds the pairs' first
    // elements, the chunk rot/16 further their second ones, and the sign of a
    // sin - b cos comes with the angles.  Interleaved pairs lie within a chunk.
    if (KIND != kValue && a.rot > 0) {
        const int half_chunks = a.rot / 16;
        turns = c < 2 * half_chunks;
        float y[8];
        if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else {
            from = lane - c + (turns ? (c < half_chunks ? c + half_chunks : c - half_chunks) : c);
            uint4 other;
            other.x = __shfl_sync(0xffffffffu, raw.x, from);
            other.y = __shfl_sync(0xffffffffu, raw.y, from);
            other.z = __shfl_sync(0xffffffffu, raw.z, from);
            other.w = __shfl_sync(0xffffffffu, raw.w, from);
            unpack8<BF16>(other, y);
        }
        if (turns) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float4 co = *reinterpret_cast<const float4*>(angles + at + 8 * u * kChunks);
                const float4 si = *reinterpret_cast<const float4*>(angles + at + (8 * u + 4) * kChunks);
                float z[4];
                mul2(z[0], z[1], x[4 * u], x[4 * u + 1], co.x, co.y);
                mul2(z[2], z[3], x[4 * u + 2], x[4 * u + 3], co.z, co.w);
                fma2(x[4 * u], x[4 * u + 1], y[4 * u], y[4 * u + 1], si.x, si.y, z[0], z[1]);
                fma2(x[4 * u + 2], x[4 * u + 3], y[4 * u + 2], y[4 * u + 3], si.z, si.w, z[2], z[3]);
            }
            rounded = pack8<BF16>(x);
        }
    }
    auto out_row = [&](void* p, uint32_t ts, uint32_t hs) {
        return reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + static_cast<uint64_t>(t) * ts +
                                        static_cast<uint64_t>(h) * hs + 8 * c);
    };
    if constexpr (KIND == kQuery) {
        if (on) *out_row(a.q_out, a.qo_ts, a.qo_hs) = rounded;
        return;
    }
    constexpr bool kIsV = KIND == kValue;
    if constexpr (KV4) {
        __half scale, zero;
        float code[8];
        const bool unsure = quantise(x, turns, from, code, scale, zero);
        for (uint32_t left = __ballot_sync(0xffffffffu, unsure && on); left != 0u;) {
            const int base = (__ffs(left) - 1) & ~3;
            left &= ~(15u << base);
            const Exact exact = requantise<BF16, kChunks>(raw, from, base, a.interleaved, turns, angles, at);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = __shfl_sync(0xffffffffu, exact.t, (lane % 4) * 8 + e);
                if ((lane & ~3) == base) code[e] = t;
            }
            if ((lane & ~3) == base) {
                scale = __ushort_as_half(static_cast<uint16_t>(exact.params));
                zero = __ushort_as_half(static_cast<uint16_t>(exact.params >> 16));
            }
        }
        uint32_t* words = static_cast<uint32_t*>(kIsV ? a.v_pages : a.k_pages) + place * (D / 8);
        if constexpr (!kIsV) {
            // Element e = 2 l + u of the chunk at nibble l + 4 u, so that a word's
            // even and odd elements unpack as 16-bit pairs.
            const uint32_t w = pack_codes(code[0], code[2], code[4], code[6], code[1], code[3], code[5], code[7]);
            if (on) words[(c % 4) * (D / 32) + c / 4] = w;
        } else {
            // Dim 16 j + 8 u + g (chunk 2 j + u, element g) at nibble j of word
            // 2 g + u (D = 128), nibble 4 u + j of word g (D = 64).
            const uint32_t w = pack_codes(code[0], code[1], code[2], code[3], code[4], code[5], code[6], code[7]);
            const uint32_t wt = D == 128 ? transpose_nibbles<2, 4, 8>(w, lane) : transpose_nibbles<2, 4, 1>(w, lane);
            if (on) words[D == 128 ? c : 4 * (c & 1) + c / 2] = wt;
        }
        if (on && c % 4 == 0)
            static_cast<__half2*>(kIsV ? a.v_scales : a.k_scales)[place * (D / 32) + c / 4] = __halves2half2(scale, zero);
        if (a.held) {
            const float s = __half2float(scale), z = __half2float(zero);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                add2(x[e], x[e + 1], code[e], code[e + 1], -kTwo23, -kTwo23);
                fma2(x[e], x[e + 1], x[e], x[e + 1], s, s, z, z);
            }
            rounded = pack8_finite<BF16>(x);
        }
    } else if (on) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(kIsV ? a.v_pages : a.k_pages) + place + 8 * c) = rounded;
    }
    void* out = kIsV ? a.v_out : a.k_out;
    if (on && out != nullptr) *out_row(out, kIsV ? a.vo_ts : a.ko_ts, kIsV ? a.vo_hs : a.ko_hs) = rounded;
}

// The rows of one kind of tokens [first, first + tokens).
template <int D, bool BF16, bool KV4, bool AXES, Kind KIND>
__device__ __forceinline__ void append_block(const AppendArgs& a, Shared<D>& sh, uint32_t first, int tokens) {
    constexpr int kChunks = D / 8;                  // threads per row
    constexpr int kLanes = kThreads / kChunks;      // row lanes of a block
    constexpr bool QUERY = KIND == kQuery;
    const int c = threadIdx.x % kChunks;
    const int rlane = threadIdx.x / kChunks;
    const int rows = QUERY ? a.H : a.Hkv;

    // Items are dealt to the row lanes in turn; from one to a lane's next:
    const int step_tl = kLanes / rows, step_h = kLanes - step_tl * rows;
    auto next = [&](Item& x) {
        x.tl += step_tl;
        x.h += step_h;
        if (x.h >= rows) {
            x.h -= rows;
            ++x.tl;
        }
    };
    // Rows on their way: an item's k and v, or those of two items.
    uint4 raw[2];
    Item ahead, now;
    now.tl = rlane / rows;
    now.h = rlane - now.tl * rows;
    ahead = now;
    auto load = [&](int u) {
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (ahead.tl < tokens) {
            const bool v = KIND == kValue || (KIND == kKeyAndValue && u == 1);
            const uint16_t* src = static_cast<const uint16_t*>(QUERY ? a.q : (v ? a.v : a.k));
            const uint32_t ts = QUERY ? a.q_ts : (v ? a.v_ts : a.k_ts);
            const uint32_t hs = QUERY ? a.q_hs : (v ? a.v_hs : a.k_hs);
            raw[u] = *reinterpret_cast<const uint4*>(src + static_cast<uint64_t>(first + ahead.tl) * ts +
                                                     static_cast<uint64_t>(ahead.h) * hs + 8 * c);
        }
        if (KIND != kKeyAndValue || u == 1) next(ahead);
    };
    load(0);
    load(1);

    // The tokens' places and angles: threads take a token each when nothing
    // turns, else one chunk of one token's angles.
    const bool turn = KIND != kValue && a.rot > 0;
    const int pieces = turn ? a.rot / 8 : 1;
    for (int x = threadIdx.x; x < tokens * pieces; x += kThreads) {
        const int tl = x / pieces, e = x - tl * pieces;
        int64_t slot = a.slots[first + tl];
        const int pos = a.rot > 0 ? a.pos[first + tl] : 0;
        bool outside = a.rot > 0 && (pos < 0 || pos >= a.max_pos);
        if constexpr (AXES) {  // (rot > 0: the launch)
            for (int ax = 1; ax < a.axes; ++ax) {
                const int p = a.pos[ax * a.T + first + tl];
                outside = outside || p < 0 || p >= a.max_pos;
            }
        }
        if (slot >= 0 && (slot >= a.num_slots || outside)) {
            if (e == 0) atomicOr(&g_append_error_word, 1u << kDevErrInvalidArg);
            slot = -1;
        }
        if (e == 0) {
            int64_t place = slot < 0 ? -1 : 0;
            if (slot >= 0 && !QUERY) {  // 32-bit division where it does
                const int64_t page = (slot >> 32) == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page_size)
                                                       : slot / a.page_size;
                const int64_t off = slot - page * a.page_size;
                place = KV4 ? page * a.Hkv * a.page_size + off : page * a.page_stride + off * D;
            }
            sh.place[tl] = place;
        }
        if (slot >= 0 && turn) {
            const int64_t at = static_cast<int64_t>(pos) * (a.rot / 2);
            float4(&cs)[4][kChunks] = sh.cs[tl];
            if constexpr (AXES) {
                // Angle i of the position on its own axis: pairs of a chunk may have
                // several, so each is looked up for itself (once a token and block;
                // 16000 tokens of 32 + 2 * 8 heads, D = 128, three axes 75.5 us, one 74).
                auto angle = [&](int i, float& co, float& si) {
                    const int64_t w = static_cast<int64_t>(a.pos[a.axis[i] * a.T + first + tl]) * (a.rot / 2) + i;
                    co = a.cos[w];
                    si = a.sin[w];
                };
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float co[4], si[4];
                    if (a.interleaved) {
                        angle(4 * e + 2 * u, co[0], si[0]);
                        angle(4 * e + 2 * u + 1, co[2], si[2]);
                        co[1] = co[0], si[1] = si[0], co[3] = co[2], si[3] = si[2];
                        si[0] = -si[0], si[2] = -si[2];
                    } else {
                        const bool second = e >= a.rot / 16;
                        const int i = 8 * (second ? e - a.rot / 16 : e) + 4 * u;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            angle(i + x, co[x], si[x]);
                            if (!second) si[x] = -si[x];
                        }
                    }
                    cs[2 * u][e] = make_float4(co[0], co[1], co[2], co[3]);
                    cs[2 * u + 1][e] = make_float4(si[0], si[1], si[2], si[3]);
                }
            } else if (a.interleaved) {  // pairs 4e .. 4e + 3, each angle for both elements
                const float4 co = *reinterpret_cast<const float4*>(a.cos + at + 4 * e);
                const float4 si = *reinterpret_cast<const float4*>(a.sin + at + 4 * e);
                cs[0][e] = make_float4(co.x, co.x, co.y, co.y);
                cs[1][e] = make_float4(-si.x, si.x, -si.y, si.y);
                cs[2][e] = make_float4(co.z, co.z, co.w, co.w);
                cs[3][e] = make_float4(-si.z, si.z, -si.w, si.w);
            } else {
                const bool second = e >= a.rot / 16;
                const int64_t i = at + 8 * (second ? e - a.rot / 16 : e);
                const float sg = second ? 1.f : -1.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float4 si = *reinterpret_cast<const float4*>(a.sin + i + 4 * u);
                    cs[2 * u][e] = *reinterpret_cast<const float4*>(a.cos + i + 4 * u);
                    cs[2 * u + 1][e] = make_float4(sg * si.x, sg * si.y, sg * si.z, sg * si.w);
                }
            }
        }
    }
    __syncthreads();

    // Every thread of a warp makes the same number of turns (shuffles inside).
    const int turns = (tokens * rows + kLanes - 1) / kLanes;
    const int64_t head = KV4 ? a.page_size : static_cast<int64_t>(a.page_size) * D;  // a head's share of a page
    constexpr int kItems = KIND == kKeyAndValue ? 1 : 2;
    for (int i = 0; i < turns; i += kItems) {
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            if (u > 0 && i + u >= turns) break;
            const int tl = min(now.tl, tokens - 1);
            const int64_t at = sh.place[tl], place = at + now.h * head;
            const uint32_t t = first + tl, h = now.h;
            const bool on = now.tl < tokens && at >= 0;
            const float* angles = reinterpret_cast<const float*>(&sh.cs[0][0][0]);
            const int angle = 16 * kChunks * tl + 4 * c;  // sh.cs[tl][0][c]
            next(now);
            append_row<D, BF16, KV4, KIND == kKeyAndValue ? kKey : KIND>(a, raw[u], t, h, on, place, angles, angle);
            load(u);
            if constexpr (KIND == kKeyAndValue) {
                append_row<D, BF16, KV4, kValue>(a, raw[1], t, h, on, place, angles, angle);
                load(1);
            }
        }
    }
}

// The first blocks take key and value rows (more work each), the rest query
// rows: spread evenly among each other they took 12 us longer at 16000 tokens,
// for the last long blocks start late.
template <int D, bool BF16, bool KV4, bool AXES>
__global__ void __launch_bounds__(kThreads, 5) cache_append_kernel(const __grid_constant__ AppendArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared<D>& sh = *reinterpret_cast<Shared<D>*>(smem);
    grid_dependency();
    const bool query = blockIdx.x >= a.kv_blocks;
    const uint32_t per = query ? a.q_tokens : a.kv_tokens;
    const uint32_t index = query ? blockIdx.x - a.kv_blocks : (a.apart ? blockIdx.x / 2 : blockIdx.x);
    const uint32_t first = index * per;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(per), a.T - first));
    if (query) {
        append_block<D, BF16, KV4, AXES, kQuery>(a, sh, first, tokens);
        return;
    }
    if constexpr (KV4) {
        if (a.apart) {
            if (blockIdx.x % 2 == 0)
                append_block<D, BF16, KV4, AXES, kKey>(a, sh, first, tokens);
            else
                append_block<D, BF16, KV4, AXES, kValue>(a, sh, first, tokens);
            return;
        }
    }
    append_block<D, BF16, KV4, AXES, kKeyAndValue>(a, sh, first, tokens);
}

template <int D, bool BF16>
cudaError_t launch_kind(const AppendArgs& a, bool kv4, unsigned grid, cudaStream_t s) {
    const size_t smem = Shared<D>::bytes(std::max(a.kv_tokens, a.q_tokens));
    if (a.axes > 0)
        return kv4 ? launch_overlapped(cache_append_kernel<D, BF16, true, true>, grid, kThreads, smem, s, a)
                   : launch_overlapped(cache_append_kernel<D, BF16, false, true>, grid, kThreads, smem, s, a);
    return kv4 ? launch_overlapped(cache_append_kernel<D, BF16, true, false>, grid, kThreads, smem, s, a)
               : launch_overlapped(cache_append_kernel<D, BF16, false, false>, grid, kThreads, smem, s, a);
}

}  // namespace

cudaError_t append_launch(AppendArgs a, int D, bool bf16, bool kv4, int sms, cudaStream_t s) {
    // Tokens of a block.  16 bits: as give its threads so many rows that all blocks
    // are on the SMs at once, five each, up to kTurns (8191 tokens of 16 + 2 * 2
    // heads, D = 64: 10.6 us; with a wave and a half of blocks 13.0).  4 bits: as
    // leave three blocks of either kind per SM, as key and value rows take several
    // times as long as query rows (4000 tokens of 32 + 2 * 8 heads 27 us; one wave
    // 34).  A block of key and value rows has one of each per thread at least.
    const int64_t lanes = kThreads / (D / 8), wave = lanes * 5 * sms;
    const int64_t turns = std::min<int64_t>((a.T * (a.H + 2 * a.Hkv) + wave - 1) / wave, kTurns);
    auto tokens = [&](int64_t rows, int64_t least) {
        auto of = [&](int64_t turns) { return std::max<int64_t>(turns * lanes / rows, 1); };
        const int64_t n = kv4 ? std::min(a.T / (3 * sms), of(kTurns)) : of(turns);
        const int64_t most = D == 128 ? Shared<128>::kMaxTokens : Shared<64>::kMaxTokens;
        return static_cast<uint32_t>(std::min(std::max(n, of(least)), most));
    };
    a.kv_tokens = tokens(2 * a.Hkv, 2);
    // Few tokens into 4 bits: one thread's k and then v would take longer than the
    // loads (64 tokens 3.6 -> 3.3 us, 300 6.6 -> 5.7; but 850 9.6 -> 11.1, and 16
    // bits, whose rows take few instructions, 2.4 -> 2.7 at 64).
    a.apart = kv4 && a.T <= 2 * sms;
    a.kv_blocks = static_cast<uint32_t>((a.T + a.kv_tokens - 1) / a.kv_tokens) * (a.apart ? 2u : 1u);
    unsigned grid = a.kv_blocks;
    a.q_tokens = 0;
    if (a.H > 0) {
        a.q_tokens = tokens(a.H, 1);
        grid += static_cast<unsigned>((a.T + a.q_tokens - 1) / a.q_tokens);
    }
    if (D == 128) return bf16 ? launch_kind<128, true>(a, kv4, grid, s) : launch_kind<128, false>(a, kv4, grid, s);
    return bf16 ? launch_kind<64, true>(a, kv4, grid, s) : launch_kind<64, false>(a, kv4, grid, s);
}

cudaError_t append_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_append_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_append_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
