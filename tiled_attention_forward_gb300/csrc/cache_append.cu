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
// value rows, of one or a few tokens; a thread starts the loads of kAhead of
// its rows before the tokens' slots, positions and angles (which depend on one
// another) have come, and the angles go through shared memory once for all
// heads.
//
// Measured (GB300): 8191 tokens of 16 + 2 * 2 heads, D = 64, 16 bits (45 MB) 13
// us, of which about 2.5 are the launch; 16000 tokens of 32 + 2 * 8 heads, D =
// 128, into 4 bits (422 MB with the values held) 106 us, 4.0 TB/s, bound by
// issue slots (about 190 instructions for 16 bytes of a key or value row).  64
// tokens take 2.6 us.  Two rows ahead and five blocks an SM: four ahead cost
// registers (115 us at four blocks), one ahead 110.  16 rows a thread: 8 took 110
// (blocks' starts), 32 the same 106.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace fattn {

// Bit k set <=> a cache kernel found fattn_status k (INVALID_ARG: an index out of range).
__device__ uint32_t g_append_error_word;

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;       // rows that a thread has on their way
constexpr int kTurns = 16;      // rows that a thread takes, where there are enough
constexpr int kMaxTokens = 16;  // tokens of a block
constexpr float kFp16Max = 65504.f;

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
// could not tell that from an error.)  Exact x needs this for the scale alone:
// its quotients are exact ties or well away from one.
__device__ __forceinline__ bool quantise(const float (&x)[8], bool rotated, int partner, float (&t)[8], __half& scale,
                                         __half& zero) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        lo = fminf(lo, x[e]);
        hi = fmaxf(hi, x[e]);
    }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    if (!(lo <= hi)) lo = hi = 0.f;  // nothing but NaN
    lo = fminf(fmaxf(lo, -kFp16Max), kFp16Max);
    hi = fminf(fmaxf(hi, -kFp16Max), kFp16Max);
    const float step = (hi - lo) / 15.f;
    scale = __float2half_rn(step);
    zero = __float2half_rn(lo);
    float most = fmaxf(-lo, hi);
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
    const float inv = s > 0.f ? 1.f / s : 0.f;
    const float top = 15.f * s;  // exact
    float worst = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float d = fminf(fmaxf(x[e] - z, 0.f), top);
        const float q = d * inv;
        const float r = fmaf(fmaf(-q, s, d), inv, q);
        t[e] = __fadd_rn(r, 8388608.f);  // 2^23 +: to the nearest, ties to even
        worst = fmaxf(worst, fabsf(r - __fsub_rn(t[e], 8388608.f)));
    }
    // The quotient's own error: 16 * 2 roundings, and that of x in steps.
    if (rotated) near = near || worst > 0.5f - fmaf(err, inv, 2.0e-6f);
    return near;
}

// The same to twice fp32's precision: values are unevaluated sums h + l of two
// floats, products by fma and sums by the two-sum of Knuth (fp64 would take 10
// times as long on this part).  From the row's raw elements: x the thread's own,
// y their partners, cs as in append_row; turns: whether they turn.  Whole
// groups call it.
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
template <bool BF16, int CHUNKS>
__device__ __noinline__ void requantise(uint4 raw, uint4 other, bool swap, bool turns, const float4* cs, uint32_t group,
                                        float* t, __half* scale, __half* zero) {
    float xf[8], yf[8];
    unpack8<BF16>(raw, xf);
    unpack8<BF16>(other, yf);
    Two x[8], lo = {INFINITY, 0.f}, hi = {-INFINITY, 0.f};
    auto less = [](const Two& a, const Two& b) { return a.h < b.h || (a.h == b.h && a.l < b.l); };
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = {xf[e], 0.f};
        if (turns) {
            const float co = reinterpret_cast<const float*>(cs + (e / 4) * 2 * CHUNKS)[e % 4];
            const float si = reinterpret_cast<const float*>(cs + ((e / 4) * 2 + 1) * CHUNKS)[e % 4];
            const float y = swap ? xf[e ^ 1] : yf[e];
            const float p = __fmul_rn(xf[e], co), q = __fmul_rn(y, si);
            const Two w = two_sum(p, q);
            x[e] = normal(w.h, __fadd_rn(w.l, __fadd_rn(__fmaf_rn(xf[e], co, -p), __fmaf_rn(y, si, -q))));
        }
        if (less(x[e], lo)) lo = x[e];
        if (less(hi, x[e])) hi = x[e];
    }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        const Two a = {__shfl_xor_sync(group, lo.h, m), __shfl_xor_sync(group, lo.l, m)};
        const Two b = {__shfl_xor_sync(group, hi.h, m), __shfl_xor_sync(group, hi.l, m)};
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
    *scale = __float2half_rn(__fadd_rn(q0, __fadd_rn(__fmaf_rn(-q0, 15.f, range.h), range.l) / 15.f));
    *zero = __float2half_rn(lo.h);
    const float s = __half2float(*scale), z = __half2float(*zero);
    const float inv = s > 0.f ? 1.f / s : 0.f, half = 0.5f * s;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // k: the code that fp32 finds; then which side of k +- 1/2 the value is on.
        const Two w = two_sum(x[e].h, -z);
        const float low = __fadd_rn(w.l, x[e].l);
        float k = rintf(fminf(fmaxf(w.h * inv, 0.f), 15.f));
        const float rest = __fmaf_rn(-k, s, w.h);
        const float above = __fadd_rn(__fsub_rn(rest, half), low), below = __fadd_rn(__fadd_rn(rest, half), low);
        const bool odd = (static_cast<int>(k) & 1) != 0;
        if (k < 15.f && (above > 0.f || (above == 0.f && odd && s > 0.f)))
            k += 1.f;
        else if (k > 0.f && (below < 0.f || (below == 0.f && odd && s > 0.f)))
            k -= 1.f;
        t[e] = 8388608.f + (s > 0.f ? k : 0.f);
    }
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

// Where an item (a row of a token) is.
struct Item {
    int tl;  // token within the block
    int r;   // row: a query head, or key heads and then value heads
};

template <int D>
struct Shared {
    static constexpr int kChunks = D / 8;
    int64_t page[kMaxTokens];  // -1: nothing of the token is written
    int off[kMaxTokens];
    // Each token's angles, as the thread of chunk c multiplies by them: cos of
    // its first 4 elements, signed sin of them, then of its other 4.
    float4 cs[kMaxTokens][4][kChunks];
};

// One row's 8 elements: rotation, outputs, cache.  Whole warps call it, with
// lanes that are not `on` repeating some row.
template <int D, bool BF16, bool KV4, bool QUERY>
__device__ __forceinline__ void append_row(const AppendArgs& a, const uint4& raw, uint32_t t, int r, bool on, int64_t page,
                                           int off, const float4* cs) {
    constexpr int kChunks = D / 8;
    const int c = threadIdx.x % kChunks, lane = threadIdx.x % 32;
    const bool is_v = !QUERY && r >= a.Hkv;
    const uint32_t h = is_v ? r - a.Hkv : r;
    uint4 rounded = raw, other = raw;
    bool turns = false;
    int from = lane;  // the lane of this thread's partner elements
    float x[8];
    if (!QUERY || a.rot > 0) unpack8<BF16>(raw, x);
    // Rotation (q and k rows).  Halves: chunk c < rot/16 holds the pairs' first
    // elements, the chunk rot/16 further their second ones, and the sign of a
    // sin - b cos comes with the angles.  Interleaved pairs lie within a chunk.
    if (a.rot > 0 && (QUERY || __any_sync(0xffffffffu, !is_v))) {
        const int half_chunks = a.rot / 16;
        turns = c < 2 * half_chunks && !is_v;
        float y[8];
        if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else {
            from = lane - c + (turns ? (c < half_chunks ? c + half_chunks : c - half_chunks) : c);
            other.x = __shfl_sync(0xffffffffu, raw.x, from);
            other.y = __shfl_sync(0xffffffffu, raw.y, from);
            other.z = __shfl_sync(0xffffffffu, raw.z, from);
            other.w = __shfl_sync(0xffffffffu, raw.w, from);
            unpack8<BF16>(other, y);
        }
        if (turns) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float4 co = cs[(2 * u) * kChunks], si = cs[(2 * u + 1) * kChunks];
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
    if constexpr (QUERY) {
        if (on) *out_row(a.q_out, a.qo_ts, a.qo_hs) = rounded;
        return;
    }
    if constexpr (KV4) {
        __half scale, zero;
        float code[8];
        const uint32_t unsure = __ballot_sync(0xffffffffu, quantise(x, turns, from, code, scale, zero));
        if (unsure != 0u) {
            const uint32_t group = 15u << (lane & ~3);
            if (unsure & group) {
                float exact[8];  // (code itself stays in registers)
                __half es, ez;
                requantise<BF16, kChunks>(raw, other, a.interleaved, turns, cs, group, exact, &es, &ez);
#pragma unroll
                for (int e = 0; e < 8; ++e) code[e] = exact[e];
                scale = es;
                zero = ez;
            }
            __syncwarp();
        }
        const int64_t row = (page * a.Hkv + h) * a.page_size + off;
        if (__any_sync(0xffffffffu, !is_v)) {
            // K: element e = 2 l + u of the chunk at nibble l + 4 u, so that a word's
            // even and odd elements unpack as 16-bit pairs.
            const uint32_t w = pack_codes(code[0], code[2], code[4], code[6], code[1], code[3], code[5], code[7]);
            if (on && !is_v) static_cast<uint32_t*>(a.k_pages)[row * (D / 8) + (c % 4) * (D / 32) + c / 4] = w;
        }
        if (__any_sync(0xffffffffu, is_v)) {
            // V: dim 16 j + 8 u + g (chunk 2 j + u, element g) at nibble j of word
            // 2 g + u (D = 128), nibble 4 u + j of word g (D = 64).
            const uint32_t w = pack_codes(code[0], code[1], code[2], code[3], code[4], code[5], code[6], code[7]);
            const uint32_t wt = D == 128 ? transpose_nibbles<2, 4, 8>(w, lane) : transpose_nibbles<2, 4, 1>(w, lane);
            if (on && is_v) static_cast<uint32_t*>(a.v_pages)[row * (D / 8) + (D == 128 ? c : 4 * (c & 1) + c / 2)] = wt;
        }
        if (on && c % 4 == 0)
            static_cast<__half2*>(is_v ? a.v_scales : a.k_scales)[row * (D / 32) + c / 4] = __halves2half2(scale, zero);
        if (a.held) {
            const float s = __half2float(scale), z = __half2float(zero);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(code[e] - 8388608.f, s, z);
            rounded = pack8<BF16>(x);
        }
    } else if (on) {
        uint16_t* pages = static_cast<uint16_t*>(is_v ? a.v_pages : a.k_pages);
        *reinterpret_cast<uint4*>(pages + page * a.page_stride + (static_cast<int64_t>(h) * a.page_size + off) * D + 8 * c) =
            rounded;
    }
    void* out = is_v ? a.v_out : a.k_out;
    if (on && out != nullptr) *out_row(out, is_v ? a.vo_ts : a.ko_ts, is_v ? a.vo_hs : a.ko_hs) = rounded;
}

// The query rows, or the key and value rows, of tokens [first, first + tokens).
template <int D, bool BF16, bool KV4, bool QUERY>
__device__ __forceinline__ void append_block(const AppendArgs& a, Shared<D>& sh, uint32_t first, int tokens) {
    constexpr int kChunks = D / 8;                  // threads per row
    constexpr int kLanes = kThreads / kChunks;      // rows in flight per block
    const int c = threadIdx.x % kChunks;
    const int rlane = threadIdx.x / kChunks;
    const int rows = QUERY ? a.H : 2 * a.Hkv;

    // Items are dealt to the row lanes in turn; from one to a lane's next:
    const int step_tl = kLanes / rows, step_r = kLanes - step_tl * rows;
    auto next = [&](Item& x) {
        x.tl += step_tl;
        x.r += step_r;
        if (x.r >= rows) {
            x.r -= rows;
            ++x.tl;
        }
    };
    uint4 raw[kAhead];
    Item ahead, now;
    now.tl = rlane / rows;
    now.r = rlane - now.tl * rows;
    ahead = now;
    auto load = [&](int u) {
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (ahead.tl < tokens) {
            const bool is_v = !QUERY && ahead.r >= a.Hkv;
            const uint16_t* src = static_cast<const uint16_t*>(QUERY ? a.q : (is_v ? a.v : a.k));
            const uint32_t ts = QUERY ? a.q_ts : (is_v ? a.v_ts : a.k_ts);
            const uint32_t hs = QUERY ? a.q_hs : (is_v ? a.v_hs : a.k_hs);
            const uint32_t h = is_v ? ahead.r - a.Hkv : ahead.r;
            raw[u] = *reinterpret_cast<const uint4*>(src + static_cast<uint64_t>(first + ahead.tl) * ts +
                                                     static_cast<uint64_t>(h) * hs + 8 * c);
        }
        next(ahead);
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(u);

    // The tokens' places and angles: threads take a token each when nothing
    // turns, else one chunk of one token's angles.
    const int pieces = a.rot > 0 ? a.rot / 8 : 1;
    for (int x = threadIdx.x; x < tokens * pieces; x += kThreads) {
        const int tl = x / pieces, e = x - tl * pieces;
        int64_t slot = a.slots[first + tl];
        const int pos = a.rot > 0 ? a.pos[first + tl] : 0;
        if (slot >= 0 && (slot >= a.num_slots || (a.rot > 0 && (pos < 0 || pos >= a.max_pos)))) {
            if (e == 0) atomicOr(&g_append_error_word, 1u << kDevErrInvalidArg);
            slot = -1;
        }
        if (e == 0) {
            int64_t page = -1;
            int off = 0;
            if (slot >= 0 && !QUERY) {  // 32-bit division where it does
                page = (slot >> 32) == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page_size)
                                         : slot / a.page_size;
                off = static_cast<int>(slot - page * a.page_size);
            }
            sh.page[tl] = QUERY ? (slot < 0 ? -1 : 0) : page;
            sh.off[tl] = off;
        }
        if (slot >= 0 && a.rot > 0) {
            const int64_t at = static_cast<int64_t>(pos) * (a.rot / 2);
            float4(&cs)[4][kChunks] = sh.cs[tl];
            if (a.interleaved) {  // pairs 4e .. 4e + 3, each angle for both elements
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
    for (int i = 0; i < turns; i += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i + u < turns) {
                const int tl = min(now.tl, tokens - 1);
                const int64_t page = sh.page[tl];
                append_row<D, BF16, KV4, QUERY>(a, raw[u], first + tl, now.r, now.tl < tokens && page >= 0, page,
                                                sh.off[tl], &sh.cs[tl][0][c]);
                next(now);
                load(u);
            }
        }
    }
}

// The first blocks take key and value rows (more work each), the rest query rows.
template <int D, bool BF16, bool KV4>
__global__ void __launch_bounds__(kThreads, 5) cache_append_kernel(const __grid_constant__ AppendArgs a) {
    __shared__ Shared<D> sh;
    grid_dependency();
    const bool query = blockIdx.x >= a.kv_blocks;
    const uint32_t per = query ? a.q_tokens : a.kv_tokens;
    const uint32_t first = (query ? blockIdx.x - a.kv_blocks : blockIdx.x) * per;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(per), a.T - first));
    if (query)
        append_block<D, BF16, KV4, true>(a, sh, first, tokens);
    else
        append_block<D, BF16, KV4, false>(a, sh, first, tokens);
}

template <int D, bool BF16>
cudaError_t launch_kind(const AppendArgs& a, bool kv4, unsigned grid, cudaStream_t s) {
    return kv4 ? launch_overlapped(cache_append_kernel<D, BF16, true>, grid, kThreads, 0, s, a)
               : launch_overlapped(cache_append_kernel<D, BF16, false>, grid, kThreads, 0, s, a);
}

}  // namespace

cudaError_t append_launch(AppendArgs a, int D, bool bf16, bool kv4, int sms, cudaStream_t s) {
    // Tokens per block: one while that leaves SMs without a block, then as many
    // as give a block's threads kTurns rows each.
    const int lanes = kThreads / (D / 8);
    auto tokens = [&](int rows) {
        const int64_t most = std::min<int64_t>(std::max(kTurns * lanes / rows, 1), kMaxTokens);
        return static_cast<uint32_t>(std::max<int64_t>(std::min(most, a.T / (3 * sms)), 1));
    };
    a.kv_tokens = tokens(2 * a.Hkv);
    a.kv_blocks = static_cast<uint32_t>((a.T + a.kv_tokens - 1) / a.kv_tokens);
    unsigned grid = a.kv_blocks;
    if (a.H > 0) {
        a.q_tokens = tokens(a.H);
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
