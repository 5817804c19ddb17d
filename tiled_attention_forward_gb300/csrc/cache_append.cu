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
// meet by shuffles within a warp.  A thread keeps its token's cos and sin in
// registers and goes over the token's rows (query heads, key heads, value
// heads), a block per token (or per few tokens, when there are few heads).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace fattn {

// Bit k set <=> a cache kernel found fattn_status k (INVALID_ARG: an index out of range).
__device__ uint32_t g_append_error_word;

namespace {

constexpr int kThreads = 256;
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

// Quantises this thread's 8 elements (4 threads hold a group): the packed
// codes (element e at nibble e), scale and zero; x becomes the values held.
__device__ __forceinline__ uint32_t quantise(float (&x)[8], __half& scale, __half& zero) {
    float lo = kFp16Max, hi = -kFp16Max;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = x[e] > kFp16Max ? kFp16Max : (x[e] < -kFp16Max ? -kFp16Max : x[e]);
        lo = fminf(lo, x[e]);  // a NaN takes no part, and gets code 0 below
        hi = fmaxf(hi, x[e]);
    }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    if (lo > hi) lo = hi = 0.f;  // nothing but NaN
    scale = __float2half_rn((hi - lo) / 15.f);
    zero = __float2half_rn(lo);
    const float s = __half2float(scale), z = __half2float(zero);
    const float inv = s > 0.f ? 1.f / s : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float c = fminf(fmaxf(rintf((x[e] - z) * inv), 0.f), 15.f);
        w |= static_cast<uint32_t>(c) << (4 * e);
        x[e] = fmaf(c, s, z);
    }
    return w;
}

template <int D, bool BF16, bool KV4>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kChunks = D / 8;                  // threads per row
    constexpr int kLanes = kThreads / kChunks;      // rows in flight per block
    const int c = threadIdx.x % kChunks;
    const int rlane = threadIdx.x / kChunks;
    const int lane = threadIdx.x % 32;
    const int rows = a.H + 2 * a.Hkv;
    // Row lanes are dealt to the block's tokens; kLanes / lanes_per_token tokens.
    const int tl = rlane / a.lanes_per_token;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kLanes / a.lanes_per_token) + tl;
    const bool in_range = t < a.T && tl < kLanes / a.lanes_per_token;

    int64_t slot = -1;
    int pos = 0;
    bool live = false;
    if (in_range) {
        slot = a.slots[t];
        pos = a.rot > 0 ? a.pos[t] : 0;
        live = slot >= 0;
        if (live && (slot >= a.num_slots || pos < 0 || (a.rot > 0 && pos >= a.max_pos))) {
            live = false;
            atomicOr(&g_append_error_word, 1u << kDevErrInvalidArg);
        }
    }
    const int64_t page = live ? slot / a.page_size : 0;
    const int off = live ? static_cast<int>(slot - page * a.page_size) : 0;

    // This thread's angles.  Halves: chunk c < rot/16 is the pairs' first
    // halves, the next rot/16 chunks their second ones.
    const int half_chunks = a.rot / 16;
    const bool rotates = c < 2 * half_chunks;
    const bool first = c < half_chunks;
    float co[8], si[8];
    if (live && rotates) {
        const int64_t base = static_cast<int64_t>(pos) * (a.rot / 2);
        if (a.interleaved) {
            const float4 x = *reinterpret_cast<const float4*>(a.cos + base + 4 * c);
            const float4 y = *reinterpret_cast<const float4*>(a.sin + base + 4 * c);
            co[0] = x.x; co[2] = x.y; co[4] = x.z; co[6] = x.w;
            si[0] = y.x; si[2] = y.y; si[4] = y.z; si[6] = y.w;
        } else {
            const int64_t i = base + 8 * (first ? c : c - half_chunks);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 x = *reinterpret_cast<const float4*>(a.cos + i + e);
                const float4 y = *reinterpret_cast<const float4*>(a.sin + i + e);
                co[e] = x.x; co[e + 1] = x.y; co[e + 2] = x.z; co[e + 3] = x.w;
                // b' = b cos + a sin, a' = a cos - b sin: the sign goes into sin
                const float sg = first ? -1.f : 1.f;
                si[e] = sg * y.x; si[e + 1] = sg * y.y; si[e + 2] = sg * y.z; si[e + 3] = sg * y.w;
            }
        }
    }
    const int partner = first ? c + half_chunks : c - half_chunks;
    const int partner_lane = (lane & ~(kChunks - 1)) + (rotates ? partner : c);

    // Every thread of a warp makes the same number of turns (shuffles below).
    const int turns = (rows + a.lanes_per_token - 1) / a.lanes_per_token;
    for (int it = 0; it < turns; ++it) {
        const int r = (rlane % a.lanes_per_token) + it * a.lanes_per_token;
        const bool is_q = r < a.H;
        const bool is_k = !is_q && r < a.H + a.Hkv;
        const int h = is_q ? r : (is_k ? r - a.H : r - a.H - a.Hkv);
        const bool on = live && r < rows && !(is_q && a.q == nullptr);
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (on) {
            const uint16_t* src = static_cast<const uint16_t*>(is_q ? a.q : (is_k ? a.k : a.v));
            const int64_t ts = is_q ? a.q_ts : (is_k ? a.k_ts : a.v_ts);
            const int64_t hs = is_q ? a.q_hs : (is_k ? a.k_hs : a.v_hs);
            raw = *reinterpret_cast<const uint4*>(src + t * ts + h * hs + 8 * c);
        }
        float x[8];
        unpack8<BF16>(raw, x);
        // Rotation (q and k rows).  Products and sums rounded one by one.
        if (a.rot > 0) {
            if (a.interleaved) {
                if (rotates && (is_q || is_k) && live) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float p = x[e], q = x[e + 1];
                        x[e] = __fsub_rn(__fmul_rn(p, co[e]), __fmul_rn(q, si[e]));
                        x[e + 1] = __fadd_rn(__fmul_rn(q, co[e]), __fmul_rn(p, si[e]));
                    }
                }
            } else {
                float y[8];
                uint4 other;
                other.x = __shfl_sync(0xffffffffu, raw.x, partner_lane);
                other.y = __shfl_sync(0xffffffffu, raw.y, partner_lane);
                other.z = __shfl_sync(0xffffffffu, raw.z, partner_lane);
                other.w = __shfl_sync(0xffffffffu, raw.w, partner_lane);
                unpack8<BF16>(other, y);
                if (rotates && (is_q || is_k) && live) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = __fadd_rn(__fmul_rn(x[e], co[e]), __fmul_rn(y[e], si[e]));
                }
            }
        }
        uint4 rounded = (is_q || is_k) && a.rot > 0 ? pack8<BF16>(x) : raw;
        if (on && is_q && a.q_out != nullptr)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + t * a.qo_ts + h * a.qo_hs + 8 * c) = rounded;
        uint32_t w = 0;
        __half scale = __float2half_rn(0.f), zero = scale;
        if (KV4) {
            w = quantise(x, scale, zero);
            // K: element e = 2 l + u of the chunk at nibble l + 4 u, so that a
            // word's even and odd elements unpack as 16-bit pairs.
            uint32_t wk = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) wk |= ((w >> (4 * e)) & 15u) << (4 * (e / 2 + 4 * (e & 1)));
            // V: dim 16 j + 8 u + g (chunk 2 j + u, element g) at nibble j of
            // word 2 g + u (D = 128), nibble 4 u + j of word g (D = 64).
            const uint32_t wv = D == 128 ? transpose_nibbles<2, 4, 8>(w, lane) : transpose_nibbles<2, 4, 1>(w, lane);
            const int word = is_k ? (c % 4) * (D / 32) + c / 4 : (D == 128 ? c : 4 * (c & 1) + c / 2);
            if (on && !is_q) {
                const int64_t row = (page * a.Hkv + h) * a.page_size + off;
                uint32_t* codes = static_cast<uint32_t*>(is_k ? a.k_pages : a.v_pages);
                codes[row * (D / 8) + word] = is_k ? wk : wv;
                if (c % 4 == 0) {
                    __half2* meta = static_cast<__half2*>(is_k ? a.k_scales : a.v_scales);
                    meta[row * (D / 32) + c / 4] = __halves2half2(scale, zero);
                }
            }
            if (a.held) rounded = pack8<BF16>(x);
        } else if (on && !is_q) {
            uint16_t* pages = static_cast<uint16_t*>(is_k ? a.k_pages : a.v_pages);
            *reinterpret_cast<uint4*>(pages + page * a.page_stride + (static_cast<int64_t>(h) * a.page_size + off) * D +
                                      8 * c) = rounded;
        }
        if (on && is_k && a.k_out != nullptr)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_out) + t * a.ko_ts + h * a.ko_hs + 8 * c) = rounded;
        if (on && !is_q && !is_k && a.v_out != nullptr)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_out) + t * a.vo_ts + h * a.vo_hs + 8 * c) = rounded;
    }
}

template <int D, bool BF16>
cudaError_t launch_kind(const AppendArgs& a, bool kv4, unsigned grid, cudaStream_t s) {
    if (kv4)
        cache_append_kernel<D, BF16, true><<<grid, kThreads, 0, s>>>(a);
    else
        cache_append_kernel<D, BF16, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t append_launch(AppendArgs a, int D, bool bf16, bool kv4, cudaStream_t s) {
    const int lanes = kThreads / (D / 8);
    const int rows = a.H + 2 * a.Hkv;
    // Lanes per token: a power of two (so that tokens split the block's lanes
    // evenly), enough for every row at once where a block has that many.
    int per = lanes;
    while (per > 1 && per / 2 >= rows) per /= 2;
    a.lanes_per_token = per;
    const int64_t tokens = lanes / per;
    const unsigned grid = static_cast<unsigned>((a.T + tokens - 1) / tokens);
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
