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
// meet by shuffles within a warp.  A block takes the rows (query heads, key
// heads, value heads) of one or a few tokens; a thread starts the loads of
// kAhead of its rows before the tokens' slots, positions and angles (which
// depend on one another) have come, and the angles go through shared memory
// once for all heads.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace fattn {

// Bit k set <=> a cache kernel found fattn_status k (INVALID_ARG: an index out of range).
__device__ uint32_t g_append_error_word;

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;       // rows that a thread has on their way
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

// Four codes (floats 0..15) as 16 bits, nibble by nibble: exact in fp32.
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
    return static_cast<uint32_t>(fmaf(d, 4096.f, fmaf(c, 256.f, fmaf(b, 16.f, a))));
}

// Quantises this thread's 8 elements (4 threads hold a group): its codes,
// scale and zero.
__device__ __forceinline__ void quantise(const float (&x)[8], float (&code)[8], __half& scale, __half& zero) {
    float y[8];
    float lo = kFp16Max, hi = -kFp16Max;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        y[e] = x[e] > kFp16Max ? kFp16Max : (x[e] < -kFp16Max ? -kFp16Max : x[e]);
        lo = fminf(lo, y[e]);  // a NaN takes no part, and gets code 0 below
        hi = fmaxf(hi, y[e]);
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
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // Adding 2^23 rounds to the nearest whole number, ties to even.
        const float c = fminf(fmaxf((y[e] - z) * inv, 0.f), 15.f);
        code[e] = __fsub_rn(__fadd_rn(c, 8388608.f), 8388608.f);
    }
}

// One row's 8 elements: rotation, outputs, cache.  Whole warps call it.
template <int D, bool BF16, bool KV4>
__device__ __forceinline__ void append_row(const AppendArgs& a, const uint4& raw, int64_t t, int r, bool on, int64_t page, int off,
                                           const float* cs) {
    constexpr int kChunks = D / 8;
    const int c = threadIdx.x % kChunks, lane = threadIdx.x % 32;
    const bool is_q = r < a.H;
    const bool is_k = !is_q && r < a.H + a.Hkv;
    const bool is_v = !is_q && !is_k;
    const int h = is_q ? r : (is_k ? r - a.H : r - a.H - a.Hkv);
    float x[8];
    unpack8<BF16>(raw, x);
    // Rotation (q and k rows): the pair's first half is chunk c < rot/16, its
    // second the chunk rot/16 further; interleaved pairs lie within a chunk.
    // Products and sums are rounded one by one.
    const int half_chunks = a.rot / 16;
    const bool turns = c < 2 * half_chunks && !is_v;
    if (a.rot > 0) {
        const float* sn = cs + a.rot / 2;
        if (a.interleaved) {
            if (turns) {
                const float4 co = *reinterpret_cast<const float4*>(cs + 4 * c);
                const float4 si = *reinterpret_cast<const float4*>(sn + 4 * c);
                const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = x[2 * e], q = x[2 * e + 1];
                    x[2 * e] = __fsub_rn(__fmul_rn(p, cv[e]), __fmul_rn(q, sv[e]));
                    x[2 * e + 1] = __fadd_rn(__fmul_rn(q, cv[e]), __fmul_rn(p, sv[e]));
                }
            }
        } else {
            const bool first = c < half_chunks;
            const int partner = turns ? (first ? c + half_chunks : c - half_chunks) : c;
            const int from = (lane & ~(kChunks - 1)) + partner;
            uint4 other;
            other.x = __shfl_sync(0xffffffffu, raw.x, from);
            other.y = __shfl_sync(0xffffffffu, raw.y, from);
            other.z = __shfl_sync(0xffffffffu, raw.z, from);
            other.w = __shfl_sync(0xffffffffu, raw.w, from);
            if (turns) {
                float y[8];
                unpack8<BF16>(other, y);
                const int i = 8 * (first ? c : c - half_chunks);
                const float sg = first ? -1.f : 1.f;  // a' = a cos - b sin, b' = b cos + a sin
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 co = *reinterpret_cast<const float4*>(cs + i + e);
                    const float4 si = *reinterpret_cast<const float4*>(sn + i + e);
                    const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        x[e + u] = __fadd_rn(__fmul_rn(x[e + u], cv[u]), __fmul_rn(y[e + u], sg * sv[u]));
                }
            }
        }
    }
    uint4 rounded = turns ? pack8<BF16>(x) : raw;
    if (on && is_q) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + t * a.qo_ts + h * a.qo_hs + 8 * c) = rounded;
    // What follows is for key and value rows: query rows are most of them, and
    // whole warps of them leave here.
    if (!__any_sync(0xffffffffu, on && !is_q)) return;
    const bool kv = on && !is_q;
    if constexpr (KV4) {
        __half scale, zero;
        float code[8];
        quantise(x, code, scale, zero);
        const int64_t row = (page * a.Hkv + h) * a.page_size + off;
        if (__any_sync(0xffffffffu, is_k)) {
            // K: element e = 2 l + u of the chunk at nibble l + 4 u, so that a word's
            // even and odd elements unpack as 16-bit pairs.
            const uint32_t w = pack_codes(code[0], code[2], code[4], code[6]) |
                               (pack_codes(code[1], code[3], code[5], code[7]) << 16);
            if (kv && is_k) static_cast<uint32_t*>(a.k_pages)[row * (D / 8) + (c % 4) * (D / 32) + c / 4] = w;
        }
        if (__any_sync(0xffffffffu, is_v)) {
            // V: dim 16 j + 8 u + g (chunk 2 j + u, element g) at nibble j of word
            // 2 g + u (D = 128), nibble 4 u + j of word g (D = 64).
            const uint32_t w = pack_codes(code[0], code[1], code[2], code[3]) |
                               (pack_codes(code[4], code[5], code[6], code[7]) << 16);
            const uint32_t wt = D == 128 ? transpose_nibbles<2, 4, 8>(w, lane) : transpose_nibbles<2, 4, 1>(w, lane);
            if (kv && is_v) static_cast<uint32_t*>(a.v_pages)[row * (D / 8) + (D == 128 ? c : 4 * (c & 1) + c / 2)] = wt;
        }
        if (kv && c % 4 == 0)
            static_cast<__half2*>(is_k ? a.k_scales : a.v_scales)[row * (D / 32) + c / 4] = __halves2half2(scale, zero);
        if (a.held) {
            const float s = __half2float(scale), z = __half2float(zero);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(code[e], s, z);
            rounded = pack8<BF16>(x);
        }
    } else if (kv) {
        uint16_t* pages = static_cast<uint16_t*>(is_k ? a.k_pages : a.v_pages);
        *reinterpret_cast<uint4*>(pages + page * a.page_stride + (static_cast<int64_t>(h) * a.page_size + off) * D + 8 * c) =
            rounded;
    }
    if (kv && is_k && a.k_out != nullptr)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_out) + t * a.ko_ts + h * a.ko_hs + 8 * c) = rounded;
    if (kv && is_v && a.v_out != nullptr)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_out) + t * a.vo_ts + h * a.vo_hs + 8 * c) = rounded;
}

template <int D, bool BF16, bool KV4>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kChunks = D / 8;                  // threads per row
    constexpr int kLanes = kThreads / kChunks;      // rows in flight per block
    __shared__ int64_t s_page[kMaxTokens];          // -1: nothing of the token is written
    __shared__ int s_off[kMaxTokens];
    __shared__ __align__(16) float s_cs[kMaxTokens][D];  // cos, then sin, of the tokens' positions
    const int c = threadIdx.x % kChunks;
    const int rlane = threadIdx.x / kChunks;
    const int rows = a.H + 2 * a.Hkv;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * a.tokens;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tokens), a.T - first));
    const int items = tokens * rows;

    uint4 raw[kAhead];
    auto load = [&](int u, int item) {
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (item < items) {
            const int tl = item / rows, r = item - tl * rows;
            const int64_t t = first + tl;
            const uint16_t* src;
            if (r < a.H)
                src = static_cast<const uint16_t*>(a.q) + t * a.q_ts + r * a.q_hs;
            else if (r < a.H + a.Hkv)
                src = static_cast<const uint16_t*>(a.k) + t * a.k_ts + (r - a.H) * a.k_hs;
            else
                src = static_cast<const uint16_t*>(a.v) + t * a.v_ts + (r - a.H - a.Hkv) * a.v_hs;
            raw[u] = *reinterpret_cast<const uint4*>(src + 8 * c);
        }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(u, rlane + u * kLanes);

    // The tokens' angles: as many threads as fit take a token each (a warp or
    // more for one token when there are few).
    const int quarter = a.rot / 4;  // 16-byte pieces of a token's angles (cos and sin)
    for (int x = threadIdx.x; x < tokens * max(quarter, 1); x += kThreads) {
        const int tl = quarter > 0 ? x / quarter : x, e = quarter > 0 ? x - tl * quarter : 0;
        int64_t slot = a.slots[first + tl];
        const int pos = a.rot > 0 ? a.pos[first + tl] : 0;
        if (slot >= 0 && (slot >= a.num_slots || (a.rot > 0 && (pos < 0 || pos >= a.max_pos)))) {
            if (e == 0) atomicOr(&g_append_error_word, 1u << kDevErrInvalidArg);
            slot = -1;
        }
        if (e == 0) {
            const int64_t page = slot < 0 ? -1 : slot / a.page_size;
            s_page[tl] = page;
            s_off[tl] = slot < 0 ? 0 : static_cast<int>(slot - page * a.page_size);
        }
        if (slot >= 0 && quarter > 0) {
            const float* table = e < quarter / 2 ? a.cos : a.sin;
            const int at = 4 * (e < quarter / 2 ? e : e - quarter / 2);
            *reinterpret_cast<float4*>(&s_cs[tl][4 * e]) =
                *reinterpret_cast<const float4*>(table + static_cast<int64_t>(pos) * (a.rot / 2) + at);
        }
    }
    __syncthreads();

    // Every thread of a warp makes the same number of turns (shuffles inside).
    for (int i = 0; i < items; i += kAhead * kLanes) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int item = i + u * kLanes + rlane;
            if (i + u * kLanes < items) {
                const int tl = min(item / rows, tokens - 1), r = item - tl * rows;
                const int64_t page = s_page[tl];
                append_row<D, BF16, KV4>(a, raw[u], first + tl, min(r, rows - 1), item < items && page >= 0, page,
                                         s_off[tl], s_cs[tl]);
                load(u, item + kAhead * kLanes);
            }
        }
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

cudaError_t append_launch(AppendArgs a, int D, bool bf16, bool kv4, int sms, cudaStream_t s) {
    // Tokens per block: one while that leaves SMs without a block, then as many
    // as give a block's threads kAhead rows each.
    const int lanes = kThreads / (D / 8);
    const int rows = a.H + 2 * a.Hkv;
    int tokens = (kAhead * lanes + rows - 1) / rows;
    tokens = std::min(std::min(tokens, kMaxTokens), static_cast<int>((a.T + 4 * sms - 1) / (4 * sms)));
    a.tokens = std::max(tokens, 1);
    const unsigned grid = static_cast<unsigned>((a.T + a.tokens - 1) / a.tokens);
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
