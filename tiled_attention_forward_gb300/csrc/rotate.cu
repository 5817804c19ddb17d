// rotate.cu -- rotation of queries and keys by positions with several axes (time,
// height and width of image and video tokens), and its gradient.
//
// A row x of a token, over its first `rot` elements: the pair (a, b) with angle
// index i = 0 .. rot/2 - 1, (x[i], x[i + rot/2]) or (x[2i], x[2i+1]), becomes
//     a' = a cos - b sin,   b' = b cos + a sin,
// cos and sin at row pos[axis[i]] of the tables, column i.  The matrix is
// orthogonal: the gradient is the same with -sin.
//
// Bound by memory (2 x 2 bytes an element, three fp32 operations).  A thread has
// eight pairs of a token, 16 elements in two 16-byte pieces, for a number of
// heads: the angles are read once and stay in registers, nothing is exchanged
// between threads, and the rows of kAtOnce heads are on their way at once.  Which
// pieces a thread has is chosen such that neighbours have neighbouring ones
// (interleaved pairs by 32 bytes a thread took 62.5 us where these take 58).
//
// Measured (GB300): 2 x 8192 tokens of 32 + 8 heads, D = 128, from a projection into
// dense tensors (344 MB), 56 us = 6.1 TB/s; 4 x 1000 tokens of 16 + 16 heads, D = 64,
// 8.0 us, 17 tokens 3.1, which is the launch.  Two heads at once and eight blocks of
// 128 threads an SM: four heads and three blocks of 256 took 57.6 and 9.3 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace fattn {
namespace {

__device__ uint32_t g_rotate_error_word;

constexpr int kThreads = 128;
constexpr int kBlocksPerSm = 8;
constexpr int kAtOnce = 2;  // heads whose rows are on their way

template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& r, float (&x)[8]) {
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
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
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

// The two pieces of a row turn: halves, u[e] with v[e] by angle e; interleaved,
// each piece by itself, u[2e] with u[2e+1] by angle e and v's by angle 4 + e.
template <bool BF16>
__device__ __forceinline__ void turn_halves(uint4& p, uint4& q, const float (&co)[8], const float (&si)[8]) {
    float u[8], v[8], x[8], y[8];
    unpack<BF16>(p, u);
    unpack<BF16>(q, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = fmaf(-v[e], si[e], u[e] * co[e]);
        y[e] = fmaf(u[e], si[e], v[e] * co[e]);
    }
    p = pack<BF16>(x);
    q = pack<BF16>(y);
}
template <bool BF16>
__device__ __forceinline__ void turn_pairs(uint4& p, const float* co, const float* si) {
    float u[8], x[8];
    unpack<BF16>(p, u);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        x[e] = fmaf(-u[e + 1], si[e / 2], u[e] * co[e / 2]);
        x[e + 1] = fmaf(u[e], si[e / 2], u[e + 1] * co[e / 2]);
    }
    p = pack<BF16>(x);
}

template <int D, bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) rotate_kernel(const __grid_constant__ RotateArgs a) {
    constexpr int kLanes = D / 16;             // threads of a token
    constexpr int kTokens = kThreads / kLanes;  // tokens of a block
    const int p = threadIdx.x % kLanes;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / kLanes;
    grid_dependency();
    if (token >= a.tokens) return;
    // The two pieces of a row that this thread has, such that a token's threads have
    // neighbouring ones.  Halves: partners, or two that do not turn.  Interleaved:
    // any two, each of which turns or not.
    const int half = a.rot / 16;
    const bool turns = INTERLEAVED ? p < 2 * half : p < half;  // the first piece
    const bool second_turns = INTERLEAVED ? p + kLanes < 2 * half : turns;
    const int first = INTERLEAVED || turns ? 8 * p : 8 * (half + p);
    const int apart = INTERLEAVED ? 8 * kLanes : (turns ? 8 * half : 8 * (kLanes - half));
    const int64_t b = token / a.N, n = token - b * a.N;
    // This block's heads, numbered over q and k.
    const int all = a.heads[0] + a.heads[1];
    const int per = ((all + gridDim.y - 1) / gridDim.y + kAtOnce - 1) / kAtOnce * kAtOnce;
    const int begin = blockIdx.y * per, end = min(all, begin + per);
    auto row_of = [&](int h, void* const (&p)[2], const int64_t (&bs)[2], const int64_t (&hs)[2], const int64_t (&ns)[2]) {
        const int k = h >= a.heads[0];
        return static_cast<uint16_t*>(p[k]) + b * bs[k] + n * ns[k] + (h - (k ? a.heads[0] : 0)) * hs[k] + first;
    };
    // Their first rows are on their way before the token's positions and angles,
    // which depend on one another, have come.
    uint4 u[kAtOnce], v[kAtOnce];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint16_t* src = row_of(min(h0 + i, end - 1), a.x, a.x_bs, a.x_hs, a.x_ns);
            u[i] = __ldcs(reinterpret_cast<const uint4*>(src));
            v[i] = __ldcs(reinterpret_cast<const uint4*>(src + apart));
        }
    };
    if (begin >= end) return;
    load(begin);
    bool outside = false;
    for (int ax = 0; ax < a.axes; ++ax) {
        const int at = a.pos[ax * a.tokens + token];
        outside = outside || at < 0 || at >= a.max_pos;
    }
    if (outside) {  // the token's rows are left as they were
        if (p == 0 && blockIdx.y == 0) atomicOr(&g_rotate_error_word, 1u << kDevErrInvalidArg);
        return;
    }
    // Angles: of pairs 8p .. 8p + 7, or interleaved of each piece's four.
    float co[8], si[8];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int i0 = INTERLEAVED ? 4 * p + g * 4 * kLanes : 8 * p + 4 * g;
        if (!(g == 0 ? turns : second_turns)) continue;
        const uint32_t which = *reinterpret_cast<const uint32_t*>(a.axis + i0);
        float4 c, s;
        if (which == (which & 0xffu) * 0x01010101u) {  // all on one axis
            const int64_t at = static_cast<int64_t>(a.pos[(which & 0xffu) * a.tokens + token]) * (a.rot / 2) + i0;
            c = *reinterpret_cast<const float4*>(a.cos + at);
            s = *reinterpret_cast<const float4*>(a.sin + at);
        } else {
            int64_t at[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                at[e] = static_cast<int64_t>(a.pos[((which >> (8 * e)) & 0xffu) * a.tokens + token]) * (a.rot / 2) + i0 + e;
            c = make_float4(a.cos[at[0]], a.cos[at[1]], a.cos[at[2]], a.cos[at[3]]);
            s = make_float4(a.sin[at[0]], a.sin[at[1]], a.sin[at[2]], a.sin[at[3]]);
        }
        const float sg = a.inverse ? -1.f : 1.f;
        co[4 * g] = c.x, co[4 * g + 1] = c.y, co[4 * g + 2] = c.z, co[4 * g + 3] = c.w;
        si[4 * g] = sg * s.x, si[4 * g + 1] = sg * s.y, si[4 * g + 2] = sg * s.z, si[4 * g + 3] = sg * s.w;
    }
    for (int h0 = begin; h0 < end; h0 += kAtOnce) {
        if (h0 > begin) load(h0);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (h0 + i >= end) break;
            if constexpr (INTERLEAVED) {
                if (turns) turn_pairs<BF16>(u[i], co, si);
                if (second_turns) turn_pairs<BF16>(v[i], co + 4, si + 4);
            } else if (turns) {
                turn_halves<BF16>(u[i], v[i], co, si);
            }
            uint16_t* dst = row_of(h0 + i, a.y, a.y_bs, a.y_hs, a.y_ns);
            *reinterpret_cast<uint4*>(dst) = u[i];
            *reinterpret_cast<uint4*>(dst + apart) = v[i];
        }
    }
}

template <int D, bool BF16>
cudaError_t launch_one(const RotateArgs& a, int sms, cudaStream_t s) {
    const int64_t blocks = (a.tokens + kThreads / (D / 16) - 1) / (kThreads / (D / 16));
    // Heads are dealt to so many blocks that the waves of blocks, each as long as its
    // heads and two turns more (the angles), are shortest; two parts also where they
    // take an eighth more than one, as their starts spread out (rotation of the 2 x
    // 8192 tokens above: 56.1 us, one part 58.0).
    const int heads = a.heads[0] + a.heads[1];
    const int64_t wave = static_cast<int64_t>(kBlocksPerSm) * sms;
    int64_t parts = 1, least = INT64_MAX;
    for (int64_t p = 1; p <= (heads + kAtOnce - 1) / kAtOnce && p <= 64; ++p) {
        const int64_t per = (heads + p - 1) / p, turns = (per + kAtOnce - 1) / kAtOnce + 2;
        const int64_t cost = (blocks * p + wave - 1) / wave * turns;
        if (cost < least || (p == 2 && 8 * cost <= 9 * least)) {
            least = cost;
            parts = p;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, a.interleaved ? rotate_kernel<D, BF16, true> : rotate_kernel<D, BF16, false>, a);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

}  // namespace

cudaError_t rotate_launch(const RotateArgs& a, int D, bool bf16, int sms, cudaStream_t s) {
    if (D == 128) return bf16 ? launch_one<128, true>(a, sms, s) : launch_one<128, false>(a, sms, s);
    return bf16 ? launch_one<64, true>(a, sms, s) : launch_one<64, false>(a, sms, s);
}

cudaError_t rotate_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_rotate_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_rotate_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
