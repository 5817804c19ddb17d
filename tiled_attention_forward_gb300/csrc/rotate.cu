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
// between threads, and the rows of kAtOnce heads are on their way at once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace fattn {
namespace {

__device__ uint32_t g_rotate_error_word;

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;  // heads whose rows are on their way

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
// u[2e] with u[2e+1] by angle e and v's by angle 4 + e.
template <bool BF16, bool INTERLEAVED>
__device__ __forceinline__ void turn(uint4& p, uint4& q, const float (&co)[8], const float (&si)[8]) {
    float u[8], v[8], x[8], y[8];
    unpack<BF16>(p, u);
    unpack<BF16>(q, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (INTERLEAVED) {
            const float sg = (e & 1) ? 1.f : -1.f;
            x[e] = fmaf(u[e ^ 1], sg * si[e / 2], u[e] * co[e / 2]);
            y[e] = fmaf(v[e ^ 1], sg * si[4 + e / 2], v[e] * co[4 + e / 2]);
        } else {
            x[e] = fmaf(-v[e], si[e], u[e] * co[e]);
            y[e] = fmaf(u[e], si[e], v[e] * co[e]);
        }
    }
    p = pack<BF16>(x);
    q = pack<BF16>(y);
}

template <int D, bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a) {
    constexpr int kLanes = D / 16;             // threads of a token
    constexpr int kTokens = kThreads / kLanes;  // tokens of a block
    const int p = threadIdx.x % kLanes;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / kLanes;
    grid_dependency();
    if (token >= a.tokens) return;
    for (int ax = 0; ax < a.axes; ++ax) {
        const int at = a.pos[ax * a.tokens + token];
        if (at < 0 || at >= a.max_pos) {  // the token's rows are left as they were
            if (p == 0 && blockIdx.y == 0) atomicOr(&g_rotate_error_word, 1u << kDevErrInvalidArg);
            return;
        }
    }
    const bool turns = p < a.rot / 16;
    float co[8], si[8];
    if (turns) {
        const uint64_t which = *reinterpret_cast<const uint64_t*>(a.axis + 8 * p);
        if (which == (which & 0xffull) * 0x0101010101010101ull) {  // all on one axis
            const int64_t at = static_cast<int64_t>(a.pos[(which & 0xffull) * a.tokens + token]) * (a.rot / 2) + 8 * p;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float4 c = *reinterpret_cast<const float4*>(a.cos + at + 4 * u);
                const float4 s = *reinterpret_cast<const float4*>(a.sin + at + 4 * u);
                co[4 * u] = c.x, co[4 * u + 1] = c.y, co[4 * u + 2] = c.z, co[4 * u + 3] = c.w;
                si[4 * u] = s.x, si[4 * u + 1] = s.y, si[4 * u + 2] = s.z, si[4 * u + 3] = s.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t row = a.pos[((which >> (8 * e)) & 0xffull) * a.tokens + token];
                co[e] = a.cos[row * (a.rot / 2) + 8 * p + e];
                si[e] = a.sin[row * (a.rot / 2) + 8 * p + e];
            }
        }
        if (a.inverse) {
#pragma unroll
            for (int e = 0; e < 8; ++e) si[e] = -si[e];
        }
    }
    // The two pieces of a row: partners where it turns in halves, else neighbours.
    const int first = turns && !INTERLEAVED ? 8 * p : 16 * p;
    const int apart = turns && !INTERLEAVED ? a.rot / 2 : 8;
    const int64_t b = token / a.N, n = token - b * a.N;
    // This block's heads, numbered over q and k.
    const int all = a.heads[0] + a.heads[1];
    const int per = (all + gridDim.y - 1) / gridDim.y;
    const int begin = blockIdx.y * per, end = min(all, begin + per);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int from = max(begin - (t ? a.heads[0] : 0), 0), to = min(end - (t ? a.heads[0] : 0), a.heads[t]);
        const uint16_t* x = static_cast<const uint16_t*>(a.x[t]) + b * a.x_bs[t] + n * a.x_ns[t] + first;
        uint16_t* y = static_cast<uint16_t*>(a.y[t]) + b * a.y_bs[t] + n * a.y_ns[t] + first;
        for (int h0 = from; h0 < to; h0 += kAtOnce) {
            uint4 u[kAtOnce], v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (h0 + i >= to) break;
                const uint16_t* src = x + (h0 + i) * a.x_hs[t];
                u[i] = __ldcs(reinterpret_cast<const uint4*>(src));
                v[i] = __ldcs(reinterpret_cast<const uint4*>(src + apart));
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (h0 + i >= to) break;
                if (turns) turn<BF16, INTERLEAVED>(u[i], v[i], co, si);
                uint16_t* dst = y + (h0 + i) * a.y_hs[t];
                *reinterpret_cast<uint4*>(dst) = u[i];
                *reinterpret_cast<uint4*>(dst + apart) = v[i];
            }
        }
    }
}

template <int D, bool BF16>
cudaError_t launch_one(const RotateArgs& a, int sms, cudaStream_t s) {
    const int64_t blocks = (a.tokens + kThreads / (D / 16) - 1) / (kThreads / (D / 16));
    // Heads are dealt to so many blocks that there are four a SM, a turn's rows at least each.
    const int heads = a.heads[0] + a.heads[1];
    int64_t parts = (4 * sms + blocks - 1) / blocks;
    const int64_t most = (heads + kAtOnce - 1) / kAtOnce;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
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
