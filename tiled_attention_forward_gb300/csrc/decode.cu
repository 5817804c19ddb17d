// decode.cu -- attention of the newest tokens of each sequence over a paged
// cache held in 16 or in 4 bits.
//
// Simple form: a block per (sequence, query row), whose four warps take the
// visible keys in turn, a lane per D/32 dims, each warp with its own running
// max and sum (online softmax), joined in shared memory at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace fattn {

__device__ uint32_t g_decode_error_word;

namespace {

constexpr float kLn2 = 0.6931471805599453f;

template <bool BF16>
__device__ __forceinline__ float load16(const void* p, int64_t i) {
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    if (BF16) return __uint_as_float(static_cast<uint32_t>(u) << 16);
    return __half2float(__ushort_as_half(u));
}

template <int D, bool BF16, bool KV4>
__global__ void __launch_bounds__(128) decode_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int E = D / 32;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int h = blockIdx.x / a.Nq, i = blockIdx.x % a.Nq, b = blockIdx.y;
    const int kvh = h / (a.H / a.Hkv);
    int64_t len = a.seq_lens[b];
    if (len < 0 || len > a.table_width * a.page_size) {
        if (threadIdx.x == 0) atomicOr(&g_decode_error_word, 1u << kDevErrInvalidArg);
        len = len < 0 ? 0 : a.table_width * a.page_size;
    }
    const int64_t end = len - a.Nq + i + 1;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = load16<BF16>(a.q, b * a.q_bs + h * a.q_hs + i * a.q_ns + lane * E + e) * a.scale_log2;
        o[e] = 0.f;
    }
    for (int64_t j = warp; j < end; j += 4) {
        const int64_t page = a.block_table[b * a.table_width + j / a.page_size];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(&g_decode_error_word, 1u << kDevErrInvalidArg);
            continue;
        }
        const int64_t in_page = static_cast<int64_t>(kvh) * a.page_size + j % a.page_size;
        float k[E], v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = lane * E + e;
            if (KV4) {
                const int64_t row = page * a.Hkv * a.page_size + in_page;
                const int nk = 8 * ((d % 32) / 8 * (D / 32) + d / 32) + (d % 8) / 2 + 4 * (d % 2);
                const int nv = (d % 8) * (D / 8) + (d % 16) / 8 * (D / 16) + d / 16;
                const int ck = (static_cast<const uint8_t*>(a.k_pages)[row * (D / 2) + nk / 2] >> (4 * (nk % 2))) & 15;
                const int cv = (static_cast<const uint8_t*>(a.v_pages)[row * (D / 2) + nv / 2] >> (4 * (nv % 2))) & 15;
                const float2 sk = __half22float2(static_cast<const __half2*>(a.k_scales)[row * (D / 32) + d / 32]);
                const float2 sv = __half22float2(static_cast<const __half2*>(a.v_scales)[row * (D / 32) + d / 32]);
                k[e] = fmaf(static_cast<float>(ck), sk.x, sk.y);
                v[e] = fmaf(static_cast<float>(cv), sv.x, sv.y);
            } else {
                k[e] = load16<BF16>(a.k_pages, page * a.page_stride + in_page * D + d);
                v[e] = load16<BF16>(a.v_pages, page * a.page_stride + in_page * D + d);
            }
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s);
        const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
        l = l * alpha + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + p * v[e];
        m = mn;
    }
    __shared__ float sm[4], sl[4], so[4][D];
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float lt = 0.f, w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        w[x] = sm[x] == -INFINITY ? 0.f : exp2f(sm[x] - mx);
        lt += w[x] * sl[x];
    }
    const float inv = lt > 0.f ? 1.f / lt : 0.f;
    if (threadIdx.x < D) {
        float acc = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) acc += w[x] * so[x][threadIdx.x];
        const int64_t at = b * a.o_bs + h * a.o_hs + i * a.o_ns + threadIdx.x;
        if (BF16)
            static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16(acc * inv);
        else
            static_cast<__half*>(a.o)[at] = __float2half(acc * inv);
    }
    if (threadIdx.x == 0 && a.lse != nullptr)
        a.lse[(static_cast<int64_t>(b) * a.H + h) * a.Nq + i] = lt > 0.f ? (mx + log2f(lt)) * kLn2 : -INFINITY;
}

template <int D, bool BF16>
cudaError_t launch_kind(const DecodeArgs& a, bool kv4, cudaStream_t s) {
    const dim3 grid(a.H * a.Nq, a.B);
    if (kv4)
        decode_kernel<D, BF16, true><<<grid, 128, 0, s>>>(a);
    else
        decode_kernel<D, BF16, false><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

int64_t decode_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 16; }

cudaError_t decode_launch(const DecodeArgs& a, int D, bool bf16, bool kv4, int, cudaStream_t s) {
    if (D == 128) return bf16 ? launch_kind<128, true>(a, kv4, s) : launch_kind<128, false>(a, kv4, s);
    return bf16 ? launch_kind<64, true>(a, kv4, s) : launch_kind<64, false>(a, kv4, s);
}

cudaError_t decode_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_decode_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_decode_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
