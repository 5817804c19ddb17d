// bwd_cross.cu -- the backward (bwd_tc_kernel.cuh) of cross attention: keys of a
// length of their own, rows by strides; and the kernel of its row statistics.
#include "bwd_tc_kernel.cuh"

namespace fattn {
namespace {

// -LSE_i * log2(e) and -Delta_i, Delta_i = dO_i . O_i, into the padded workspace
// [B*H][2][Npad]; rows past Nq, and rows that saw no key (LSE = -inf), get -inf
// and 0.  A row is read as 16-byte pieces by D/8 lanes, kStatLoads such rows of O
// and of dO in flight a lane.
constexpr int kStatLoads = 4;
template <int D>
constexpr int kStatRows = (32 / (D / 8)) * kStatLoads;  // of a warp

template <int D, bool BF16>
__global__ void __launch_bounds__(256) cross_stats_kernel(const __grid_constant__ CrossBwdArgs a) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int64_t rows = static_cast<int64_t>(a.BH) * a.Npad;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
    const int lane = threadIdx.x % 32, piece = lane % kLanes;
    uint4 o[kStatLoads], g[kStatLoads];
    grid_dependency();
#pragma unroll
    for (int k = 0; k < kStatLoads; ++k) {
        const int64_t row = warp * kStatRows<D> + k * kRows + lane / kLanes;
        o[k] = g[k] = make_uint4(0u, 0u, 0u, 0u);
        const int64_t bh = row / a.Npad;
        const int i = static_cast<int>(row - bh * a.Npad);
        if (row < rows && i < a.N) {
            const int64_t b = bh / a.H, h = bh - b * a.H;
            o[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o) + b * a.o_bs + h * a.o_hs +
                                                   i * a.o_ns + 8 * piece);
            g[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dout) + b * a.do_bs + h * a.do_hs +
                                                   i * a.do_ns + 8 * piece);
        }
    }
#pragma unroll
    for (int k = 0; k < kStatLoads; ++k) {
        const uint32_t x[4] = {o[k].x, o[k].y, o[k].z, o[k].w}, y[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float2 u, v;
            if (BF16) {
                u = make_float2(__uint_as_float(x[w] << 16), __uint_as_float(x[w] & 0xffff0000u));
                v = make_float2(__uint_as_float(y[w] << 16), __uint_as_float(y[w] & 0xffff0000u));
            } else {
                u = __half22float2(*reinterpret_cast<const __half2*>(&x[w]));
                v = __half22float2(*reinterpret_cast<const __half2*>(&y[w]));
            }
            sum = fmaf(u.x, v.x, sum);
            sum = fmaf(u.y, v.y, sum);
        }
#pragma unroll
        for (int d = kLanes / 2; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const int64_t row = warp * kStatRows<D> + k * kRows + lane / kLanes;
        if (piece == 0 && row < rows) {
            const int64_t bh = row / a.Npad;
            const int i = static_cast<int>(row - bh * a.Npad);
            float nlse2 = -INFINITY, ndelta = 0.f;
            if (i < a.N) {
                const float lse = a.lse[bh * a.N + i];
                if (lse != -INFINITY) {
                    nlse2 = -lse * 1.4426950408889634f;
                    ndelta = -sum;
                }
            }
            a.ws[bh * 2 * a.Npad + i] = nlse2;
            a.ws[(bh * 2 + 1) * a.Npad + i] = ndelta;
        }
    }
}

template <int D, bool BF16>
cudaError_t launch_all(const CrossBwdArgs& a, cudaStream_t s) {
    // (Without queries the key kernel, without keys the query kernel writes zeros.)
    const int64_t warps = (static_cast<int64_t>(a.BH) * a.Npad + kStatRows<D> - 1) / kStatRows<D>;
    cudaError_t e = cudaSuccess;
    if (a.N > 0 && a.Nk > 0) {
        e = launch_overlapped(cross_stats_kernel<D, BF16>, static_cast<unsigned>((warps + 7) / 8), 256, 0, s, a);
        if (e != cudaSuccess) return e;
    }
    static std::atomic<bool> kv_done[kMaxDevices] = {};
    static std::atomic<bool> q_done[kMaxDevices] = {};
    auto* kkv = attn_bwd_kernel<D, BF16, true, false, true>;
    if ((e = opt_in_smem_once(kkv, BwdLayout<D, true>::kBytes, kv_done)) != cudaSuccess) return e;
    if (a.tiles_k > 0) {
        e = launch_overlapped(kkv, static_cast<unsigned>(a.tiles_k * a.BHkv), kBwdThreads, BwdLayout<D, true>::kBytes, s, a);
        if (e != cudaSuccess) return e;
    }
    if (a.num_tiles == 0) return cudaSuccess;
    auto* kq = attn_bwd_kernel<D, BF16, false, false, true>;
    if ((e = opt_in_smem_once(kq, BwdLayout<D, false>::kBytes, q_done)) != cudaSuccess) return e;
    const unsigned grid_q = static_cast<unsigned>(a.num_tiles * a.BH);
    // (Behind the key kernel only: it reads and writes without waiting first.)
    if (a.tiles_k > 0) return launch_overlapped(kq, grid_q, kBwdThreads, BwdLayout<D, false>::kBytes, s, a);
    kq<<<grid_q, kBwdThreads, BwdLayout<D, false>::kBytes, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t bwd_cross_launch(const CrossBwdArgs& a, int D, bool bf16, cudaStream_t s) {
    if (D == 128) return bf16 ? launch_all<128, true>(a, s) : launch_all<128, false>(a, s);
    return bf16 ? launch_all<64, true>(a, s) : launch_all<64, false>(a, s);
}

cudaError_t bwd_cross_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
