// bwd_tc.cu -- the backward (bwd_tc_kernel.cuh) of dense [B,H,N,D] batches, and the
// kernel of its row statistics.
#include "bwd_tc_kernel.cuh"

namespace fattn {
namespace {

// -LSE_i * log2(e) and -Delta_i, Delta_i = dO_i . O_i (fp32 over the 16-bit
// inputs), into the padded workspace [B*H][2][Npad]; rows past N get -inf
// and 0.  A row is read as 16-byte pieces by D/8 lanes, a warp covers
// 32/(D/8) rows per load and keeps kPrepLoads such loads of O and of dO in
// flight (kPrepRows rows per warp), so the kernel streams at memory rate.
constexpr int kPrepLoads = 4;
template <int D>
__host__ __device__ constexpr int prep_rows_per_warp() { return (32 / (D / 8)) * kPrepLoads; }

template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_bwd_prep_kernel(const void* __restrict__ o,
                                                            const void* __restrict__ dout,
                                                            const float* __restrict__ lse,
                                                            float* __restrict__ ws, int N, int Npad,
                                                            int64_t rows_padded) {
    constexpr int kLanesPerRow = D / 8;               // 16-byte pieces per row
    constexpr int kRowsPerLoad = 32 / kLanesPerRow;
    const int64_t gw = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
    const int lane = threadIdx.x % 32;
    const int sub = lane / kLanesPerRow, piece = lane % kLanesPerRow;
    uint4 ov[kPrepLoads], dv[kPrepLoads];
    int64_t prow[kPrepLoads];
#pragma unroll
    for (int k = 0; k < kPrepLoads; ++k) {
        prow[k] = gw * prep_rows_per_warp<D>() + k * kRowsPerLoad + sub;  // padded row
        ov[k] = make_uint4(0u, 0u, 0u, 0u);
        dv[k] = ov[k];
        if (prow[k] < rows_padded) {
            const int64_t bh = prow[k] / Npad;
            const int i = static_cast<int>(prow[k] % Npad);
            if (i < N) {
                const int64_t off = ((bh * N + i) * D) * 2 + piece * 16;
                ov[k] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(o) + off);
                dv[k] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(dout) + off);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kPrepLoads; ++k) {
        const uint32_t ow[4] = {ov[k].x, ov[k].y, ov[k].z, ov[k].w};
        const uint32_t dw[4] = {dv[k].x, dv[k].y, dv[k].z, dv[k].w};
        float acc = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float x0, x1, y0, y1;
            if (BF16) {
                const __nv_bfloat162 xb = *reinterpret_cast<const __nv_bfloat162*>(&ow[w]);
                const __nv_bfloat162 yb = *reinterpret_cast<const __nv_bfloat162*>(&dw[w]);
                x0 = __low2float(xb); x1 = __high2float(xb);
                y0 = __low2float(yb); y1 = __high2float(yb);
            } else {
                const __half2 xh = *reinterpret_cast<const __half2*>(&ow[w]);
                const __half2 yh = *reinterpret_cast<const __half2*>(&dw[w]);
                x0 = __low2float(xh); x1 = __high2float(xh);
                y0 = __low2float(yh); y1 = __high2float(yh);
            }
            acc = fmaf(x0, y0, acc);
            acc = fmaf(x1, y1, acc);
        }
#pragma unroll
        for (int off = kLanesPerRow / 2; off > 0; off >>= 1)
            acc += __shfl_xor_sync(0xffffffffu, acc, off, kLanesPerRow);
        if (piece == 0 && prow[k] < rows_padded) {
            const int64_t bh = prow[k] / Npad;
            const int i = static_cast<int>(prow[k] % Npad);
            float nlse2 = -INFINITY, ndelta = 0.f;
            if (i < N) {
                ndelta = -acc;
                nlse2 = -lse[bh * N + i] * 1.4426950408889634f;
            }
            ws[bh * 2 * Npad + i] = nlse2;
            ws[(bh * 2 + 1) * Npad + i] = ndelta;
        }
    }
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t bwd_launch_all(const BwdArgs& a, const void* o, const void* dout, const float* lse,
                           cudaStream_t stream) {
    const int64_t rows_padded = static_cast<int64_t>(a.BH) * a.Npad;
    const int64_t prep_warps = (rows_padded + prep_rows_per_warp<D>() - 1) / prep_rows_per_warp<D>();
    attn_bwd_prep_kernel<D, BF16><<<static_cast<unsigned>((prep_warps + 7) / 8), 256, 0, stream>>>(
        o, dout, lse, a.ws, a.N, a.Npad, rows_padded);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const unsigned grid_kv = static_cast<unsigned>(static_cast<int64_t>(a.num_tiles) * a.BHkv);
    const unsigned grid_q = static_cast<unsigned>(static_cast<int64_t>(a.num_tiles) * a.BH);
    static std::atomic<bool> kv_done[kMaxDevices] = {};
    static std::atomic<bool> q_done[kMaxDevices] = {};
    auto* kkv = attn_bwd_kernel<D, BF16, true, CAUSAL, false>;
    if ((e = opt_in_smem_once(kkv, BwdLayout<D, true>::kBytes, kv_done)) != cudaSuccess) return e;
    kkv<<<grid_kv, kBwdThreads, BwdLayout<D, true>::kBytes, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    auto* kq = attn_bwd_kernel<D, BF16, false, CAUSAL, false>;
    if ((e = opt_in_smem_once(kq, BwdLayout<D, false>::kBytes, q_done)) != cudaSuccess) return e;
    kq<<<grid_q, kBwdThreads, BwdLayout<D, false>::kBytes, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

int64_t bwd_padded_rows(int64_t N) { return (N + kBT - 1) / kBT * kBT; }

cudaError_t bwd_launch(const BwdArgs& a, const void* o, const void* dout, const float* lse, int D,
                       bool bf16, bool causal, cudaStream_t s) {
    if (D == 128) {
        if (bf16) return causal ? bwd_launch_all<128, true, true>(a, o, dout, lse, s)
                                : bwd_launch_all<128, true, false>(a, o, dout, lse, s);
        return causal ? bwd_launch_all<128, false, true>(a, o, dout, lse, s)
                      : bwd_launch_all<128, false, false>(a, o, dout, lse, s);
    }
    if (bf16) return causal ? bwd_launch_all<64, true, true>(a, o, dout, lse, s)
                            : bwd_launch_all<64, true, false>(a, o, dout, lse, s);
    return causal ? bwd_launch_all<64, false, true>(a, o, dout, lse, s)
                  : bwd_launch_all<64, false, false>(a, o, dout, lse, s);
}

cudaError_t bwd_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
