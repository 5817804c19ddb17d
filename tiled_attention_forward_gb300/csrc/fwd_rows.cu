// fwd_rows.cu -- the tensor-core forward (fwd_tc_kernel.cuh) on query rows over
// keys of a length of their own, and the kernel that joins the parts of rows whose
// keys were cut.
#include "fwd_tc_kernel.cuh"

namespace fattn {
namespace {

constexpr int kJoinThreads = 256;

// A warp a row of the output: the parts in the order of their keys.
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) rows_join_kernel(const __grid_constant__ RowsArgs a) {
    constexpr int kPer = D / 32;  // elements a lane
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x) / 32;
    const int lane = threadIdx.x % 32;
    grid_dependency();
    if (w >= static_cast<int64_t>(a.B) * a.H * a.Nq) return;
    const int i = static_cast<int>(w % a.Nq);
    const int64_t bh = w / a.Nq;
    const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
    const int kvh = h / a.share, hq = h % a.share;
    const int u = (hq / a.box_h) * a.n_i + i / a.box_i, trow = (hq % a.box_h) * a.box_i + i % a.box_i;
    const int64_t at = (((static_cast<int64_t>(b) * a.Hkv + kvh) * a.tiles + u) * kTcBM + trow) * a.part_pitch;
    float m = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) m = fmaxf(m, __ldcg(a.part_ml + at + s).x);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const bool none = m == -INFINITY;
    float sum = 0.f, acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float2 ml = __ldcg(a.part_ml + at + s);
        const float wt = none ? 0.f : ex2_approx(ml.x - m);
        sum = fmaf(wt, ml.y, sum);
        const float* src = a.part_o + (at + s) * D + lane * kPer;
        float v[kPer];
        if constexpr (kPer == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
            v[0] = x.x, v[1] = x.y;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(wt, v[e], acc[e]);
    }
    const float inv = none ? 0.f : 1.f / sum;
    uint16_t* o = static_cast<uint16_t*>(a.o) + b * a.o_bs + h * a.o_hs + i * a.o_ns + lane * kPer;
    if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(o) =
            make_uint2(pack2(acc[0] * inv, acc[1] * inv, BF16), pack2(acc[2] * inv, acc[3] * inv, BF16));
    else
        *reinterpret_cast<uint32_t*>(o) = pack2(acc[0] * inv, acc[1] * inv, BF16);
    if (lane == 0 && a.lse != nullptr) a.lse[w] = none ? -INFINITY : (m + log2f(sum)) * kLn2;
}

template <int D, bool BF16>
cudaError_t launch_one(const RowsArgs& a, int grid, cudaStream_t stream) {
    using L = TcLayout<D>;
    auto* fn = attn_fwd_tc_kernel<D, BF16, false, kRows>;
    static std::atomic<bool> done[kMaxDevices] = {};
    const cudaError_t e = opt_in_smem_once(fn, L::kAlloc, done);
    if (e != cudaSuccess) return e;
    return launch_overlapped(fn, grid, kTcThreads, L::kAlloc, stream, a);
}

}  // namespace

cudaError_t rows_launch(const RowsArgs& a, int D, bool bf16, int grid, cudaStream_t s) {
    if (D == 128) return bf16 ? launch_one<128, true>(a, grid, s) : launch_one<128, false>(a, grid, s);
    return bf16 ? launch_one<64, true>(a, grid, s) : launch_one<64, false>(a, grid, s);
}

cudaError_t rows_join_launch(const RowsArgs& a, int D, bool bf16, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.H * a.Nq;
    const unsigned grid = static_cast<unsigned>((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
    auto* fn = D == 128 ? (bf16 ? rows_join_kernel<128, true> : rows_join_kernel<128, false>)
                        : (bf16 ? rows_join_kernel<64, true> : rows_join_kernel<64, false>);
    return launch_overlapped(fn, grid, kJoinThreads, 0, s, a);
}

cudaError_t rows_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
