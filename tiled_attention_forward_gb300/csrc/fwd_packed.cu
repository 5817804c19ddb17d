// fwd_packed.cu -- the tensor-core forward (fwd_tc_kernel.cuh) on packed
// sequences of different lengths, and the kernel that lists their Q blocks.
//
// Sequences s = cu[b] .. cu[b+1] of one [T, H, D] tensor become Q blocks of 256
// rows.  Only the device knows the lengths, so a first launch of one CTA writes
// the list, sorted by the K/V tiles a block visits, longest first: CTAs of the
// second launch take (block, head) tasks from a counter in that order, so that
// the short ones fill in the tail whatever the mix of lengths.  The sort is a
// counting sort over at most 1024 bins; the order within a bin depends on
// atomics, which moves tasks in time and changes no result (a task's rows are
// written by one CTA, from its own inputs).
#include "fwd_tc_kernel.cuh"

namespace fattn {
namespace {

constexpr int kPlanThreads = 1024;

// K/V tiles that Q block `blk` of a sequence of n tokens visits.
template <bool CAUSAL>
__device__ __forceinline__ int block_tiles(int n, int blk) {
    const int keys = CAUSAL ? min(n, (blk + 1) * (kTcBM * kTcQTiles)) : n;
    return (keys + kTcBN - 1) / kTcBN;
}

template <bool CAUSAL>
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const int* __restrict__ cu, int B, int T,
                                                                   int capacity, PackedPlan* plan) {
    __shared__ int bins[kPlanThreads];
    __shared__ int warp_sums[32];
    __shared__ int most, bad;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    if (tid == 0) most = bad = 0;
    bins[tid] = 0;
    __syncthreads();
    int local_most = 0, local_bad = 0;
    for (int b = tid; b < B; b += kPlanThreads) {
        const int s = cu[b], e = cu[b + 1];
        if (s < 0 || e < s || e > T)
            local_bad = 1;
        else
            local_most = max(local_most, (e - s + kTcBN - 1) / kTcBN);
    }
    if (local_bad) bad = 1;
    atomicMax(&most, local_most);
    __syncthreads();
    if (bad) {  // nothing is computed; the host learns it from the device status
        if (tid == 0) {
            plan->blocks = 0;
            atomicOr(&g_error_word, 1u << kDevErrInvalidArg);
        }
        return;
    }
    int shift = 0;
    while ((most >> shift) >= kPlanThreads) ++shift;
    constexpr int kRows = kTcBM * kTcQTiles;
    for (int b = warp; b < B; b += kPlanThreads / 32) {
        const int n = cu[b + 1] - cu[b];
        for (int blk = lane; blk * kRows < n; blk += 32)
            atomicAdd(&bins[kPlanThreads - 1 - (block_tiles<CAUSAL>(n, blk) >> shift)], 1);
    }
    __syncthreads();
    // Exclusive scan of the bins (largest first).
    const int own = bins[tid];
    int x = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const int total = warp_sums[31];
    bins[tid] = x - own + (warp > 0 ? warp_sums[warp - 1] : 0);
    if (tid == 0) plan->blocks = min(total, capacity);
    __syncthreads();
    for (int b = warp; b < B; b += kPlanThreads / 32) {
        const int s = cu[b], n = cu[b + 1] - s;
        for (int blk = lane; blk * kRows < n; blk += 32) {
            const int at = atomicAdd(&bins[kPlanThreads - 1 - (block_tiles<CAUSAL>(n, blk) >> shift)], 1);
            if (at < capacity) plan->list[at] = make_int4(s, n, blk, 0);
        }
    }
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t launch_one(const PackedArgs& a, const int32_t* cu, int B, int capacity, int grid, cudaStream_t stream) {
    using L = TcLayout<D>;
    auto* fn = attn_fwd_tc_kernel<D, BF16, CAUSAL, true>;
    static std::atomic<bool> done[kMaxDevices] = {};
    cudaError_t e = opt_in_smem_once(fn, L::kAlloc, done);
    if (e != cudaSuccess) return e;
    packed_plan_kernel<CAUSAL><<<1, kPlanThreads, 0, stream>>>(cu, B, static_cast<int>(a.T), capacity, a.plan);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    fn<<<grid, kTcThreads, L::kAlloc, stream>>>(a);
    return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_causal(const PackedArgs& a, const int32_t* cu, int B, bool causal, int capacity, int grid,
                          cudaStream_t s) {
    return causal ? launch_one<D, BF16, true>(a, cu, B, capacity, grid, s)
                  : launch_one<D, BF16, false>(a, cu, B, capacity, grid, s);
}

}  // namespace

cudaError_t packed_launch(const PackedArgs& a, const int32_t* cu, int B, int D, bool bf16, bool causal, int capacity,
                          int grid, cudaStream_t s) {
    if (D == 128)
        return bf16 ? launch_causal<128, true>(a, cu, B, causal, capacity, grid, s)
                    : launch_causal<128, false>(a, cu, B, causal, capacity, grid, s);
    return bf16 ? launch_causal<64, true>(a, cu, B, causal, capacity, grid, s)
                : launch_causal<64, false>(a, cu, B, causal, capacity, grid, s);
}

cudaError_t packed_read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace fattn
