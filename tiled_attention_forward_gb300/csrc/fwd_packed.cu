// fwd_packed.cu -- the tensor-core forward (fwd_tc_kernel.cuh) on packed
// sequences of different lengths, and the kernel that lists their Q blocks.
//
// Sequences s = cu[b] .. cu[b+1] of one [T, H, D] tensor become Q blocks of 256
// rows.  Only the device knows the lengths.  Where T/256 + B is at most 64 each
// CTA lists the blocks for itself; else a first launch of one CTA writes the
// list, sorted by the K/V tiles a block visits, longest first: CTAs of the
// forward take (block, head) tasks from a counter in that order, so that
// the short ones fill in the tail whatever the mix of lengths.  The sort is a
// counting sort over at most 1024 bins; the order within a bin depends on
// atomics, which moves tasks in time and changes no result (a task's rows are
// written by one CTA, from its own inputs).
//
// Measured (GB300, bf16, 32 heads on 8, D = 128, causal, in a stream of calls on
// changing inputs): a prompt of 16000 tokens beside three short ones 1.30 to 1.32
// ms = 1590 to 1610 TFLOP/s, the dense forward's rate (0.83 of the measured peak);
// 16 prompts of 1 to 4096 tokens 298 us = 1195 TFLOP/s (replayed from a graph 281).
// The forward's own chain bounds both (fwd_tc_kernel.cuh); the mix
// pays about 2.8 us at each of the 15 task changes of a CTA, and 8 % more scores
// than the mask leaves (whole 128 x 128 tiles).  Five prompts of up to 128
// tokens take 9.2 us (graph 8.5), of which the list is about 1.
#include "fwd_tc_kernel.cuh"

namespace fattn {
namespace {

constexpr int kPlanThreads = 1024;
struct PlanArgs {
    const int* cu;
    int B, T, capacity;
    PackedPlan* plan;
};

// Warp w keeps sequences w, w + 32, .. in its lanes (1024 of them at once, read
// once where there are no more) and takes them one after the other, lanes over
// blocks.
template <bool CAUSAL>
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PlanArgs args) {
    const int* __restrict__ cu = args.cu;
    const int B = args.B, T = args.T, capacity = args.capacity;
    PackedPlan* plan = args.plan;
    __shared__ int bins[kPlanThreads];
    __shared__ int warp_sums[32];
    __shared__ int most, bad;
    grid_dependency();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    if (tid == 0) most = bad = 0;
    bins[tid] = 0;
    int start = 0, n = 0;
    auto read = [&](int b0) -> bool {  // this lane's sequence of the 1024 from b0 on; false: it breaks the rules
        const int b = b0 + warp + 32 * lane;
        start = n = 0;
        if (b >= B) return true;
        const int s = cu[b], e = cu[b + 1];
        if (s < 0 || e < s || e > T) return false;
        start = s;
        n = e - s;
        return true;
    };
    int local_most = 0;
    bool fine = true;
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
        fine = read(b0) && fine;
        local_most = max(local_most, (n + kTcBN - 1) / kTcBN);
    }
    __syncthreads();
    if (!fine) bad = 1;
    local_most = __reduce_max_sync(0xffffffffu, local_most);
    if (lane == 0) atomicMax(&most, local_most);
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
    auto for_blocks = [&](auto&& take) {
        for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
            if (B > kPlanThreads) read(b0);
            for (uint32_t left = __ballot_sync(0xffffffffu, n > 0); left != 0u; left &= left - 1u) {
                const int from = __ffs(left) - 1;
                const int s = __shfl_sync(0xffffffffu, start, from), m = __shfl_sync(0xffffffffu, n, from);
                for (int blk = lane; blk * kRows < m; blk += 32)
                    take(s, m, blk, &bins[kPlanThreads - 1 - (block_tiles<CAUSAL>(m, blk) >> shift)]);
            }
        }
    };
    for_blocks([&](int, int, int, int* bin) { atomicAdd(bin, 1); });
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
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
        const int s = warp_sums[w];
        if (w < warp) before += s;
        total += s;
    }
    bins[tid] = x - own + before;
    if (tid == 0) plan->blocks = min(total, capacity);
    __syncthreads();
    for_blocks([&](int s, int m, int blk, int* bin) {
        const int at = atomicAdd(bin, 1);
        if (at < capacity) plan->list[at] = make_int4(s, m, blk, 0);
    });
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t launch_one(const PackedArgs& a, int capacity, int grid, cudaStream_t stream) {
    using L = TcLayout<D>;
    auto* fn = attn_fwd_tc_kernel<D, BF16, CAUSAL, kPacked>;
    static std::atomic<bool> done[kMaxDevices] = {};
    cudaError_t e = opt_in_smem_once(fn, L::kAlloc, done);
    if (e != cudaSuccess) return e;
    if (a.plan_stride == 0) {
        const PlanArgs p = {a.cu, a.B, static_cast<int>(a.T), capacity, a.plan};
        e = launch_overlapped(packed_plan_kernel<CAUSAL>, 1, kPlanThreads, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    // The forward's own setup runs while the list is written.
    return launch_overlapped(fn, grid, kTcThreads, L::kAlloc, stream, a);
}

template <int D, bool BF16>
cudaError_t launch_causal(const PackedArgs& a, bool causal, int capacity, int grid, cudaStream_t s) {
    return causal ? launch_one<D, BF16, true>(a, capacity, grid, s) : launch_one<D, BF16, false>(a, capacity, grid, s);
}

}  // namespace

cudaError_t packed_launch(const PackedArgs& a, int D, bool bf16, bool causal, int capacity, int grid, cudaStream_t s) {
    if (D == 128)
        return bf16 ? launch_causal<128, true>(a, causal, capacity, grid, s)
                    : launch_causal<128, false>(a, causal, capacity, grid, s);
    return bf16 ? launch_causal<64, true>(a, causal, capacity, grid, s)
                : launch_causal<64, false>(a, causal, capacity, grid, s);
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
