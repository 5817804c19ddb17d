// fwd_tc.cu -- the tensor-core forward (fwd_tc_kernel.cuh) on dense [B,H,N,D]
// batches, and the self test of the bounded wait.
#include "fwd_tc_kernel.cuh"

namespace fattn {
namespace {

__global__ void wait_selftest_kernel(uint64_t timeout_ns) {
    __shared__ uint64_t bar;
    __shared__ uint32_t abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0u;
        fence_barrier_init();
    }
    __syncthreads();
    // Nothing ever arrives on `bar`: the bounded wait must give up, record
    // the timeout in the error word and return.
    if (threadIdx.x == 0)
        (void)mbar_wait_bounded(&bar, 0u, &abort_flag, &g_error_word, timeout_ns);
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t launch_one(const TcArgs& a, int grid, cudaStream_t stream) {
    using L = TcLayout<D>;
    auto* fn = attn_fwd_tc_kernel<D, BF16, CAUSAL, false>;
    // The opt-in above 48 KB of dynamic shared memory is per device: set it
    // once for every device this instantiation is launched on.
    static std::atomic<bool> done[kMaxDevices] = {};
    cudaError_t e = opt_in_smem_once(fn, L::kAlloc, done);
    if (e != cudaSuccess) return e;
    fn<<<grid, kTcThreads, L::kAlloc, stream>>>(a);
    return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_causal(const TcArgs& a, bool causal, int grid, cudaStream_t s) {
    return causal ? launch_one<D, BF16, true>(a, grid, s) : launch_one<D, BF16, false>(a, grid, s);
}

}  // namespace

int tc_smem_bytes(int D) { return D == 128 ? TcLayout<128>::kAlloc : TcLayout<64>::kAlloc; }
int tc_num_stages(int D) { return D == 128 ? TcLayout<128>::kStages : TcLayout<64>::kStages; }

cudaError_t tc_launch(const TcArgs& a, int D, bool bf16, bool causal, int grid,
                      cudaStream_t stream) {
    if (D == 128)
        return bf16 ? launch_causal<128, true>(a, causal, grid, stream)
                    : launch_causal<128, false>(a, causal, grid, stream);
    return bf16 ? launch_causal<64, true>(a, causal, grid, stream)
                : launch_causal<64, false>(a, causal, grid, stream);
}

cudaError_t read_and_clear_error_word(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
    *out = v;
    return e;
}

cudaError_t launch_wait_selftest(uint64_t timeout_ns, cudaStream_t stream) {
    wait_selftest_kernel<<<1, 32, 0, stream>>>(timeout_ns);
    return cudaGetLastError();
}

}  // namespace fattn
