// decode.cu -- decode_kernel.cuh over a paged cache in 16 or in 4 bits.
#include "decode_kernel.cuh"

namespace fattn {
namespace {

template <int D, bool BF16>
cudaError_t launch_kv4(const DecodeArgs& a, int sms, cudaStream_t s) {
    return launch_rows<D, BF16, true, kCache>(a, sms, s);
}

}  // namespace

int64_t decode_workspace_bytes(int64_t, int64_t H, int64_t Hkv, int64_t Nq, int64_t D) {
    const int64_t rows = 8 * row_tiles(H / Hkv * Nq);
    return 16 * kMaxCtas + 2 * kMaxCtas * rows * (D + 2) * static_cast<int64_t>(sizeof(float));
}

cudaError_t decode_launch(const DecodeArgs& a, int D, bool bf16, bool kv4, int sms, cudaStream_t s) {
    if (!kv4) return launch16<kCache>(a, D, bf16, sms, s);
    if (D == 128) return bf16 ? launch_kv4<128, true>(a, sms, s) : launch_kv4<128, false>(a, sms, s);
    return bf16 ? launch_kv4<64, true>(a, sms, s) : launch_kv4<64, false>(a, sms, s);
}

cudaError_t decode_read_and_clear_error_word(uint32_t* out) { return read_and_clear(out); }

}  // namespace fattn
