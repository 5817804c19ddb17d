// decode_shared.cu -- decode_kernel.cuh for sequences that share a prefix: over their
// own keys, as a part beside those that the prefix's kernel leaves (fwd_rows.cu), and
// over the prefix and their own keys in one.
#include "decode_kernel.cuh"

namespace fattn {

cudaError_t decode_shared_launch(const SharedDecodeArgs& a, int D, bool bf16, int sms, cudaStream_t s) {
    return launch16<kBehindPrefix>(a, D, bf16, sms, s);
}

cudaError_t decode_prefix_launch(const PrefixDecodeArgs& a, int D, bool bf16, int sms, cudaStream_t s) {
    return launch16<kWithPrefix>(a, D, bf16, sms, s);
}

cudaError_t decode_shared_read_and_clear_error_word(uint32_t* out) { return read_and_clear(out); }

}  // namespace fattn
