// decode_shared.cu -- decode_kernel.cuh over the sequences' own keys, joined to the
// parts that the prefix they share has left (fwd_rows.cu).
#include "decode_kernel.cuh"

namespace fattn {

cudaError_t decode_shared_launch(const SharedDecodeArgs& a, int D, bool bf16, int sms, cudaStream_t s) {
    return launch16<kBehindPrefix>(a, D, bf16, sms, s);
}

cudaError_t decode_shared_read_and_clear_error_word(uint32_t* out) { return read_and_clear(out); }

}  // namespace fattn
