// decode_cross.cu -- decode_kernel.cuh over an encoder's states: dense tensors by
// strides, every key of a batch entry visible to all its rows.
#include "decode_kernel.cuh"

namespace fattn {

cudaError_t decode_cross_launch(const CrossDecodeArgs& a, int D, bool bf16, int sms, cudaStream_t s) {
    return launch16<kCross>(a, D, bf16, sms, s);
}

cudaError_t decode_cross_read_and_clear_error_word(uint32_t* out) { return read_and_clear(out); }

}  // namespace fattn
