// decode_cross.cu -- decode_kernel.cuh over an encoder's states: dense tensors by
// strides, every key of a batch entry visible to all its rows.
//
// Measured (GB300): 24 entries of up to 4096 keys, one token, 32 heads on 8, D = 128,
// bf16 (274 MB) 47.4 us = 5.8 TB/s, memory and about 7 us of start and joins; one
// entry of 1000 keys 8.2 us.
#include "decode_kernel.cuh"

namespace fattn {

cudaError_t decode_cross_launch(const CrossDecodeArgs& a, int D, bool bf16, int sms, cudaStream_t s) {
    return launch16<kCross>(a, D, bf16, sms, s);
}

cudaError_t decode_cross_read_and_clear_error_word(uint32_t* out) { return read_and_clear(out); }

}  // namespace fattn
