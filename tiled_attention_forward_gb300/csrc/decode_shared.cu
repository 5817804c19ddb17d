// decode_shared.cu -- decode_kernel.cuh for sequences that share a prefix: over their
// own keys, as a part beside those that the prefix's kernel leaves (fwd_rows.cu), and
// over the prefix and their own keys in one.
//
// Measured (GB300, 32 heads on 8, D = 128, bf16): 64 sequences of up to 1024 own
// tokens (121 MB) behind 16000 shared ones 62 us, own keys 26, prefix 22, join 7 and
// the starts of three kernels; plain decode over the same keys would read 4.3 GB.  16
// sequences of two rows behind 120001 tokens 100 us.  Short targets are a chain of
// latencies (700 instructions to start and join one, 150 a stage of 16 keys), so
// the own keys take six warps a CTA, two CTAs an SM (65 -> 62 us; the few of the
// second case are joined a little later, 98 -> 100).  The own keys come first: behind
// the prefix their K and V pushed its parts out of L2 (76 -> 63 us).  4 sequences of
// up to 100 tokens behind 2000, 16 heads on 4, D = 64, in one launch: 9.5 us.
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
