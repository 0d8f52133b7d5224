// decode_scaled_int8.cu -- decode attention over int8 pools with a scale per
// block, in a translation unit of its own.
#include "decode_scaled.cuh"

namespace pkv {

cudaError_t launch_decode_scaled_int8(const DecodeArgs& a, bool stall, cudaStream_t stream) {
    return launch_decode_scaled_kind<kKindInt8Blocks>(a, stall, stream);
}

}  // namespace pkv
