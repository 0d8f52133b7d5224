// decode_scaled_e4m3.cu -- decode attention over e4m3 pools with a scale per
// block, in a translation unit of its own.
#include "decode_scaled.cuh"

namespace pkv {

cudaError_t launch_decode_scaled_e4m3(const DecodeArgs& a, bool stall, cudaStream_t stream) {
    return launch_decode_scaled_kind<kKindE4m3Blocks>(a, stall, stream);
}

}  // namespace pkv
