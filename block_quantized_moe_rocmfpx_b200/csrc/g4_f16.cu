// g4_f16.cu -- 4-bit group-scale products of fp16 activations (g4.cuh).
#include "g4.cuh"

namespace rfx {
cudaError_t g4_launch_f16(G4Params p, int G, bool zeros, cudaStream_t stream) {
    return g4_launch_x<2>(p, G, zeros, stream);
}
}  // namespace rfx
