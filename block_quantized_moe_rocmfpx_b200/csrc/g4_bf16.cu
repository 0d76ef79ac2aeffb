// g4_bf16.cu -- 4-bit group-scale products of bf16 activations (g4.cuh).
#include "g4.cuh"

namespace rfx {
cudaError_t g4_launch_bf16(G4Params p, int G, bool zeros, cudaStream_t stream) {
    return g4_launch_x<0>(p, G, zeros, stream);
}
}  // namespace rfx
