// g4_f32.cu -- 4-bit group-scale products of fp32 activations (g4.cuh).
#include "g4.cuh"

namespace rfx {
cudaError_t g4_launch_f32(G4Params p, int G, bool zeros, cudaStream_t stream) {
    return g4_launch_x<1>(p, G, zeros, stream);
}
}  // namespace rfx
