// rows.h -- launch parameters of the token grouping, the weighted combine and
// their gradients (rows.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rfx {

struct GroupParams {
    const uint8_t* x;      // [T] rows of row_bytes, or null: no rows are copied
    uint8_t* xs;           // [T * k] rows
    long long row_bytes;
    const int32_t* idx;    // [T][k]
    int T, k, E;
    int32_t* pos;          // [T][k]
    int32_t* rows;         // [T * k]
    int32_t* offsets;      // [E + 1]
    uint32_t* ctrl;        // workspace control words
    int32_t* part;         // [slices][group_pitch(E)] entries per expert and slice
    int slices;            // token slices, one CTA each
    int per;               // tokens per slice
};

constexpr int GROUP_CTRL_BYTES = 256;
constexpr int group_pitch(int E) { return (E + 3) & ~3; }
// Slices of a call, and whether it takes the two-launch plan; the same rule
// sizes the workspace.
int group_slices(int T, int k);
bool group_two_launches(int T, int k);

cudaError_t group_launch(const GroupParams& p, cudaStream_t stream);

// dtype: 0 bf16, 1 fp32, 2 fp16
cudaError_t combine_launch(const void* ys, int dtype, int T, int H, const int32_t* pos, int k, const float* w,
                           const void* base, void* y, int y_dtype, cudaStream_t stream);
cudaError_t combine_backward_launch(const void* dy, int y_dtype, const void* ys, int dtype, int T, int H,
                                    const int32_t* pos, int k, const float* w, void* dys, float* dw,
                                    cudaStream_t stream);
cudaError_t router_backward_launch(const int32_t* idx, const float* w, const float* dw, int T, int E, int k,
                                   float* dlogits, cudaStream_t stream);

}  // namespace rfx
