// g4.h -- launch parameters of the 4-bit group-scale products (g4.cuh).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rfx {

struct G4Params {
    const uint8_t* W0;        // packed matrix, or the experts' matrices at a stride (gate of gate/up)
    const uint8_t* W1;        // up matrices of gate/up, else null
    long long stride;         // bytes between experts
    const int32_t* offsets;   // [E + 1] rows of x by expert, or null: one matrix for all R rows
    int E, R, N, K;
    const void* x;            // [R][K]
    float* y;                 // [R][N]
    // set by the launcher
    long long rg_bytes;       // bytes of a row-group
    int c0, c1;               // chunks of this launch; c0 > 0 adds to y
    int units;                // units of a matrix
    int team, teams, inv_team;   // warps that share a unit, such teams in a CTA, 65536 / team
    int split;                // CTAs of a cluster that share a unit's K (1 to 8)
    int cols, shift;          // rows of x per pass over a matrix, at most (experts: 1 << shift)
    int x_room;               // shared memory for x
};

// x_dtype: 0 bf16, 1 fp32, 2 fp16
cudaError_t g4_launch_bf16(G4Params p, int G, bool zeros, cudaStream_t stream);
cudaError_t g4_launch_f32(G4Params p, int G, bool zeros, cudaStream_t stream);
cudaError_t g4_launch_f16(G4Params p, int G, bool zeros, cudaStream_t stream);
cudaError_t g4_pack_launch(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, long long rows,
                           long long cols, int G, uint8_t* dst, cudaStream_t stream);

}  // namespace rfx
