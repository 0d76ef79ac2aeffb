// g4_pack.cu -- packers of the 4-bit group-scale layout (g4_layout.h): on the
// host, its inverse, and on the device.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/rfx.h"
#include "g4.h"
#include "g4_layout.h"
#include "launch_util.h"
#include "rfx_device.cuh"

namespace rfx {
namespace {

// Word of lane quarter t for 8 codes (columns 8t .. 8t + 7, low nibbles of b).
__host__ __device__ __forceinline__ uint32_t g4_word(const uint8_t b[8]) {
    uint32_t w = 0;
    for (int j = 0; j < 2; ++j) {
        const uint32_t h = (b[j] & 15u) | (b[2 + j] & 15u) << 4 | (b[4 + j] & 15u) << 8 | (b[6 + j] & 15u) << 12;
        w |= ((h << 3 | h >> 13) & 0xFFFFu) << (16 * j);
    }
    return w;
}

// One warp per chunk.  WIDE: codes are read 8 at a time (base 8-byte aligned).
template <bool WIDE>
__global__ void __launch_bounds__(256) g4_pack_kernel(const uint8_t* __restrict__ codes,
                                                      const uint16_t* __restrict__ scales,
                                                      const uint8_t* __restrict__ zeros, long long rows, long long cols,
                                                      int G, long long rg_bytes, int chunks, long long total,
                                                      uint8_t* __restrict__ dst) {
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long ng = cols / G;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
        const long long rg = i / chunks;
        const int c = (int)(i % chunks);
        const int nc = (int)min((long long)G4_CHUNK, cols - (long long)c * G4_CHUNK);
        uint8_t* out = dst + rg * rg_bytes + (long long)c * g4_chunk_bytes(G4_CHUNK, G, zeros != nullptr);
        for (int p = 0; p < g4_slabs(nc); ++p) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const long long row = rg * 16 + g + 8 * (q & 1);
                const int k = p * 64 + (q >> 1) * 32 + 8 * t;
                uint8_t b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (row < rows && k < nc) {
                    const uint8_t* s = codes + row * cols + (long long)c * G4_CHUNK + k;
                    if constexpr (WIDE) {
                        const uint2 v = *reinterpret_cast<const uint2*>(s);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            b[j] = (uint8_t)(v.x >> (8 * j));
                            b[4 + j] = (uint8_t)(v.y >> (8 * j));
                        }
                    } else {
                        for (int j = 0; j < 8; ++j) b[j] = s[j];
                    }
                }
                w[q] = g4_word(b);
            }
            *reinterpret_cast<uint4*>(out + p * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const int groups = nc / G;
        const long long g0 = (long long)c * G4_CHUNK / G;
        for (int j = lane; j < groups * 8; j += 32) {
            const long long r0 = rg * 16 + j / groups, r1 = r0 + 8;
            const long long at = g0 + j % groups;
            const uint32_t s0 = r0 < rows ? scales[r0 * ng + at] : 0u, s1 = r1 < rows ? scales[r1 * ng + at] : 0u;
            *reinterpret_cast<uint32_t*>(out + g4_scale_off(nc) + j * 4) = s0 | s1 << 16;
        }
        if (zeros) {
            const int bytes = g4_chunk_bytes(nc, G, 1) - g4_zero_off(nc, G);
            for (int j = lane; j < bytes; j += 32) {
                uint32_t v = 0;
                if (j < groups * 8) {
                    const long long r0 = rg * 16 + j / groups, r1 = r0 + 8;
                    const long long at = g0 + j % groups;
                    if (r0 < rows) v |= zeros[r0 * ng + at] & 15u;
                    if (r1 < rows) v |= (zeros[r1 * ng + at] & 15u) << 4;
                }
                out[g4_zero_off(nc, G) + j] = (uint8_t)v;
            }
        }
    }
}

}  // namespace

cudaError_t g4_pack_launch(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, long long rows,
                           long long cols, int G, uint8_t* dst, cudaStream_t stream) {
    const int chunks = (int)((cols + G4_CHUNK - 1) / G4_CHUNK);
    const long long total = (rows + 15) / 16 * chunks;
    const unsigned grid = (unsigned)std::min<long long>((total + 7) / 8, 1 << 20);
    const long long rgb = g4_rowgroup_bytes(cols, G, zeros != nullptr);
    if (((uintptr_t)codes & 7u) == 0)
        return launch_dependent(g4_pack_kernel<true>, grid, 256, 0, stream, codes, scales, zeros, rows, cols, G, rgb,
                                chunks, total, dst);
    return launch_dependent(g4_pack_kernel<false>, grid, 256, 0, stream, codes, scales, zeros, rows, cols, G, rgb,
                            chunks, total, dst);
}

void g4_pack_host(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t rows, int64_t cols, int G,
                  uint8_t* dst) {
    const int64_t ng = cols / G, rgb = g4_rowgroup_bytes(cols, G, zeros != nullptr), nrg = (rows + 15) / 16;
    std::fill(dst, dst + nrg * rgb, (uint8_t)0);
#pragma omp parallel for
    for (int64_t r = 0; r < rows; ++r) {
        const int g = (int)(r & 7), h = (int)(r >> 3 & 1);
        uint8_t* out = dst + r / 16 * rgb;
        for (int64_t k0 = 0; k0 < cols; k0 += G4_CHUNK) {
            const int nc = (int)std::min<int64_t>(G4_CHUNK, cols - k0);
            for (int k = 0; k < nc; k += 8) {
                const uint32_t w = g4_word(codes + r * cols + k0 + k);
                uint8_t* d = out + k / 64 * 512 + (4 * g + (k / 8 & 3)) * 16 + ((k / 32 & 1) * 2 + h) * 4;
                for (int i = 0; i < 4; ++i) d[i] = (uint8_t)(w >> (8 * i));
            }
            out += g4_chunk_bytes(nc, G, zeros != nullptr);
        }
    }
    // scales and zeros by row-group: two rows share a byte of zeros
#pragma omp parallel for
    for (int64_t rg = 0; rg < nrg; ++rg) {
        uint8_t* out = dst + rg * rgb;
        for (int64_t k0 = 0; k0 < cols; k0 += G4_CHUNK) {
            const int nc = (int)std::min<int64_t>(G4_CHUNK, cols - k0);
            for (int j = 0; j < nc / G; ++j)
                for (int i = 0; i < 16 && rg * 16 + i < rows; ++i) {
                    const int64_t at = (rg * 16 + i) * ng + k0 / G + j;
                    uint8_t* d = out + g4_scale_off(nc) + ((i & 7) * (nc / G) + j) * 4 + (i >> 3) * 2;
                    d[0] = (uint8_t)scales[at];
                    d[1] = (uint8_t)(scales[at] >> 8);
                    if (zeros) out[g4_zero_off(nc, G) + (i & 7) * (nc / G) + j] |= (uint8_t)(zeros[at] << (i >> 3) * 4);
                }
            out += g4_chunk_bytes(nc, G, zeros != nullptr);
        }
    }
}

void g4_unpack_host(const uint8_t* src, int64_t rows, int64_t cols, int G, uint8_t* codes, uint16_t* scales,
                    uint8_t* zeros) {
    const int64_t ng = cols / G, rgb = g4_rowgroup_bytes(cols, G, zeros != nullptr);
#pragma omp parallel for
    for (int64_t r = 0; r < rows; ++r) {
        const int g = (int)(r & 7), h = (int)(r >> 3 & 1);
        const uint8_t* in = src + r / 16 * rgb;
        for (int64_t k0 = 0; k0 < cols; k0 += G4_CHUNK) {
            const int nc = (int)std::min<int64_t>(G4_CHUNK, cols - k0);
            for (int k = 0; k < nc; ++k) {
                const uint8_t* s = in + k / 64 * 512 + (4 * g + (k / 8 & 3)) * 16 + ((k / 32 & 1) * 2 + h) * 4;
                const uint32_t half = s[2 * (k & 1)] | (uint32_t)s[2 * (k & 1) + 1] << 8;
                codes[r * cols + k0 + k] = (uint8_t)((half >> 3 | half << 13) >> (k & 6) * 2 & 15);
            }
            for (int j = 0; j < nc / G; ++j) {
                const uint8_t* s = in + g4_scale_off(nc) + (g * (nc / G) + j) * 4 + h * 2;
                const int64_t at = r * ng + k0 / G + j;
                scales[at] = (uint16_t)(s[0] | s[1] << 8);
                if (zeros) zeros[at] = (uint8_t)(in[g4_zero_off(nc, G) + g * (nc / G) + j] >> h * 4 & 15);
            }
            in += g4_chunk_bytes(nc, G, zeros != nullptr);
        }
    }
}

}  // namespace rfx
