// g4.cuh -- products with 4-bit weights in groups (layout: g4_layout.h), for
// up to 8 columns a pass: y[c][n] = sum_g scale[n][g] sum_k (code - zero) x[c][k].
//
// The bracket is taken on the tensor cores (mma.sync m16n8k16, 16 rows x 8
// columns) with exact operands: code - zero is a small integer, formed in
// registers by or-ing the code into the mantissa of 128 (bf16) or 1024 (fp16)
// and subtracting 128 + zero or 1024 + zero; x enters as it is (bf16, fp16) or
// as three bf16 parts that add up to it (fp32).  So the only roundings are the
// fp32 sums and the scale's product.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "g4.h"
#include "g4_layout.h"
#include "launch_util.h"
#include "rfx_device.cuh"

namespace rfx {
namespace {

constexpr int G4_THREADS = 512;
constexpr int G4_WARPS = G4_THREADS / 32;
constexpr int G4_MAXE = 1024;

__device__ __forceinline__ uint32_t g4_bf16_sub(uint32_t a, uint32_t b) {
    __nv_bfloat162 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = __hsub2(x, y);
    memcpy(&a, &x, 4);
    return a;
}
__device__ __forceinline__ uint32_t g4_f16_sub(uint32_t a, uint32_t b) {
    __half2 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = __hsub2(x, y);
    memcpy(&a, &x, 4);
    return a;
}
// a / 16 - b, exact here
__device__ __forceinline__ uint32_t g4_f16_sub16(uint32_t a, uint32_t b) {
    __half2 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = __hfma2(x, __float2half2_rn(0.0625f), __hneg2(y));
    memcpy(&a, &x, 4);
    return a;
}

// The four A registers of one word: codes 2i, 2i + 1 of the lane minus z, as
// bf16 or fp16 pairs.
template <bool F16>
__device__ __forceinline__ void g4_unpack(uint32_t w, uint32_t z, uint32_t a[4]) {
    if constexpr (F16) {
        const uint32_t lo = 0x64006400u + z * 0x00010001u;            // 1024 + z
        const uint32_t hi = 0x54005400u + z * 0x00100010u;            // 64 + z
        const uint32_t w8 = w >> 8;
        a[0] = g4_f16_sub((w & 0x000F000Fu) | 0x64006400u, lo);
        a[1] = g4_f16_sub16((w & 0x00F000F0u) | 0x64006400u, hi);
        a[2] = g4_f16_sub((w8 & 0x000F000Fu) | 0x64006400u, lo);
        a[3] = g4_f16_sub16((w8 & 0x00F000F0u) | 0x64006400u, hi);
    } else {
        const uint32_t c = 0x43004300u + z * 0x00010001u;             // 128 + z
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = g4_bf16_sub(((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, c);
    }
}

// The B operands of one tile for the lane: columns 8t .. 8t + 7 of its x row.
// fp32 x = p0 + p1 + p2 with bf16 parts cut off the top of the significand
// (8 + 8 + 8 bits), so the three products add up to the exact one.
template <int XT>
struct G4B {
    static constexpr int PARTS = XT == 1 ? 3 : 1;
    uint32_t v[PARTS][4];
    __device__ __forceinline__ void load(const void* x, long long at, bool live) {
        if constexpr (XT != 1) {
            uint4 q = {0u, 0u, 0u, 0u};
            if (live) q = __ldg(reinterpret_cast<const uint4*>((const uint16_t*)x + at));
            v[0][0] = q.x; v[0][1] = q.y; v[0][2] = q.z; v[0][3] = q.w;
        } else {
            float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (live) {
                const float4 a = __ldg(reinterpret_cast<const float4*>((const float*)x + at));
                const float4 b = __ldg(reinterpret_cast<const float4*>((const float*)x + at) + 1);
                f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
                f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t u0 = __float_as_uint(f[2 * i]), u1 = __float_as_uint(f[2 * i + 1]);
                v[0][i] = __byte_perm(u0, u1, 0x7632);
                float r0 = f[2 * i] - __uint_as_float(u0 & 0xFFFF0000u);
                float r1 = f[2 * i + 1] - __uint_as_float(u1 & 0xFFFF0000u);
                u0 = __float_as_uint(r0);
                u1 = __float_as_uint(r1);
                v[1][i] = __byte_perm(u0, u1, 0x7632);
                r0 -= __uint_as_float(u0 & 0xFFFF0000u);
                r1 -= __uint_as_float(u1 & 0xFFFF0000u);
                v[2][i] = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
            }
        }
    }
};

// One chunk of nc columns of two row-groups into acc.
template <int XT, int G, bool Z>
__device__ __forceinline__ void g4_chunk(const uint8_t* c0, const uint8_t* c1, int nc, const void* x, long long xat,
                                         bool live, int lane, float acc[2][4]) {
    constexpr bool F16 = XT == 2;
    const int g = lane >> 2;
    const int soff = g4_scale_off(nc), zoff = g4_zero_off(nc, G);
    const uint8_t* const ch[2] = {c0, c1};
    float s[2][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        if (p * 64 < nc) {
            uint4 w[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) w[r] = *reinterpret_cast<const uint4*>(ch[r] + p * 512 + lane * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = p * 64 + h * 32;
                if (col < nc) {
                    G4B<XT> b;
                    b.load(x, xat + col, live);
                    const int grp = col / G;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (col % G == 0)
                            for (int i = 0; i < 4; ++i) s[r][i] = 0.f;
                        uint32_t z0 = 8, z1 = 8;
                        if constexpr (Z) {
                            const uint32_t zz = ch[r][zoff + grp * 8 + g];
                            z0 = zz & 15u;
                            z1 = zz >> 4;
                        }
                        uint32_t a0[4], a1[4];
                        g4_unpack<F16>(h ? w[r].z : w[r].x, z0, a0);
                        g4_unpack<F16>(h ? w[r].w : w[r].y, z1, a1);
                        const uint32_t m0[4] = {a0[0], a1[0], a0[1], a1[1]};
                        const uint32_t m1[4] = {a0[2], a1[2], a0[3], a1[3]};
#pragma unroll
                        for (int q = 0; q < G4B<XT>::PARTS; ++q) {
                            mma16816<F16>(s[r], m0, b.v[q][0], b.v[q][1], s[r]);
                            mma16816<F16>(s[r], m1, b.v[q][2], b.v[q][3], s[r]);
                        }
                        if ((col + 32) % G == 0) {
                            const __half2 sc = *reinterpret_cast<const __half2*>(ch[r] + soff + (grp * 8 + g) * 4);
                            const float2 f = __half22float2(sc);
                            acc[r][0] = fmaf(f.x, s[r][0], acc[r][0]);
                            acc[r][1] = fmaf(f.x, s[r][1], acc[r][1]);
                            acc[r][2] = fmaf(f.y, s[r][2], acc[r][2]);
                            acc[r][3] = fmaf(f.y, s[r][3], acc[r][3]);
                        }
                    }
                }
            }
        }
    }
}

__device__ __forceinline__ float g4_silu_mul(float g, float u) {
    return g < -64.f ? silu_mul_tail(g, u) : g / (1.f + expf(-g)) * u;
}

// A unit is two row-groups against up to 8 rows of x: rows 32u .. 32u + 31 of
// the matrix, or (PAIR) the gate and the up rows 16u .. 16u + 15.  A team of
// p.team warps shares a unit, warp i of it the chunks i, i + team, ...; the
// partial sums meet in shared memory and are added in warp order.
template <int XT, int G, bool Z, bool PAIR>
__global__ void __launch_bounds__(G4_THREADS, 1) g4_kernel(G4Params p) {
    __shared__ float red[2][G4_WARPS][8][32];
    __shared__ int32_t blk[G4_MAXE + 1];   // column blocks before expert e
    __shared__ int32_t wsum[G4_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_launch();
    grid_dep_wait();
    int blocks = 1;
    if (p.offsets) {
        auto rows_of = [&](int e) {
            if (e >= p.E) return 0;
            const int lo = max(0, min(p.offsets[e], p.R)), hi = max(0, min(p.offsets[e + 1], p.R));
            return max(0, hi - lo);
        };
        const int a = (rows_of(2 * tid) + 7) >> 3, b = (rows_of(2 * tid + 1) + 7) >> 3;
        int s = a + b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += v;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        int before = 0;
#pragma unroll
        for (int w = 0; w < G4_WARPS; ++w) before += w < warp ? wsum[w] : 0;
        blk[2 * tid] = before + s - a - b;
        blk[2 * tid + 1] = before + s - b;
        if (tid == G4_THREADS - 1) blk[G4_MAXE] = before + s;
        __syncthreads();
        blocks = blk[G4_MAXE];
    }
    const int team = warp / p.team, member = warp % p.team, teams = G4_WARPS / p.team;
    const long long total = (long long)blocks * p.units;
    const long long step = (long long)gridDim.x * teams;
    const int rgs = (p.N + 15) / 16;
    const int full = g4_chunk_bytes(G4_CHUNK, G, Z);
    int par = 0;
    for (long long u = (long long)blockIdx.x + (long long)team * gridDim.x; u < total; u += step) {
        const int slot = (int)(u / p.units), unit = (int)(u % p.units);
        int e = 0, row0 = 0, cols = p.R;
        if (p.offsets) {
            int lo = 0, hi = p.E;   // the largest e with blk[e] <= slot
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (blk[mid] <= slot) lo = mid;
                else hi = mid;
            }
            e = lo;
            row0 = max(0, min(p.offsets[e], p.R)) + 8 * (slot - blk[e]);
            cols = min(8, max(0, min(p.offsets[e + 1], p.R)) - row0);
        }
        const uint8_t* r0;
        const uint8_t* r1;
        if constexpr (PAIR) {
            r0 = p.W0 + e * p.stride + unit * p.rg_bytes;
            r1 = p.W1 + e * p.stride + unit * p.rg_bytes;
        } else {
            r0 = p.W0 + e * p.stride + 2LL * unit * p.rg_bytes;
            r1 = 2 * unit + 1 < rgs ? r0 + p.rg_bytes : r0;   // past the end: read again, dropped below
        }
        const int g = lane >> 2, t = lane & 3;
        const bool live = g < cols;
        const long long xrow = (long long)(row0 + g) * p.K + 8 * t;
        float acc[2][4] = {};
        for (int c = member; c < p.chunks; c += p.team) {
            const int nc = min(G4_CHUNK, p.K - c * G4_CHUNK);
            g4_chunk<XT, G, Z>(r0 + (long long)c * full, r1 + (long long)c * full, nc, p.x, xrow + c * G4_CHUNK, live,
                               lane, acc);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) red[par][warp][i][lane] = acc[i >> 2][i & 3];
        if (p.team > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * p.team) : "memory");
        else __syncwarp();
        constexpr int OUT = PAIR ? 128 : 256;
        for (int o = member * 32 + lane; o < OUT; o += 32 * p.team) {
            const int i = o >> 5, l = o & 31;
            const int col = 2 * (l & 3) + (i & 1);
            const int row = (PAIR ? 16 : 32) * unit + (i >> 2) * 16 + ((i & 2) ? 8 : 0) + (l >> 2);
            if (col < cols && row < p.N) {
                float a = 0.f, b = 0.f;
                for (int w = 0; w < p.team; ++w) {
                    a += red[par][team * p.team + w][i][l];
                    if constexpr (PAIR) b += red[par][team * p.team + w][i + 4][l];
                }
                p.y[(long long)(row0 + col) * p.N + row] = PAIR ? g4_silu_mul(a, b) : a;
            }
        }
        par ^= 1;
    }
}

// Warps per unit: the fewest rounds of chunks, and of equals the fewest warps
// (less to add up).
inline int g4_team(long long units, int chunks, int sms) {
    int best = 1;
    long long cost = -1;
    for (int s = 1; s <= G4_WARPS; s *= 2) {
        if (s > 1 && s > chunks) break;
        const long long teams = (long long)sms * (G4_WARPS / s);
        const long long c = (units + teams - 1) / teams * ((chunks + s - 1) / s);
        if (cost < 0 || c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

template <int XT, int G, bool Z>
cudaError_t g4_launch_t(G4Params p, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = device_sms(sms);
    if (e != cudaSuccess) return e;
    p.rg_bytes = g4_rowgroup_bytes(p.K, G, Z);
    p.chunks = (p.K + G4_CHUNK - 1) / G4_CHUNK;
    p.units = p.W1 ? (p.N + 15) / 16 : (p.N + 31) / 32;
    const long long units = (long long)p.units * (p.offsets ? std::min(p.E, p.R) : 1);
    p.team = g4_team(units, p.chunks, sms);
    // at most one column block per row, so never more units than this
    const long long most = (long long)p.units * (p.offsets ? p.R : 1);
    const int grid = (int)std::min<long long>(sms, most);
    return p.W1 ? launch_dependent(g4_kernel<XT, G, Z, true>, grid, G4_THREADS, 0, stream, p)
                : launch_dependent(g4_kernel<XT, G, Z, false>, grid, G4_THREADS, 0, stream, p);
}

template <int XT>
cudaError_t g4_launch_x(const G4Params& p, int G, bool zeros, cudaStream_t stream) {
    switch (G) {
        case 32: return zeros ? g4_launch_t<XT, 32, true>(p, stream) : g4_launch_t<XT, 32, false>(p, stream);
        case 64: return zeros ? g4_launch_t<XT, 64, true>(p, stream) : g4_launch_t<XT, 64, false>(p, stream);
        default: return zeros ? g4_launch_t<XT, 128, true>(p, stream) : g4_launch_t<XT, 128, false>(p, stream);
    }
}

}  // namespace
}  // namespace rfx
