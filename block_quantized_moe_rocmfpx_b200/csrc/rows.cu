// rows.cu -- token rows grouped by expert and brought back, with gradients.
//
// Entry i = t * k + j routes token t to expert idx[t][j].  The rows of the
// grouped order are the entries sorted by (expert, i): row pos[t][j] holds
// x[t], expert e owns rows offsets[e] .. offsets[e+1].  The way back is
// y[t] = base[t] + sum_j w[t][j] ys[pos[t][j]].
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch_util.h"
#include "moe_decode.h"
#include "rfx_device.cuh"
#include "rows.h"

namespace rfx {
namespace {

constexpr int GT = 512;          // threads of a grouping CTA
constexpr int GROUP_MAXE = 1024;
constexpr int GROUP_BATCH = 512; // entries placed per batch
constexpr int GROUP_ONE = 4096;  // entries up to which every CTA counts all of idx itself

// ------------------------------------------------------------- grouping ---

__global__ void __launch_bounds__(GT) group_count_kernel(GroupParams p) {
    __shared__ int32_t hist[GROUP_MAXE];
    grid_dep_launch();
    for (int e = threadIdx.x; e < p.E; e += GT) hist[e] = 0;
    __syncthreads();
    grid_dep_wait();
    const long long i0 = (long long)blockIdx.x * p.per * p.k;
    const long long i1 = min(i0 + (long long)p.per * p.k, (long long)p.T * p.k);
    for (long long i = i0 + threadIdx.x; i < i1; i += GT) {
        const int e = p.idx[i];
        if ((unsigned)e < (unsigned)p.E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    int32_t* out = p.part + (long long)blockIdx.x * group_pitch(p.E);
    for (int e = threadIdx.x; e < group_pitch(p.E); e += GT) out[e] = e < p.E ? hist[e] : 0;
}

// One CTA per slice: first rows of the slice's experts (ONE: by counting all
// of idx; else from the counts of the slices), the places of its entries in
// order, and the copies of its tokens' rows.
template <bool ONE, typename V>
__global__ void __launch_bounds__(GT) group_place_kernel(GroupParams p) {
    __shared__ __align__(16) int32_t tot[GROUP_MAXE];
    __shared__ __align__(16) int32_t cur[GROUP_MAXE];
    __shared__ int32_t wsum[GT / 32];
    __shared__ int32_t s_pos[GROUP_BATCH];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_launch();
    for (int e = tid; e < GROUP_MAXE; e += GT) {
        tot[e] = 0;
        cur[e] = 0;
    }
    __syncthreads();
    grid_dep_wait();
    const long long n = (long long)p.T * p.k;
    const int t0 = blockIdx.x * p.per;
    const int t1 = min(t0 + p.per, p.T);
    const long long first = (long long)t0 * p.k;
    if constexpr (ONE) {
        for (long long i = tid; i < n; i += GT) {
            const int e = p.idx[i];
            if ((unsigned)e < (unsigned)p.E) {
                atomicAdd(&tot[e], 1);
                if (i < first) atomicAdd(&cur[e], 1);
            }
        }
    } else {
        const int pitch = group_pitch(p.E), quads = pitch >> 2;
        const int lines = GT / quads;      // quads <= 256: at least two lines
        const int q = tid % quads, l = tid / quads;
        if (l < lines) {
            int4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
#pragma unroll 8
            for (int s = l; s < p.slices; s += lines) {
                const int4 v = *reinterpret_cast<const int4*>(p.part + (long long)s * pitch + 4 * q);
                a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
                if (s < (int)blockIdx.x) { b.x += v.x; b.y += v.y; b.z += v.z; b.w += v.w; }
            }
            atomicAdd(&tot[4 * q + 0], a.x); atomicAdd(&tot[4 * q + 1], a.y);
            atomicAdd(&tot[4 * q + 2], a.z); atomicAdd(&tot[4 * q + 3], a.w);
            atomicAdd(&cur[4 * q + 0], b.x); atomicAdd(&cur[4 * q + 1], b.y);
            atomicAdd(&cur[4 * q + 2], b.z); atomicAdd(&cur[4 * q + 3], b.w);
        }
    }
    __syncthreads();
    // exclusive sum of tot over the experts, two per thread
    {
        const int a = tot[2 * tid], b = tot[2 * tid + 1];
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
        for (int w = 0; w < GT / 32; ++w) before += w < warp ? wsum[w] : 0;
        const int ex = before + s - a - b;
        cur[2 * tid] += ex;
        cur[2 * tid + 1] += ex + a;
        if (blockIdx.x == 0) {
            if (2 * tid < p.E) p.offsets[2 * tid] = ex;
            if (2 * tid + 1 < p.E) p.offsets[2 * tid + 1] = ex + a;
            if (tid == GT - 1) p.offsets[p.E] = before + s;
        }
    }
    __syncthreads();
    const int tb = GROUP_BATCH / p.k;   // tokens per batch
    for (int ta = t0; ta < t1; ta += tb) {
        const int nt = min(tb, t1 - ta);
        if (warp == 0) {
            // 32 entries a step: lanes of one expert rank themselves by lane
            bool bad = false;
            for (int i = 0; i < nt * p.k; i += 32) {
                const int m = i + lane;
                const long long ent = (long long)ta * p.k + m;
                int e = -1;
                if (m < nt * p.k) {
                    e = p.idx[ent];
                    if ((unsigned)e >= (unsigned)p.E) {
                        bad |= e != -1;
                        e = -1;
                    }
                }
                const unsigned same = __match_any_sync(0xffffffffu, e);
                const int rank = __popc(same & ((1u << lane) - 1u));
                int at = -1;
                if (e >= 0) at = cur[e] + rank;
                __syncwarp();
                if (e >= 0 && rank == 0) cur[e] += __popc(same);
                __syncwarp();
                if (m < nt * p.k) {
                    s_pos[m] = at;
                    p.pos[ent] = at;
                    if (at >= 0) p.rows[at] = (int32_t)ent;
                }
            }
            if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.ctrl + MOE_CTRL_ERR, MOE_ERR_EXPERT);
        }
        __syncthreads();
        if (p.x) {
            const int nv = (int)(p.row_bytes / (long long)sizeof(V));
            const long long items = (long long)nt * nv;
            for (long long i = tid; i < items; i += GT) {
                const int t = (int)(i / nv), c = (int)(i % nv);
                const V v = reinterpret_cast<const V*>(p.x + (long long)(ta + t) * p.row_bytes)[c];
                for (int j = 0; j < p.k; ++j) {
                    const int at = s_pos[t * p.k + j];
                    if (at >= 0) reinterpret_cast<V*>(p.xs + (long long)at * p.row_bytes)[c] = v;
                }
            }
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------- conversions ---

template <typename E> __device__ __forceinline__ float to_f(E v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename E> __device__ __forceinline__ E from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

template <typename E, int N>
struct alignas(sizeof(E) * N < 16 ? sizeof(E) * N : 16) Vec { E v[N]; };

// -------------------------------------------------------------- combine ---

template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(256) combine_kernel(const TI* __restrict__ ys, int T, int H,
                                                      const int32_t* __restrict__ pos, int k,
                                                      const float* __restrict__ w, const TO* base, TO* y,
                                                      int blocks_per_row) {
    grid_dep_launch();
    grid_dep_wait();
    const int t = blockIdx.x / blocks_per_row;
    const int c = ((int)(blockIdx.x % blocks_per_row) * 256 + threadIdx.x) * N;
    if (c >= H) return;
    const long long R = (long long)T * k;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int j = 0; j < k; ++j) {
        const int at = pos[(long long)t * k + j];
        if ((unsigned long long)(long long)at >= (unsigned long long)R) continue;
        const Vec<TI, N> v = *reinterpret_cast<const Vec<TI, N>*>(ys + (long long)at * H + c);
        if (w) {
            const float wj = w[(long long)t * k + j];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(wj, to_f(v.v[i]), acc[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += to_f(v.v[i]);
        }
    }
    Vec<TO, N> o;
    if (base) {
        const Vec<TO, N> b = *reinterpret_cast<const Vec<TO, N>*>(base + (long long)t * H + c);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += to_f(b.v[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f<TO>(acc[i]);
    *reinterpret_cast<Vec<TO, N>*>(y + (long long)t * H + c) = o;
}

template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(256) combine_backward_kernel(const TO* __restrict__ dy, const TI* __restrict__ ys,
                                                               int T, int H, const int32_t* __restrict__ pos, int k,
                                                               const float* __restrict__ w, TI* __restrict__ dys,
                                                               float* __restrict__ dw) {
    __shared__ float part[8];
    grid_dep_launch();
    grid_dep_wait();
    const int t = blockIdx.x;
    const long long R = (long long)T * k;
    for (int j = 0; j < k; ++j) {
        const int at = pos[(long long)t * k + j];
        const bool live = (unsigned long long)(long long)at < (unsigned long long)R;
        float s = 0.f;
        if (live) {
            const float wj = w[(long long)t * k + j];
            for (int c = threadIdx.x * N; c < H; c += 256 * N) {
                const Vec<TO, N> d = *reinterpret_cast<const Vec<TO, N>*>(dy + (long long)t * H + c);
                const Vec<TI, N> v = *reinterpret_cast<const Vec<TI, N>*>(ys + (long long)at * H + c);
                Vec<TI, N> o;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    s = fmaf(to_f(d.v[i]), to_f(v.v[i]), s);
                    o.v[i] = from_f<TI>(wj * to_f(d.v[i]));
                }
                *reinterpret_cast<Vec<TI, N>*>(dys + (long long)at * H + c) = o;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            float z = 0.f;
            for (int i = 0; i < 8; ++i) z += part[i];
            dw[(long long)t * k + j] = z;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------- router gradient ---

// w = softmax of the k selected logits: d l_j = w_j (dw_j - sum_i w_i dw_i),
// nothing for the others.  One warp per token.
__global__ void __launch_bounds__(256) router_backward_kernel(const int32_t* __restrict__ idx,
                                                              const float* __restrict__ w,
                                                              const float* __restrict__ dw, int T, int E, int k,
                                                              float* __restrict__ dlogits) {
    grid_dep_launch();
    grid_dep_wait();
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= T) return;
    float* out = dlogits + (long long)t * E;
    int e = -1;
    float wj = 0.f, gj = 0.f;
    if (lane < k) {
        e = idx[(long long)t * k + lane];
        wj = w[(long long)t * k + lane];
        gj = dw[(long long)t * k + lane];
    }
    float s = wj * gj;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float d = wj * (gj - s);
    // an id that appears twice receives the sum of its entries
    float sum = 0.f;
    for (int j = 0; j < k; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, j);
        const float dj = __shfl_sync(0xffffffffu, d, j);
        if (ej == e) sum += dj;
    }
    for (int i = lane; i < E; i += 32) out[i] = 0.f;
    __syncwarp();
    if (lane < k && (unsigned)e < (unsigned)E) out[e] = sum;
}

template <typename TI, typename TO>
cudaError_t combine_t(const void* ys, int T, int H, const int32_t* pos, int k, const float* w, const void* base,
                      void* y, cudaStream_t stream) {
    constexpr int N = 8;
    const uintptr_t a = (uintptr_t)ys | (uintptr_t)base | (uintptr_t)y;
    if (H % N == 0 && (a & 15u) == 0) {
        const int bpr = (H / N + 255) / 256;
        return launch_dependent(combine_kernel<TI, TO, N>, (unsigned)T * bpr, 256, 0, stream, (const TI*)ys, T, H, pos,
                                k, w, (const TO*)base, (TO*)y, bpr);
    }
    const int bpr = (H + 255) / 256;
    return launch_dependent(combine_kernel<TI, TO, 1>, (unsigned)T * bpr, 256, 0, stream, (const TI*)ys, T, H, pos, k,
                            w, (const TO*)base, (TO*)y, bpr);
}

template <typename TI, typename TO>
cudaError_t combine_backward_t(const void* dy, const void* ys, int T, int H, const int32_t* pos, int k, const float* w,
                               void* dys, float* dw, cudaStream_t stream) {
    constexpr int N = 8;
    const uintptr_t a = (uintptr_t)ys | (uintptr_t)dy | (uintptr_t)dys;
    if (H % N == 0 && (a & 15u) == 0)
        return launch_dependent(combine_backward_kernel<TI, TO, N>, (unsigned)T, 256, 0, stream, (const TO*)dy,
                                (const TI*)ys, T, H, pos, k, w, (TI*)dys, dw);
    return launch_dependent(combine_backward_kernel<TI, TO, 1>, (unsigned)T, 256, 0, stream, (const TO*)dy,
                            (const TI*)ys, T, H, pos, k, w, (TI*)dys, dw);
}

}  // namespace

int group_slices(int T, int k) {
    (void)k;
    return std::min(T, 296);
}
bool group_two_launches(int T, int k) { return (long long)T * k > GROUP_ONE; }

cudaError_t group_launch(const GroupParams& p0, cudaStream_t stream) {
    GroupParams p = p0;
    const bool two = group_two_launches(p.T, p.k);
    const int want = group_slices(p.T, p.k);
    p.per = (p.T + want - 1) / want;
    p.slices = (p.T + p.per - 1) / p.per;
    if (two) {
        cudaError_t e = launch_dependent(group_count_kernel, p.slices, GT, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    const uintptr_t a = (uintptr_t)p.x | (uintptr_t)p.xs | (uintptr_t)p.row_bytes;
    if ((a & 15u) == 0)
        return two ? launch_dependent(group_place_kernel<false, uint4>, p.slices, GT, 0, stream, p)
                   : launch_dependent(group_place_kernel<true, uint4>, p.slices, GT, 0, stream, p);
    if ((a & 3u) == 0)
        return two ? launch_dependent(group_place_kernel<false, uint32_t>, p.slices, GT, 0, stream, p)
                   : launch_dependent(group_place_kernel<true, uint32_t>, p.slices, GT, 0, stream, p);
    return two ? launch_dependent(group_place_kernel<false, uint16_t>, p.slices, GT, 0, stream, p)
               : launch_dependent(group_place_kernel<true, uint16_t>, p.slices, GT, 0, stream, p);
}

cudaError_t combine_launch(const void* ys, int dtype, int T, int H, const int32_t* pos, int k, const float* w,
                           const void* base, void* y, int y_dtype, cudaStream_t stream) {
    if (dtype == 1) return combine_t<float, float>(ys, T, H, pos, k, w, base, y, stream);
    if (dtype == 0)
        return y_dtype == 1 ? combine_t<__nv_bfloat16, float>(ys, T, H, pos, k, w, base, y, stream)
                            : combine_t<__nv_bfloat16, __nv_bfloat16>(ys, T, H, pos, k, w, base, y, stream);
    return y_dtype == 1 ? combine_t<__half, float>(ys, T, H, pos, k, w, base, y, stream)
                        : combine_t<__half, __half>(ys, T, H, pos, k, w, base, y, stream);
}

cudaError_t combine_backward_launch(const void* dy, int y_dtype, const void* ys, int dtype, int T, int H,
                                    const int32_t* pos, int k, const float* w, void* dys, float* dw,
                                    cudaStream_t stream) {
    if (dtype == 1) return combine_backward_t<float, float>(dy, ys, T, H, pos, k, w, dys, dw, stream);
    if (dtype == 0)
        return y_dtype == 1 ? combine_backward_t<__nv_bfloat16, float>(dy, ys, T, H, pos, k, w, dys, dw, stream)
                            : combine_backward_t<__nv_bfloat16, __nv_bfloat16>(dy, ys, T, H, pos, k, w, dys, dw, stream);
    return y_dtype == 1 ? combine_backward_t<__half, float>(dy, ys, T, H, pos, k, w, dys, dw, stream)
                        : combine_backward_t<__half, __half>(dy, ys, T, H, pos, k, w, dys, dw, stream);
}

cudaError_t router_backward_launch(const int32_t* idx, const float* w, const float* dw, int T, int E, int k,
                                   float* dlogits, cudaStream_t stream) {
    return launch_dependent(router_backward_kernel, (unsigned)(T + 7) / 8, 256, 0, stream, idx, w, dw, T, E, k,
                            dlogits);
}

}  // namespace rfx
