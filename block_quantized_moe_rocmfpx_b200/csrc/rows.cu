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
constexpr int GROUP_BATCH = GT;  // entries placed per batch, one per thread
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

// 8192 tokens x 6 rows of 8 KB: 95 us, of which the places are 9; 403 MB written and 67 read, so the writes are
// what it waits for (each x row is read once; stores by threads took as long).
//
// Copies of a CTA's rows by bulk stores: a warp brings a piece of a token's row into
// one of its GROUP_SLOTS buffers in shared memory (cp.async), and lanes 0 .. k - 1 each
// store it whole to one of the rows that it goes to.  Pieces of later tokens are on their
// way meanwhile; a buffer is filled again once its stores have read it.
constexpr int GROUP_PIECE = 4096;
constexpr int GROUP_SLOTS = 3;
constexpr int GROUP_SMEM = GT / 32 * GROUP_SLOTS * GROUP_PIECE;

__device__ __forceinline__ void group_copy(const GroupParams& p, int ta, int nt, const int32_t* s_pos, uint8_t* ring) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pieces = (int)((p.row_bytes + GROUP_PIECE - 1) / GROUP_PIECE), items = nt * pieces;
    uint8_t* mine = ring + warp * (GROUP_SLOTS * GROUP_PIECE);
    const uint32_t mine_s = smem_u32(mine);
    auto bytes_of = [&](int q) { return (int)min((long long)GROUP_PIECE, p.row_bytes - (long long)q * GROUP_PIECE); };
    auto load = [&](int i, int slot) {
        if (i < items) {
            const int t = i / pieces, q = i - t * pieces, n = bytes_of(q);
            const uint8_t* src = p.x + (long long)(ta + t) * p.row_bytes + (long long)q * GROUP_PIECE;
            for (int o = lane * 16; o < n; o += 512)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine_s + slot * GROUP_PIECE + o), "l"(src + o)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load(warp, 0);
    load(warp + GT / 32, 1);
    int slot = 0;
    for (int i = warp; i < items; i += GT / 32) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // every lane's copies, before the bulk stores read them
        __syncwarp();
        const int t = i / pieces, q = i - t * pieces;
        if (lane < p.k) {
            const int r = s_pos[t * p.k + lane];
            if (r >= 0) {
                uint8_t* dst = p.xs + (long long)r * p.row_bytes + (long long)q * GROUP_PIECE;
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                             "r"(mine_s + slot * GROUP_PIECE), "r"(bytes_of(q))
                             : "memory");
            }
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        // the buffer of the piece after next is the one stored before this: all but the last group have been read
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
        load(i + 2 * (GT / 32), slot >= 1 ? slot - 1 : GROUP_SLOTS - 1);
        slot = slot + 1 == GROUP_SLOTS ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// One CTA per slice: first rows of the slice's experts (ONE: by counting all
// of idx; else from the counts of the slices), the places of its entries in
// order, and the copies of its tokens' rows.
template <bool ONE, bool BULK, typename V>
__global__ void __launch_bounds__(GT) group_place_kernel(GroupParams p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) int32_t tot[GROUP_MAXE];
    __shared__ __align__(16) int32_t cur[GROUP_MAXE];
    __shared__ int32_t wsum[GT / 32];
    __shared__ int32_t s_pos[GROUP_BATCH];   // places of a batch's entries
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
    const int tb = GROUP_BATCH / p.k;   // tokens per batch
    int next = tid < min(tb, t1 - t0) * p.k ? p.idx[first + tid] : -1;   // the thread's entry of the next batch
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
            for (int s0 = l; s0 < p.slices; s0 += 10 * lines) {
                int4 v[10];   // all on their way at once
#pragma unroll
                for (int i = 0; i < 10; ++i) {
                    const int s = s0 + i * lines;
                    v[i] = make_int4(0, 0, 0, 0);
                    if (s < p.slices) v[i] = __ldcg(reinterpret_cast<const int4*>(p.part + (long long)s * pitch) + q);
                }
#pragma unroll
                for (int i = 0; i < 10; ++i) {
                    const int4 u = v[i];
                    a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
                    if (s0 + i * lines < (int)blockIdx.x) { b.x += u.x; b.y += u.y; b.z += u.z; b.w += u.w; }
                }
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
    for (int ta = t0; ta < t1; ta += tb) {
        const int nt = min(tb, t1 - ta);
        // an entry per thread: lanes of one expert rank themselves by lane, the warps take their turns
        const int m = nt * p.k;
        const long long ent = (long long)ta * p.k + tid;
        int e = next;
        const bool bad = tid < m && e != -1 && (unsigned)e >= (unsigned)p.E;
        if (tid >= m || bad) e = -1;
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.ctrl + MOE_CTRL_ERR, MOE_ERR_EXPERT);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int at = -1;
        for (int w = 0; w < (m + 31) >> 5; ++w) {
            if (warp == w) {
                if (e >= 0) at = cur[e] + rank;
                __syncwarp();
                if (e >= 0 && rank == 0) cur[e] += __popc(same);
            }
            __syncthreads();
        }
        if (tid < m) {
            s_pos[tid] = at;
            p.pos[ent] = at;
            if (at >= 0) p.rows[at] = (int32_t)ent;
        }
        const int tn = ta + tb;
        if (tn < t1) next = tid < min(tb, t1 - tn) * p.k ? p.idx[(long long)tn * p.k + tid] : -1;
        __syncthreads();
        if constexpr (BULK) {
            group_copy(p, ta, nt, s_pos, ring);
        } else if (p.x) {
            // `span` threads a token (a power of two, a warp at least), U vectors of its row in flight each
            constexpr int U = 4;
            const int nv = (int)(p.row_bytes / (long long)sizeof(V));
            int span = GT;
            while (span > 32 && GT / span < nt) span >>= 1;
            for (int t = tid / span; t < nt; t += GT / span) {
                const V* src = reinterpret_cast<const V*>(p.x + (long long)(ta + t) * p.row_bytes);
                const int32_t* at = s_pos + t * p.k;
                for (int c0 = tid & (span - 1); c0 < nv; c0 += U * span) {
                    V v[U];
#pragma unroll
                    for (int i = 0; i < U; ++i)
                        if (c0 + i * span < nv) v[i] = __ldg(src + c0 + i * span);
                    for (int j = 0; j < p.k; ++j) {
                        const int r = at[j];
                        if (r < 0) continue;
                        V* dst = reinterpret_cast<V*>(p.xs + (long long)r * p.row_bytes) + c0;
#pragma unroll
                        for (int i = 0; i < U; ++i)
                            if (c0 + i * span < nv) dst[i * span] = v[i];
                    }
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

// A thread takes N neighbouring elements of a token: the k rows' loads are issued
// together (ROWS at a time), then added in the order of j.  Bound by memory: each
// row is read once, in pieces of 16 bytes a thread.  1999 tokens x 8 rows of 5 KB (92 MB): 18.7 us, 4.9 TB/s with the
// launch; one piece a thread in short-lived CTAs took 19.6, rows one after the other 21.
constexpr int ROWS = 8;
constexpr int COMBINE_CTAS = 3;   // CTAs per SM: 24 warps with 8 rows in flight each

template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(256, COMBINE_CTAS) combine_kernel(const TI* __restrict__ ys, int T, int H,
                                                          const int32_t* __restrict__ pos, int k,
                                                          const float* __restrict__ w, const TO* base, TO* y) {
    const int per = H / N;                                     // pieces of a row
    const unsigned long long R = (unsigned long long)T * k;
    // the thread's first piece, and how far it is to the next (in tokens and pieces)
    const long long item = (long long)blockIdx.x * 256 + threadIdx.x, step = (long long)gridDim.x * 256;
    long long t = item / per;
    int c = (int)(item - t * per);
    const long long dt = step / per;
    const int dc = (int)(step - dt * per);
    grid_dep_launch();
    grid_dep_wait();
    int at[ROWS];
    auto places = [&](long long t, int j0) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const long long r = t < T && j0 + j < k ? pos[t * k + j0 + j] : -1;
            at[j] = (unsigned long long)r < R ? (int)r : -1;
        }
    };
    places(t, 0);
    while (t < T) {
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        const long long here = t * H + (long long)c * N;
        long long tn = t + dt;
        int cn = c + dc;
        if (cn >= per) {
            cn -= per;
            ++tn;
        }
        for (int j0 = 0; j0 < k; j0 += ROWS) {
            float wj[ROWS];
            Vec<TI, N> v[ROWS];
            unsigned live = 0;
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                if (at[j] >= 0) {
                    v[j] = *reinterpret_cast<const Vec<TI, N>*>(ys + (long long)at[j] * H + c * N);
                    wj[j] = w ? w[t * k + j0 + j] : 1.f;
                    live |= 1u << j;
                }
            // the places of the next rows come while these are on their way
            if (j0 + ROWS < k) places(t, j0 + ROWS);
            else places(tn, 0);
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                if (live >> j & 1u)
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[i] = fmaf(wj[j], to_f(v[j].v[i]), acc[i]);
        }
        Vec<TO, N> o;
        if (base) {
            const Vec<TO, N> b = *reinterpret_cast<const Vec<TO, N>*>(base + here);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += to_f(b.v[i]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) o.v[i] = from_f<TO>(acc[i]);
        *reinterpret_cast<Vec<TO, N>*>(y + here) = o;
        t = tn;
        c = cn;
    }
}

// One CTA per token; a thread reads its pieces of dy once for all k rows.  The k dot
// products are summed per thread, then over the warp and the warps in a fixed order.
// Bound by memory: 4096 tokens x 6 rows of 8 KB (470 MB): 84.8 us, 5.5 TB/s; with three CTAs a SM (fewer registers,
// spills) 108, dy read again for every row 88.
template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(256, 2) combine_backward_kernel(const TO* __restrict__ dy, const TI* ys, int T, int H,
                                                               const int32_t* __restrict__ pos, int k,
                                                               const float* __restrict__ w, TI* dys,
                                                               float* __restrict__ dw) {
    __shared__ float part[8][16];
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const unsigned long long R = (unsigned long long)T * k;
    grid_dep_launch();
    grid_dep_wait();
    pos += (long long)t * k;
    w += (long long)t * k;
    dy += (long long)t * H;
    for (int j0 = 0; j0 < k; j0 += ROWS) {
        long long at[ROWS];
        float wj[ROWS], s[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const long long r = j0 + j < k ? pos[j0 + j] : -1;
            at[j] = (unsigned long long)r < R ? r * H : -1;
            wj[j] = j0 + j < k ? w[j0 + j] : 0.f;
            s[j] = 0.f;
        }
        for (int c = threadIdx.x * N; c < H; c += blockDim.x * N) {
            const Vec<TO, N> d = *reinterpret_cast<const Vec<TO, N>*>(dy + c);
            Vec<TI, N> v[ROWS];
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                if (at[j] >= 0) v[j] = *reinterpret_cast<const Vec<TI, N>*>(ys + at[j] + c);
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                if (at[j] >= 0) {
                    Vec<TI, N> o;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        s[j] = fmaf(to_f(d.v[i]), to_f(v[j].v[i]), s[j]);
                        o.v[i] = from_f<TI>(wj[j] * to_f(d.v[i]));
                    }
                    *reinterpret_cast<Vec<TI, N>*>(dys + at[j] + c) = o;
                }
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
            if (lane == 0) part[warp][(j0 + j) & 15] = s[j];
        }
    }
    __syncthreads();
    if (threadIdx.x < k) {
        float z = 0.f;
        for (int i = 0; i < warps; ++i) z += part[i][threadIdx.x];
        dw[(long long)t * k + threadIdx.x] = z;
    }
}

// ------------------------------------------------------- router gradient ---

// w = softmax of the k selected logits: d l_j = w_j (dw_j - sum_i w_i dw_i),
// nothing for the others.  One warp per token: zeros by 16 bytes a lane, then the k entries.  8192 x 256: 3.1 us
// (8.4 MB written; a launch alone is 1.2).
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
    if ((E & 3) == 0 && ((uintptr_t)dlogits & 15u) == 0)
        for (int i = lane; i < E / 4; i += 32) reinterpret_cast<float4*>(out)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    else
        for (int i = lane; i < E; i += 32) out[i] = 0.f;
    __syncwarp();
    if (lane < k && (unsigned)e < (unsigned)E) out[e] = sum;
}

// Elements a thread takes at a time: 16 bytes of a row where rows and pointers allow,
// else two elements, else one.
template <typename TI, typename TO>
int piece(uintptr_t all, uintptr_t rows, uintptr_t outs, int H) {
    constexpr int N = 16 / sizeof(TI);
    if (H % N == 0 && (all & 15u) == 0) return N;
    return H % 2 == 0 && (rows & (2 * sizeof(TI) - 1)) == 0 && (outs & (2 * sizeof(TO) - 1)) == 0 ? 2 : 1;
}

template <typename TI, typename TO>
cudaError_t combine_t(const void* ys, int T, int H, const int32_t* pos, int k, const float* w, const void* base,
                      void* y, cudaStream_t stream) {
    const int n = piece<TI, TO>((uintptr_t)ys | (uintptr_t)base | (uintptr_t)y, (uintptr_t)ys, (uintptr_t)base | (uintptr_t)y, H);
    const long long items = (long long)T * (H / n);
    int sms = 0;
    cudaError_t e = device_sms(sms);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::min<long long>((items + 255) / 256, (long long)sms * COMBINE_CTAS);
    auto kernel = n == 1 ? combine_kernel<TI, TO, 1> : n == 2 ? combine_kernel<TI, TO, 2> : combine_kernel<TI, TO, 16 / sizeof(TI)>;
    return launch_dependent(kernel, grid, 256, 0, stream, (const TI*)ys, T, H, pos, k, w, (const TO*)base, (TO*)y);
}

template <typename TI, typename TO>
cudaError_t combine_backward_t(const void* dy, const void* ys, int T, int H, const int32_t* pos, int k, const float* w,
                               void* dys, float* dw, cudaStream_t stream) {
    const int n = piece<TI, TO>((uintptr_t)ys | (uintptr_t)dy | (uintptr_t)dys, (uintptr_t)ys | (uintptr_t)dys, (uintptr_t)dy, H);
    const unsigned block = (unsigned)std::min(256, (H / n + 31) / 32 * 32);
    auto kernel = n == 1   ? combine_backward_kernel<TI, TO, 1>
                  : n == 2 ? combine_backward_kernel<TI, TO, 2>
                           : combine_backward_kernel<TI, TO, 16 / sizeof(TI)>;
    return launch_dependent(kernel, (unsigned)T, block, 0, stream, (const TO*)dy, (const TI*)ys, T, H, pos, k, w, (TI*)dys, dw);
}

}  // namespace

// One slice per SM: the grouping of a slice is one CTA's work.
int group_slices(int T, int k) {
    (void)k;
    return std::min(T, 148);
}
bool group_two_launches(int T, int k) { return (long long)T * k > GROUP_ONE; }

namespace {
template <bool BULK, typename V>
cudaError_t group_place(const GroupParams& p, bool two, cudaStream_t stream) {
    const int smem = BULK ? GROUP_SMEM : 0;
    static SmemLimit limit[2];
    auto kernel = two ? group_place_kernel<false, BULK, V> : group_place_kernel<true, BULK, V>;
    cudaError_t e = BULK ? limit[two].ensure((const void*)kernel, smem) : cudaSuccess;
    return e != cudaSuccess ? e : launch_dependent(kernel, p.slices, GT, smem, stream, p);
}
}  // namespace

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
    // bulk stores for the longer batches; for a few tokens all threads of a CTA copy a row (T = 4, k = 6, rows of
    // 8 KB: 2.95 us against 3.2 by bulk stores)
    if (p.x && (a & 15u) == 0)
        return two ? group_place<true, uint4>(p, two, stream) : group_place<false, uint4>(p, two, stream);
    return (a & 3u) == 0 ? group_place<false, uint32_t>(p, two, stream) : group_place<false, uint16_t>(p, two, stream);
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
