// g4.cuh -- products with 4-bit weights in groups (layout: g4_layout.h):
//   y[c][n] = sum_g scale[n][g] sum_k (code - zero) x[c][k].
//
// The inner sums run on the tensor cores as fp16 products (mma.sync m16n8k16,
// 16 rows x 8 columns, fp32 sums) with exact operands.
//   Codes: a 16-bit half whose bits 3..6 (or 7..10) are a code and whose other bits are
//   zero is, as fp16, 8 (or 128) code * 2^-24: subnormal or, for both values of bit
//   10, of the lowest exponent, which has the same scale.  The four codes of a half
//   lie so that the half and the half turned by a byte have one at either place: a PRMT and
//   four ANDs make eight operands of a word, and the x that meet codes at bits 7..10 are
//   stored divided by 16.
//   x: brought to max|x| in [2^13, 2^14) by a power of two (per column, over the launch's
//   part of K) and rounded to fp16.  That keeps bf16 and fp16 values whole down to
//   2^-23 of the largest, and 2^-34 of the largest below that (fp32 sums keep 2^-24).
//   fp32 x is cut into three such parts of 11 bits, which are columns of the product.
//   zero: the sums start from -zero * sum_k x.
// So the only roundings that count are the fp32 sums and the scale's product.  They go with
// scale (code + zero) |x|, the size of what is summed, not with |W x|: weights near their zero point lose
// up to 5 bits to that, and a weight of 0 adds a rounding instead of 0.  (code - zero) as operands would
// not, for 8 more operations per 16 x 32 weights.
//
// Why mma.sync and not tcgen05: with 8 columns a 128 x 8 x 16 tcgen05.mma takes as long as one
// with 128 columns (about 89 cycles, 23 weights a cycle and SM, where the weights arrive at 46),
// its A operand would have to be written to shared memory decoded, and each group's sums read back from
// tensor memory to be scaled.  Forms that were built and measured slower at 131072 x 4096 (G = 64,
// zeros, q = 4; this one 61 us on the same kind of box): bf16 code - zero by subtraction, 79 us; e4m3 operands,
// which mma.sync takes apart into fp16 ones, 107 us; weights straight into registers, two chunks ahead, 66 us, and with
// an L2 prefetch of the next unit, 87 us; 16 or 32 warps instead of 24, 67 and 70 us; a third stage, 63 us.
//
// Bound at large sizes by memory (G = 128, q = 1: 4.8 TB/s of weights) with the instruction slots close
// behind (G = 64, zeros, q = 4: 40 instructions per 16 x 32 weights, 68 % of the issue slots); at small ones by the
// launch and its start (3 us for one 64 x 512 matrix).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "g4.h"
#include "g4_layout.h"
#include "launch_util.h"
#include "rfx_device.cuh"

namespace rfx {
namespace {

constexpr int G4_NR = 2;                        // row-groups a warp takes at a time
constexpr int G4_MAXE = 1024;
constexpr int G4_SPLIT = 8;                     // CTAs of a cluster, at most
constexpr int G4_SMEM = 232448 - 1024;          // dynamic and static shared memory of a block, less what the system takes

// x in shared memory, for the columns (rows of x) of one or more passes.  A row of
// it is a column, or (fp32) one of a column's three parts; a product (8 columns) takes the
// columns of one pass, at most 8, or 2 of them with their parts (parts 0, 1, 2 and
// a column that does not count).  A chunk: [tile][row][t][8 values], then -sum of each
// group [group][product][8 columns], fp32 (times 2^-21, and times 8 without zeros).
template <int XT> struct G4X {
    static constexpr int PARTS = XT == 1 ? 3 : 1;
    static constexpr int COLS = XT == 1 ? 2 : 8;
    static constexpr int BYTES = XT == 1 ? 4 : 2;
};
// Warps of a CTA, by the products a pass may take: registers for two leave room for 16.
constexpr int g4_warps(int nb) { return nb == 2 ? 16 : 24; }
__host__ __device__ constexpr int g4_x_bytes(int G, int products, int rows) {
    return rows * (G4_CHUNK * 2) + G4_CHUNK / G * products * 32;
}

__device__ __forceinline__ void g4_cp16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// (w & mask) | base in one instruction
__device__ __forceinline__ uint32_t g4_field(uint32_t w, uint32_t mask, uint32_t base) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(base));
    return d;
}

__device__ __forceinline__ void g4_mma(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1, const float c[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Eight x values as they lie in memory, and as fp32.
template <int XT> struct G4Raw { uint4 v[XT == 1 ? 2 : 1]; };

template <int XT>
__device__ __forceinline__ void g4_x_values(const G4Raw<XT>& r, float f[8]) {
    if constexpr (XT == 1) {
        memcpy(f, r.v, 32);
    } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (XT == 0) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                __half2 h;
                memcpy(&h, &w[i], 4);
                const float2 g = __half22float2(h);
                f[2 * i] = g.x;
                f[2 * i + 1] = g.y;
            }
        }
    }
}

// The lane's part of a chunk of G4_NR row-groups, from its stage.
template <int G, bool Z>
struct G4Stage {
    static constexpr int NG = G4_CHUNK / G, FULL = g4_chunk_bytes(G4_CHUNK, G, Z);
    uint4 w[G4_NR][2];
    uint32_t s[G4_NR][NG];   // scales of rows g and g + 8
    uint32_t z[G4_NR];       // a byte per group: zeros of rows g and g + 8

    __device__ __forceinline__ void load(const uint8_t* st, int nc, int lane) {
        const int g = lane >> 2;
        if (nc >= G4_CHUNK) {
#pragma unroll
            for (int i = 0; i < G4_NR; ++i) {
                const uint8_t* r = st + i * FULL;
                w[i][0] = *reinterpret_cast<const uint4*>(r + lane * 16);
                w[i][1] = *reinterpret_cast<const uint4*>(r + 512 + lane * 16);
                const uint8_t* sc = r + g4_scale_off(G4_CHUNK) + g * (4 * NG);
                if constexpr (NG == 4) {
                    const uint4 v = *reinterpret_cast<const uint4*>(sc);
                    s[i][0] = v.x; s[i][1] = v.y; s[i][2] = v.z; s[i][3] = v.w;
                } else if constexpr (NG == 2) {
                    const uint2 v = *reinterpret_cast<const uint2*>(sc);
                    s[i][0] = v.x; s[i][1] = v.y;
                } else {
                    s[i][0] = *reinterpret_cast<const uint32_t*>(sc);
                }
                if constexpr (Z) {
                    const uint8_t* zp = r + g4_zero_off(G4_CHUNK, G) + g * NG;
                    if constexpr (NG == 4) z[i] = *reinterpret_cast<const uint32_t*>(zp);
                    else if constexpr (NG == 2) z[i] = *reinterpret_cast<const uint16_t*>(zp);
                    else z[i] = *zp;
                }
            }
        } else {   // the last chunk of a K that is no multiple of 128: what is missing counts as zero
            const int ng = nc / G;
#pragma unroll
            for (int i = 0; i < G4_NR; ++i) {
                const uint8_t* r = st + i * FULL;
                w[i][0] = *reinterpret_cast<const uint4*>(r + lane * 16);
                w[i][1] = make_uint4(0u, 0u, 0u, 0u);
                if (nc > 64) w[i][1] = *reinterpret_cast<const uint4*>(r + 512 + lane * 16);
                z[i] = 0;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    s[i][j] = 0;
                    if (j < ng) {
                        s[i][j] = reinterpret_cast<const uint32_t*>(r + g4_scale_off(nc))[g * ng + j];
                        if (Z) z[i] |= (uint32_t)r[g4_zero_off(nc, G) + g * ng + j] << (8 * j);
                    }
                }
            }
        }
    }
};

// A chunk of G4_NR row-groups into acc; xs: the chunk's x, at[nb] the lane's place
// in a tile of it, tile the bytes of a tile; sums: the lane's sums of the first group,
// sum_step bytes to the next.
template <int G, bool Z, int NB>
__device__ __forceinline__ void g4_chunk(const G4Stage<G, Z>& st, const uint8_t* xs, const int at[NB], int tile,
                                         const uint8_t* sums, int sum_step, float acc[G4_NR][NB][4]) {
    constexpr int NG = G4_CHUNK / G;
    float s[G4_NR][NB][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {      // tiles of 32 columns
        const int j = k * 32 / G;      // the group
        if (k * 32 % G == 0) {
            float z[G4_NR][2];
#pragma unroll
            for (int r = 0; r < G4_NR; ++r) {
                z[r][0] = z[r][1] = 1.f;
                if constexpr (Z) {   // as floats: or-ed into the mantissa of 2^23, there worth z or 16 z times 256^(j % 2)
                    const uint32_t zz = j >= 2 ? st.z[r] >> 16 : st.z[r], magic = 0x4B000000u;
                    const float f = j & 1 ? 0x1.0p-8f : 1.f;
                    z[r][0] = fmaf(__uint_as_float(g4_field(zz, j & 1 ? 0xF00u : 0xFu, magic)), f, -8388608.f * f);
                    z[r][1] = fmaf(__uint_as_float(g4_field(zz, j & 1 ? 0xF000u : 0xF0u, magic)), f * 0.0625f,
                                   -524288.f * f);
                }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float2 sx = *reinterpret_cast<const float2*>(sums + j * sum_step + b * 32);
#pragma unroll
                for (int r = 0; r < G4_NR; ++r) {
                    s[r][b][0] = Z ? z[r][0] * sx.x : sx.x; s[r][b][1] = Z ? z[r][0] * sx.y : sx.y;
                    s[r][b][2] = Z ? z[r][1] * sx.x : sx.x; s[r][b][3] = Z ? z[r][1] * sx.y : sx.y;
                }
            }
        }
        uint4 x[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) x[b] = *reinterpret_cast<const uint4*>(xs + k * tile + at[b]);
#pragma unroll
        for (int r = 0; r < G4_NR; ++r) {
            const uint32_t w0 = k & 1 ? st.w[r][k >> 1].z : st.w[r][k >> 1].x;
            const uint32_t w1 = k & 1 ? st.w[r][k >> 1].w : st.w[r][k >> 1].y;
            const uint32_t v0 = __byte_perm(w0, 0, 0x2301), v1 = __byte_perm(w1, 0, 0x2301);
            const uint32_t a0[4] = {w0 & 0x00780078u, w1 & 0x00780078u, w0 & 0x07800780u, w1 & 0x07800780u};
            const uint32_t a1[4] = {v0 & 0x00780078u, v1 & 0x00780078u, v0 & 0x07800780u, v1 & 0x07800780u};
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                g4_mma(s[r][b], a0, x[b].x, x[b].y, s[r][b]);
                g4_mma(s[r][b], a1, x[b].z, x[b].w, s[r][b]);
            }
        }
        if ((k + 1) * 32 % G == 0) {
#pragma unroll
            for (int r = 0; r < G4_NR; ++r) {
                __half2 h;
                memcpy(&h, &st.s[r][j], 4);
                const float2 f = __half22float2(h);
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r][b][i] = fmaf(i < 2 ? f.x : f.y, s[r][b][i], acc[r][b][i]);
            }
        }
    }
    static_assert(NG >= 1, "a group is at most a chunk");
}

__device__ __forceinline__ float g4_silu_mul(float g, float u) {
    return g < -64.f ? silu_mul_tail(g, u) : g / (1.f + expf(-g)) * u;
}

// A value that is the same in all lanes, told to the compiler (it then lives in a
// uniform register and its branches need no reconvergence).
__device__ __forceinline__ int g4_uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Rows of x by expert, read once per CTA: blk[e] slots (passes of p.cols = 1 << p.shift
// rows) before expert e, and its rows lo[e] .. hi[e].
struct G4Rows {
    int32_t blk[G4_MAXE + 1];
    int32_t lo[G4_MAXE], hi[G4_MAXE];
    int32_t wsum[32];
    int32_t first, near[32];   // the CTA's first slot; the experts of it and the next
};

// The CTA's units u0 .. u1 - 1 of all of `slots` slots.
__device__ __forceinline__ void g4_share(int slots, int groups, int b, const G4Params& p, int& u0, int& u1) {
    const int total = slots * p.units, each = total / groups, more = total - each * groups;
    u0 = each * b + min(b, more);
    u1 = u0 + each + (b < more);
}

template <int WARPS>
__device__ __forceinline__ int g4_rows(G4Rows& s, const G4Params& p) {
    constexpr int PER = (G4_MAXE + 32 * WARPS - 1) / (32 * WARPS);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = PER * tid + i;
        n[i] = 0;
        if (e < p.E) {
            const int lo = max(0, min(p.offsets[e], p.R)), hi = max(lo, min(p.offsets[e + 1], p.R));
            s.lo[e] = lo;
            s.hi[e] = hi;
            n[i] = (hi - lo + p.cols - 1) >> p.shift;
        }
        sum += n[i];
    }
    const int own = sum;
    auto scan = [&](int v) {
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };
    sum = scan(sum);
    if (lane == 31) s.wsum[warp] = sum;
    __syncthreads();
    const int sums = scan(lane < WARPS ? s.wsum[lane] : 0);
    int at = sum - own + (warp ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0);
    const int all = __shfl_sync(0xffffffffu, sums, 31);
    int u0, u1;
    g4_share(all, gridDim.x, blockIdx.x, p, u0, u1);
    const int first = u0 / p.units;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (PER * tid + i <= p.E) s.blk[PER * tid + i] = at;
#pragma unroll 1
        for (int slot = max(at, first); slot < min(at + n[i], first + 32); ++slot) s.near[slot - first] = PER * tid + i;
        at += n[i];
    }
    if (tid == 0) {
        s.blk[p.E] = all;
        s.first = first;
    }
    __syncthreads();
    return all;
}

// A unit: row-groups of a matrix against the columns of a slot (one pass over the
// matrix of expert e).
template <bool EXPERTS>
struct G4Walk {
    int slot, unit, e;
    static __device__ __forceinline__ int find(int slot, const G4Rows* s, const G4Params& p) {
        if constexpr (!EXPERTS) return 0;
        if ((unsigned)(slot - s->first) < 32) return s->near[slot - s->first];
        int e = 0;          // the largest e with blk[e] <= slot
#pragma unroll 1
        for (int hi = p.E; hi - e > 1;) {
            const int mid = (e + hi) >> 1;
            if (s->blk[mid] <= slot) e = mid;
            else hi = mid;
        }
        return e;
    }
    __device__ __forceinline__ void step(int by, const G4Rows* s, const G4Params& p) {
        unit += by;
        if (!EXPERTS || unit < p.units) return;
        do {
            unit -= p.units;
            ++slot;
        } while (unit >= p.units);
        e = g4_uniform(find(slot, s, p));
    }
    __device__ __forceinline__ int row(const G4Rows* s, const G4Params& p) const {
        return EXPERTS ? s->lo[e] + ((slot - s->blk[e]) << p.shift) : 0;
    }
    __device__ __forceinline__ int cols(const G4Rows* s, const G4Params& p, int row) const {
        return EXPERTS ? min(p.cols, s->hi[e] - row) : p.R;
    }
};

// The x that is in shared memory: the columns of slots first .. end - 1.
constexpr int G4_COLS = 32;
struct G4Phase {
    int end, cols, products;
    int row[G4_COLS];                // of a column: its row of x, the place of its (first) sum
    int sum[G4_COLS];
    uint32_t top[G4_COLS];           // largest |x|, as fp32 bits
    float down[G4_COLS];             // 2^-E (NaN for a column with an infinity or a NaN)
    int slot_col[G4_COLS], slot_prod[G4_COLS];   // of a slot: its first column and product
};

// As many slots from `first` on as there is room for, up to the one of unit u1 - 1: one
// warp, a lane per slot.  (One matrix: its only slot.)
template <int XT, int G, bool EXPERTS>
__device__ __forceinline__ void g4_plan(G4Phase& ph, int first, int u1, int chunks, const G4Rows* s, const G4Params& p) {
    constexpr int P = G4X<XT>::PARTS, CO = G4X<XT>::COLS;
    const int lane = threadIdx.x & 31;
    if constexpr (!EXPERTS) {
        if (lane < p.R) {
            ph.row[lane] = lane;
            ph.sum[lane] = lane / CO * 8 + lane % CO * (8 / CO);
            ph.top[lane] = 0;
        }
        if (lane == 0) {
            ph.end = 1;
            ph.cols = p.R;
            ph.products = (p.R + CO - 1) / CO + 1;
            ph.slot_col[0] = ph.slot_prod[0] = 0;
        }
        return;
    }
    const int slot = first + lane;
    const bool in = (long long)slot * p.units < u1;
    int row = 0, c = 0;
    if (in) {
        const G4Walk<true> f = {slot, 0, G4Walk<true>::find(slot, s, p)};
        row = f.row(s, p);
        c = f.cols(s, p, row);
    }
    const int q = (c + CO - 1) / CO;
    int both = c | q << 16;   // at most 32 * 8 of either
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, both, o);
        if (lane >= o) both += x;
    }
    const int cols = both & 0xFFFF, products = both >> 16;
    // a second product may be read where a slot has only one
    const bool fits = in && (lane == 0 || (cols <= G4_COLS && chunks * g4_x_bytes(G, products + 1, cols * P) <= p.x_room));
    const unsigned no = ~__ballot_sync(0xffffffffu, fits);
    const int n = no ? __ffs(no) - 1 : 32;
    if (lane < n) {
        ph.slot_col[lane] = cols - c;
        ph.slot_prod[lane] = products - q;
#pragma unroll 1
        for (int j = 0; j < c; ++j) {
            ph.row[cols - c + j] = row + j;
            ph.sum[cols - c + j] = (products - q + j / CO) * 8 + j % CO * (8 / CO);
            ph.top[cols - c + j] = 0;
        }
    }
    if (lane == n - 1) {
        ph.end = first + n;
        ph.cols = cols;
        ph.products = products + 1;
    }
}

// Their largest, as the bits of its fp32 magnitude (any NaN: above the infinity).
template <int XT>
__device__ __forceinline__ uint32_t g4_x_largest(const G4Raw<XT>& r) {
    if constexpr (XT == 1) {
        const uint4 a = r.v[0], b = r.v[1];
        constexpr uint32_t M = 0x7FFFFFFFu;
        return max(max(max(a.x & M, a.y & M), max(a.z & M, a.w & M)), max(max(b.x & M, b.y & M), max(b.z & M, b.w & M)));
    } else {   // magnitudes of 16 bits are in the order of their bits
        const uint4 a = r.v[0];
        constexpr uint32_t M = 0x7FFF7FFFu;
        const uint32_t m = __vmaxu2(__vmaxu2(a.x & M, a.y & M), __vmaxu2(a.z & M, a.w & M));
        const uint32_t h = max(m >> 16, m & 0xFFFFu);
        if constexpr (XT == 0) return h << 16;
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
    }
}

// Where a lane works while x is staged: a warp takes two chunks of a column at a time, all pairs of all columns
// in turn, a lane 8 values (its place of 16 bytes, or two of a column's three for fp32).
template <int XT, bool EXPERTS, int WARPS>
struct G4XPlace {
    int col, i, pairs, turn_col, turn_i;
    __device__ __forceinline__ explicit G4XPlace(int chunks) {
        const int warp = g4_uniform(threadIdx.x >> 5);
        pairs = (chunks + 1) >> 1;
        if constexpr (EXPERTS) {   // on the path of their start, and short of registers (one token's gate/up: 16.6 / 17.2 us)
            col = 0;
            i = warp - WARPS;
            next();
        } else {
            col = warp / pairs;
            i = warp - col * pairs;
            turn_col = WARPS / pairs;
            turn_i = WARPS - turn_col * pairs;
        }
    }
    __device__ __forceinline__ void next() {
        if constexpr (EXPERTS) {
            i += WARPS;
            while (i >= pairs) {
                i -= pairs;
                ++col;
            }
        } else {
            i += turn_i;
            const int over = i >= pairs;
            i -= over ? pairs : 0;
            col += turn_col + over;
        }
    }
    // the lane's 8 values of chunk 2i or 2i + 1 of a row of x (0 behind the last)
    __device__ __forceinline__ G4Raw<XT> load(const G4Params& p, int row, int c0, int chunks) const {
        const int lane = threadIdx.x & 31, c = 2 * i + (lane >> 4), k = (c0 + c) * G4_CHUNK + (lane & 15) * 8;
        G4Raw<XT> r = {};
        if (c < chunks && k < p.K) {
            const uint4* src = reinterpret_cast<const uint4*>((const uint8_t*)p.x + ((long long)row * p.K + k) * G4X<XT>::BYTES);
            r.v[0] = __ldg(src);
            if constexpr (XT == 1) r.v[1] = __ldg(src + 1);
        }
        return r;
    }
};

// One matrix: a warp's first part of x, asked for before anything else.
template <int XT, int WARPS> struct G4XFirst { G4XPlace<XT, false, WARPS> at; G4Raw<XT> v; };

// x of the planned columns into shared memory, by all warps: first as it is (the next part on its way
// while one is looked at for its largest value), then in place as the products take it.
// The instruction slots bound it (about 100 a warp and turn, of either pass), and behind them the chain of a turn: few
// wide turns win (two chunks and 8 values a lane against one and 4, 4096 x 4096, q = 8: 11.1 / 14.2 us).
template <int XT, int G, bool Z, bool EXPERTS, int WARPS>
__device__ __forceinline__ void g4_stage_x(const G4Params& p, G4Phase& ph, int c0, int chunks, uint8_t* xs, const G4XFirst<XT, WARPS>* begun) {
    using Place = G4XPlace<XT, EXPERTS, WARPS>;
    constexpr int P = G4X<XT>::PARTS;
    const int lane = threadIdx.x & 31, l = lane & 15;
    const int cols = EXPERTS ? g4_uniform(ph.cols) : p.R, products = g4_uniform(ph.products);
    const int tile = cols * P * 64, x_chunk = g4_x_bytes(G, products, cols * P);
    // the lane's values of chunk 2i + lane / 16: columns 8l .. 8l + 7
    uint8_t* const mine = xs + (lane >> 4) * x_chunk + (l >> 2) * tile + (l & 3) * 16;
    uint8_t* const my_sums = xs + (lane >> 4) * x_chunk + 4 * tile + l / (G / 8) * products * 32;
    auto load = [&](const Place& at) {
        return at.col < cols ? at.load(p, EXPERTS ? ph.row[at.col] : at.col, c0, chunks) : G4Raw<XT>();
    };
    auto start = [&]() {
        if constexpr (EXPERTS) return Place(chunks);
        else return begun->at;
    };
    Place at = start();
    G4Raw<XT> v;
    if constexpr (EXPERTS) v = load(at);
    else v = begun->v;
#pragma unroll 1
    while (at.col < cols) {
        const int here = at.col, i = at.i;
        at.next();
        const G4Raw<XT> u = load(at);
        const uint32_t m = __reduce_max_sync(0xffffffffu, g4_x_largest<XT>(v));
        if (lane == 0 && m) atomicMax(&ph.top[here], m);
        if (2 * i + (lane >> 4) < chunks) {
            uint8_t* bytes = mine + i * 2 * x_chunk + here * (P * 64);
            *reinterpret_cast<uint4*>(bytes) = v.v[0];
            if constexpr (XT == 1) *reinterpret_cast<uint4*>(bytes + 64) = v.v[1];
        }
        v = u;
    }
    __syncthreads();
#pragma unroll 1
    for (at = start(); at.col < cols; at.next()) {
        const bool in = 2 * at.i + (lane >> 4) < chunks;
        uint8_t* bytes = mine + at.i * 2 * x_chunk + at.col * (P * 64);
        G4Raw<XT> r = {};
        if (in) {
            r.v[0] = *reinterpret_cast<const uint4*>(bytes);
            if constexpr (XT == 1) r.v[1] = *reinterpret_cast<const uint4*>(bytes + 64);
        }
        float f[8];
        g4_x_values<XT>(r, f);
        const uint32_t top = ph.top[at.col];
        // the largest lands in [2^13, 2^14); at most 2^126, which still keeps the smallest columns whole
        const int E = min(126, 13 + 127 - (int)(top >> 23));
        const float up = __uint_as_float((uint32_t)(127 + E) << 23);
        if (at.i == 0 && lane == 0)
            ph.down[at.col] = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : (uint32_t)(127 - E) << 23);
        // columns 0, 1, 4, 5 times 1, columns 2, 3, 6, 7 by 16
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= j & 2 ? up * 0.0625f : up;
        float* sums = reinterpret_cast<float*>(my_sums + at.i * 2 * x_chunk) + ph.sum[at.col];
#pragma unroll 1
        for (int q = 0; q < P; ++q) {
            uint32_t o[4];
            float s[2] = {0.f, 0.f};   // of the values times 1, and by 16
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 h = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
                memcpy(&o[j], &h, 4);
                if constexpr (P > 1) {
                    const float2 g = __half22float2(h);
                    s[j & 1] += g.x + g.y;
                    f[2 * j] = (f[2 * j] - g.x) * 2048.f;
                    f[2 * j + 1] = (f[2 * j + 1] - g.y) * 2048.f;
                } else {   // before rounding: the same but for what the smallest values lose, 2^-34 of the largest
                    s[j & 1] += f[2 * j] + f[2 * j + 1];
                }
            }
            if (in) *reinterpret_cast<uint4*>(bytes + q * 64) = make_uint4(o[0], o[1], o[2], o[3]);
            float sum = fmaf(s[1], 16.f, s[0]);
#pragma unroll
            for (int d = 1; d < G / 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (in && l % (G / 8) == 0) sums[q] = sum * (Z ? -0x1.0p-21f : -0x1.0p-18f);
        }
    }
    __syncthreads();
}

// A unit is two row-groups against up to p.cols rows of x: rows 32u .. 32u + 31
// of the matrix, or (PAIR) the gate and the up rows 16u .. 16u + 15.  A CTA takes a
// contiguous range of all units (so that it meets few slots), its teams of p.team warps
// the units of the range in turn; warp i of a team takes the chunks i, i + team, ...
//
// Every warp streams its own chunks through its own ring of two stages in shared
// memory (cp.async), across the ends of units.  The partial sums meet in shared memory
// and are added in warp order.  That is put off until the team's buffer is full (8 units
// of one column, 1 of 8), so that the warps of a team wait for one another as rarely
// as they can.
// MODE: 0 one matrix, 1 experts, 2 gate and up of experts (PAIR)
template <int XT, int G, bool Z, int MODE, int NBMAX>
__global__ void __launch_bounds__(g4_warps(NBMAX) * 32, 1) g4_kernel(G4Params p) {
    constexpr int FULL = g4_chunk_bytes(G4_CHUNK, G, Z);
    constexpr int P = G4X<XT>::PARTS, WARPS = g4_warps(NBMAX);
    constexpr bool EXPERTS = MODE > 0, PAIR = MODE == 2;
    using Walk = G4Walk<EXPERTS>;
    constexpr int STAGE = G4_NR * FULL, RING = 2 * STAGE;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int2 wait_all[WARPS][8];   // (unit, row of y) of the blocks of 32 sums that wait
    __shared__ G4Phase ph;
    __shared__ float parts[EXPERTS ? 1 : G4_SPLIT][8][32];   // of a cluster's CTAs, in its first one
    // shared memory: sums, rings, x, rows by expert
    float* const red_all = reinterpret_cast<float*>(smem);
    uint8_t* const xs = smem + WARPS * 1024 + WARPS * RING;
    G4Rows* const rows = reinterpret_cast<G4Rows*>(xs + p.x_room);
    const int lane = threadIdx.x & 31, warp = g4_uniform(threadIdx.x >> 5);
    const int team = warp * p.inv_team >> 16, member = warp - team * p.team, teams = p.teams;
    float* const red = red_all + team * p.team * 256;
    // one matrix of few rows: the p.split CTAs of a cluster share a unit, each a part of K
    const int split = EXPERTS ? 1 : p.split, rank = EXPERTS ? 0 : blockIdx.x % split;
    const int c0 = EXPERTS ? p.c0 : p.c0 + (p.c1 - p.c0) * rank / split;
    const int chunks = EXPERTS ? p.c1 - p.c0 : p.c0 + (p.c1 - p.c0) * (rank + 1) / split - c0;
    if (!EXPERTS && split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this CTA is there
    grid_dep_launch();
    if (EXPERTS) grid_dep_wait();   // for offsets; one matrix waits below
    const int slots = EXPERTS ? g4_uniform(g4_rows<WARPS>(*rows, p)) : 1;
    // the CTA's units u0 .. u1 - 1
    const int groups = EXPERTS ? gridDim.x : gridDim.x / split;
    int u0, u1;
    g4_share(slots, groups, EXPERTS ? blockIdx.x : blockIdx.x / split, p, u0, u1);
    if (u0 == u1) return;

    // loads: the next chunk of this warp, in order
    Walk w;
    const int first_slot = EXPERTS ? u0 / p.units : 0;
    w.slot = first_slot;
    w.unit = u0 - first_slot * p.units;
    w.e = g4_uniform(Walk::find(w.slot, rows, p));
    if (team) w.step(team, rows, p);
    const uint8_t* const ring = smem + WARPS * 1024 + warp * RING;
    const uint32_t ring_s = smem_u32(ring) + lane * 16;
    const int o_tail = (lane >> 4) * (FULL - 256) + 1024;              // the lane's piece behind the codes of either row-group
    const bool has_tail = (lane & 15) * 16 < FULL - 1024;
    // the warp's chunks of a unit; the last of them may be the short end of K
    const int n = (chunks - member + p.team - 1) * p.inv_team >> 16;
    const int last = p.K - (c0 + member + (n - 1) * p.team) * G4_CHUNK;
    const int end = last < G4_CHUNK ? 1 : 0;                           // chunks to go when the short one is next, 0: there is none
    const int jump = p.team * FULL;
    int fu = u0 + team, fl = fu < u1 ? n : 0, fstage = 0;               // unit and chunks of it still to load, 0: nothing left
    const uint8_t *f0 = nullptr, *f1 = nullptr, *f2 = nullptr;         // the lane's pieces: codes of both, and behind
    Walk f = w;
    auto aim = [&]() {
        const long long at = f.e * p.stride + (long long)(c0 + member) * FULL;
        const uint8_t *r0, *r1;
        if constexpr (PAIR) {
            r0 = p.W0 + at + f.unit * p.rg_bytes;
            r1 = p.W1 + at + f.unit * p.rg_bytes;
        } else {
            r0 = p.W0 + at + 2LL * f.unit * p.rg_bytes;
            r1 = 2 * f.unit + 1 < (p.N + 15) / 16 ? r0 + p.rg_bytes : r0;   // past the end: read again, dropped below
        }
        f0 = r0 + lane * 16;
        f1 = r1 + lane * 16;
        f2 = (lane >> 4 ? r1 : r0) + 1024 + (lane & 15) * 16;
    };
    auto fetch = [&]() {
        if (fl) {
            const uint32_t d = ring_s + fstage;
            if (fl != end) {
                g4_cp16(d, f0);
                g4_cp16(d + 512, f0 + 512);
                g4_cp16(d + FULL, f1);
                g4_cp16(d + FULL + 512, f1 + 512);
                if (has_tail) g4_cp16(d + o_tail, f2);
            } else {
                const int bytes = g4_chunk_bytes(last, G, Z) - lane * 16;
                for (int i = 0; i < bytes; i += 512) {
                    g4_cp16(d + i, f0 + i);
                    g4_cp16(d + FULL + i, f1 + i);
                }
            }
            f0 += jump;
            f1 += jump;
            f2 += jump;
            if (--fl == 0 && (fu += teams) < u1) {
                f.step(teams, rows, p);
                fl = n;
                aim();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        fstage ^= STAGE;
    };
    if (fl) aim();
    G4XFirst<XT, WARPS> begun = {G4XPlace<XT, false, WARPS>(chunks), {}};   // (experts: not used, and gone)
    if constexpr (!EXPERTS) {
        // One matrix: all up to here may run beside the kernel before (512 x 2048: 4.8 -> 4.3 us; the weights' way
        // into the L2 from here on too: 0.1 us slower).
        grid_dep_wait();
        // the warp's first part of x, on its way while the rest is set up (x by asynchronous copies ahead of the
        // weights: 4096 x 4096, q = 8, 11.8 / 10.3 us)
        if (begun.at.col < p.R) begun.v = begun.at.load(p, begun.at.col, c0, chunks);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) fetch();

    const int g = lane >> 2, t = lane & 3;
    int used = 0, stage = 0;   // used: blocks of 32 sums in the buffer
    auto meet = [&]() {
        if (p.team > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * p.team) : "memory");
        else __syncwarp();
    };
    // add up what waits in the team's buffer, a block of 32 sums per warp and turn
    auto flush = [&]() {
        meet();
        for (int i = member; i < used; i += p.team) {
            const int2 q = wait_all[team][i];
            float a = 0.f;
            for (int m = 0; m < p.team; ++m) a += red[(i * p.team + m) * 32 + lane];
            int row = (PAIR ? 16 : 32) * q.x + lane;
            if constexpr (PAIR) {
                const float b = __shfl_down_sync(0xffffffffu, a, 16);
                a = g4_silu_mul(a, b);
                if (lane >= 16) row = p.N;
            }
            if (!EXPERTS && split > 1) {   // to the cluster's first CTA
                uint32_t to = smem_u32(&parts[rank][i][lane]);
                asm volatile("mapa.shared::cluster.u32 %0, %0, 0;" : "+r"(to));
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(a) : "memory");
            } else if (row < p.N) {
                float* out = p.y + (long long)q.y * p.N + row;
                *out = p.c0 ? *out + a : a;
            }
        }
        meet();   // the buffer is written again
        used = 0;
    };
    int phase_end = -1, first = 0, tile = 0, x_chunk = 0, products = 0;
    // one unit with NB products
    auto unit = [&](auto nb, int cols, int col0, int prod0) {
        constexpr int NB = decltype(nb)::value;
        float acc[G4_NR][NB][4] = {};
        int at[NB];   // the row of x that the lane multiplies with (there may be fewer: the last one, and not counted)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            at[b] = (P == 1 ? col0 + min(g, cols - 1) : (col0 + min(2 * b + (g >> 2), cols - 1)) * 3 + min(g & 3, 2)) * 64 + t * 16;
        const uint8_t* xc = xs + member * x_chunk;
        const int xjump = p.team * x_chunk;
        const int sum0 = 4 * tile + prod0 * 32 + 8 * t, sum_step = products * 32;
#pragma unroll 1
        for (int i = n; i > 0; --i) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();   // the scales and zeros came by other lanes' copies
            G4Stage<G, Z> st;
            st.load(ring + stage, i != end ? G4_CHUNK : last, lane);
            g4_chunk<G, Z, NB>(st, xc, at, tile, xc + sum0, sum_step, acc);
            xc += xjump;
            __syncwarp();   // every lane has read the stage
            fetch();
            stage ^= STAGE;
        }
        // sums are 2^-21 of theirs, part q of a column 2^(-21 - 11q)
        float* const mine = red + (used * p.team + member) * 32 + g;
        const float* const down = ph.down + col0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < (P == 1 ? 2 : 1); ++i) {
                const int col = P == 1 ? 2 * t + i : 2 * b + (t >> 1);
                const float dn = down[min(col, cols - 1)];
#pragma unroll
                for (int r = 0; r < G4_NR; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v = acc[r][b][2 * h + i] * 0x1.0p21f;
                        if constexpr (P > 1) {
                            v = t & 1 ? v * 0x1.0p-22f : fmaf(acc[r][b][2 * h + 1], 0x1.0p10f, v);
                            v += __shfl_xor_sync(0xffffffffu, v, 1);
                        }
                        if (col < cols && (P == 1 || !(t & 1))) mine[col * p.team * 32 + 16 * r + 8 * h] = v * dn;
                    }
            }
    };
    if (!EXPERTS && split > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");      // all are there
    for (int u = u0 + team;;) {
        // x of the next slots, when the CTA is through with the last ones
        first = phase_end < 0 ? first_slot : phase_end;
        if (warp == 0) g4_plan<XT, G, EXPERTS>(ph, first, u1, chunks, rows, p);
        __syncthreads();
        phase_end = g4_uniform(ph.end);
        products = g4_uniform(ph.products);
        tile = g4_uniform(ph.cols) * P * 64;
        x_chunk = g4_x_bytes(G, products, g4_uniform(ph.cols) * P);
        g4_stage_x<XT, G, Z, EXPERTS, WARPS>(p, ph, c0, chunks, xs, EXPERTS ? nullptr : &begun);
        const bool done = !EXPERTS || phase_end * (long long)p.units >= u1;   // the CTA's last slots
#pragma unroll 1
        while (true) {
            const bool more = u < u1 && (!EXPERTS || w.slot < phase_end);
            int row0 = 0, cols = 0;
            if (more) {
                row0 = g4_uniform(w.row(rows, p));
                cols = g4_uniform(w.cols(rows, p, row0));
            }
            if (more ? used + cols > 8 : done && used) flush();
            if (!more) break;
            const int col0 = EXPERTS ? g4_uniform(ph.slot_col[w.slot - first]) : 0;
            const int prod0 = EXPERTS ? g4_uniform(ph.slot_prod[w.slot - first]) : 0;
            if (NBMAX == 1 || cols <= 2) unit(std::integral_constant<int, 1>(), cols, col0, prod0);
            else unit(std::integral_constant<int, NBMAX>(), cols, col0, prod0);
            if (member == 0 && lane < cols) wait_all[team][used + lane] = make_int2(w.unit, row0 + lane);
            used += cols;
            u += teams;
            w.step(teams, rows, p);
        }
        if (done) break;
        __syncthreads();   // x is written again
    }
    if (!EXPERTS && split > 1) {
        // the parts of K, added in the order of the CTAs
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        const int row = 32 * u0 + lane;
        if (rank == 0 && warp < p.R && row < p.N) {
            float a = 0.f;
            for (int r = 0; r < split; ++r) a += parts[r][warp][lane];
            float* out = p.y + (long long)warp * p.N + row;
            *out = p.c0 ? *out + a : a;
        }
    }
}

// Warps per unit: the least time of the busiest team, a unit costing its chunks and
// about one and a half more (walking, adding up).  Measured with every team size (us, teams of
// 24 / 12 / 8 / 6 / 4 / 3 / 2 warps): 131072 x 4096, G = 64, zeros, q = 4: 88 / 70 / 65 / 64 /
// 62 / 62 / 64; 37 experts of 4096 x 2048, G = 32, fp32 x: 78 / 62 / 53 / 52 / 48 / 48 / 46.
inline int g4_team(long long units, int chunks, int sms, int warps) {
    int best = warps;
    long long cost = -1;
    for (int s = warps; s >= 1; --s) {
        if (warps % s || warps / s > 15) continue;   // a named barrier per team
        const long long teams = (long long)sms * (warps / s);
        const long long c = (units + teams - 1) / teams * (2 * ((chunks + s - 1) / s) + 3);
        if (cost < 0 || c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

// Shared memory of a CTA beside x, and what is left for x.
template <int G, bool Z, int MODE, int NBMAX>
constexpr int g4_fixed() {
    constexpr int WARPS = g4_warps(NBMAX), FULL = g4_chunk_bytes(G4_CHUNK, G, Z);
    return WARPS * 1024 + WARPS * 2 * G4_NR * FULL + (MODE ? (int)sizeof(G4Rows) : 0);
}
template <int G, bool Z, int MODE, int NBMAX>
constexpr int g4_room() {   // less the kernel's static part
    return (G4_SMEM - (int)sizeof(G4Phase) - g4_warps(NBMAX) * 64 - (MODE ? 0 : G4_SPLIT * 1024) - 640 - g4_fixed<G, Z, MODE, NBMAX>()) & ~127;
}

template <int XT, int G, bool Z, int MODE, int NBMAX>
cudaError_t g4_launch_n(G4Params p, cudaStream_t stream) {
    constexpr bool EXPERTS = MODE > 0, PAIR = MODE == 2;
    int sms = 0;
    cudaError_t e = device_sms(sms);
    if (e != cudaSuccess) return e;
    constexpr int P = G4X<XT>::PARTS, CO = G4X<XT>::COLS, WARPS = g4_warps(NBMAX);
    constexpr int fixed = g4_fixed<G, Z, MODE, NBMAX>(), room = g4_room<G, Z, MODE, NBMAX>();
    p.rg_bytes = g4_rowgroup_bytes(p.K, G, Z);
    p.units = PAIR ? (p.N + 15) / 16 : (p.N + 31) / 32;
    const int chunks = (p.K + G4_CHUNK - 1) / G4_CHUNK;
    // columns of a pass: as many as there can be, with the x of all of K in shared memory.  Where that
    // does not fit, fewer columns a pass (gate/up, whose sums have to be whole before silu) or K in
    // parts, one launch each (the weights are then still read once).  (Experts: a power of two, so that
    // rows are counted by shifts.)
    int span = 0, x_chunk = 0;
    for (p.shift = 0; EXPERTS && (1 << p.shift) < std::min(p.R, NBMAX * CO); ++p.shift) {}
    p.cols = EXPERTS ? 1 << p.shift : std::min(p.R, NBMAX * CO);
    auto kernel = g4_kernel<XT, G, Z, MODE, NBMAX>;
    static SmemLimit limit;   // one per instantiation
    static ClusterFit fit;
    // One matrix of few rows: clusters of up to G4_SPLIT CTAs share a unit, down to 8 chunks a CTA (few
    // turns of staging x), as long as all clusters run at once; odd sizes leave halves of SM pairs idle and take longer
    // than the occupancy says when nearly all of theirs are needed.  us, one CTA a unit / clusters of 2 / these:
    // 500 x 14336, q = 4: 22.5 / - / 6.9 (16 clusters of 8 do not fit: 12.4); 1024 x 4096, q = 8: 9.8 / 7.5 / 6.4; 200 x 8192,
    // fp32 x, q = 2: 15.8 / - / 5.0; 1400 x 4096, q = 8 (44 units): - / 7.6 / 7.6, of 3: 8.1.
    p.split = 1;
    if (!EXPERTS && p.units < sms) {
        int split = std::min(G4_SPLIT, (chunks + 7) / 8);   // not by the columns: a column's sums do not depend on the others
        if (split > 1) e = limit.ensure((const void*)kernel, fixed + room);
        for (int clusters = 0; split > 1 && e == cudaSuccess; --split) {
            e = fit.get(kernel, split, WARPS * 32, fixed + room, clusters);
            if (p.units <= (split & 1 ? clusters * 7 / 8 : clusters)) break;
        }
        if (e != cudaSuccess) return e;
        p.split = split;
    }
    while (true) {
        x_chunk = g4_x_bytes(G, (p.cols + CO - 1) / CO + 1, p.cols * P);
        span = (int)std::min<long long>(chunks, (long long)p.split * (room / x_chunk));
        if (span == chunks || !PAIR || p.cols == 1) break;
        p.cols = 1 << --p.shift;
    }
    if (span < 1 || (PAIR && span < chunks) || (span < chunks && span < 2 * p.split)) return cudaErrorNotSupported;
    // one matrix has one slot; experts up to one per row, and room for several
    p.x_room = EXPERTS ? room : (span + p.split - 1) / p.split * x_chunk;
    p.team = p.split > 1 ? WARPS : g4_team((long long)p.units * (EXPERTS ? std::min(p.E, p.R) : 1), span, sms, WARPS);
    p.teams = WARPS / p.team;
    p.inv_team = (65536 + p.team - 1) / p.team;   // warp / team = warp * inv_team >> 16 for fewer than 32 warps
    const long long total = (long long)p.units * (EXPERTS ? p.R : 1);
    const int grid = p.split > 1 ? p.units * p.split : (int)std::min<long long>(sms, total);
    const int smem = fixed + p.x_room;
    e = limit.ensure((const void*)kernel, smem);
    const int all = p.R;
    for (int r = 0; r < all && e == cudaSuccess; r += p.R) {
        if (!EXPERTS) {   // one matrix: a launch serves p.cols columns
            p.R = std::min(p.cols, all - r);
            p.x = (const uint8_t*)p.x + (r ? (long long)p.cols * p.K * G4X<XT>::BYTES : 0);
            p.y += r ? (long long)p.cols * p.N : 0;
        }
        for (p.c0 = 0; p.c0 < chunks && e == cudaSuccess; p.c0 = p.c1) {
            p.c1 = std::min(chunks, p.c0 + span);
            // every CTA of a cluster has a chunk at least, in the last part too (its span is 2 a CTA or more)
            if (p.c1 < chunks && chunks - p.c1 < p.split) p.c1 = chunks - p.split;
            e = p.split > 1 ? launch_clusters(kernel, grid, p.split, WARPS * 32, smem, stream, p)
                            : launch_dependent(kernel, grid, WARPS * 32, smem, stream, p);
        }
    }
    return e;
}

template <int XT, int G, bool Z, int MODE>
cudaError_t g4_launch_p(const G4Params& p, cudaStream_t stream) {
    // fp32 x: two products a pass (4 columns) where there are that many columns to an expert.  Gate/up also where one
    // column of all of K does not fit beside the rings of 24 warps (G = 32: K above 9984, with zeros 9600; G = 64
    // with zeros: 12160): those of 16 warps leave room for K = 15488 and more
    if constexpr (XT == 1) {
        const int chunks = (p.K + G4_CHUNK - 1) / G4_CHUNK;
        if (p.R > 2 * (MODE ? p.E : 1) || (MODE == 2 && chunks * g4_x_bytes(G, 2, G4X<XT>::PARTS) > g4_room<G, Z, MODE, 1>()))
            return g4_launch_n<XT, G, Z, MODE, 2>(p, stream);
    }
    return g4_launch_n<XT, G, Z, MODE, 1>(p, stream);
}

template <int XT, int G, bool Z>
cudaError_t g4_launch_m(const G4Params& p, cudaStream_t stream) {
    return p.W1 ? g4_launch_p<XT, G, Z, 2>(p, stream)
                : p.offsets ? g4_launch_p<XT, G, Z, 1>(p, stream) : g4_launch_p<XT, G, Z, 0>(p, stream);
}

template <int XT, int G>
cudaError_t g4_launch_g(const G4Params& p, bool zeros, cudaStream_t stream) {
    return zeros ? g4_launch_m<XT, G, true>(p, stream) : g4_launch_m<XT, G, false>(p, stream);
}

template <int XT>
cudaError_t g4_launch_x(const G4Params& p, int G, bool zeros, cudaStream_t stream) {
    return G == 32   ? g4_launch_g<XT, 32>(p, zeros, stream)
           : G == 64 ? g4_launch_g<XT, 64>(p, zeros, stream)
                     : g4_launch_g<XT, 128>(p, zeros, stream);
}

}  // namespace
}  // namespace rfx
