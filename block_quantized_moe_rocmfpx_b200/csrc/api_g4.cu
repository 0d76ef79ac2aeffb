// api_g4.cu -- C ABI entry points (include/rfx.h) of the 4-bit group-scale
// weights: packers, the mat-vec and the experts' products.
#include <cuda_runtime.h>

#include <string>

#include "../../include/rfx.h"
#include "g4.h"
#include "g4_layout.h"

int rfx_fail(int code, const std::string& msg);  // rfx_pack.cpp

namespace rfx {
void g4_pack_host(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t rows, int64_t cols, int G,
                  uint8_t* dst);
void g4_unpack_host(const uint8_t* src, int64_t rows, int64_t cols, int G, uint8_t* codes, uint16_t* scales,
                    uint8_t* zeros);
}  // namespace rfx

namespace {

int cuda_fail(const char* where, cudaError_t e) {
    return rfx_fail(RFX_ECUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool group_ok(int G) { return G == 32 || G == 64 || G == 128; }
// rows and columns whose packed size and indexes stay far below 2^63
bool shape_ok(int64_t rows, int64_t cols, int G) {
    return group_ok(G) && rows >= 0 && rows <= 2147483647LL && cols > 0 && cols % G == 0 && cols <= 1073741824LL;
}

// units of 32 rows are counted in 32 bits, the rows behind the last included
constexpr int64_t kMaxN = 2147483647LL - 31;

const char* const kShape = ": need group 32, 64 or 128, 0 <= rows < 2^31 and cols a positive multiple of group, <= 2^30";

int launch(const rfx::G4Params& p, int dtype, int G, bool zeros, void* stream, const char* who) {
    cudaError_t e = dtype == RFX_BF16  ? rfx::g4_launch_bf16(p, G, zeros, (cudaStream_t)stream)
                    : dtype == RFX_F32 ? rfx::g4_launch_f32(p, G, zeros, (cudaStream_t)stream)
                                       : rfx::g4_launch_f16(p, G, zeros, (cudaStream_t)stream);
    return e == cudaSuccess ? RFX_OK : cuda_fail(who, e);
}

int experts(const char* who, const void* W0, const void* W1, bool pair, size_t stride, int E, int64_t N, int64_t K, int G,
            int has_zeros, const void* x, int x_dtype, const int32_t* offsets, int R, float* y, void* stream) {
    if (!shape_ok(N, K, G) || N < 1) return rfx_fail(RFX_EINVAL, std::string(who) + kShape + " (and N >= 1)");
    if (x_dtype != RFX_BF16 && x_dtype != RFX_F32 && x_dtype != RFX_F16)
        return rfx_fail(RFX_EINVAL, std::string(who) + ": bad x_dtype");
    if (N > kMaxN) return rfx_fail(RFX_EUNSUPPORTED, std::string(who) + ": N <= 2^31 - 32");
    if (E < 1 || E > 1024 || R < 0) return rfx_fail(RFX_EINVAL, std::string(who) + ": need 1 <= E <= 1024 and R >= 0");
    if (pair && K > 12288) return rfx_fail(RFX_EUNSUPPORTED, std::string(who) + ": K <= 12288");
    if ((N + 15) / 16 * R > 2147483000LL)   // units are counted in 32 bits, a team's step past the last included
        return rfx_fail(RFX_EUNSUPPORTED, std::string(who) + ": ceil(N / 16) * R must be at most 2147483000");
    if (R == 0) return RFX_OK;
    if (!W0 || (pair && !W1) || !x || !offsets || !y) return rfx_fail(RFX_EINVAL, std::string(who) + ": null pointer");
    if (!aligned16(W0) || !aligned16(W1) || stride % 16 || !aligned16(x))
        return rfx_fail(RFX_EINVAL, std::string(who) + ": weights, stride and x must be 16-byte aligned");
    if (!aligned4(offsets) || !aligned4(y))
        return rfx_fail(RFX_EINVAL, std::string(who) + ": offsets and the output must be 4-byte aligned");
    if (E > 1 && stride < rfx_g4_packed_bytes(N, K, G, has_zeros))
        return rfx_fail(RFX_EINVAL, std::string(who) + ": stride smaller than the packed matrix");
    rfx::G4Params p = {};
    p.W0 = (const uint8_t*)W0;
    p.W1 = (const uint8_t*)W1;
    p.stride = (long long)stride;
    p.offsets = offsets;
    p.E = E; p.R = R; p.N = (int)N; p.K = (int)K;
    p.x = x;
    p.y = y;
    return launch(p, x_dtype, G, has_zeros != 0, stream, who);
}

}  // namespace

extern "C" size_t rfx_g4_packed_bytes(int64_t rows, int64_t cols, int group, int has_zeros) {
    if (!shape_ok(rows, cols, group)) return 0;
    return (size_t)g4_matrix_bytes(rows, cols, group, has_zeros != 0);
}

extern "C" int rfx_g4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t rows, int64_t cols,
                           int group, void* dst, size_t dst_bytes) {
    if (!shape_ok(rows, cols, group)) return rfx_fail(RFX_EINVAL, std::string("rfx_g4_pack") + kShape);
    if (rows == 0) return RFX_OK;
    if (!codes || !scales || !dst) return rfx_fail(RFX_EINVAL, "rfx_g4_pack: null pointer");
    if (dst_bytes < rfx_g4_packed_bytes(rows, cols, group, zeros != nullptr))
        return rfx_fail(RFX_EINVAL, "rfx_g4_pack: dst_bytes smaller than rfx_g4_packed_bytes");
    for (int64_t i = 0; i < rows * cols; ++i)
        if (codes[i] > 15) return rfx_fail(RFX_EINVAL, "rfx_g4_pack: a code is above 15");
    for (int64_t i = 0; i < rows * (cols / group); ++i) {
        if ((scales[i] & 0x7C00u) == 0x7C00u) return rfx_fail(RFX_EINVAL, "rfx_g4_pack: scales must be finite");
        if (zeros && zeros[i] > 15) return rfx_fail(RFX_EINVAL, "rfx_g4_pack: a zero point is above 15");
    }
    rfx::g4_pack_host(codes, scales, zeros, rows, cols, group, (uint8_t*)dst);
    return RFX_OK;
}

extern "C" int rfx_g4_unpack(const void* src, int64_t rows, int64_t cols, int group, uint8_t* codes, uint16_t* scales,
                             uint8_t* zeros) {
    if (!shape_ok(rows, cols, group)) return rfx_fail(RFX_EINVAL, std::string("rfx_g4_unpack") + kShape);
    if (rows == 0) return RFX_OK;
    if (!src || !codes || !scales) return rfx_fail(RFX_EINVAL, "rfx_g4_unpack: null pointer");
    rfx::g4_unpack_host((const uint8_t*)src, rows, cols, group, codes, scales, zeros);
    return RFX_OK;
}

extern "C" int rfx_g4_pack_device(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t rows,
                                  int64_t cols, int group, void* dst, void* stream) {
    if (!shape_ok(rows, cols, group)) return rfx_fail(RFX_EINVAL, std::string("rfx_g4_pack_device") + kShape);
    if (rows == 0) return RFX_OK;
    if (!codes || !scales || !dst) return rfx_fail(RFX_EINVAL, "rfx_g4_pack_device: null pointer");
    if (!aligned16(dst) || ((uintptr_t)scales & 1u))
        return rfx_fail(RFX_EINVAL, "rfx_g4_pack_device: dst must be 16-byte and scales 2-byte aligned");
    cudaError_t e = rfx::g4_pack_launch(codes, scales, zeros, rows, cols, group, (uint8_t*)dst, (cudaStream_t)stream);
    return e == cudaSuccess ? RFX_OK : cuda_fail("rfx_g4_pack_device", e);
}

extern "C" int rfx_gemv_g4(const void* W, int64_t N, int64_t K, int group, int has_zeros, const void* x,
                           rfx_dtype x_dtype, int q, float* y, void* stream) {
    if (!shape_ok(N, K, group) || N < 1) return rfx_fail(RFX_EINVAL, std::string("rfx_gemv_g4") + kShape + " (and N >= 1)");
    if (x_dtype != RFX_BF16 && x_dtype != RFX_F32 && x_dtype != RFX_F16)
        return rfx_fail(RFX_EINVAL, "rfx_gemv_g4: bad x_dtype");
    if (N > kMaxN) return rfx_fail(RFX_EUNSUPPORTED, "rfx_gemv_g4: N <= 2^31 - 32");
    if (q < 1 || q > 8) return rfx_fail(RFX_EUNSUPPORTED, "rfx_gemv_g4: 1 <= q <= 8");
    if (!W || !x || !y) return rfx_fail(RFX_EINVAL, "rfx_gemv_g4: null pointer");
    if (!aligned16(W) || !aligned16(x)) return rfx_fail(RFX_EINVAL, "rfx_gemv_g4: W and x must be 16-byte aligned");
    if (!aligned4(y)) return rfx_fail(RFX_EINVAL, "rfx_gemv_g4: y must be 4-byte aligned");
    rfx::G4Params p = {};
    p.W0 = (const uint8_t*)W;
    p.E = 1; p.R = q; p.N = (int)N; p.K = (int)K;
    p.x = x;
    p.y = y;
    return launch(p, x_dtype, group, has_zeros != 0, stream, "rfx_gemv_g4");
}

extern "C" int moe_gemv_g4(const void* W, size_t stride, int E, int64_t N, int64_t K, int group, int has_zeros,
                           const void* x, rfx_dtype x_dtype, const int32_t* offsets, int R, float* y, void* stream) {
    return experts("moe_gemv_g4", W, nullptr, false, stride, E, N, K, group, has_zeros, x, x_dtype, offsets, R, y, stream);
}

extern "C" int moe_gate_up_g4(const void* gate, const void* up, size_t stride, int E, int64_t N, int64_t K, int group,
                              int has_zeros, const void* x, rfx_dtype x_dtype, const int32_t* offsets, int R, float* h,
                              void* stream) {
    return experts("moe_gate_up_g4", gate, up, true, stride, E, N, K, group, has_zeros, x, x_dtype, offsets, R, h, stream);
}
