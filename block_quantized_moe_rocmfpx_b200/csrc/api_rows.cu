// api_rows.cu -- C ABI entry points (include/rfx.h) of the token grouping, the
// weighted combine and their gradients, and the router's gradient: argument
// checks and launches.
#include <cuda_runtime.h>

#include <string>

#include "../../include/rfx.h"
#include "rows.h"

int rfx_fail(int code, const std::string& msg);  // rfx_pack.cpp

namespace {

int cuda_fail(const char* where, cudaError_t e) {
    return rfx_fail(RFX_ECUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

bool dtype_ok(int d) { return d == RFX_BF16 || d == RFX_F32 || d == RFX_F16; }
size_t dtype_bytes(int d) { return d == RFX_F32 ? 4 : 2; }
bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
template <typename... P>
bool aligned4(const P*... p) { return ((((uintptr_t)p & 3u) == 0) && ...); }

// Shared limits of the row calls; RFX_OK or the error.
int check_rows(const char* who, int dtype, int T, int H, int k) {
    if (!dtype_ok(dtype)) return rfx_fail(RFX_EINVAL, std::string(who) + ": bad dtype");
    if (T < 0 || H < 1 || k < 1 || k > 16)
        return rfx_fail(RFX_EINVAL, std::string(who) + ": need T >= 0, H >= 1 and 1 <= k <= 16");
    if ((long long)T * k > 2147483647LL || H > (1 << 24))
        return rfx_fail(RFX_EUNSUPPORTED, std::string(who) + ": T * k must be below 2^31 and H at most 2^24");
    return RFX_OK;
}

}  // namespace

extern "C" size_t moe_group_workspace_bytes(int T, int k, int E) {
    if (T < 1 || k < 1 || k > 16 || E < 1 || E > 1024 || (long long)T * k > 2147483647LL) return 0;
    size_t n = rfx::GROUP_CTRL_BYTES;
    if (rfx::group_two_launches(T, k))
        n += (size_t)rfx::group_slices(T, k) * rfx::group_pitch(E) * sizeof(int32_t);
    return (n + 255) / 256 * 256;
}

extern "C" int moe_group_tokens(const void* x, rfx_dtype dtype, int T, int H, const int32_t* idx, int k, int E, void* xs,
                                int32_t* pos, int32_t* rows, int32_t* offsets, void* ws, size_t ws_bytes,
                                void* stream) {
    int rc = check_rows("moe_group_tokens", dtype, T, H, k);
    if (rc != RFX_OK) return rc;
    if (E < 1 || E > 1024) return rfx_fail(RFX_EINVAL, "moe_group_tokens: need 1 <= E <= 1024");
    if (T == 0) return RFX_OK;
    if (!idx || !pos || !rows || !offsets || !ws || !x != !xs)
        return rfx_fail(RFX_EINVAL, "moe_group_tokens: null pointer (x and xs may both be null)");
    if (!aligned_to(x, dtype_bytes(dtype)) || !aligned_to(xs, dtype_bytes(dtype)))
        return rfx_fail(RFX_EINVAL, "moe_group_tokens: x and xs must be aligned to their element");
    if (!aligned4(idx, pos, rows, offsets))
        return rfx_fail(RFX_EINVAL, "moe_group_tokens: idx, pos, rows and offsets must be 4-byte aligned");
    if (!aligned_to(ws, 256)) return rfx_fail(RFX_EINVAL, "moe_group_tokens: ws must be 256-byte aligned");
    if (ws_bytes < moe_group_workspace_bytes(T, k, E))
        return rfx_fail(RFX_EINVAL, "moe_group_tokens: workspace smaller than moe_group_workspace_bytes");
    rfx::GroupParams p = {};
    p.x = (const uint8_t*)x;
    p.xs = (uint8_t*)xs;
    p.row_bytes = (long long)H * (long long)dtype_bytes(dtype);
    p.idx = idx;
    p.T = T; p.k = k; p.E = E;
    p.pos = pos; p.rows = rows; p.offsets = offsets;
    p.ctrl = (uint32_t*)ws;
    p.part = (int32_t*)((uint8_t*)ws + rfx::GROUP_CTRL_BYTES);
    cudaError_t e = rfx::group_launch(p, (cudaStream_t)stream);
    return e == cudaSuccess ? RFX_OK : cuda_fail("moe_group_tokens", e);
}

extern "C" int moe_group_tokens_backward(const void* dxs, rfx_dtype dtype, int T, int H, const int32_t* pos, int k,
                                         void* dx, void* stream) {
    int rc = check_rows("moe_group_tokens_backward", dtype, T, H, k);
    if (rc != RFX_OK) return rc;
    if (T == 0) return RFX_OK;
    if (!dxs || !pos || !dx) return rfx_fail(RFX_EINVAL, "moe_group_tokens_backward: null pointer");
    if (!aligned_to(dxs, dtype_bytes(dtype)) || !aligned_to(dx, dtype_bytes(dtype)))
        return rfx_fail(RFX_EINVAL, "moe_group_tokens_backward: dxs and dx must be aligned to their element");
    if (!aligned4(pos)) return rfx_fail(RFX_EINVAL, "moe_group_tokens_backward: pos must be 4-byte aligned");
    cudaError_t e = rfx::combine_launch(dxs, dtype, T, H, pos, k, nullptr, nullptr, dx, dtype, (cudaStream_t)stream);
    return e == cudaSuccess ? RFX_OK : cuda_fail("moe_group_tokens_backward", e);
}

extern "C" int moe_combine_rows(const void* ys, rfx_dtype dtype, int T, int H, const int32_t* pos, int k, const float* w,
                                const void* base, void* y, rfx_dtype y_dtype, void* stream) {
    int rc = check_rows("moe_combine_rows", dtype, T, H, k);
    if (rc != RFX_OK) return rc;
    if (y_dtype != dtype && y_dtype != RFX_F32)
        return rfx_fail(RFX_EINVAL, "moe_combine_rows: y must have the type of ys or fp32");
    if (T == 0) return RFX_OK;
    if (!ys || !pos || !w || !y) return rfx_fail(RFX_EINVAL, "moe_combine_rows: null pointer");
    if (!aligned_to(ys, dtype_bytes(dtype)) || !aligned_to(y, dtype_bytes(y_dtype)) ||
        !aligned_to(base, dtype_bytes(y_dtype)))
        return rfx_fail(RFX_EINVAL, "moe_combine_rows: ys, base and y must be aligned to their element");
    if (!aligned4(pos, w)) return rfx_fail(RFX_EINVAL, "moe_combine_rows: pos and w must be 4-byte aligned");
    cudaError_t e = rfx::combine_launch(ys, dtype, T, H, pos, k, w, base, y, y_dtype, (cudaStream_t)stream);
    return e == cudaSuccess ? RFX_OK : cuda_fail("moe_combine_rows", e);
}

extern "C" int moe_combine_rows_backward(const void* dy, rfx_dtype y_dtype, const void* ys, rfx_dtype dtype, int T, int H,
                                         const int32_t* pos, int k, const float* w, void* dys, float* dw,
                                         void* stream) {
    int rc = check_rows("moe_combine_rows_backward", dtype, T, H, k);
    if (rc != RFX_OK) return rc;
    if (y_dtype != dtype && y_dtype != RFX_F32)
        return rfx_fail(RFX_EINVAL, "moe_combine_rows_backward: dy must have the type of ys or fp32");
    if (T == 0) return RFX_OK;
    if (!dy || !ys || !pos || !w || !dys || !dw)
        return rfx_fail(RFX_EINVAL, "moe_combine_rows_backward: null pointer");
    if (!aligned_to(ys, dtype_bytes(dtype)) || !aligned_to(dys, dtype_bytes(dtype)) ||
        !aligned_to(dy, dtype_bytes(y_dtype)))
        return rfx_fail(RFX_EINVAL, "moe_combine_rows_backward: dy, ys and dys must be aligned to their element");
    if (!aligned4(pos, w, dw)) return rfx_fail(RFX_EINVAL, "moe_combine_rows_backward: pos, w and dw must be 4-byte aligned");
    cudaError_t e = rfx::combine_backward_launch(dy, y_dtype, ys, dtype, T, H, pos, k, w, dys, dw, (cudaStream_t)stream);
    return e == cudaSuccess ? RFX_OK : cuda_fail("moe_combine_rows_backward", e);
}

extern "C" int moe_router_topk_backward(const int32_t* idx, const float* w, const float* dw, int T, int E, int k,
                                        float* dlogits, void* stream) {
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > E || k > 16)
        return rfx_fail(RFX_EINVAL, "moe_router_topk_backward: need T >= 0, 1 <= E <= 1024, 1 <= k <= min(E, 16)");
    if (T == 0) return RFX_OK;
    if (!idx || !w || !dw || !dlogits) return rfx_fail(RFX_EINVAL, "moe_router_topk_backward: null pointer");
    if (!aligned4(idx, w, dw, dlogits))
        return rfx_fail(RFX_EINVAL, "moe_router_topk_backward: idx, w, dw and dlogits must be 4-byte aligned");
    cudaError_t e = rfx::router_backward_launch(idx, w, dw, T, E, k, dlogits, (cudaStream_t)stream);
    return e == cudaSuccess ? RFX_OK : cuda_fail("moe_router_topk_backward", e);
}
