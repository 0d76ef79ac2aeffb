"""B200 (sm_100a) block-quantised MoE FFN: thin Python binding of ``librfx.so``.

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels (``csrc/``); PyTorch supplies device memory and streams.  The
binding keeps the C ABI's names (``include/rfx.h``).  There is no CPU fallback:
importing fails if the library is missing and every call raises on a non-OK
status.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librfx.so")

RFX_OK, RFX_EINVAL, RFX_EUNSUPPORTED, RFX_ECUDA, RFX_EDEVICE, RFX_ERANGE = 0, -1, -2, -3, -4, -5
RFX_FP2, RFX_FP3, RFX_FP4 = 2, 3, 4
MAX_T = 8

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python block_quantized_moe_rocmfpx_b200/build.py` "
                      "(nvcc, sm_100a); there is no fallback implementation")

_lib = ctypes.CDLL(LIB_PATH)
_i32, _i64, _sz, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p


class moe_layer_desc(ctypes.Structure):
    _fields_ = [("H", _i32), ("I", _i32), ("E", _i32), ("k", _i32),
                ("f_gate", _i32), ("f_up", _i32), ("f_down", _i32),
                ("gate", _vp), ("up", _vp), ("down", _vp),
                ("stride_gate", _sz), ("stride_up", _sz), ("stride_down", _sz),
                ("has_shared", _i32),
                ("f_sh_gate", _i32), ("f_sh_up", _i32), ("f_sh_down", _i32),
                ("sh_gate", _vp), ("sh_up", _vp), ("sh_down", _vp)]


class moe_expert_mix(ctypes.Structure):
    _fields_ = [("f_gate_up", _i32), ("f_down", _i32),
                ("off_gate", ctypes.c_uint64), ("off_up", ctypes.c_uint64), ("off_down", ctypes.c_uint64)]


def _proto(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_lib_last_error = _proto("rfx_last_error", ctypes.c_char_p, [])
_packed_bytes = _proto("rfx_packed_bytes", _sz, [_i32, _i64, _i64])
_pack = _proto("rfx_pack", _i32, [_i32, _vp, _vp, _i64, _i64, _vp, _sz])
_unpack = _proto("rfx_unpack", _i32, [_i32, _vp, _i64, _i64, _vp, _vp])
_pack_device = _proto("rfx_pack_device", _i32, [_i32, _vp, _vp, _i64, _i64, _vp, _vp])
_router = _proto("moe_router_topk", _i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp])
_router_logits = _proto("moe_router_logits", _i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp])
_router_proj_topk = _proto("moe_router_project_topk", _i32,
                           [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp])
_gemv = _proto("rfx_gemv_q", _i32, [_i32, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _vp])
_layer_create = _proto("moe_layer_create", _i32, [ctypes.POINTER(moe_layer_desc), ctypes.POINTER(_vp)])
_layer_create_mix = _proto("moe_layer_create_mix", _i32,
                           [ctypes.POINTER(moe_layer_desc), ctypes.POINTER(moe_expert_mix), ctypes.POINTER(_vp)])
_layer_destroy = _proto("moe_layer_destroy", None, [_vp])
_ws_bytes = _proto("moe_ffn_workspace_bytes", _sz, [_vp, _i32])
_ws_init = _proto("rfx_ws_init", _i32, [_vp, _sz, _vp])
_ws_status = _proto("rfx_ws_status", _i32, [_vp, _vp])
_forward = _proto("moe_ffn_forward", _i32, [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp])
_forward_logits = _proto("moe_ffn_forward_logits", _i32, [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp])
_host_scratch = _proto("moe_ffn_host_scratch_bytes", _sz, [_vp, _i32])
_forward_host = _proto("moe_ffn_forward_host", _i32, [_vp, _vp, _vp, _i32, _vp, _vp, _sz, _vp])
_forward_static = _proto("moe_ffn_forward_static", _i32, [_vp, _vp, _i32, _vp, _vp, _vp, _vp])
_rms = _proto("moe_rms_norm_bf16", _i32, [_vp, _i32, _i32, _vp, _vp])
_stack_ws = _proto("moe_stack_workspace_bytes", _sz, [_vp, _i32, _i32])
_stack = _proto("moe_stack_forward", _i32, [_vp, _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp])
_pf_ws_bytes = _proto("moe_prefill_workspace_bytes", _sz, [_vp, _i32])
_debug_fault = _proto("rfx_debug_set_fault", _i32, [_i32, ctypes.c_longlong])
_prefill = _proto("moe_ffn_prefill", _i32, [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp])
_pf_ws_bytes_ex = _proto("moe_prefill_workspace_bytes_ex", _sz, [_vp, _i32, _i32])
_prefill_ex = _proto("moe_ffn_prefill_ex", _i32, [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _i32, _vp])
_group_ws = _proto("moe_group_workspace_bytes", _sz, [_i32, _i32, _i32])
_group = _proto("moe_group_tokens", _i32,
                [_vp, _i32, _i32, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp])
_group_bwd = _proto("moe_group_tokens_backward", _i32, [_vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp])
_combine = _proto("moe_combine_rows", _i32, [_vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _i32, _vp])
_combine_bwd = _proto("moe_combine_rows_backward", _i32,
                      [_vp, _i32, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp])
_router_bwd = _proto("moe_router_topk_backward", _i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp])
_g4_bytes = _proto("rfx_g4_packed_bytes", _sz, [_i64, _i64, _i32, _i32])
_g4_pack = _proto("rfx_g4_pack", _i32, [_vp, _vp, _vp, _i64, _i64, _i32, _vp, _sz])
_g4_unpack = _proto("rfx_g4_unpack", _i32, [_vp, _i64, _i64, _i32, _vp, _vp, _vp])
_g4_pack_device = _proto("rfx_g4_pack_device", _i32, [_vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp])
_gemv_g4 = _proto("rfx_gemv_g4", _i32, [_vp, _i64, _i64, _i32, _i32, _vp, _i32, _i32, _vp, _vp])
_moe_g4 = _proto("moe_gemv_g4", _i32,
                 [_vp, _sz, _i32, _i64, _i64, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp])
_moe_gate_up_g4 = _proto("moe_gate_up_g4", _i32,
                         [_vp, _vp, _sz, _i32, _i64, _i64, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp])
RFX_PREFILL_BF16, RFX_PREFILL_EXACT = 0, 1
RFX_BF16, RFX_F32, RFX_F16 = 0, 1, 2


class moe_prefill_ws_view(ctypes.Structure):
    _fields_ = [("counts", _vp), ("row_token", _vp), ("row_weight", _vp), ("h", _vp),
                ("routed_rows", _i64), ("h_rows", _i64), ("h_lo", _vp)]


_pf_view = _proto("moe_prefill_view", _i32, [_vp, _i32, _vp, ctypes.POINTER(moe_prefill_ws_view)])

EXPORTED = ["rfx_last_error", "rfx_packed_bytes", "rfx_pack", "rfx_unpack", "rfx_pack_device", "moe_router_topk",
            "rfx_gemv_q", "moe_layer_create", "moe_layer_create_mix", "moe_layer_destroy", "moe_ffn_workspace_bytes", "rfx_ws_init",
            "rfx_ws_status", "moe_ffn_forward", "moe_ffn_forward_logits", "moe_ffn_forward_static", "moe_rms_norm_bf16",
            "moe_stack_workspace_bytes", "moe_stack_forward", "moe_prefill_workspace_bytes", "moe_ffn_prefill",
            "moe_prefill_workspace_bytes_ex", "moe_ffn_prefill_ex",
            "moe_prefill_view", "moe_router_logits", "moe_router_project_topk", "moe_router_topk_backward",
            "moe_group_workspace_bytes", "moe_group_tokens", "moe_group_tokens_backward", "moe_combine_rows",
            "moe_combine_rows_backward", "rfx_g4_packed_bytes", "rfx_g4_pack", "rfx_g4_unpack", "rfx_g4_pack_device",
            "rfx_gemv_g4", "moe_gemv_g4", "moe_gate_up_g4",
            "moe_ffn_host_scratch_bytes", "moe_ffn_forward_host", "rfx_debug_set_fault"]


class RfxError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"rfx status {code}: {msg}")
        self.code = code


def rfx_last_error() -> str:
    return _lib_last_error().decode()


def _check(rc: int):
    if rc != RFX_OK:
        raise RfxError(rc, rfx_last_error())


def _ptr(t) -> int | None:
    """Device pointer of a torch tensor, host pointer of a numpy array, or an int."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ format ---

def rfx_packed_bytes(fmt: int, rows: int, cols: int) -> int:
    return int(_packed_bytes(fmt, rows, cols))


def rfx_pack(fmt: int, codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    rows, cols = codes.shape
    scales = np.ascontiguousarray(scales, dtype=np.uint8 if fmt == RFX_FP4 else np.uint16)
    out = np.empty(rfx_packed_bytes(fmt, rows, cols), dtype=np.uint8)
    _check(_pack(fmt, _ptr(codes), _ptr(scales), rows, cols, _ptr(out), out.nbytes))
    return out


def rfx_unpack(fmt: int, packed: np.ndarray, rows: int, cols: int):
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    codes = np.empty((rows, cols), dtype=np.uint8)
    scales = np.empty((rows, cols // 32), dtype=np.uint8 if fmt == RFX_FP4 else np.uint16)
    _check(_unpack(fmt, _ptr(packed), rows, cols, _ptr(codes), _ptr(scales)))
    return codes, scales


def rfx_pack_device(fmt: int, codes, scales, rows: int, cols: int, dst, stream=None):
    """Pack device arrays (torch uint8 codes [rows][cols], scales) into device dst."""
    _check(_pack_device(fmt, _ptr(codes), _ptr(scales), rows, cols, _ptr(dst), _stream(stream)))


# ---------------------------------------------------------------- kernels ---

def moe_router_topk(logits, k: int, idx, w, stream=None):
    """logits fp32 [T][E] (device) -> idx int32 [T][k], w fp32 [T][k] (device, preallocated)."""
    T, E = logits.shape
    _check(_router(_ptr(logits), T, E, k, _ptr(idx), _ptr(w), _stream(stream)))


def moe_router_logits(w_router, bias, x, logits, stream=None):
    """logits fp32 [T][E] = W x + bias for w_router bf16 [E][H], bias fp32 [E] or
    None, x bf16 [T][H] (device tensors)."""
    E, H = w_router.shape
    T = x.shape[0]
    _check(_router_logits(_ptr(w_router), _ptr(bias), _ptr(x), T, H, E, _ptr(logits), _stream(stream)))


def moe_router_project_topk(w_router, bias, x, k: int, logits, idx, w, stream=None):
    """moe_router_logits, then moe_router_topk: fills logits [T][E], idx [T][k], w [T][k]."""
    E, H = w_router.shape
    T = x.shape[0]
    _check(_router_proj_topk(_ptr(w_router), _ptr(bias), _ptr(x), T, H, E, k, _ptr(logits), _ptr(idx), _ptr(w),
                             _stream(stream)))


_RT = None   # torch and what the row and 4-bit calls need of it at every call, looked up once


class _Runtime:
    def __init__(self):
        import torch
        self.i32, self.f32, self.u8, self.f16 = torch.int32, torch.float32, torch.uint8, torch.float16
        self.codes = {torch.bfloat16: RFX_BF16, torch.float32: RFX_F32, torch.float16: RFX_F16}
        self.device = torch.cuda.current_device
        # the stream's handle without making a Stream object, where torch offers it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream = raw if raw is not None else (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _runtime() -> _Runtime:
    global _RT
    if _RT is None:
        _RT = _Runtime()
    return _RT


def _on(name: str, t) -> int:
    """The device of a call: that of its tensor `t`, which has to be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != _runtime().device():
        raise ValueError(f"{name}: must be on the current CUDA device, not {t.device}")
    return dev


def _dense(name: str, t, dev: int, shape, dtype=None):
    """Check a tensor of a row or 4-bit call: on device dev, contiguous, of this
    shape and type (the C call sees only its pointer)."""
    if t.get_device() == dev and t.shape == shape and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return
    if t.get_device() != dev:
        raise ValueError(f"{name}: must be on the current CUDA device, not {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name}: must be contiguous")


_I32_MAX = 2147483647   # ctypes cuts larger sizes to 32 bits


def _too_large(*sizes):
    raise ValueError(f"sizes {sizes}: each must be below 2^31")


def _bytes_at_least(name: str, t, dev: int, n: int):
    if t.get_device() != dev:
        raise ValueError(f"{name}: must be on the current CUDA device, not {t.device}")
    if t.numel() * t.element_size() < n:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, at least {n} expected")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _type_code(name: str, t) -> int:
    """rfx_dtype of a tensor's elements."""
    code = _RT.codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: dtype {t.dtype}, expected bfloat16, float16 or float32")
    return code


def _on_stream(stream, dev: int) -> int:
    return _RT.stream(dev) if stream is None else _stream(stream)


def moe_router_topk_backward(idx, w, dw, dlogits, stream=None):
    """dlogits fp32 [T][E] from dw fp32 [T][k], the gradient of moe_router_topk's w
    (idx int32 / w fp32 [T][k] as it wrote them)."""
    dev = _on("dlogits", dlogits)
    T, E = dlogits.shape
    k = idx.shape[-1]
    if T > _I32_MAX or k > _I32_MAX or E > _I32_MAX:
        _too_large(T, k, E)
    rt, tk = _RT, (T, k)
    _dense("dlogits", dlogits, dev, (T, E), rt.f32)
    _dense("idx", idx, dev, tk, rt.i32)
    _dense("w", w, dev, tk, rt.f32)
    _dense("dw", dw, dev, tk, rt.f32)
    rc = _router_bwd(idx.data_ptr(), w.data_ptr(), dw.data_ptr(), T, E, k, dlogits.data_ptr(), _on_stream(stream, dev))
    if rc:
        _check(rc)


def moe_group_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(_group_ws(T, k, E))


def moe_group_tokens(x, idx, E: int, xs, pos, rows, offsets, ws, stream=None):
    """Rows of x [T][H] sorted by expert: xs [T*k][H], pos int32 [T][k], rows int32
    [T*k], offsets int32 [E+1] from idx int32 [T][k] (device tensors; x and xs may
    both be None).  ws: moe_group_workspace_bytes(T, k, E) bytes, rfx_ws_init once."""
    dev = _on("idx", idx)
    T, k = idx.shape
    i32 = _RT.i32
    _dense("idx", idx, dev, (T, k), i32)
    _dense("pos", pos, dev, (T, k), i32)
    _dense("rows", rows, dev, (T * k,), i32)
    _dense("offsets", offsets, dev, (E + 1,), i32)
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws: must be contiguous and on the current CUDA device")
    if (x is None) != (xs is None):
        raise ValueError("x and xs: both or neither")
    H, dt, px, pxs = 1, RFX_F32, None, None
    if x is not None:
        H, dt = x.shape[-1], _type_code("x", x)
        _dense("x", x, dev, (T, H))
        _dense("xs", xs, dev, (T * k, H), x.dtype)
        px, pxs = x.data_ptr(), xs.data_ptr()
    if T > _I32_MAX or k > _I32_MAX or E > _I32_MAX or H > _I32_MAX:
        _too_large(T, k, E, H)
    rc = _group(px, dt, T, H, idx.data_ptr(), k, E, pxs, pos.data_ptr(), rows.data_ptr(), offsets.data_ptr(),
                ws.data_ptr(), ws.numel() * ws.element_size(), _on_stream(stream, dev))
    if rc:
        _check(rc)


def moe_group_tokens_backward(dxs, pos, dx, stream=None):
    """dx [T][H] = sum over j of dxs[pos[t][j]] (dxs [T*k][H] of dx's type, pos int32 [T][k])."""
    dev = _on("pos", pos)
    T, k = pos.shape
    H = dx.shape[-1]
    if T > _I32_MAX or k > _I32_MAX or H > _I32_MAX:
        _too_large(T, k, H)
    _dense("pos", pos, dev, (T, k), _RT.i32)
    _dense("dxs", dxs, dev, (T * k, H), dx.dtype)
    _dense("dx", dx, dev, (T, H))
    rc = _group_bwd(dxs.data_ptr(), _type_code("dx", dx), T, H, pos.data_ptr(), k, dx.data_ptr(),
                    _on_stream(stream, dev))
    if rc:
        _check(rc)


def moe_combine_rows(ys, pos, w, y, base=None, stream=None):
    """y [T][H] = base + sum over j of w[t][j] * ys[pos[t][j]] (ys [T*k][H], pos int32
    and w fp32 [T][k]; y and base of ys's type or fp32)."""
    dev = _on("pos", pos)
    T, k = pos.shape
    H = y.shape[-1]
    if T > _I32_MAX or k > _I32_MAX or H > _I32_MAX:
        _too_large(T, k, H)
    _dense("pos", pos, dev, (T, k), _RT.i32)
    _dense("w", w, dev, (T, k), _RT.f32)
    _dense("ys", ys, dev, (T * k, H))
    _dense("y", y, dev, (T, H))
    if base is not None:
        _dense("base", base, dev, (T, H), y.dtype)
        base = base.data_ptr()
    rc = _combine(ys.data_ptr(), _type_code("ys", ys), T, H, pos.data_ptr(), k, w.data_ptr(), base, y.data_ptr(),
                  _type_code("y", y), _on_stream(stream, dev))
    if rc:
        _check(rc)


def moe_combine_rows_backward(dy, ys, pos, w, dys, dw, stream=None):
    """dys [T*k][H] and dw fp32 [T][k], the gradients of moe_combine_rows from dy [T][H]
    (of ys's type or fp32)."""
    dev = _on("pos", pos)
    T, k = pos.shape
    H = dy.shape[-1]
    if T > _I32_MAX or k > _I32_MAX or H > _I32_MAX:
        _too_large(T, k, H)
    _dense("pos", pos, dev, (T, k), _RT.i32)
    _dense("w", w, dev, (T, k), _RT.f32)
    _dense("ys", ys, dev, (T * k, H))
    _dense("dys", dys, dev, (T * k, H), ys.dtype)
    _dense("dy", dy, dev, (T, H))
    _dense("dw", dw, dev, (T, k), _RT.f32)
    rc = _combine_bwd(dy.data_ptr(), _type_code("dy", dy), ys.data_ptr(), _type_code("ys", ys), T, H, pos.data_ptr(), k,
                      w.data_ptr(), dys.data_ptr(), dw.data_ptr(), _on_stream(stream, dev))
    if rc:
        _check(rc)


def rfx_gemv_q(fmt: int, W, N: int, K: int, x, y, stream=None):
    """y fp32 [q][N] = dequant(W) x for x bf16 [q][K] or fp32 [q][K] (device tensors)."""
    import torch
    q = x.shape[0]
    x_is_fp32 = 1 if x.dtype == torch.float32 else 0
    _check(_gemv(fmt, _ptr(W), N, K, _ptr(x), x_is_fp32, q, _ptr(y), _stream(stream)))


# ------------------------------------------- 4-bit weights, group scales ---

def rfx_g4_packed_bytes(rows: int, cols: int, group: int, zeros: bool = False) -> int:
    return int(_g4_bytes(rows, cols, group, 1 if zeros else 0))


def _whole(name: str, a, dtype) -> np.ndarray:
    """A contiguous array of whole numbers as dtype; refused where a cast would change a value."""
    a = np.ascontiguousarray(a)
    if a.dtype == dtype:
        return a
    if a.dtype.kind not in "iu" or (a.size and (a.min() < 0 or a.max() > np.iinfo(dtype).max)):
        raise ValueError(f"{name}: whole numbers from 0 to {np.iinfo(dtype).max} expected (dtype {a.dtype})")
    return a.astype(dtype)


def rfx_g4_pack(codes: np.ndarray, scales: np.ndarray, group: int, zeros: np.ndarray | None = None) -> np.ndarray:
    """codes uint8 [rows][cols] (< 16), scales binary16 (float16 or its bits) and zeros
    uint8 (< 16) or None, both [rows][cols/group] -> packed bytes (host)."""
    codes = _whole("codes", codes, np.uint8)
    rows, cols = codes.shape
    scales = np.ascontiguousarray(scales)
    scales = scales.view(np.uint16) if scales.dtype in (np.float16, np.int16) else _whole("scales", scales, np.uint16)
    nbytes = rfx_g4_packed_bytes(rows, cols, group, zeros is not None)
    if nbytes and scales.shape != (rows, cols // group):
        raise ValueError(f"scales: shape {scales.shape}, expected {(rows, cols // group)}")
    if zeros is not None:
        zeros = _whole("zeros", zeros, np.uint8)
        if zeros.shape != scales.shape:
            raise ValueError(f"zeros: shape {zeros.shape}, expected {scales.shape}")
    out = np.empty(nbytes, dtype=np.uint8)
    _check(_g4_pack(_ptr(codes), _ptr(scales), _ptr(zeros), rows, cols, group, _ptr(out), out.nbytes))
    return out


def rfx_g4_unpack(packed: np.ndarray, rows: int, cols: int, group: int, zeros: bool = False):
    """(codes, scale bits, zeros or None) of rfx_g4_pack's bytes."""
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    if packed.nbytes < rfx_g4_packed_bytes(rows, cols, group, zeros):
        raise ValueError(f"packed: {packed.nbytes} bytes, expected {rfx_g4_packed_bytes(rows, cols, group, zeros)}")
    codes = np.empty((rows, cols), dtype=np.uint8)
    scales = np.empty((rows, cols // max(group, 1)), dtype=np.uint16)
    z = np.empty(scales.shape, dtype=np.uint8) if zeros else None
    _check(_g4_unpack(_ptr(packed), rows, cols, group, _ptr(codes), _ptr(scales), _ptr(z)))
    return codes, scales, z


def rfx_g4_pack_device(codes, scales, zeros, rows: int, cols: int, group: int, dst, stream=None):
    """Pack device tensors (codes uint8 [rows][cols], scales float16 and zeros uint8 or
    None [rows][cols/group]) into device dst (rfx_g4_packed_bytes bytes)."""
    dev = _on("codes", codes)
    per = (rows, cols // max(group, 1))
    _dense("codes", codes, dev, (rows, cols), _RT.u8)
    _dense("scales", scales, dev, per, _RT.f16)
    if zeros is not None:
        _dense("zeros", zeros, dev, per, _RT.u8)
    _bytes_at_least("dst", dst, dev, rfx_g4_packed_bytes(rows, cols, group, zeros is not None))
    _check(_g4_pack_device(_ptr(codes), _ptr(scales), _ptr(zeros), rows, cols, group, _ptr(dst),
                           _on_stream(stream, dev)))


def rfx_gemv_g4(W, N: int, K: int, group: int, x, y, zeros: bool = False, stream=None):
    """y fp32 [q][N] = W x for packed G4 weights W [N][K] and x [q][K] (bf16, fp16 or
    fp32, q <= 8; device tensors).  zeros: W was packed with zero points."""
    dev = _on("x", x)
    q, z = x.shape[0], 1 if zeros else 0
    _dense("x", x, dev, (q, K))
    _dense("y", y, dev, (q, N), _RT.f32)
    _bytes_at_least("W", W, dev, _g4_bytes(N, K, group, z))
    rc = _gemv_g4(W.data_ptr(), N, K, group, z, x.data_ptr(), _type_code("x", x), q, y.data_ptr(),
                  _on_stream(stream, dev))
    if rc:
        _check(rc)


def _experts_g4(x, offsets, y, N, K):
    dev = _on("x", x)
    R, E = x.shape[0], offsets.shape[0] - 1
    _dense("x", x, dev, (R, K))
    _dense("offsets", offsets, dev, (E + 1,), _RT.i32)
    _dense("y", y, dev, (R, N), _RT.f32)
    return dev, R, E


def moe_gemv_g4(W, stride: int, N: int, K: int, group: int, x, offsets, y, zeros: bool = False, stream=None):
    """y[r] = W_e x[r] for the rows r of expert e (offsets int32 [E+1]): x [R][K] bf16,
    fp16 or fp32, y fp32 [R][N], W: E packed G4 matrices `stride` bytes apart."""
    dev, R, E = _experts_g4(x, offsets, y, N, K)
    z = 1 if zeros else 0
    _bytes_at_least("W", W, dev, (E - 1) * stride + _g4_bytes(N, K, group, z))
    rc = _moe_g4(W.data_ptr(), stride, E, N, K, group, z, x.data_ptr(), _type_code("x", x), offsets.data_ptr(), R,
                 y.data_ptr(), _on_stream(stream, dev))
    if rc:
        _check(rc)


def moe_gate_up_g4(gate, up, stride: int, N: int, K: int, group: int, x, offsets, h, zeros: bool = False, stream=None):
    """h[r] = silu(gate_e x[r]) * (up_e x[r]) for the rows r of expert e; arguments as moe_gemv_g4."""
    dev, R, E = _experts_g4(x, offsets, h, N, K)
    z = 1 if zeros else 0
    n = (E - 1) * stride + _g4_bytes(N, K, group, z)
    _bytes_at_least("gate", gate, dev, n)
    _bytes_at_least("up", up, dev, n)
    rc = _moe_gate_up_g4(gate.data_ptr(), up.data_ptr(), stride, E, N, K, group, z, x.data_ptr(), _type_code("x", x),
                         offsets.data_ptr(), R, h.data_ptr(), _on_stream(stream, dev))
    if rc:
        _check(rc)


def moe_layer_create(desc: moe_layer_desc) -> int:
    h = _vp()
    _check(_layer_create(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def moe_layer_create_mix(desc: moe_layer_desc, mix) -> int:
    """mix: E tuples (f_gate_up, f_down, off_gate, off_up, off_down)."""
    arr = (moe_expert_mix * len(mix))(*[moe_expert_mix(*m) for m in mix])
    h = _vp()
    _check(_layer_create_mix(ctypes.byref(desc), arr, ctypes.byref(h)))
    return h.value


def moe_layer_destroy(handle: int):
    _layer_destroy(handle)


def moe_ffn_workspace_bytes(handle: int, T: int) -> int:
    return int(_ws_bytes(handle, T))


def rfx_ws_init(ws, stream=None):
    _check(_ws_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def rfx_ws_status(ws, stream=None) -> int:
    rc = int(_ws_status(_ptr(ws), _stream(stream)))
    return rc


def moe_ffn_forward(handle: int, x, T: int, idx, w, y, ws, stream=None):
    _check(_forward(handle, _ptr(x), T, _ptr(idx), _ptr(w), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                    _stream(stream)))


def moe_ffn_forward_logits(handle: int, x, T: int, logits, idx, w, y, ws, stream=None):
    """Router top-k of logits (fp32 [T][E]) into idx / w, then the MoE FFN
    (moe_router_topk + moe_ffn_forward in one call)."""
    _check(_forward_logits(handle, _ptr(x), T, _ptr(logits), _ptr(idx), _ptr(w), _ptr(y), _ptr(ws),
                           ws.numel() * ws.element_size(), _stream(stream)))


def moe_ffn_host_scratch_bytes(handle: int, T: int) -> int:
    return int(_host_scratch(handle, T))


def moe_ffn_forward_host(handle: int, x, logits, T: int, y, scratch, stream=None):
    """Router + MoE FFN from host buffers (x bf16 [T][H], logits fp32 [T][E], y fp32
    [T][H], pinned CPU tensors or arrays); scratch: device, zeroed once."""
    _check(_forward_host(handle, _ptr(x), _ptr(logits), T, _ptr(y), _ptr(scratch),
                         scratch.numel() * scratch.element_size(), _stream(stream)))


def moe_ffn_forward_static(handle: int, x, T: int, idx, w, y, stream=None):
    """moe_ffn_forward with the library's built-in 16 MiB workspace, for callers
    that cannot allocate device memory (see include/rfx.h)."""
    _check(_forward_static(handle, _ptr(x), T, _ptr(idx), _ptr(w), _ptr(y), _stream(stream)))


def rfx_debug_set_fault(fault: int, wait_cycles: int = 0):
    """Test hook of the device error path (rfx.h): plant a wait that cannot end
    and shorten every bounded wait; fault=0, wait_cycles=0 restores normal use."""
    _check(_debug_fault(fault, wait_cycles))


def moe_rms_norm_bf16(y, x_next, stream=None):
    """y fp32 [T][H] -> x_next bf16 [T][H] = bf16(y / sqrt(mean(y^2))) per column (device tensors)."""
    T, H = y.shape
    _check(_rms(_ptr(y), T, H, _ptr(x_next), _stream(stream)))


def _handles(layers):
    arr = (_vp * len(layers))(*[(l.handle if hasattr(l, "handle") else l) for l in layers])
    return arr


def moe_stack_workspace_bytes(layers, T: int) -> int:
    return int(_stack_ws(_handles(layers), len(layers), T))


def moe_stack_forward(layers, logits, x, y, ws, stream=None):
    """L layers (MoeLayer or handles); logits fp32 [L][T][E], x bf16 [T][H], y fp32 [T][H] (device)."""
    T = x.shape[0]
    _check(_stack(_handles(layers), len(layers), _ptr(logits), _ptr(x), T, _ptr(y), _ptr(ws),
                  ws.numel() * ws.element_size(), _stream(stream)))


def moe_prefill_workspace_bytes(handle: int, T: int) -> int:
    return int(_pf_ws_bytes(handle, T))


def moe_ffn_prefill(handle: int, x, T: int, idx, w, y, ws, stream=None):
    """Grouped-GEMM prefill (bf16 operands, tcgen05): x bf16 [T][H], idx int32 [T][k],
    w fp32 [T][k], y fp32 [T][H], ws uint8 (moe_prefill_workspace_bytes), all device."""
    _check(_prefill(handle, _ptr(x), T, _ptr(idx), _ptr(w), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                    _stream(stream)))


def moe_prefill_workspace_bytes_ex(handle: int, T: int, precision: int) -> int:
    return int(_pf_ws_bytes_ex(handle, T, precision))


def moe_ffn_prefill_ex(handle: int, x, T: int, idx, w, y, ws, precision: int, stream=None):
    """moe_ffn_prefill at a chosen precision (RFX_PREFILL_BF16 or RFX_PREFILL_EXACT)."""
    _check(_prefill_ex(handle, _ptr(x), T, _ptr(idx), _ptr(w), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                       precision, _stream(stream)))


def moe_prefill_view(handle: int, T: int, ws, I: int, E: int):
    """Tensors viewing a prefill workspace after a call: counts int32 [E], row_token
    int32 [T*k], row_weight fp32 [T*k], h bf16 bits int16 [T*k + T][I]."""
    import torch
    v = moe_prefill_ws_view()
    _check(_pf_view(handle, T, _ptr(ws), ctypes.byref(v)))
    base = ws.data_ptr()

    def sub(ptr, nbytes, dtype):
        off = int(ptr) - base
        return ws[off:off + nbytes].view(dtype)

    rr, hr = int(v.routed_rows), int(v.h_rows)
    return {"counts": sub(v.counts, 4 * E, torch.int32), "row_token": sub(v.row_token, 4 * rr, torch.int32),
            "row_weight": sub(v.row_weight, 4 * rr, torch.float32),
            "h": sub(v.h, 2 * hr * I, torch.int16).view(hr, I),
            "h_lo": sub(v.h_lo, 2 * hr * I, torch.int16).view(hr, I) if int(v.h_lo) + 2 * hr * I <= base + ws.numel()
            else None}


# --------------------------------------------------------- convenience ---

class MoeLayer:
    """One MoE layer over caller-owned packed device buffers.

    ``gate``/``up``/``down`` are uint8 device tensors holding E packed experts
    at a fixed stride (or, with ``mix``, at the table's offsets in the table's
    formats); ``shared`` is (gate, up, down) or None.  Creates the
    host handle and a zeroed workspace for up to ``max_T`` token columns.
    """

    def __init__(self, H, I, E, k, fmts, gate, up, down, strides, shared=None, shared_fmts=(4, 4, 4), max_T=MAX_T,
                 mix=None):
        import torch
        self.H, self.I, self.E, self.k = H, I, E, k
        self._keep = [gate, up, down] + (list(shared) if shared else [])
        d = moe_layer_desc()
        d.H, d.I, d.E, d.k = H, I, E, k
        d.f_gate, d.f_up, d.f_down = fmts
        d.gate, d.up, d.down = _ptr(gate), _ptr(up), _ptr(down)
        d.stride_gate, d.stride_up, d.stride_down = strides
        d.has_shared = 1 if shared else 0
        if shared:
            d.f_sh_gate, d.f_sh_up, d.f_sh_down = shared_fmts
            d.sh_gate, d.sh_up, d.sh_down = (_ptr(s) for s in shared)
        self.desc = d
        # mix: ROCmFPX MIX table, E tuples (f_gate_up, f_down, off_gate, off_up, off_down)
        self.handle = moe_layer_create(d) if mix is None else moe_layer_create_mix(d, mix)
        self.max_T = max_T
        self._used_on = {}   # streams that a kept workspace was used on
        # of a call of any T up to max_T: a short prefill's may be smaller than decode's
        nbytes = max(moe_ffn_workspace_bytes(self.handle, max_T), moe_ffn_workspace_bytes(self.handle, min(max_T, 8)))
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=gate.device)
        rfx_ws_init(self.ws)

    def _kept(self, name: str, nbytes: int, stream: int):
        """The workspace kept as `name`, grown to nbytes, for a call on `stream`: its memory comes from that
        stream and is zeroed there, and goes back when every stream that used it is through."""
        import torch
        dev, ws = self.ws.device, getattr(self, name, None)

        def known():   # 0 to 2: the default streams, which wait for one another
            return torch.cuda.default_stream(dev) if stream <= 2 else torch.cuda.ExternalStream(stream, device=dev)

        if ws is None or ws.numel() < nbytes:
            with torch.cuda.stream(known()):
                ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            rfx_ws_init(ws, stream)
            setattr(self, name, ws)
            self._used_on[name] = {stream}
        elif stream not in self._used_on[name]:
            ws.record_stream(known())
            self._used_on[name].add(stream)
        return ws

    def forward(self, x, idx, w, y, stream=None):
        T = x.shape[0]
        if T > self.max_T:
            raise ValueError(f"T={T} > max_T={self.max_T}")
        moe_ffn_forward(self.handle, x, T, idx, w, y, self.ws, stream)

    def forward_logits(self, x, logits, idx, w, y, stream=None):
        """Routing from the logits, then the FFN (moe_ffn_forward_logits)."""
        T = x.shape[0]
        if T > self.max_T:
            raise ValueError(f"T={T} > max_T={self.max_T}")
        moe_ffn_forward_logits(self.handle, x, T, logits, idx, w, y, self.ws, stream)

    def forward_host(self, x, logits, y, stream=None):
        """Router + FFN from host buffers (see moe_ffn_forward_host); the device
        scratch is kept on the layer (grown on demand, zeroed when made)."""
        T = x.shape[0]
        nbytes = moe_ffn_host_scratch_bytes(self.handle, T)
        if nbytes == 0:
            raise RfxError(-2, f"unsupported T={T}")
        stream = _stream(stream)
        moe_ffn_forward_host(self.handle, x, logits, T, y, self._kept("host_scratch", nbytes, stream), stream)

    def host_status(self, stream=None) -> int:
        """Device flag of the host-call scratch (its workspace comes first)."""
        return rfx_ws_status(self.host_scratch, stream)

    def prefill(self, x, idx, w, y, stream=None, exact=False):
        """moe_ffn_prefill (exact: moe_ffn_prefill_ex at RFX_PREFILL_EXACT) with a
        workspace kept on the layer (grown on demand)."""
        T = x.shape[0]
        prec = RFX_PREFILL_EXACT if exact else RFX_PREFILL_BF16
        nbytes = moe_prefill_workspace_bytes_ex(self.handle, T, prec)
        if nbytes == 0:
            raise RfxError(-2, f"prefill unsupported for T={T}, H={self.H}, I={self.I}")
        stream = _stream(stream)
        ws = self._kept("pf_ws", nbytes, stream)
        if exact:
            moe_ffn_prefill_ex(self.handle, x, T, idx, w, y, ws, prec, stream)
        else:
            moe_ffn_prefill(self.handle, x, T, idx, w, y, ws, stream)

    def prefill_view(self, T: int):
        return moe_prefill_view(self.handle, T, self.pf_ws, self.I, self.E)

    def prefill_status(self, stream=None) -> int:
        return rfx_ws_status(self.pf_ws, stream)

    def status(self, stream=None) -> int:
        return rfx_ws_status(self.ws, stream)

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                moe_layer_destroy(self.handle)
                self.handle = None
        except Exception:
            pass
