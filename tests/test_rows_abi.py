"""Argument checks of the row operators: every refusal is made before any CUDA
call, so the tests run without a GPU."""
import ctypes

import pytest
import torch

import block_quantized_moe_rocmfpx_b200 as rfx

A = 4096          # a made-up aligned address; no refused call reads it


def code(rc):
    if rc != rfx.RFX_OK:
        assert rfx.rfx_last_error()
    return rc


def group(x=A, dt=0, T=4, H=8, idx=A, k=2, E=4, xs=A, pos=A, rows=A, off=A, ws=A, n=1 << 20):
    return code(rfx._group(x, dt, T, H, idx, k, E, xs, pos, rows, off, ws, n, None))


def test_group_refusals():
    E = rfx.RFX_EINVAL
    for bad in ({"dt": 3}, {"dt": -1}, {"T": -1}, {"H": 0}, {"k": 0}, {"k": 17}, {"E": 0}, {"E": 1025}, {"idx": None},
                {"pos": None}, {"rows": None}, {"off": None}, {"ws": None}, {"x": None}, {"xs": None},
                {"x": A + 1}, {"xs": A + 1}, {"dt": 1, "x": A + 2}, {"ws": A + 16}, {"n": 255}):
        assert group(**bad) == E, bad
    assert group(T=2 ** 30, k=16) == rfx.RFX_EUNSUPPORTED
    assert group(T=0, idx=None, ws=None) == rfx.RFX_OK


def test_group_workspace_bytes():
    assert rfx.moe_group_workspace_bytes(4, 6, 256) == 256
    assert rfx.moe_group_workspace_bytes(8192, 6, 256) > 256
    for T, k, E in ((0, 1, 1), (1, 0, 1), (1, 17, 1), (1, 1, 0), (1, 1, 1025), (2 ** 30, 16, 4)):
        assert rfx.moe_group_workspace_bytes(T, k, E) == 0


def test_group_backward_refusals():
    def call(dxs=A, dt=0, T=4, H=8, pos=A, k=2, dx=A):
        return code(rfx._group_bwd(dxs, dt, T, H, pos, k, dx, None))
    for bad in ({"dt": 5}, {"T": -1}, {"H": 0}, {"k": 0}, {"k": 17}, {"dxs": None}, {"pos": None}, {"dx": None},
                {"dxs": A + 1}, {"dx": A + 1}):
        assert call(**bad) == rfx.RFX_EINVAL, bad
    assert call(T=0, dx=None) == rfx.RFX_OK


def test_combine_refusals():
    def call(ys=A, dt=0, T=4, H=8, pos=A, k=2, w=A, base=None, y=A, yd=1):
        return code(rfx._combine(ys, dt, T, H, pos, k, w, base, y, yd, None))
    for bad in ({"dt": 5}, {"yd": 2}, {"dt": 1, "yd": 0}, {"yd": 7}, {"T": -1}, {"H": 0}, {"k": 0}, {"k": 17},
                {"ys": None}, {"pos": None}, {"w": None}, {"y": None}, {"ys": A + 1}, {"y": A + 2}, {"base": A + 2}):
        assert call(**bad) == rfx.RFX_EINVAL, bad
    assert call(T=0, y=None) == rfx.RFX_OK
    assert call(H=2 ** 24 + 1) == rfx.RFX_EUNSUPPORTED
    assert call(T=2 ** 30, k=2) == rfx.RFX_EUNSUPPORTED


def test_combine_backward_refusals():
    def call(dy=A, yd=1, ys=A, dt=0, T=4, H=8, pos=A, k=2, w=A, dys=A, dw=A):
        return code(rfx._combine_bwd(dy, yd, ys, dt, T, H, pos, k, w, dys, dw, None))
    for bad in ({"dt": 5}, {"yd": 2}, {"T": -1}, {"H": 0}, {"k": 17}, {"dy": None}, {"ys": None}, {"pos": None},
                {"w": None}, {"dys": None}, {"dw": None}, {"dy": A + 2}, {"ys": A + 1}, {"dys": A + 1}):
        assert call(**bad) == rfx.RFX_EINVAL, bad
    assert call(T=0, dw=None) == rfx.RFX_OK


def test_router_backward_refusals():
    def call(idx=A, w=A, dw=A, T=4, E=8, k=2, dl=A):
        return code(rfx._router_bwd(idx, w, dw, T, E, k, dl, None))
    for bad in ({"T": -1}, {"E": 0}, {"E": 1025}, {"k": 0}, {"k": 9}, {"E": 64, "k": 17}, {"idx": None}, {"w": None},
                {"dw": None}, {"dl": None}):
        assert call(**bad) == rfx.RFX_EINVAL, bad
    assert call(T=0, dl=None) == rfx.RFX_OK


@pytest.mark.parametrize("off", [1, 2, 3])
def test_indexes_and_weights_must_be_aligned_to_4_bytes(off):
    E, B = rfx.RFX_EINVAL, A + off
    for name in ("idx", "pos", "rows", "off"):
        assert group(**{name: B}) == E, name
    assert code(rfx._group_bwd(A, 0, 4, 8, B, 2, A, None)) == E
    assert code(rfx._combine(A, 0, 4, 8, B, 2, A, None, A, 1, None)) == E
    assert code(rfx._combine(A, 0, 4, 8, A, 2, B, None, A, 1, None)) == E
    for at in (6, 8, 10):       # pos, w, dw
        args = [A, 1, A, 0, 4, 8, A, 2, A, A, A, None]
        args[at] = B
        assert code(rfx._combine_bwd(*args)) == E, at
    for at in (0, 1, 2, 6):     # idx, w, dw, dlogits
        args = [A, A, A, 4, 8, 2, A, None]
        args[at] = B
        assert code(rfx._router_bwd(*args)) == E, at


def test_python_refuses_host_tensors():
    t = torch.zeros((2, 2))
    with pytest.raises(ValueError):
        rfx.moe_router_topk_backward(t.int(), t, t, torch.zeros((2, 4)))
    with pytest.raises(ValueError):
        rfx.moe_combine_rows(torch.zeros((4, 8)), t.int(), t, torch.zeros((2, 8)))


class Fake:
    """What the binding sees of a device tensor, of any size."""

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, "cuda:0"

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 4


@pytest.mark.parametrize("T,H", [(2 ** 32, 8), (2 ** 32 + 5, 1), (2 ** 31, 1), (1, 2 ** 32 + 8)])
def test_python_refuses_sizes_that_do_not_fit_the_call(T, H, monkeypatch):
    class Runtime:
        i32, f32, codes = torch.int32, torch.float32, {torch.float32: rfx.RFX_F32}
        device, stream = staticmethod(lambda: 0), staticmethod(lambda dev: 0)

    monkeypatch.setattr(rfx, "_RT", Runtime)
    for name in ("_group", "_group_bwd", "_combine", "_combine_bwd", "_router_bwd"):
        monkeypatch.setattr(rfx, name, lambda *args: pytest.fail("the sizes reached the call cut to 32 bits"))
    i = Fake(T, 1, dtype=torch.int32)
    w, x, xs, off = Fake(T, 1), Fake(T, H), Fake(T, H), Fake(9, dtype=torch.int32)
    for call in (lambda: rfx.moe_group_tokens(x, i, 8, xs, i, Fake(T, dtype=torch.int32), off, Fake(1 << 20)),
                 lambda: rfx.moe_group_tokens_backward(xs, i, x), lambda: rfx.moe_combine_rows(xs, i, w, x),
                 lambda: rfx.moe_combine_rows_backward(x, xs, i, w, xs, w)):
        with pytest.raises(ValueError):
            call()
    many = 2 ** 32 + 2       # experts, or entries of a token
    one, ids, w1 = Fake(1, H), Fake(1, many, dtype=torch.int32), Fake(1, many)
    for call in (lambda: rfx.moe_router_topk_backward(Fake(1, 2, dtype=torch.int32), Fake(1, 2), Fake(1, 2), w1),
                 lambda: rfx.moe_router_topk_backward(ids, w1, w1, Fake(1, 8)),
                 lambda: rfx.moe_combine_rows(Fake(many, H), ids, w1, one),
                 lambda: rfx.moe_group_tokens(None, Fake(1, 2, dtype=torch.int32), many, None, Fake(1, 2, dtype=torch.int32),
                                              Fake(2, dtype=torch.int32), Fake(many + 1, dtype=torch.int32), Fake(1 << 20))):
        with pytest.raises(ValueError):
            call()
    if H == 1:
        with pytest.raises(ValueError):
            rfx.moe_router_topk_backward(i, w, w, Fake(T, 1))
        with pytest.raises(ValueError):
            rfx.moe_group_tokens(None, i, 8, None, i, Fake(T, dtype=torch.int32), off, Fake(1 << 20))


def test_dtype_codes_match_the_header():
    assert (rfx.RFX_BF16, rfx.RFX_F32, rfx.RFX_F16) == (0, 1, 2)
    assert ctypes.sizeof(ctypes.c_int) == 4
