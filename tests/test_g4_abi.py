"""4-bit group-scale weights on the host: the packed layout as the header
states it, the inverse, and argument checks made before any CUDA call."""
import numpy as np
import pytest
import torch

import block_quantized_moe_rocmfpx_b200 as rfx

A = 4096          # a made-up aligned address; no refused call reads it


def weights(rows, cols, G, zeros, seed=0):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    scales = (rng.random((rows, cols // G)) + 0.5).astype(np.float16)
    z = rng.integers(0, 16, (rows, cols // G)).astype(np.uint8) if zeros else None
    return codes, scales, z


SHAPES = [(1, 32, 32), (16, 256, 32), (17, 288, 32), (33, 320, 64), (48, 384, 128), (5, 128, 128), (31, 4096, 64)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,cols,G", SHAPES)
def test_pack_round_trip(rows, cols, G, zeros):
    c, s, z = weights(rows, cols, G, zeros)
    packed = rfx.rfx_g4_pack(c, s, G, z)
    assert packed.nbytes == rfx.rfx_g4_packed_bytes(rows, cols, G, zeros)
    c2, s2, z2 = rfx.rfx_g4_unpack(packed, rows, cols, G, zeros)
    assert np.array_equal(c, c2) and np.array_equal(s.view(np.uint16), s2)
    assert z2 is None if z is None else np.array_equal(z, z2)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,cols,G", SHAPES)
def test_layout_matches_header_description(rows, cols, G, zeros):
    c, s, z = weights(rows, cols, G, zeros, 3)
    packed = rfx.rfx_g4_pack(c, s, G, z)
    want = bytearray()
    sb = s.view(np.uint16)

    def at(a, r, k):
        return int(a[r, k]) if r < rows and k < a.shape[1] else 0

    for rg in range((rows + 15) // 16):
        for k0 in range(0, cols, 128):
            nc = min(128, cols - k0)
            for p in range((nc + 63) // 64):
                for L in range(32):
                    g, t = L >> 2, L & 3
                    for tile in (0, 1):
                        for row in (16 * rg + g, 16 * rg + g + 8):
                            word = 0
                            for j in (0, 1):
                                half = 0
                                for i in range(4):
                                    k = p * 64 + tile * 32 + 8 * t + 2 * i + j
                                    if k < nc:
                                        half |= at(c, row, k0 + k) << (4 * i)
                                word |= ((half << 3 | half >> 13) & 0xFFFF) << (16 * j)
                            want += word.to_bytes(4, "little")
            for g in range(8):
                for j in range(nc // G):
                    word = at(sb, 16 * rg + g, k0 // G + j) | at(sb, 16 * rg + g + 8, k0 // G + j) << 16
                    want += word.to_bytes(4, "little")
            if zeros:
                part = bytearray()
                for g in range(8):
                    for j in range(nc // G):
                        part.append(at(z, 16 * rg + g, k0 // G + j) | at(z, 16 * rg + g + 8, k0 // G + j) << 4)
                part += bytes(-len(part) % 16)
                want += part
    assert bytes(want) == packed.tobytes()


def test_packed_bytes():
    # per 128 columns and 16 rows: 1024 of codes, 32 of scales and 8 of zeros (padded to 16) a group
    assert rfx.rfx_g4_packed_bytes(4096, 4096, 128) == 256 * 32 * (1024 + 32)
    assert rfx.rfx_g4_packed_bytes(17, 256, 32, True) == 2 * 2 * (1024 + 128 + 32)
    assert rfx.rfx_g4_packed_bytes(16, 128, 128, True) == 1024 + 32 + 16
    for rows, cols, G in ((16, 256, 16), (16, 200, 32), (16, 64, 128), (-1, 64, 64), (2 ** 31, 64, 64), (16, 0, 32)):
        assert rfx.rfx_g4_packed_bytes(rows, cols, G) == 0


def test_pack_refuses_bad_values():
    c, s, z = weights(16, 64, 32, True)
    for which in range(4):
        c2, s2, z2 = c.copy(), s.copy(), z.copy()
        if which == 0:
            c2[3, 5] = 16
        elif which == 1:
            s2[15, 1] = np.inf
        elif which == 2:
            s2[0, 0] = np.nan
        else:
            z2[7, 1] = 16
        with pytest.raises(rfx.RfxError) as e:
            rfx.rfx_g4_pack(c2, s2, 32, z2)
        assert e.value.code == rfx.RFX_EINVAL
    with pytest.raises(rfx.RfxError):
        rfx.rfx_g4_pack(c, s, 48, z)
    with pytest.raises(ValueError):
        rfx.rfx_g4_pack(c, s[:, :1], 32, z)
    with pytest.raises(ValueError):
        rfx.rfx_g4_unpack(np.zeros(10, np.uint8), 16, 64, 32)


def test_python_pack_refuses_arrays_that_a_cast_would_change():
    c, s, z = weights(16, 64, 32, True)
    want = rfx.rfx_g4_pack(c, s, 32, z)
    # other integer types that hold the same values, and the scales' bits as such
    assert np.array_equal(rfx.rfx_g4_pack(c.astype(np.int64), s.view(np.uint16), 32, z.astype(np.int32)), want)
    assert np.array_equal(rfx.rfx_g4_pack(c.tolist(), s.view(np.int16), 32, z.tolist()), want)
    big = c.astype(np.int64)
    big[2, 3] = 256 + 5
    for bad in ((big, s, z), (c - np.int64(300), s, z), (c, s, z.astype(np.int64) + 256), (c.astype(np.float32), s, z),
                (c, s, z.astype(np.float64)), (c, s.astype(np.float32), z), (c, s.astype(np.float64), z),
                (c, s.view(np.uint16).astype(np.int64) + 65536, z)):
        with pytest.raises(ValueError):
            rfx.rfx_g4_pack(bad[0], bad[1], 32, bad[2])


def test_gemv_refusals():
    def call(W=A, N=64, K=256, G=64, z=0, x=A, dt=0, q=1, y=A):
        return rfx._gemv_g4(W, N, K, G, z, x, dt, q, y, None)
    for bad in ({"N": 0}, {"N": 2 ** 31}, {"K": 0}, {"K": 96}, {"G": 16}, {"dt": 3}, {"W": None}, {"x": None},
                {"y": None}, {"W": A + 8}, {"x": A + 8}):
        assert call(**bad) == rfx.RFX_EINVAL, bad
        assert rfx.rfx_last_error()
    assert call(q=0) == rfx.RFX_EUNSUPPORTED and call(q=9) == rfx.RFX_EUNSUPPORTED


def test_expert_product_refusals():
    n = rfx.rfx_g4_packed_bytes(64, 256, 64)

    def plain(W=A, st=n, E=4, N=64, K=256, G=64, z=0, x=A, dt=0, off=A, R=3, y=A):
        return rfx._moe_g4(W, st, E, N, K, G, z, x, dt, off, R, y, None)

    def pair(W=A, up=A, st=n, E=4, N=64, K=256, G=64, z=0, x=A, dt=0, off=A, R=3, y=A):
        return rfx._moe_gate_up_g4(W, up, st, E, N, K, G, z, x, dt, off, R, y, None)

    for f in (plain, pair):
        for bad in ({"N": 0}, {"K": 96}, {"G": 0}, {"dt": 9}, {"E": 0}, {"E": 1025}, {"R": -1}, {"W": None},
                    {"x": None}, {"off": None}, {"y": None}, {"W": A + 4}, {"x": A + 2}, {"st": n + 8},
                    {"st": n - 16}, {"z": 1}):
            assert f(**bad) == rfx.RFX_EINVAL, bad
        assert f(R=0, y=None) == rfx.RFX_OK
    assert pair(up=None) == rfx.RFX_EINVAL and pair(up=A + 8) == rfx.RFX_EINVAL
    big = rfx.rfx_g4_packed_bytes(64, 12544, 64)
    assert pair(K=12544, st=big) == rfx.RFX_EUNSUPPORTED
    assert plain(N=2 ** 20, st=rfx.rfx_g4_packed_bytes(2 ** 20, 256, 64), R=2 ** 15) == rfx.RFX_EUNSUPPORTED


@pytest.mark.parametrize("N", [2 ** 31 - 31, 2 ** 31 - 1])
def test_products_refuse_rows_that_do_not_fit_32_bits(N):
    # units of 32 rows are counted in 32 bits, the rows behind the last included
    assert rfx.rfx_g4_packed_bytes(N, 32, 32) > 0
    assert rfx._gemv_g4(A, N, 32, 32, 0, A, 0, 1, A, None) == rfx.RFX_EUNSUPPORTED
    n = rfx.rfx_g4_packed_bytes(N, 32, 32)
    assert rfx._moe_g4(A, n, 1, N, 32, 32, 0, A, 0, A, 1, A, None) == rfx.RFX_EUNSUPPORTED
    assert rfx._moe_gate_up_g4(A, A, n, 1, N, 32, 32, 0, A, 0, A, 1, A, None) == rfx.RFX_EUNSUPPORTED


@pytest.mark.parametrize("off", [1, 2, 3])
def test_offsets_and_outputs_must_be_aligned_to_4_bytes(off):
    n, B = rfx.rfx_g4_packed_bytes(64, 256, 64), A + off
    assert rfx._gemv_g4(A, 64, 256, 64, 0, A, 0, 1, B, None) == rfx.RFX_EINVAL
    for offsets, y in ((B, A), (A, B)):
        assert rfx._moe_g4(A, n, 4, 64, 256, 64, 0, A, 0, offsets, 3, y, None) == rfx.RFX_EINVAL
        assert rfx._moe_gate_up_g4(A, A, n, 4, 64, 256, 64, 0, A, 0, offsets, 3, y, None) == rfx.RFX_EINVAL


def test_device_pack_refusals():
    def call(c=A, s=A, z=None, rows=16, cols=64, G=64, dst=A):
        return rfx._g4_pack_device(c, s, z, rows, cols, G, dst, None)
    for bad in ({"c": None}, {"s": None}, {"dst": None}, {"dst": A + 8}, {"s": A + 1}, {"rows": -1}, {"cols": 32},
                {"G": 31}):
        assert call(**bad) == rfx.RFX_EINVAL, bad
    assert call(rows=0, dst=None) == rfx.RFX_OK


def test_python_refuses_host_tensors():
    with pytest.raises(ValueError):
        rfx.rfx_gemv_g4(torch.zeros(4096, dtype=torch.uint8), 16, 64, 64, torch.zeros((1, 64)), torch.zeros((1, 16)))
