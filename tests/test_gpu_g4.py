"""4-bit group-scale products against 64-bit sums.

Two kinds of check.  Integer inputs (x small integers, scales powers of two):
every sum is an integer multiple of the scale below 2^24 in size, so fp32 holds
every partial sum and the result must be equal bit for bit, in any order.
Random inputs: an m16n8k16 step adds 16 products to its accumulator; if the
tensor core cut each addend to 24 bits of the largest one, a step would err by
at most 16 * 2^-23 times the magnitude M = sum |w x|.  K / 16 steps (three
times that for fp32 x, whose parts add up to at most 1.01 |x|) then stay below
3 * K * 2^-23 * M, and scaling and adding the groups and the warps' shares adds
(K / G + 17) * 2^-24 * M; beside that bound the library's acceptance holds,
relative L2 <= 1e-5.
"""
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_quantized_moe_rocmfpx_b200 as rfx
from conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


class G4:
    """E random matrices [N][K], packed `stride` bytes apart, and their 64-bit values."""

    def __init__(self, N, K, G, zeros, seed, E=1, integer=False, pad=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.N, self.K, self.G, self.zeros, self.E = N, K, G, zeros, E
        self.stride = rfx.rfx_g4_packed_bytes(N, K, G, zeros) + pad
        self.codes = torch.randint(0, 16, (E, N, K), generator=g, device=DEV, dtype=torch.uint8)
        u = torch.rand((E, N, K // G), generator=g, device=DEV)
        self.scales = (torch.exp2(torch.floor(u * 3) - 1) if integer else 0.01 * torch.exp2(2 * u - 1)).half()
        self.z = torch.randint(0, 16, self.scales.shape, generator=g, device=DEV, dtype=torch.uint8) if zeros else None
        self.packed = torch.full((E * self.stride,), 0xA5, dtype=torch.uint8, device=DEV)
        for e in range(E):
            rfx.rfx_g4_pack_device(self.codes[e], self.scales[e], self.z[e] if zeros else None, N, K, G,
                                   self.packed[e * self.stride:])

    def dense(self, e=0):
        c = self.codes[e].double().view(self.N, -1, self.G)
        z = self.z[e].double()[..., None] if self.zeros else 8.0
        return ((c - z) * self.scales[e].double()[..., None]).view(self.N, self.K)


def x_of(shape, dtype, seed, integer):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if integer:
        return torch.randint(-8, 9, shape, generator=g, device=DEV).to(dtype)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def check(y, W, x, G, integer=False):
    ref = x.double() @ W.t()
    if integer:
        assert torch.equal(y.double(), ref)
        return
    K = x.shape[1]
    m = x.double().abs() @ W.abs().t()
    err = (y.double() - ref).abs()
    assert torch.isfinite(y).all()
    assert bool((err <= (3 * K * 2.0 ** -23 + (K / G + 17) * 2.0 ** -24) * m + 1e-37).all())
    assert float((y.double() - ref).norm() / ref.norm()) <= 1e-5


SHAPES = [(1, 32, 32), (16, 64, 64), (17, 288, 32), (33, 128, 128), (100, 320, 64), (64, 4096, 128), (250, 2048, 32),
          (4096, 256, 64), (5000, 96, 32), (48, 14336, 128), (31, 7168, 64), (20000, 512, 128), (70, 12320, 32), (2300, 3200, 64)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,G", SHAPES)
def test_device_pack_equals_host_pack(N, K, G, zeros):
    w = G4(N, K, G, zeros, N)
    host = rfx.rfx_g4_pack(w.codes[0].cpu().numpy(), w.scales[0].cpu().numpy(), G,
                           w.z[0].cpu().numpy() if zeros else None)
    assert np.array_equal(w.packed.cpu().numpy(), host)
    # codes at an odd address, and values above 15 taken modulo 16
    raw = torch.zeros(N * K + 3, dtype=torch.uint8, device=DEV)
    raw[3:] = w.codes[0].flatten() | 0xC0
    again = torch.zeros_like(w.packed)
    rfx.rfx_g4_pack_device(raw[3:].view(N, K), w.scales[0], w.z[0] if zeros else None, N, K, G, again)
    assert torch.equal(again, w.packed)


@pytest.mark.parametrize("integer", [True, False])
@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,G", SHAPES)
def test_gemv(N, K, G, zeros, dtype, integer):
    w = G4(N, K, G, zeros, N + K, integer=integer)
    W = w.dense()
    for q in (1, 3, 8):
        x = x_of((q, K), dtype, q, integer)
        out = torch.full((q * N + 64,), float("nan"), device=DEV)
        y = out[:q * N].view(q, N)
        rfx.rfx_gemv_g4(w.packed, N, K, G, x, y, zeros=zeros)
        check(y, W, x, G, integer)
        assert torch.isnan(out[q * N:]).all()


@pytest.mark.parametrize("dtype", [BF, HF, FF])
def test_gemv_columns_are_independent(dtype):
    N, K, G = 300, 1024, 64
    w = G4(N, K, G, True, 5)
    x = x_of((8, K), dtype, 1, False)
    y8 = torch.empty((8, N), device=DEV)
    rfx.rfx_gemv_g4(w.packed, N, K, G, x, y8, zeros=True)
    for c in (0, 3, 7):
        y1 = torch.empty((1, N), device=DEV)
        rfx.rfx_gemv_g4(w.packed, N, K, G, x[c:c + 1].contiguous(), y1, zeros=True)
        assert torch.equal(y1[0], y8[c])
    bad = x.clone()
    bad[2, 17], bad[5, 1000] = float("nan"), float("inf")
    yb = torch.empty((8, N), device=DEV)
    rfx.rfx_gemv_g4(w.packed, N, K, G, bad, yb, zeros=True)
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(yb[keep], y8[keep])
    assert torch.isnan(yb[2]).all() and not torch.isfinite(yb[5]).any()


@pytest.mark.parametrize("dtype,q,zeros,chunks", [(BF, 8, False, 352), (HF, 7, True, 344), (FF, 4, False, 344), (FF, 2, True, 456)])
def test_gemv_of_several_parts_of_K(dtype, q, zeros, chunks):
    # x of all K does not fit the shared memory of a cluster: the last part may be shorter than the cluster is wide.
    # |w x| <= 15 * 2 * 4, in units of 1/2: sums below 2^24 up to K = 69,000
    N, G = 40, 128
    for n in range(chunks - 12, chunks + 20):
        K = 128 * n
        w = G4(N, K, G, zeros, n, integer=True)
        x = x_of((q, K), dtype, n, True).clamp(-4, 4)
        y = torch.full((q, N), float("nan"), device=DEV)
        rfx.rfx_gemv_g4(w.packed, N, K, G, x, y, zeros=zeros)
        check(y, w.dense(), x, G, integer=True)


@pytest.mark.parametrize("N", [1180, 2400, 4800])
@pytest.mark.parametrize("dtype,q", [(BF, 8), (FF, 8), (FF, 2)])
def test_gemv_of_many_rows_and_several_parts_of_K(N, dtype, q):
    # as above without clusters, or in narrow ones: parts of about 44 (fp32, q = 2: 58) chunks a CTA
    G = 128
    for n in (45, 89, 90, 133):
        K = 128 * n
        w = G4(N, K, G, True, n, integer=True)
        x = x_of((q, K), dtype, n, True)
        y = torch.full((q, N), float("nan"), device=DEV)
        rfx.rfx_gemv_g4(w.packed, N, K, G, x, y, zeros=True)
        check(y, w.dense(), x, G, integer=True)


@pytest.mark.parametrize("N,K", [(40, 4096), (500, 14336), (800, 8192), (1400, 4096), (4096, 2048)])
def test_gemv_columns_are_independent_in_clusters(N, K):
    w = G4(N, K, 64, False, 6)
    x = x_of((8, K), BF, 1, False)
    y8 = torch.empty((8, N), device=DEV)
    rfx.rfx_gemv_g4(w.packed, N, K, 64, x, y8)
    check(y8, w.dense(), x, 64)
    for c in (0, 7):
        y1 = torch.empty((1, N), device=DEV)
        rfx.rfx_gemv_g4(w.packed, N, K, 64, x[c:c + 1].contiguous(), y1)
        assert torch.equal(y1[0], y8[c])


def test_gemv_fp32_x_of_any_size():
    # 24-bit significands from 2^-60 to 2^60 in one row: the parts lose nothing
    N, K, G = 64, 512, 32
    w = G4(N, K, G, True, 8)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    for lo, hi in ((-60, -40), (0, 1), (40, 60)):
        x = torch.randn((4, K), generator=g, device=DEV) * torch.exp2(
            torch.randint(lo, hi, (4, K), generator=g, device=DEV).float())
        y = torch.empty((4, N), device=DEV)
        rfx.rfx_gemv_g4(w.packed, N, K, G, x, y, zeros=True)
        check(y, w.dense(), x, G)
    # one column of x at a time picks one weight: x * w exactly rounded
    x = torch.zeros((8, K), device=DEV)
    v = torch.tensor([1 + 2.0 ** -23, 3.1415927, -0.1, 1e-30, 7e25, 16777215.0, -1.9999999, 2.0 ** -100], device=DEV)
    cols = [0, 31, 32, 77, 255, 256, 300, 511]
    for i, c in enumerate(cols):
        x[i, c] = v[i]
    y = torch.empty((8, N), device=DEV)
    rfx.rfx_gemv_g4(w.packed, N, K, G, x, y, zeros=True)
    W = w.dense()
    want = torch.stack([W[:, c] * v[i].double() for i, c in enumerate(cols)])
    # (code - zero) * x needs up to 28 bits: one rounding to fp32, one more for the scale
    assert bool(((y.double() - want).abs() <= 4 * 2.0 ** -23 * want.abs()).all())


def true_bound(w, x, e=0):
    """The error that the form of the sums allows, in 64 bits.  A group is summed as code * x - zero * sum x, of
    magnitude S = sum (code + zero) |x|: G / 16 steps of the tensor core with 17 addends, each cut to 24 bits of the
    largest (17 * G / 16 * 2^-23 S); the sum of x in at most 10 roundings and its product with zero in one; then scaled
    and added, K / G roundings in a warp and at most 24 + 8 + 8 over warps, CTAs and parts of K.  16-bit values of x far below their
    column's largest enter within 2^-34 of that, times a code of at most 15."""
    c = w.codes[e].double().view(w.N, -1, w.G)
    z = w.z[e].double()[..., None] if w.zeros else 8.0
    s = w.scales[e].double()[..., None].abs()
    K, G = w.K, w.G
    m = x.double().abs() @ ((c + z) * s).view(w.N, K).t()
    err = (17 * G / 16 * 2.0 ** -23 + (11 + K / G + 40) * 2.0 ** -24) * 1.01 * m
    if x.dtype is not FF:
        err = err + 15 * 2.0 ** -34 * x.double().abs().amax(1)[:, None] * (s.sum(1) * G).T
    return err + 1e-37


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("K,G,zeros", [(512, 32, True), (4096, 128, False), (4096, 64, True), (352, 32, False), (20480, 128, True)])
def test_weights_of_zero_and_near_it(K, G, zeros, dtype):
    # pruned rows and groups (every code the zero point), rows next to their zero point, outliers of x that
    # meet weights of 0, and x over the whole range that 16-bit types hold a column's largest and smallest in
    N = 96
    w = G4(N, K, G, zeros, 61)
    z = w.z[0].view(N, -1, 1).expand(N, K // G, G).reshape(N, K) if zeros else torch.full_like(w.codes[0], 8)
    g = torch.Generator(device=DEV)
    g.manual_seed(62)
    c = w.codes[0]
    c[0:16] = z[0:16]                                                   # pruned rows
    near = torch.randint(-1, 2, c.shape, generator=g, device=DEV, dtype=torch.int16)
    c[16:48] = (z[16:48].to(torch.int16) + near[16:48]).clamp(0, 15).to(torch.uint8)
    c[48:64, K // 2 // G * G:] = z[48:64, K // 2 // G * G:]             # pruned groups
    far = torch.tensor([3, K // 3, K - 1], device=DEV)
    c[:80, far] = z[:80, far]                                           # the outliers' weights
    rfx.rfx_g4_pack_device(c, w.scales[0], w.z[0] if zeros else None, N, K, G, w.packed)
    W = w.dense()
    assert bool((W[:16] == 0).all() and (W[:80, far] == 0).all())
    x = torch.randn((6, K), generator=g, device=DEV)
    x[1, far] = 3.0e3
    x[2, far] = 6.0e4
    x[3] *= torch.exp2(torch.randint(-13, 14, (K,), generator=g, device=DEV).float())
    x[4] *= torch.exp2(torch.randint(-24, 1, (K,), generator=g, device=DEV).float())
    x[5] *= 2.0 ** -14
    x[5, far] = 6.0e4
    x = x.to(dtype)
    y = torch.empty((6, N), device=DEV)
    rfx.rfx_gemv_g4(w.packed, N, K, G, x, y, zeros=zeros)
    ye = torch.empty((6, N), device=DEV)
    rfx.moe_gemv_g4(w.packed, w.stride, N, K, G, x, offsets_of([6]), ye, zeros=zeros)
    want, bound = x.double() @ W.t(), true_bound(w, x)
    for got in (y, ye):
        assert bool(((got.double() - want).abs() <= bound).all()), float(((got.double() - want).abs() / bound).max())


# ------------------------------------------------------------- experts ---

def offsets_of(counts):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(counts), 0)
    return off.to(DEV)


COUNTS = {"one": [1], "first_last": [1, 0, 0, 2], "wide": [0, 9, 0, 0, 23, 8, 1, 0], "empty": [0, 0, 0],
          "all": [3, 1, 2, 1, 4, 1]}


@pytest.mark.parametrize("integer", [True, False])
@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("N,K,G,zeros", [(64, 256, 128, False), (50, 352, 32, True), (300, 2048, 64, True)])
@pytest.mark.parametrize("which", sorted(COUNTS))
def test_expert_products(which, N, K, G, zeros, dtype, integer):
    counts = COUNTS[which]
    E, R = len(counts), sum(counts) + 3        # three rows behind the last expert
    w = G4(N, K, G, zeros, 3, E=E, integer=integer, pad=48)
    off = offsets_of(counts)
    x = x_of((R, K), dtype, 4, integer)
    x[R - 3:] = float("nan")
    y = torch.full((R, N), -5.0, device=DEV)
    rfx.moe_gemv_g4(w.packed, w.stride, N, K, G, x, off, y, zeros=zeros)
    lo = 0
    for e, n in enumerate(counts):
        if n:
            check(y[lo:lo + n], w.dense(e), x[lo:lo + n], G, integer)
        lo += n
    assert (y[lo:] == -5.0).all()


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("N,K,G,zeros", [(64, 256, 128, True), (50, 352, 32, False), (300, 2048, 64, True)])
@pytest.mark.parametrize("which", sorted(COUNTS))
def test_gate_up(which, N, K, G, zeros, dtype):
    counts = COUNTS[which]
    E, R = len(counts), sum(counts) + 1
    gate, up = G4(N, K, G, zeros, 11, E=E), G4(N, K, G, zeros, 12, E=E)
    off = offsets_of(counts)
    x = x_of((R, K), dtype, 6, False)
    h = torch.full((R, N), -5.0, device=DEV)
    rfx.moe_gate_up_g4(gate.packed, up.packed, gate.stride, N, K, G, x, off, h, zeros=zeros)
    d = 3 * K * 2.0 ** -23 + (K / G + 17) * 2.0 ** -24
    lo = 0
    for e, n in enumerate(counts):
        if n:
            xe = x[lo:lo + n].double()
            g, u = xe @ gate.dense(e).t(), xe @ up.dense(e).t()
            mg, mu = xe.abs() @ gate.dense(e).abs().t(), xe.abs() @ up.dense(e).abs().t()
            want = g * torch.sigmoid(g) * u
            # |silu'| < 1.1 and |silu(g)| <= |g|: the products' errors, then four roundings and expf's 2 ulp
            bound = 1.1 * d * mg * u.abs() + d * mu * g.abs() + 1.1 * d * d * mg * mu + 8 * 2.0 ** -23 * want.abs()
            got = h[lo:lo + n].double()
            assert bool(((got - want).abs() <= bound + 1e-37).all())
            assert float((got - want).norm() / want.norm()) <= 1e-5
        lo += n
    assert (h[lo:] == -5.0).all()


@pytest.mark.parametrize("counts", [[0, 1, 0, 2], [3, 0, 9, 1]])      # R below and above 2 E
@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("K,G", [(9632, 32), (9984, 32), (10016, 32), (12288, 32), (12160, 64), (12224, 64), (12288, 64),
                                 (12288, 128)])
def test_gate_up_of_long_rows(K, G, zeros, dtype, counts):
    # up to the limit of K, with every type: x of all K is in shared memory, of one column at least
    N, E, R = 40, len(counts), sum(counts) + 1
    gate, up = G4(N, K, G, zeros, 11, E=E), G4(N, K, G, zeros, 12, E=E)
    x = x_of((R, K), dtype, 6, False)
    h = torch.full((R, N), -5.0, device=DEV)
    rfx.moe_gate_up_g4(gate.packed, up.packed, gate.stride, N, K, G, x, offsets_of(counts), h, zeros=zeros)
    # the bound of test_gate_up
    d = 3 * K * 2.0 ** -23 + (K / G + 17) * 2.0 ** -24
    lo = 0
    for e, n in enumerate(counts):
        if n:
            xe = x[lo:lo + n].double()
            g, u = xe @ gate.dense(e).t(), xe @ up.dense(e).t()
            mg, mu = xe.abs() @ gate.dense(e).abs().t(), xe.abs() @ up.dense(e).abs().t()
            want = g * torch.sigmoid(g) * u
            bound = 1.1 * d * mg * u.abs() + d * mu * g.abs() + 1.1 * d * d * mg * mu + 8 * 2.0 ** -23 * want.abs()
            got = h[lo:lo + n].double()
            assert bool(((got - want).abs() <= bound + 1e-37).all())
            assert float((got - want).norm() / want.norm()) <= 1e-5
        lo += n
    assert (h[lo:] == -5.0).all()


@pytest.mark.parametrize("counts", [[0, 9, 1, 23], [2, 0, 1, 0, 0, 0, 3, 0]])      # R above and below 2 E
@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("K,G,zeros", [(4640, 32, True), (5504, 128, False), (7168, 64, True), (12352, 64, False),
                                       (14336, 128, True), (14368, 32, True), (30112, 32, False)])
def test_expert_products_of_long_rows(K, G, zeros, dtype, counts):
    # x of all K does not fit a CTA's shared memory (8 columns of 16 bits: K above 4224 to 5376; fp32, 2 or 4
    # columns: 4480 to 7168): K in parts, added in y by one launch after the other, the last part and its last chunk
    # shorter.  |w x| <= 480 in units of 1/2: integer sums below 2^24 up to K = 34,000
    N, E, R = 50, len(counts), sum(counts) + 2
    w = G4(N, K, G, zeros, 23, E=E, integer=True, pad=16)
    x = x_of((R, K), dtype, 4, True)
    x[R - 2:] = float("nan")
    y = torch.full((R, N), -5.0, device=DEV)
    rfx.moe_gemv_g4(w.packed, w.stride, N, K, G, x, offsets_of(counts), y, zeros=zeros)
    lo = 0
    for e, n in enumerate(counts):
        if n:
            check(y[lo:lo + n], w.dense(e), x[lo:lo + n], G, integer=True)
        lo += n
    assert (y[lo:] == -5.0).all()


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("K,G,zeros", [(4640, 32, True), (5504, 128, False), (7168, 64, True), (9600, 32, False)])
def test_gate_up_of_long_rows_with_many_of_them(K, G, zeros, dtype):
    # x of all K leaves room for 4, 2 or 1 columns a pass instead of 8 (fp32: of 4).  Integer inputs, so that the products are
    # exact: of the size of fp32's whole numbers, so only silu's tail and roundings remain
    counts, N = [0, 9, 1, 23], 40
    E, R = len(counts), sum(counts) + 1
    gate, up = G4(N, K, G, zeros, 31, E=E, integer=True), G4(N, K, G, zeros, 32, E=E, integer=True)
    x = x_of((R, K), dtype, 4, True)
    x[R - 1:] = float("nan")
    h = torch.full((R, N), -5.0, device=DEV)
    rfx.moe_gate_up_g4(gate.packed, up.packed, gate.stride, N, K, G, x, offsets_of(counts), h, zeros=zeros)
    lo = 0
    for e, n in enumerate(counts):
        if n:
            xe = x[lo:lo + n].double()
            g, u = xe @ gate.dense(e).t(), xe @ up.dense(e).t()
            want = g * torch.sigmoid(g) * u
            # as in test_expert_products_of_many_passes
            bound = (6 + 2 * g.abs().clamp(max=104)) * 2.0 ** -23 * want.abs() + 1e-37 * (1 + u.abs())
            assert bool(((h[lo:lo + n].double() - want).abs() <= bound).all())
        lo += n
    assert (h[lo:] == -5.0).all()


def test_gate_up_far_tail_of_silu():
    # one weight per row picks g and u: silu at the ends of fp32's range of exp
    N, K, G = 16, 32, 32
    codes = torch.full((N, K), 8, dtype=torch.uint8, device=DEV)
    codes[:, 0] = 9                                  # weight 1 in column 0
    s = torch.ones((N, 1), dtype=torch.float16, device=DEV)
    packed = torch.zeros(rfx.rfx_g4_packed_bytes(N, K, G), dtype=torch.uint8, device=DEV)
    rfx.rfx_g4_pack_device(codes, s, None, N, K, G, packed)
    x = torch.zeros((6, K), device=DEV)
    x[:, 0] = torch.tensor([0.0, -87.0, -95.0, 88.0, 3000.0, -3000.0])
    h = torch.empty((6, N), device=DEV)
    rfx.moe_gate_up_g4(packed, packed, packed.numel(), N, K, G, x, offsets_of([6]), h)
    v = x[:, :1].double()
    want = (v * v / (1 + torch.exp(-v))).expand(6, N)
    # exp(g) near -90 carries |g| * 2^-24 * 2 of its argument's rounding
    assert bool(((h.double() - want).abs() <= 4e-5 * want.abs() + 1e-38).all())


def test_expert_products_many_experts_and_bad_offsets():
    E, N, K, G = 1024, 32, 64, 32
    w = G4(N, K, G, False, 2, E=1, integer=True)
    packed = w.packed.repeat(E)
    counts = [0] * E
    for e in (0, 1, 511, 777, 1023):
        counts[e] = 1 + e % 3
    R = sum(counts)
    x = x_of((R, K), BF, 1, True)
    y = torch.empty((R, N), device=DEV)
    rfx.moe_gemv_g4(packed, w.stride, N, K, G, x, offsets_of(counts), y)
    check(y, w.dense(), x, G, integer=True)
    # offsets outside [0, R] are taken as the nearer end, a descending pair as no rows
    off = torch.tensor([-4, 2, 1, R + 9], dtype=torch.int32, device=DEV)
    y2 = torch.full((R, N), -5.0, device=DEV)
    rfx.moe_gemv_g4(packed, w.stride, N, K, G, x, off, y2)
    assert torch.equal(y2, y)


@pytest.mark.parametrize("K,dtype,rows", [(64, BF, (8, 9)), (4096, HF, (7, 8)), (2048, FF, (1, 5))])
def test_expert_products_of_many_passes(K, dtype, rows):
    # a CTA meets more columns than fit shared memory at once: x comes in several turns
    E, N, G = 300 if K > 64 else 1024, 32, 64
    w = G4(N, K, G, True, 2, E=1, integer=True)
    packed = w.packed.repeat(E)
    counts = [rows[e % 2] for e in range(E)]
    R = sum(counts)
    x = x_of((R, K), dtype, 1, True)
    y = torch.full((R, N), float("nan"), device=DEV)
    rfx.moe_gemv_g4(packed, w.stride, N, K, G, x, offsets_of(counts), y, zeros=True)
    check(y, w.dense(), x, G, integer=True)
    h = torch.full((R, N), float("nan"), device=DEV)
    rfx.moe_gate_up_g4(packed, packed, w.stride, N, K, G, x, offsets_of(counts), h, zeros=True)
    a = x.double() @ w.dense().t()
    want = a * torch.sigmoid(a) * a
    # the products are exact: silu's division and exponential (2 ulp of it, |a| * 2^-24 * 2 of its argument) remain
    bound = (6 + 2 * a.abs().clamp(max=104)) * 2.0 ** -23 * want.abs() + 1e-37
    assert bool(((h.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("E,R,K,G,zeros", [(6, 16, 1024, 64, True), (12, 16, 1024, 64, False), (6, 16, 7168, 32, True)])
def test_bits_of_a_row_depend_on_no_other_row(E, R, K, G, zeros, dtype):
    # one row through expert 3, wherever its place and whatever the other experts have: the same bits in every call of
    # the same E and R (K = 7168: in parts)
    N = 130
    w, up = G4(N, K, G, zeros, 41, E=E), G4(N, K, G, zeros, 42, E=E)
    v = x_of((1, K), dtype, 43, False)[0]
    first = None
    for seed, (before, mine, at) in enumerate([(0, 1, 0), (0, R, 7), (5, 3, 2), (9, 2, 0), (1, 9, 8), (R - 1, 1, 0)]):
        counts = [0] * E
        counts[3] = mine
        g = torch.Generator().manual_seed(seed)
        for e in torch.randint(0, 3, (before,), generator=g).tolist():
            counts[e] += 1
        for e in torch.randint(4, E, (R - before - mine,), generator=g).tolist():
            counts[e] += 1
        x = x_of((R, K), dtype, 50 + seed, False) * (seed + 1)
        r = before + at
        x[r] = v
        y, h = torch.empty((R, N), device=DEV), torch.empty((R, N), device=DEV)
        rfx.moe_gemv_g4(w.packed, w.stride, N, K, G, x, offsets_of(counts), y, zeros=zeros)
        rfx.moe_gate_up_g4(w.packed, up.packed, w.stride, N, K, G, x, offsets_of(counts), h, zeros=zeros)
        if first is None:
            first = y[r].clone(), h[r].clone()
            check(y[r:r + 1], w.dense(3), v[None], G)
        assert torch.equal(y[r], first[0]) and torch.equal(h[r], first[1])


def test_experts_past_4_gib_and_no_rows():
    N, K, G = 48, 256, 64
    w = G4(N, K, G, True, 7, E=3, integer=True)
    stride = (5 << 30) // 2                            # the third matrix begins at 5 GiB
    far = torch.empty(2 * stride + w.stride, dtype=torch.uint8, device=DEV)
    for e in range(3):
        far[e * stride:e * stride + w.stride] = w.packed[e * w.stride:(e + 1) * w.stride]
    counts = [2, 1, 3]
    x = x_of((6, K), BF, 3, True)
    y = torch.empty((6, N), device=DEV)
    rfx.moe_gemv_g4(far, stride, N, K, G, x, offsets_of(counts), y, zeros=True)
    for e, lo in ((0, 0), (1, 2), (2, 3)):
        check(y[lo:lo + counts[e]], w.dense(e), x[lo:lo + counts[e]], G, integer=True)
    none = torch.empty((0, K), dtype=BF, device=DEV)
    rfx.moe_gemv_g4(far, stride, N, K, G, none, offsets_of([0, 0, 0]), torch.empty((0, N), device=DEV), zeros=True)


def test_first_call_inside_a_capture():
    # in a process of its own: nothing of the library has run before the capture
    code = (
        "import torch, block_quantized_moe_rocmfpx_b200 as rfx\n"
        "d = 'cuda'\n"
        "W = torch.zeros(rfx.rfx_g4_packed_bytes(64, 128, 64), dtype=torch.uint8, device=d)\n"
        "x, y = torch.ones((1, 128), device=d).bfloat16(), torch.ones((1, 64), device=d)\n"
        "pos, w = torch.zeros((1, 1), dtype=torch.int32, device=d), torch.ones((1, 1), device=d)\n"
        "z = torch.zeros((1, 64), device=d)\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    rfx.rfx_gemv_g4(W, 64, 128, 64, x, y)\n"
        "    rfx.moe_combine_rows(y, pos, w, z)\n"
        "z.fill_(5)\n"
        "g.replay()\n"
        "torch.cuda.synchronize()\n"
        "assert (y == 0).all() and (z == 0).all()\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_first_clusters_inside_a_capture():
    code = (
        "import torch, block_quantized_moe_rocmfpx_b200 as rfx\n"
        "d = 'cuda'\n"
        "W = torch.zeros(rfx.rfx_g4_packed_bytes(64, 4096, 64), dtype=torch.uint8, device=d)\n"
        "x, y = torch.ones((2, 4096), device=d).bfloat16(), torch.ones((2, 64), device=d)\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    rfx.rfx_gemv_g4(W, 64, 4096, 64, x, y)\n"
        "y.fill_(5)\n"
        "g.replay()\n"
        "torch.cuda.synchronize()\n"
        "assert (y == 0).all()\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_python_checks_on_the_device():
    w = G4(32, 64, 32, False, 1)
    x, y = x_of((2, 64), BF, 1, False), torch.empty((2, 32), device=DEV)
    for bad in ({"x": x[:, :32]}, {"x": x.t().contiguous().t()}, {"y": y.half()}, {"x": x.double()}, {"y": y.cpu()},
                {"W": w.packed[:-1]}):
        a = {"W": w.packed, "x": x, "y": y, **bad}
        with pytest.raises(ValueError):
            rfx.rfx_gemv_g4(a["W"], 32, 64, 32, a["x"], a["y"])
    with pytest.raises(ValueError):                   # packed without zeros, read with
        rfx.rfx_gemv_g4(w.packed, 32, 64, 32, x, y, zeros=True)


# ------------------------------------------------- the operators together ---

def moe_step(x, logits, gate, up, down, k, base, bufs):
    """Route, group, gate/up, down and combine with 4-bit experts."""
    H, I, E = down.N, gate.N, gate.E
    rfx.moe_router_topk(logits, k, bufs["idx"], bufs["w"])
    rfx.moe_group_tokens(x, bufs["idx"], E, bufs["xs"], bufs["pos"], bufs["rows"], bufs["off"], bufs["ws"])
    rfx.moe_gate_up_g4(gate.packed, up.packed, gate.stride, I, H, gate.G, bufs["xs"], bufs["off"], bufs["h"],
                       zeros=gate.zeros)
    rfx.moe_gemv_g4(down.packed, down.stride, H, I, down.G, bufs["h"], bufs["off"], bufs["d"], zeros=down.zeros)
    rfx.moe_combine_rows(bufs["d"], bufs["pos"], bufs["w"], bufs["y"], base=base)


def make_bufs(T, k, E, H, I):
    i32 = dict(dtype=torch.int32, device=DEV)
    R = T * k
    return {"idx": torch.empty((T, k), **i32), "w": torch.empty((T, k), device=DEV),
            "xs": torch.empty((R, H), dtype=BF, device=DEV), "pos": torch.empty((T, k), **i32),
            "rows": torch.empty(R, **i32), "off": torch.empty(E + 1, **i32), "h": torch.empty((R, I), device=DEV),
            "d": torch.empty((R, H), device=DEV), "y": torch.empty((T, H), device=DEV),
            "ws": torch.zeros(rfx.moe_group_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)}


@pytest.mark.parametrize("T", [1, 4, 40])
def test_moe_step_and_its_router_gradient(T):
    H, I, E, k = 512, 256, 8, 2
    gate, up, down = (G4(n, c, 64, True, s, E=E) for n, c, s in ((I, H, 1), (I, H, 2), (H, I, 3)))
    x = x_of((T, H), BF, T, False)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    logits = torch.randn((T, E), generator=g, device=DEV)
    base = torch.randn((T, H), generator=g, device=DEV)
    b = make_bufs(T, k, E, H, I)
    moe_step(x, logits, gate, up, down, k, base, b)
    assert rfx.rfx_ws_status(b["ws"]) == rfx.RFX_OK
    dy = torch.randn((T, H), generator=g, device=DEV)
    dd, dw, dl = torch.empty_like(b["d"]), torch.empty_like(b["w"]), torch.empty_like(logits)
    rfx.moe_combine_rows_backward(dy, b["d"], b["pos"], b["w"], dd, dw)
    rfx.moe_router_topk_backward(b["idx"], b["w"], dw, dl)
    # the same in 64 bits through autograd, experts frozen
    l64 = logits.double().requires_grad_()
    sel = torch.topk(l64, k, dim=1)
    assert torch.equal(sel.indices.int(), b["idx"])
    w = torch.softmax(sel.values, dim=1)
    y = base.double()
    for t in range(T):
        for j in range(k):
            e = int(sel.indices[t, j])
            gg, uu = gate.dense(e) @ x[t].double(), up.dense(e) @ x[t].double()
            hh = gg * torch.sigmoid(gg) * uu
            y = y.index_add(0, torch.tensor([t], device=DEV), (w[t, j] * (down.dense(e) @ hh))[None])
    assert float((b["y"].double() - y.detach()).norm() / y.detach().norm()) <= 1e-5
    y.backward(dy.double())
    assert float((dl.double() - l64.grad).norm() / l64.grad.norm()) <= 1e-4


def test_moe_step_in_a_graph_and_two_streams_at_once():
    H, I, E, k, T = 1024, 256, 16, 4, 8
    gate, up, down = (G4(n, c, 32, False, s, E=E) for n, c, s in ((I, H, 1), (I, H, 2), (H, I, 3)))
    xa, xb = x_of((T, H), BF, 1, False), x_of((T, H), BF, 2, False)
    la, lb = (torch.randn((T, E), device=DEV) for _ in range(2))
    a, b = make_bufs(T, k, E, H, I), make_bufs(T, k, E, H, I)
    moe_step(xa, la, gate, up, down, k, None, a)
    moe_step(xb, lb, gate, up, down, k, None, b)
    torch.cuda.synchronize()
    ya, yb = a["y"].clone(), b["y"].clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a["y"].zero_()
        b["y"].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            moe_step(xa, la, gate, up, down, k, None, a)
        with torch.cuda.stream(s2):
            moe_step(xb, lb, gate, up, down, k, None, b)
        torch.cuda.synchronize()
        assert torch.equal(a["y"], ya) and torch.equal(b["y"], yb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe_step(xa, la, gate, up, down, k, None, a)
    xa.copy_(xb)
    la.copy_(lb)
    for _ in range(3):
        a["y"].zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a["y"], yb)
