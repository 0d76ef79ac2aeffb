"""Token rows grouped by expert, the weighted combine, their gradients and the
router's gradient, against plain 64-bit forms.

Tolerances, with u = 2^-24 (half an fp32 step, relative): a sum of k products
in fp32 by fma has k roundings, each at most u times the running magnitude
M = sum |w v| (+ |base|), so |error| <= (k + 1) u M; the one rounding to the
output type adds half a step of it, eps(type) / 2 times the value.  The dot
products sum H terms in an unspecified but fixed tree: at most H roundings,
|error| <= H u M.  Copies and integers are exact.
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_rocmfpx_b200 as rfx

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def plan_numpy(idx, E):
    flat = idx.reshape(-1)
    good = (flat >= 0) & (flat < E)
    ent = np.nonzero(good)[0]
    order = ent[np.argsort(flat[ent], kind="stable")]
    pos = np.full(flat.size, -1, np.int32)
    pos[order] = np.arange(order.size, dtype=np.int32)
    offsets = np.zeros(E + 1, np.int32)
    offsets[1:] = np.cumsum(np.bincount(flat[ent], minlength=E))
    return pos.reshape(idx.shape), order.astype(np.int32), offsets


def make_idx(rng, T, k, E, mode):
    if mode == "one":
        return np.full((T, k), E - 1, np.int32)
    if mode == "skew":
        return np.minimum((rng.random((T, k)) ** 4 * E).astype(np.int32), E - 1)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if mode == "padded":       # whole tokens and single entries without an expert
        idx[rng.random(T) < 0.3] = -1
        idx[rng.random((T, k)) < 0.1] = -1
    if mode == "none":
        idx[:] = -1
    return idx


def group(x, idx, E, ws=None, stream=None):
    T, k = idx.shape
    H = x.shape[1]
    xs = torch.full((T * k, H), 7.0, dtype=x.dtype, device=DEV)
    pos = torch.full((T, k), -9, dtype=torch.int32, device=DEV)
    rows = torch.full((T * k,), -9, dtype=torch.int32, device=DEV)
    off = torch.full((E + 1,), -9, dtype=torch.int32, device=DEV)
    if ws is None:
        ws = torch.empty(rfx.moe_group_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)
        rfx.rfx_ws_init(ws, stream)
    rfx.moe_group_tokens(x, idx, E, xs, pos, rows, off, ws, stream)
    return xs, pos, rows, off, ws


def check_group(x, idx_np, E):
    T, k = idx_np.shape
    xs, pos, rows, off, ws = group(x, torch.from_numpy(idx_np).to(DEV), E)
    torch.cuda.synchronize()
    p, r, o = plan_numpy(idx_np, E)
    n = int(o[-1])
    assert np.array_equal(off.cpu().numpy(), o)
    assert np.array_equal(pos.cpu().numpy(), p)
    assert np.array_equal(rows.cpu().numpy()[:n], r)
    assert (rows.cpu().numpy()[n:] == -9).all()
    want = torch.full_like(xs, 7.0)
    want[:n] = x[torch.from_numpy(r.astype(np.int64) // k).to(DEV)]
    assert torch.equal(xs.view(torch.uint8), want.view(torch.uint8))
    return ws


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("T,H,k,E", [(1, 8, 1, 1), (1, 4096, 6, 256), (4, 4096, 6, 256), (3, 1, 2, 5), (7, 33, 3, 4),
                                     (64, 250, 8, 9), (700, 72, 6, 300), (1500, 64, 8, 1024), (5000, 17, 2, 3),
                                     (9001, 40, 4, 64), (5, 8, 4, 2), (700, 2056, 6, 3), (60000, 16, 8, 256),
                                     (30000, 9, 16, 1000)])
def test_group_places_and_rows(T, H, k, E, dtype):
    rng = np.random.default_rng(T * 31 + H)
    x = torch.randn((T, H), device=DEV).to(dtype)
    ws = check_group(x, make_idx(rng, T, k, E, "uniform"), E)
    assert rfx.rfx_ws_status(ws) == rfx.RFX_OK


@pytest.mark.parametrize("mode", ["one", "skew", "padded", "none"])
@pytest.mark.parametrize("T,k", [(5, 6), (40, 3), (600, 7), (2000, 16)])
def test_group_routings(T, k, mode):
    rng = np.random.default_rng(T + k)
    x = torch.randn((T, 96), device=DEV).to(BF)
    ws = check_group(x, make_idx(rng, T, k, 33, mode), 33)
    assert rfx.rfx_ws_status(ws) == rfx.RFX_OK      # -1 is no error


@pytest.mark.parametrize("T,k", [(6, 4), (3000, 3)])
def test_group_bad_ids_set_the_flag_and_get_no_row(T, k):
    rng = np.random.default_rng(5)
    idx = make_idx(rng, T, k, 10, "uniform")
    idx[1, 0], idx[T - 1, k - 1], idx[2, 1] = 10, -2, 2 ** 31 - 1
    x = torch.randn((T, 64), device=DEV)
    ws = check_group(x, idx, 10)
    assert rfx.rfx_ws_status(ws) == rfx.RFX_EDEVICE
    assert rfx.rfx_ws_status(ws) == rfx.RFX_OK      # read and cleared


@pytest.mark.parametrize("off", [1, 3, 8])
def test_group_rows_at_any_element_alignment(off):
    T, H, k, E = 33, 64, 3, 7
    idx = torch.from_numpy(make_idx(np.random.default_rng(1), T, k, E, "uniform")).to(DEV)
    raw = torch.randn(T * H + off, device=DEV).to(BF)
    x = raw[off:].view(T, H)
    out = torch.zeros(T * k * H + off, dtype=BF, device=DEV)
    xs = out[off:].view(T * k, H)
    pos = torch.empty((T, k), dtype=torch.int32, device=DEV)
    rows = torch.empty(T * k, dtype=torch.int32, device=DEV)
    offs = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    ws = torch.zeros(rfx.moe_group_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)
    rfx.moe_group_tokens(x, idx, E, xs, pos, rows, offs, ws)
    assert torch.equal(xs, x[rows.long() // k])
    assert (out[:off] == 0).all()


def test_group_places_only():
    T, k, E = 900, 8, 60
    idx = make_idx(np.random.default_rng(2), T, k, E, "padded")
    pos = torch.empty((T, k), dtype=torch.int32, device=DEV)
    rows = torch.empty(T * k, dtype=torch.int32, device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    ws = torch.zeros(rfx.moe_group_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)
    rfx.moe_group_tokens(None, torch.from_numpy(idx).to(DEV), E, None, pos, rows, off, ws)
    p, r, o = plan_numpy(idx, E)
    assert np.array_equal(pos.cpu().numpy(), p) and np.array_equal(off.cpu().numpy(), o)
    assert np.array_equal(rows.cpu().numpy()[:o[-1]], r)


def test_rows_past_4_gib():
    T, H, k, E = 70000, 4096, 8, 64                 # 4.6 GB of grouped rows
    rng = np.random.default_rng(12)
    idx_np = make_idx(rng, T, k, E, "uniform")
    x = torch.randn((T, H), device=DEV).to(BF)
    xs, pos, rows, off, ws = group(x, torch.from_numpy(idx_np).to(DEV), E)
    p, r, o = plan_numpy(idx_np, E)
    assert np.array_equal(pos.cpu().numpy(), p) and np.array_equal(off.cpu().numpy(), o)
    some = torch.from_numpy(np.unique(np.concatenate([rng.integers(0, T * k, 500), [0, T * k - 1]]))).to(DEV)
    assert torch.equal(xs[some], x[rows[some].long() // k])
    w = torch.rand((T, k), device=DEV)
    y = torch.empty((T, H), dtype=BF, device=DEV)
    rfx.moe_combine_rows(xs, pos, w, y)
    t = torch.from_numpy(np.concatenate([rng.integers(0, T, 50), [T - 1]])).to(DEV)
    # every row of a token is the token itself: y = (sum_j w_j) x
    check_sum(y[t], w[t].double().sum(1, keepdim=True) * x[t].double(),
              w[t].double().sum(1, keepdim=True) * x[t].double().abs(), terms=k + 1)
    dw = torch.empty_like(w)
    rfx.moe_combine_rows_backward(x, xs, pos, w, xs, dw)      # gradients over the rows themselves
    sq = (x[t].double() ** 2).sum(1, keepdim=True)
    assert bool(((dw[t].double() - sq).abs() <= H * U * sq).all())
    got = xs[pos[t].long()].double()
    want = w[t].double()[..., None] * x[t].double()[:, None, :]
    assert bool(((got - want).abs() <= (half_step(BF) + U) * (1 + half_step(BF)) * want.abs()).all())


def test_no_tokens_is_a_no_op():
    i = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    f = torch.empty((0, 4), device=DEV)
    x = torch.empty((0, 16), device=DEV)
    off = torch.full((9,), 3, dtype=torch.int32, device=DEV)
    flat = torch.empty(0, dtype=torch.int32, device=DEV)
    rfx.moe_group_tokens(x, i, 8, x.clone(), i, flat, off, torch.empty(0, dtype=torch.uint8, device=DEV))
    rfx.moe_combine_rows(x, i, f, x.clone())
    rfx.moe_combine_rows_backward(x, x, i, f, x.clone(), f)
    rfx.moe_group_tokens_backward(x, i, x.clone())
    rfx.moe_router_topk_backward(i, f, f, torch.empty((0, 8), device=DEV))
    torch.cuda.synchronize()
    assert (off == 3).all()


# ------------------------------------------------------------- combine ---

def random_case(T, H, k, dtype, out, seed, drop=0.2, base=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    R = T * k
    perm = torch.randperm(R, generator=g, device=DEV).to(torch.int32)
    pos = perm.view(T, k).clone()
    pos[torch.rand((T, k), generator=g, device=DEV) < drop] = -1
    ys = torch.randn((R, H), generator=g, device=DEV).to(dtype)
    w = torch.rand((T, k), generator=g, device=DEV)
    b = torch.randn((T, H), generator=g, device=DEV).to(out) if base else None
    return ys, pos, w, b


def combine64(ys, pos, w, base):
    """y and sum of magnitudes in 64 bits; rows that pos does not name are never read."""
    T, k = pos.shape
    live = (pos >= 0).double()
    rows = ys.double()[pos.clamp(min=0).long()]
    rows = torch.where(live[..., None] > 0, rows, torch.zeros_like(rows))
    ww = torch.ones_like(live) if w is None else w.double()
    ww = torch.where(live > 0, ww, torch.zeros_like(ww))
    y = (ww[..., None] * rows).sum(1)
    m = (ww[..., None] * rows).abs().sum(1)
    if base is not None:
        y = y + base.double()
        m = m + base.double().abs()
    return y, m


def check_sum(got, y, m, terms):
    err = (got.double() - y).abs()
    s = half_step(got.dtype) if got.dtype != FF else 0.0
    tiny = torch.finfo(got.dtype).smallest_normal * 2 ** -8
    bound = terms * U * m * (1 + s) + s * y.abs() + tiny
    assert torch.isfinite(got).all()
    assert bool((err <= bound).all()), float((err / bound).max())


SHAPES = [(1, 1, 1), (1, 4096, 6), (4, 4096, 6), (3, 7, 2), (17, 264, 8), (130, 1000, 16), (333, 72, 5), (9, 8200, 3)]


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, FF), (HF, HF), (HF, FF), (FF, FF)])
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_combine(T, H, k, dtype, out):
    for base in (False, True):
        ys, pos, w, b = random_case(T, H, k, dtype, out, T + H, base=base)
        y = torch.full((T, H), float("nan"), dtype=out, device=DEV)
        rfx.moe_combine_rows(ys, pos, w, y, base=b)
        check_sum(y, *combine64(ys, pos, w, b), terms=k + 1)


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_group_backward(T, H, k, dtype):
    ys, pos, _, _ = random_case(T, H, k, dtype, dtype, 3 * T + H)
    dx = torch.full((T, H), float("nan"), dtype=dtype, device=DEV)
    rfx.moe_group_tokens_backward(ys, pos, dx)
    check_sum(dx, *combine64(ys, pos, None, None), terms=k)


def test_combine_leaves_dropped_rows_unread():
    # a row without an entry may hold anything, and a dropped entry's weight too
    T, H, k = 12, 512, 4
    ys, pos, w, b = random_case(T, H, k, BF, FF, 9, drop=0.5)
    named = torch.zeros(T * k, dtype=torch.bool, device=DEV)
    named[pos[pos >= 0].long()] = True
    ys[~named] = float("nan")
    w[pos < 0] = float("inf")
    pos[0] = -1                                    # a token with no row at all
    pos[1, 0] = T * k                              # beyond the rows: as -1
    y = torch.empty((T, H), dtype=FF, device=DEV)
    rfx.moe_combine_rows(ys, pos, w, y, base=b)
    p2 = pos.clone()
    p2[1, 0] = -1
    check_sum(y, *combine64(ys, p2, w, b), terms=k + 1)
    assert torch.equal(y[0], b[0])
    # in place: y is base
    y2 = b.clone()
    rfx.moe_combine_rows(ys, pos, w, y2, base=y2)
    assert torch.equal(y2, y)


def test_combine_keeps_nan_and_inf_of_named_rows():
    T, H, k = 2, 64, 2
    ys = torch.ones((4, H), device=DEV)
    ys[1, 3], ys[2, 5] = float("nan"), float("inf")
    pos = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    w = torch.full((2, 2), 0.5, device=DEV)
    y = torch.empty((2, H), device=DEV)
    rfx.moe_combine_rows(ys, pos, w, y)
    assert torch.isnan(y[0, 3]) and torch.isinf(y[1, 5])
    assert int(torch.isfinite(y).sum()) == 2 * H - 2


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, FF), (HF, HF), (HF, FF), (FF, FF)])
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_combine_backward(T, H, k, dtype, out):
    ys, pos, w, _ = random_case(T, H, k, dtype, out, 7 * T + H, base=False)
    g = torch.Generator(device=DEV)
    g.manual_seed(H)
    dy = torch.randn((T, H), generator=g, device=DEV).to(out)
    dys = torch.full_like(ys, 5.0)
    dw = torch.full((T, k), float("nan"), device=DEV)
    rfx.moe_combine_rows_backward(dy, ys, pos, w, dys, dw)
    want = torch.full(ys.shape, 5.0, dtype=torch.float64, device=DEV)
    live = pos >= 0
    prod = w.double()[..., None] * dy.double()[:, None, :]
    want[pos[live].long()] = prod[live]
    err = (dys.double() - want).abs()
    s = half_step(dtype)
    # w * dy is rounded to fp32 first, then once to the type
    bound = (s + U) * (1 + s) * want.abs() + torch.finfo(dtype).smallest_normal * 2 ** -8
    assert bool((err <= bound).all())
    rows = ys.double()[pos.clamp(min=0).long()]
    terms = torch.where(live[..., None], dy.double()[:, None, :] * rows, torch.zeros_like(rows))
    err = (dw.double() - terms.sum(2)).abs()
    assert bool((err <= H * U * terms.abs().sum(2) + 1e-38).all())
    assert (dw[~live] == 0).all()
    # dys written over ys, and the same bits again
    over, dw2 = ys.clone(), torch.empty_like(dw)
    rfx.moe_combine_rows_backward(dy, over, pos, w, over, dw2)
    assert torch.equal(dw, dw2) and torch.equal(over[pos[live].long()], dys[pos[live].long()])


def shifted(t, off):
    """A copy of t that begins `off` elements past a 16-byte boundary, and the buffer it lies in."""
    raw = torch.full((t.numel() + off + 16,), 3.0, dtype=t.dtype, device=DEV)
    v = raw[off:off + t.numel()].view(t.shape)
    v.copy_(t)
    assert v.data_ptr() == raw.data_ptr() + off * t.element_size()
    return v, raw


def untouched(v, raw, off):
    return bool((raw[:off] == 3.0).all() and (raw[off + v.numel():] == 3.0).all())


# elements that ys (or dxs), the token side (base, y, dy, dx) and dys lie off a 16-byte boundary: pieces of 16 bytes,
# of two elements and of one
OFFS = [(0, 0, 0), (0, 2, 0), (2, 0, 2), (4, 4, 4), (1, 0, 0), (0, 1, 0), (0, 0, 1), (2, 2, 3), (3, 5, 7)]


@pytest.mark.parametrize("ro,to,do", OFFS)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, FF), (FF, FF)])
def test_combine_and_gradients_at_any_element_alignment(dtype, out, ro, to, do):
    T, H, k = 21, 264, 5
    ys, pos, w, b = random_case(T, H, k, dtype, out, 31, base=True)
    ys, _ = shifted(ys, ro)
    b, _ = shifted(b, to)
    y, yraw = shifted(torch.full((T, H), float("nan"), dtype=out, device=DEV), to)
    rfx.moe_combine_rows(ys, pos, w, y, base=b)
    check_sum(y, *combine64(ys, pos, w, b), terms=k + 1)
    assert untouched(y, yraw, to)
    dx, dxraw = shifted(torch.full((T, H), float("nan"), dtype=dtype, device=DEV), to)
    rfx.moe_group_tokens_backward(ys, pos, dx)
    check_sum(dx, *combine64(ys, pos, None, None), terms=k)
    assert untouched(dx, dxraw, to)
    # the gradients: the same bits for dys as without the shift, dw's sums in another order
    dy = torch.randn((T, H), device=DEV).to(out)
    want, dw = torch.full_like(ys, 5.0), torch.empty_like(w)
    rfx.moe_combine_rows_backward(dy, ys.clone(), pos, w, want, dw)
    dys, dysraw = shifted(torch.full_like(ys, 5.0), do)
    dw2 = torch.full_like(w, float("nan"))
    rfx.moe_combine_rows_backward(shifted(dy, to)[0], ys, pos, w, dys, dw2)
    assert torch.equal(dys, want) and untouched(dys, dysraw, do)
    live = pos >= 0
    rows = torch.where(live[..., None], ys.double()[pos.clamp(min=0).long()], torch.zeros((), dtype=torch.float64, device=DEV))
    terms = dy.double()[:, None, :] * rows
    assert bool(((dw2.double() - terms.sum(2)).abs() <= H * U * terms.abs().sum(2) + 1e-38).all())
    assert (dw2[~live] == 0).all()


def test_combine_gradients_against_differences():
    # L = <c, combine(ys, w)> is linear in ys and in w: its difference quotient is exact up to rounding
    T, H, k = 5, 96, 3
    ys, pos, w, _ = random_case(T, H, k, FF, FF, 21, base=False)
    c = torch.randn((T, H), device=DEV)
    dys, dw = torch.zeros_like(ys), torch.empty_like(w)
    rfx.moe_combine_rows_backward(c, ys, pos, w, dys, dw)
    dirs, dirw = torch.randn_like(ys), torch.randn_like(w)

    def loss(a, b):
        y = torch.empty((T, H), device=DEV)
        rfx.moe_combine_rows(a, pos, b, y)
        return float((y.double() * c.double()).sum())

    slope_y = loss(ys + dirs, w) - loss(ys, w)
    slope_w = loss(ys, w + dirw) - loss(ys, w)
    # inputs and outputs of magnitude < 16 rounded to fp32, T*H*k of them: 2e-4 covers 1440 * 16 * 2^-24 * 8
    tol = 8 * T * H * k * 16 * 16 * U
    assert abs(slope_y - float((dys.double() * dirs.double()).sum())) <= tol
    live = (pos >= 0).double()
    assert abs(slope_w - float((dw.double() * dirw.double() * live).sum())) <= tol


# ------------------------------------------------------ router gradient ---

@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 6), (5, 256, 6), (9, 7, 7), (300, 33, 2), (64, 1024, 16),
                                   (1000, 250, 8), (3, 130, 5)])
def test_router_backward_matches_autograd_in_64_bits(T, E, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(T * E)
    logits = torch.randn((T, E), generator=g, device=DEV)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    rfx.moe_router_topk(logits, k, idx, w)
    dw = torch.randn((T, k), generator=g, device=DEV)
    dl = torch.full((T, E), float("nan"), device=DEV)
    rfx.moe_router_topk_backward(idx, w, dw, dl)
    l64 = logits.double().requires_grad_()
    torch.softmax(l64.gather(1, idx.long()), dim=1).backward(dw.double())
    # w is within 2^-20 of the softmax (its own tolerance, 1e-6); the k-term sum and two products add (k + 3) u
    m = w.double() * (dw.abs().double() + (w.abs() * dw.abs()).double().sum(1, keepdim=True))
    bound = torch.zeros_like(l64).scatter_(1, idx.long(), (4e-6 + (k + 3) * U) * m) + 1e-38
    assert bool(((dl.double() - l64.grad).abs() <= bound).all())


def test_router_backward_repeated_and_missing_ids():
    idx = torch.tensor([[2, 2, 0], [-1, 3, 1], [4, 9, 4]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, 0.25, 0.25]] * 3, device=DEV)
    dw = torch.tensor([[1.0, 2.0, -1.0]] * 3, device=DEV)
    dl = torch.full((3, 5), float("nan"), device=DEV)
    rfx.moe_router_topk_backward(idx, w, dw, dl)
    s = 0.5 + 0.5 - 0.25
    d = [0.5 * (1 - s), 0.25 * (2 - s), 0.25 * (-1 - s)]
    want = torch.tensor([[d[2], 0, d[0] + d[1], 0, 0], [0, d[2], 0, d[1], 0], [0, 0, 0, 0, d[0] + d[2]]], device=DEV)
    assert torch.equal(dl, want)      # every value is a short binary fraction: exact


# --------------------------------------------------- streams and graphs ---

def test_rows_on_a_side_stream_and_in_a_graph():
    T, H, k, E = 700, 256, 6, 40          # two launches
    rng = np.random.default_rng(8)
    idx = torch.from_numpy(make_idx(rng, T, k, E, "skew")).to(DEV)
    x = torch.randn((T, H), device=DEV).to(BF)
    w = torch.rand((T, k), device=DEV)
    ws = torch.zeros(rfx.moe_group_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)
    xs = torch.empty((T * k, H), dtype=BF, device=DEV)
    pos = torch.empty((T, k), dtype=torch.int32, device=DEV)
    rows = torch.empty(T * k, dtype=torch.int32, device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    y = torch.empty((T, H), device=DEV)
    dys, dw, dx = torch.empty_like(xs), torch.empty_like(w), torch.empty_like(x)
    dl = torch.empty((T, E), device=DEV)

    def step():
        rfx.moe_group_tokens(x, idx, E, xs, pos, rows, off, ws)
        rfx.moe_combine_rows(xs, pos, w, y)
        rfx.moe_combine_rows_backward(y, xs, pos, w, dys, dw)
        rfx.moe_group_tokens_backward(dys, pos, dx)
        rfx.moe_router_topk_backward(idx, w, dw, dl)

    outs = (xs, pos, rows, off, y, dys, dw, dx, dl)
    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in outs:
            t.zero_()
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # new inputs in the same buffers, replayed twice
    idx2 = make_idx(rng, T, k, E, "padded")
    idx.copy_(torch.from_numpy(idx2))
    x.copy_(torch.randn((T, H), device=DEV).to(BF))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    p, r, o = plan_numpy(idx2, E)
    assert np.array_equal(got[1].cpu().numpy(), p) and np.array_equal(got[3].cpu().numpy(), o)
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a[:int(o[-1])] if i in (0, 2, 5) else a, b[:int(o[-1])] if i in (0, 2, 5) else b)
               for i, (a, b) in enumerate(zip(got, outs)))
