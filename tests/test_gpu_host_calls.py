"""Host-buffer calls (moe_ffn_forward_host) whose uploads run on a side stream:
no upload may pass work that still uses the memory it writes to.

The calls of a test are issued back to back behind a busy stream, then every y is compared with
the device path (moe_router_topk and moe_ffn_forward on a workspace of its own) on the same inputs: decode bit
for bit; prefill adds with fp32 atomics, so equal up to the order of the adds.
"""
import pytest
import torch

import block_quantized_moe_rocmfpx_b200 as rfx
import synth
from synth.layers import SynthLayer

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, I, E, K = 512, 256, 16, 4
BUSY = 100_000_000          # cycles, about 50 ms


def layers(n, seed=71):
    lays = [SynthLayer(seed + i, 0, H, I, E, K) for i in range(n)]
    return lays, [lay.moe_layer() for lay in lays]


def host_inputs(T, seed):
    x = torch.from_numpy(synth.x_bf16(71, seed, T, H)).view(torch.bfloat16).pin_memory()
    logits = torch.from_numpy(synth.logits(71, 0, seed, T, E, 1.1)).pin_memory()
    return x, logits, torch.full((T, H), float("nan")).pin_memory()


def scratch_for(ml, *Ts):
    s = torch.empty(max(rfx.moe_ffn_host_scratch_bytes(ml.handle, T) for T in Ts), dtype=torch.uint8, device=DEV)
    rfx.rfx_ws_init(s)
    return s


def check(ml, x, logits, y):
    T = x.shape[0]
    ws = torch.zeros(rfx.moe_ffn_workspace_bytes(ml.handle, T), dtype=torch.uint8, device=DEV)
    idx = torch.empty((T, K), dtype=torch.int32, device=DEV)
    w = torch.empty((T, K), device=DEV)
    want = torch.empty((T, H), device=DEV)
    rfx.moe_router_topk(logits.to(DEV), K, idx, w)
    rfx.moe_ffn_forward(ml.handle, x.to(DEV), T, idx, w, want, ws)
    want = want.cpu()
    if T <= 8:
        assert torch.equal(y, want), T
    else:
        assert torch.allclose(y, want, rtol=1e-5, atol=1e-5 * float(want.abs().max())), T


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_calls_of_changing_T_on_one_scratch(seed):
    _, (ml,) = layers(1)
    Ts = [300, 2, 8, 1, 8, 300, 40, 1, 40, 8, 8, 2, 300, 1, 1, 1, 300, 300, 3, 5]
    Ts = Ts[seed:] + Ts[:seed]
    scratch = scratch_for(ml, *Ts)
    ins = [host_inputs(T, 1000 * seed + 37 * i) for i, T in enumerate(Ts)]
    torch.cuda._sleep(BUSY)
    for (x, logits, y), T in zip(ins, Ts):
        rfx.moe_ffn_forward_host(ml.handle, x, logits, T, y, scratch)
    torch.cuda.synchronize()
    assert rfx.rfx_ws_status(scratch) == rfx.RFX_OK
    for x, logits, y in ins:
        check(ml, x, logits, y)


def test_a_layer_keeps_its_larger_scratch():
    # MoeLayer.forward_host grows its scratch and uses the larger one for every smaller T
    _, (ml,) = layers(1)
    ins = [host_inputs(T, 11 * i) for i, T in enumerate((300, 2, 2, 8, 1, 300, 1))]
    torch.cuda._sleep(BUSY)
    for x, logits, y in ins:
        ml.forward_host(x, logits, y)
    torch.cuda.synchronize()
    assert ml.host_status() == rfx.RFX_OK
    for x, logits, y in ins:
        check(ml, x, logits, y)


@pytest.mark.parametrize("T", [1, 8, 40])
def test_layers_that_share_a_scratch(T):
    _, mls = layers(3)
    scratch = scratch_for(mls[0], T)
    order = [0, 1, 0, 1, 0, 0, 2, 1, 2, 0, 1, 1]
    ins = [host_inputs(T, 500 + 13 * i) for i in range(len(order))]
    torch.cuda._sleep(BUSY)
    for (x, logits, y), l in zip(ins, order):
        rfx.moe_ffn_forward_host(mls[l].handle, x, logits, T, y, scratch)
    torch.cuda.synchronize()
    for (x, logits, y), l in zip(ins, order):
        check(mls[l], x, logits, y)


def test_a_scratch_after_its_last_layer_is_gone():
    lays, mls = layers(2)
    T = 4
    scratch = scratch_for(mls[0], T)
    ins = [host_inputs(T, 700 + i) for i in range(4)]
    torch.cuda._sleep(BUSY)
    for i in (0, 1):
        rfx.moe_ffn_forward_host(mls[0].handle, *ins[i][:2], T, ins[i][2], scratch)
    torch.cuda.synchronize()
    for i in (0, 1):
        check(mls[0], *ins[i])
    mls[0] = lays[0].moe_layer()           # the old handle is destroyed, a new one may get its address
    torch.cuda._sleep(BUSY)
    for i in (2, 3):
        rfx.moe_ffn_forward_host(mls[i - 2].handle, *ins[i][:2], T, ins[i][2], scratch)
    torch.cuda.synchronize()
    for i in (2, 3):
        check(mls[i - 2], *ins[i])


@pytest.mark.parametrize("T", [2, 40])
def test_replayed_and_eager_calls_on_one_scratch(T):
    _, (ml,) = layers(1)
    scratch = scratch_for(ml, T)
    x, logits, y = host_inputs(T, 3)
    for _ in range(2):                     # eager first: both sets and the streams exist
        rfx.moe_ffn_forward_host(ml.handle, x, logits, T, y, scratch)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rfx.moe_ffn_forward_host(ml.handle, x, logits, T, y, scratch)
    y.fill_(float("nan"))
    ins = [host_inputs(T, 900 + 17 * i) for i in range(6)]
    torch.cuda._sleep(BUSY)
    for i, (a, b, out) in enumerate(ins):
        if i != 3:
            graph.replay()
        rfx.moe_ffn_forward_host(ml.handle, a, b, T, out, scratch)
    torch.cuda.synchronize()
    check(ml, x, logits, y)
    for a, b, out in ins:
        check(ml, a, b, out)


def test_one_layer_on_two_streams_with_a_scratch_each():
    _, (ml,) = layers(1)
    T = 40
    scratch = [scratch_for(ml, T) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    order = [0, 1, 1, 0, 1, 0, 0, 0, 1, 1, 0]
    ins = [host_inputs(T, 1300 + 19 * i) for i in range(len(order))]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
    for (x, logits, y), i in zip(ins, order):
        rfx.moe_ffn_forward_host(ml.handle, x, logits, T, y, scratch[i], streams[i])
    torch.cuda.synchronize()
    for x, logits, y in ins:
        check(ml, x, logits, y)


@pytest.mark.parametrize("part", [None, "all", "end"])
def test_uploads_run_ahead_unless_the_scratch_itself_was_zeroed(part):
    # behind a busy stream: a workspace of something else that is zeroed does not hold the uploads up, the
    # scratch (or a part of it) does
    _, (ml,) = layers(1)
    T = 4
    scratch = scratch_for(ml, T)
    other = torch.empty(4096, dtype=torch.uint8, device=DEV)
    ins = [host_inputs(T, 1500 + 23 * i) for i in range(3)]
    for x, logits, y in ins[:2]:
        rfx.moe_ffn_forward_host(ml.handle, x, logits, T, y, scratch)
    torch.cuda.synchronize()
    x, logits, y = ins[2]
    at = (rfx.moe_ffn_workspace_bytes(ml.handle, T) + 255) // 256 * 256      # the first set's x: the third call's
    there = scratch[at:at + 2 * T * H].view(torch.bfloat16).view(T, H)
    assert not torch.equal(there.cpu(), x)
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    torch.cuda._sleep(8 * BUSY)
    done.record()
    rfx.rfx_ws_init(other if part is None else scratch if part == "all" else scratch[-256:])
    rfx.moe_ffn_forward_host(ml.handle, x, logits, T, y, scratch)
    seen, copy = False, torch.empty((T, H), dtype=torch.bfloat16).pin_memory()
    while not seen and not done.query():
        with torch.cuda.stream(side):
            copy.copy_(there, non_blocking=True)
        side.synchronize()
        seen = torch.equal(copy, x) and not done.query()
    torch.cuda.synchronize()
    assert seen == (part is None)
    check(ml, x, logits, y)


def device_inputs(T, seed):
    x, logits, _ = host_inputs(T, seed)
    idx = torch.empty((T, K), dtype=torch.int32, device=DEV)
    w = torch.empty((T, K), device=DEV)
    rfx.moe_router_topk(logits.to(DEV), K, idx, w)
    return x.to(DEV), idx, w


def test_a_kept_workspace_is_made_on_the_stream_of_its_call():
    """MoeLayer's own workspaces on a side stream while the current one is busy: neither the zeroing nor what the
    current stream still has to write to memory that torch gave back may fall into the call."""
    _, (ml,) = layers(1)
    T = 40
    x, idx, w = device_inputs(T, 5)
    want, y = torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV)
    ml.prefill(x, idx, w, want)
    counts = ml.prefill_view(T)["counts"].clone()
    _, (ml,) = layers(1)
    hx, hl, hy = host_inputs(T, 6)
    side = torch.cuda.Stream()
    n = max(rfx.moe_prefill_workspace_bytes(ml.handle, T), rfx.moe_ffn_host_scratch_bytes(ml.handle, T))
    old = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in old:
        t.fill_(0xFF)
    del old, t
    ml.prefill(x, idx, w, y, stream=side)
    ml.forward_host(hx, hl, hy, stream=side)
    side.synchronize()
    first = hy.clone()
    hy.fill_(float("nan"))
    torch.cuda.synchronize()
    assert torch.equal(ml.prefill_view(T)["counts"], counts)
    torch.testing.assert_close(y, want, rtol=1e-5, atol=1e-5 * float(want.abs().max()))
    ml.forward_host(hx, hl, hy, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert ml.host_status() == rfx.RFX_OK and ml.prefill_status() == rfx.RFX_OK
    check(ml, hx, hl, first)
    check(ml, hx, hl, hy)


def test_a_grown_workspace_does_not_take_the_old_one_from_its_stream():
    # the old scratch goes back to torch while a side stream's call still works in it
    _, (ml,) = layers(1)
    small, big = host_inputs(8, 21), host_inputs(300, 22)
    n = rfx.moe_ffn_host_scratch_bytes(ml.handle, 8)
    ml.forward_host(*host_inputs(8, 20))             # the scratch comes from the current stream ...
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    ml.forward_host(*small, stream=side)             # ... is used on the other ...
    ml.forward_host(*big, stream=side)               # ... and outgrown
    for _ in range(8):
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xFF)
    torch.cuda.synchronize()
    assert ml.host_status() == rfx.RFX_OK
    check(ml, *small)
    check(ml, *big)


@pytest.mark.parametrize("T", [4, 40])
def test_kept_workspaces_in_a_captured_call(T):
    _, (ml,) = layers(1)
    hx, hl, hy = host_inputs(T, 31)
    x, idx, w = device_inputs(T, 32)
    y, want = torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV)
    ml.forward_host(hx, hl, hy)
    ml.prefill(x, idx, w, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ml.forward_host(hx, hl, hy)
        ml.prefill(x, idx, w, y)
    new = host_inputs(T, 33)
    hx.copy_(new[0])
    hl.copy_(new[1])
    hy.fill_(float("nan"))
    y.fill_(float("nan"))
    graph.replay()
    ml.forward_host(*new)
    torch.cuda.synchronize()
    check(ml, hx, hl, hy)
    check(ml, *new)
    torch.testing.assert_close(y, want, rtol=1e-5, atol=1e-5 * float(want.abs().max()))


@pytest.mark.parametrize("stream", [0, 1, 2])
def test_kept_workspaces_on_the_default_streams(stream):
    # the handles of the legacy and the per-thread default stream
    _, (ml,) = layers(1)
    for T in (2, 40, 2):
        x, logits, y = host_inputs(T, 50 + T)
        torch.cuda.synchronize()
        ml.forward_host(x, logits, y, stream=stream)
        torch.cuda.synchronize()
        check(ml, x, logits, y)
    assert ml.host_status() == rfx.RFX_OK
