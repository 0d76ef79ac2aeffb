"""Cases of the token-grouping, weighted-combine and 4-bit group-scale operators.

Each case names an operator, its sizes and its types.  With ``own`` false,
``run`` computes the operator in elementary torch operations in 32 bits; with
``own`` true it makes the library's calls.  ``exact`` gives the same outputs
from the definitions in 64 bits.

Operators (T tokens, k experts per token, R = T*k routed rows, E experts):

  group        rows sorted by expert: xs[pos[t][j]] = x[t], offsets, pos, rows
  group_bwd    its gradient: dx[t] = sum_j dxs[pos[t][j]]
  combine      rows back to tokens: y[t] = base[t] + sum_j w[t][j] ys[pos[t][j]]
  combine_bwd  its gradients: dys[pos[t][j]] = w[t][j] dy[t], dw[t][j] = dy[t].ys[pos[t][j]]
  gemv_g4      y = W x, W[n][c] = scale[n][c/G] (code - zero[n][c/G]), codes of 4 bits
  experts_g4   the same product for rows sorted by expert, one matrix per expert;
               "gate_up": h = silu(Wg x) * (Wu x)
  router_bwd   gradient of the router's softmax over the selected logits
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # speculative verify of four columns: the smallest call, only latency counts
        {"name": "group_verify_q4", "op": "group", "T": 4, "H": 4096, "E": 256, "k": 6, "dtype": "bf16"},
        # a long prompt's prefill batch: every token copied to its six experts' segments
        {"name": "group_prefill_8192", "op": "group", "T": 8192, "H": 4096, "E": 256, "k": 6, "dtype": "bf16"},
        # a training step's gradient of the grouping, an odd batch in half precision
        {"name": "group_grad_2047", "op": "group_bwd", "T": 2047, "H": 2560, "E": 64, "k": 8, "dtype": "fp16"},
        # verify columns: fp32 expert outputs, the shared expert's output as the base
        {"name": "combine_verify_q4", "op": "combine", "T": 4, "H": 4096, "E": 256, "k": 6, "dtype": "fp32",
         "out": "fp32", "base": True},
        # a ragged prefill batch in half precision, top-8 of 64
        {"name": "combine_ragged_1999", "op": "combine", "T": 1999, "H": 2560, "E": 64, "k": 8, "dtype": "fp16",
         "out": "fp16", "base": False},
        # a training step over frozen experts: gradients of their outputs and of the router's weights
        {"name": "combine_grad_4096", "op": "combine_bwd", "T": 4096, "H": 4096, "E": 256, "k": 6, "dtype": "bf16",
         "out": "fp32"},
        # one token through a square projection
        {"name": "gemv_g4_q1_4096", "op": "gemv_g4", "N": 4096, "K": 4096, "G": 128, "zeros": False, "q": 1,
         "dtype": "bf16"},
        # four verify columns through a vocabulary-sized matrix with zero points
        {"name": "gemv_g4_q4_131072", "op": "gemv_g4", "N": 131072, "K": 4096, "G": 64, "zeros": True, "q": 4,
         "dtype": "bf16"},
        # one token's six experts: gate and up with SwiGLU
        {"name": "experts_gate_up_q1", "op": "experts_g4", "kind": "gate_up", "E": 256, "hit": 6, "R": 6, "N": 2048,
         "K": 4096, "G": 128, "zeros": False, "dtype": "bf16"},
        # eight verify columns' experts: down products of fp32 activations, small groups with zero points
        {"name": "experts_down_q8", "op": "experts_g4", "kind": "plain", "E": 256, "hit": 37, "R": 48, "N": 4096,
         "K": 2048, "G": 32, "zeros": True, "dtype": "fp32"},
        # the router's gradient for a few tokens and for a long batch
        {"name": "router_grad_5", "op": "router_bwd", "T": 5, "E": 256, "k": 6},
        {"name": "router_grad_8192", "op": "router_bwd", "T": 8192, "E": 256, "k": 6},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group", "group_bwd", "combine", "combine_bwd", "gemv_g4", "gemv_g4", "experts_g4", "experts_g4",
                     "router_bwd"])
    if op == "router_bwd":
        E = _log_int(rng, 2, 512)
        return {"op": op, "T": _log_int(rng, 1, 8192 * 256 // max(E, 256)), "E": E, "k": rng.randint(2, min(E, 16))}
    if op in ("group", "group_bwd", "combine", "combine_bwd"):
        E = _log_int(rng, 2, 512)
        k = rng.randint(1, min(E, 10))
        H = _log_int(rng, 48, 8192)
        if rng.random() < 0.75:
            H = (H + 15) // 16 * 16
        most = 8192 * 6 * 4096 if op in ("group", "combine_bwd") else 4096 * 6 * 4096
        c = {"op": op, "T": _log_int(rng, 1, min(16384, max(1, most // (2 * k * H)))), "H": H, "E": E, "k": k,
             "dtype": rng.choice(["bf16", "fp16", "fp32"])}
        if op.startswith("combine"):
            c["out"] = rng.choice([c["dtype"], "fp32"])
            if op == "combine":
                c["base"] = rng.random() < 0.5
        return c
    G = rng.choice([32, 64, 128])
    zeros = rng.random() < 0.5
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    K = max(1, _log_int(rng, 128, 14336) // G) * G
    if op == "gemv_g4":
        return {"op": op, "N": _log_int(rng, 33, min(131072, 131072 * 4096 // K)), "K": K, "G": G, "zeros": zeros,
                "q": rng.randint(1, 8), "dtype": dtype}
    R = _log_int(rng, 1, 64)
    E = _log_int(rng, 8, 256)
    kind = rng.choice(["plain", "gate_up"])
    K = min(K, 4096)
    N = _log_int(rng, 64, min(4096, 2048 * 4096 // K))
    return {"op": op, "kind": kind, "E": E, "hit": rng.randint(1, min(E, R, 37)), "R": R, "N": N, "K": K, "G": G,
            "zeros": zeros, "dtype": dtype}


# ------------------------------------------------------------------ inputs ---

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFFFFFFFFFF)
    return g


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(DTYPES[dtype])


def _routing(c, seed):
    """idx int32 [T][k] (distinct experts per token) and w fp32 [T][k] of a skewed router."""
    T, E, k = c["T"], c["E"], c["k"]
    g = _gen(seed, 11)
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1.0
    logits = torch.randn((T, E), generator=g, device=DEV) - 1.1 * torch.log(rank)
    top = torch.topk(logits, k, dim=1)
    return top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, dim=1).contiguous()


def _places(idx):
    """Row of every entry in the order (expert, entry)."""
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(flat.numel(), device=DEV)
    return pos.to(torch.int32).reshape(idx.shape)


def _weights(c, seed, salt, count):
    """count matrices of N rows: two codes a byte (low one first) [count*N][K/2], scales, zeros or None."""
    g = _gen(seed, salt)
    rows, K, G = count * c["N"], c["K"], c["G"]
    b = torch.randint(0, 256, (rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = (0.005 * torch.exp2(2.0 * torch.rand((rows, K // G), generator=g, device=DEV) - 1.0)).half()
    z = None
    if c["zeros"]:
        z = (8.0 + 1.5 * torch.randn((rows, K // G), generator=g, device=DEV)).round().clamp(0, 15).to(torch.uint8)
    return b, s, z


def _sorted_rows(c, seed):
    """offsets int32 [E+1] of R rows over exactly `hit` experts, some of them with many rows."""
    g = _gen(seed, 17)
    E, hit, R = c["E"], c["hit"], c["R"]
    chosen = torch.randperm(E, generator=g, device=DEV)[:hit]
    u = torch.rand((R - hit,), generator=g, device=DEV)
    more = (u * u * hit).long().clamp(max=hit - 1)
    counts = torch.zeros(E, dtype=torch.int64, device=DEV)
    counts[chosen] = 1
    counts.scatter_add_(0, chosen[more], torch.ones_like(more))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return offsets


def _inputs(c, seed):
    op = c["op"]
    s = {}
    if op == "gemv_g4":
        s["x"] = _normal((c["q"], c["K"]), _gen(seed, 1), c["dtype"])
        s["w0"] = _weights(c, seed, 21, 1)
        return s
    if op == "experts_g4":
        s["x"] = _normal((c["R"], c["K"]), _gen(seed, 1), c["dtype"])
        s["offsets"] = _sorted_rows(c, seed)
        s["w0"] = _weights(c, seed, 21, c["E"])
        if c["kind"] == "gate_up":
            s["w1"] = _weights(c, seed, 22, c["E"])
        return s
    s["idx"], s["w"] = _routing(c, seed)
    T, k = c["T"], c["k"]
    if op == "router_bwd":
        s["dw"] = _normal((T, k), _gen(seed, 1), "fp32")
        return s
    H = c["H"]
    if op == "group":
        s["x"] = _normal((T, H), _gen(seed, 1), c["dtype"])
        return s
    s["pos"] = _places(s["idx"])
    s["rows"] = _normal((T * k, H), _gen(seed, 2), c["dtype"])
    if op == "combine" and c["base"]:
        s["base"] = _normal((T, H), _gen(seed, 3), c["out"])
    if op == "combine_bwd":
        s["dy"] = _normal((T, H), _gen(seed, 4), c["out"])
    return s


def _codes(b):
    return torch.stack((b & 15, b >> 4), dim=-1).reshape(b.shape[0], -1)


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    s["case"] = c
    if not own:
        return s
    import block_quantized_moe_rocmfpx_b200 as rfx
    s["rfx"] = rfx
    op = c["op"]

    def new(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device=DEV)

    if op in ("gemv_g4", "experts_g4"):
        count = c.get("E", 1)
        rows = (c["N"] + 15) // 16 * 16          # a matrix begins on a packed row-group
        stride = rfx.rfx_g4_packed_bytes(c["N"], c["K"], c["G"], c["zeros"])
        s["stride"] = stride
        for name in ("w0", "w1"):
            if name not in s:
                continue
            b, sc, z = s.pop(name)
            packed = new(count * stride, dtype=torch.uint8)
            per = c["N"] if rows != c["N"] else count * c["N"]
            for i in range(count * c["N"] // per):
                a = slice(i * per, (i + 1) * per)
                rfx.rfx_g4_pack_device(_codes(b[a]), sc[a], None if z is None else z[a], per, c["K"], c["G"],
                                       packed[i * stride:])
            s[name] = packed
        n = c["q"] if op == "gemv_g4" else c["R"]
        s["y"] = new(n, c["N"], dtype=torch.float32)
        return s
    T, k = c["T"], c["k"]
    if op == "group":
        s["xs"] = new(T * k, c["H"], dtype=DTYPES[c["dtype"]])
        s["pos"] = new(T, k, dtype=torch.int32)
        s["row_entry"] = new(T * k, dtype=torch.int32)
        s["offsets"] = new(c["E"] + 1, dtype=torch.int32)
        s["ws"] = new(rfx.moe_group_workspace_bytes(T, k, c["E"]), dtype=torch.uint8)
        rfx.rfx_ws_init(s["ws"])
    elif op == "group_bwd":
        s["dx"] = new(T, c["H"], dtype=DTYPES[c["dtype"]])
    elif op == "combine":
        s["y"] = new(T, c["H"], dtype=DTYPES[c["out"]])
    elif op == "combine_bwd":
        s["dys"] = new(T * k, c["H"], dtype=DTYPES[c["dtype"]])
        s["dw"] = new(T, k, dtype=torch.float32)
    else:
        s["dlogits"] = new(T, c["E"], dtype=torch.float32)
    return s


# -------------------------------------------------------------------- run ---

def _dense(w, G):
    """fp32 weights of two codes a byte, scales and zeros (8 where there are none)."""
    b, s, z = w
    v = _codes(b).float().reshape(b.shape[0], -1, G)
    v = v - (8.0 if z is None else z.float()[..., None])
    return (v * s.float()[..., None]).reshape(b.shape[0], -1)


def _expert_rows(w, c, offsets, x):
    """W_e x for every row, one row at a time, its expert's matrix picked on the device."""
    E, N, R = c["E"], c["N"], c["R"]
    row = torch.arange(R, device=DEV)
    expert = (row[:, None] >= offsets[None, 1:].long()).sum(1)
    out = []
    for r in range(R):
        e = expert[r:r + 1]
        part = tuple(None if a is None else a.reshape(E, N, -1).index_select(0, e)[0] for a in w)
        out.append(_dense(part, c["G"]) @ x[r].float())
    return torch.stack(out)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "gemv_g4":
        return s["x"].float() @ _dense(s["w0"], c["G"]).t()
    if op == "experts_g4":
        g = _expert_rows(s["w0"], c, s["offsets"], s["x"])
        if c["kind"] == "plain":
            return g
        u = _expert_rows(s["w1"], c, s["offsets"], s["x"])
        return g / (1.0 + torch.exp(-g)) * u
    T, k, E = c["T"], c["k"], c["E"]
    if op == "group":
        flat = s["idx"].reshape(-1).long()
        order = torch.argsort(flat, stable=True)
        pos = torch.empty_like(order)
        pos[order] = torch.arange(T * k, device=DEV)
        counts = torch.zeros(E, dtype=torch.int64, device=DEV)
        counts.scatter_add_(0, flat, torch.ones_like(flat))
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
        return {"xs": s["x"][order // k], "pos": pos.to(torch.int32).reshape(T, k), "rows": order.to(torch.int32),
                "offsets": offsets}
    if op == "router_bwd":
        w, dw = s["w"], s["dw"]
        d = w * (dw - (w * dw).sum(1, keepdim=True))
        out = torch.zeros((T, E), dtype=torch.float32, device=DEV)
        return out.scatter_(1, s["idx"].long(), d)
    pos = s["pos"].long()
    if op == "group_bwd":
        return s["rows"].float()[pos].sum(1).to(DTYPES[c["dtype"]])
    if op == "combine":
        y = (s["w"][..., None] * s["rows"].float()[pos]).sum(1)
        if c["base"]:
            y = s["base"].float() + y
        return y.to(DTYPES[c["out"]])
    dy = s["dy"].float()
    dys = torch.empty_like(s["rows"])
    dys[pos.reshape(-1)] = (s["w"][..., None] * dy[:, None, :]).reshape(T * k, -1).to(DTYPES[c["dtype"]])
    dw = (dy[:, None, :] * s["rows"].float()[pos]).sum(2)
    return {"dys": dys, "dw": dw}


def run(state):
    s = state
    if not own:
        return _run_plain(s)
    c, rfx = s["case"], s["rfx"]
    op = c["op"]
    if op == "gemv_g4":
        rfx.rfx_gemv_g4(s["w0"], c["N"], c["K"], c["G"], s["x"], s["y"], zeros=c["zeros"])
        return s["y"]
    if op == "experts_g4":
        if c["kind"] == "plain":
            rfx.moe_gemv_g4(s["w0"], s["stride"], c["N"], c["K"], c["G"], s["x"], s["offsets"], s["y"],
                            zeros=c["zeros"])
        else:
            rfx.moe_gate_up_g4(s["w0"], s["w1"], s["stride"], c["N"], c["K"], c["G"], s["x"], s["offsets"], s["y"],
                               zeros=c["zeros"])
        return s["y"]
    if op == "group":
        rfx.moe_group_tokens(s["x"], s["idx"], c["E"], s["xs"], s["pos"], s["row_entry"], s["offsets"], s["ws"])
        return {"xs": s["xs"], "pos": s["pos"], "rows": s["row_entry"], "offsets": s["offsets"]}
    if op == "group_bwd":
        rfx.moe_group_tokens_backward(s["rows"], s["pos"], s["dx"])
        return s["dx"]
    if op == "combine":
        rfx.moe_combine_rows(s["rows"], s["pos"], s["w"], s["y"], base=s.get("base"))
        return s["y"]
    if op == "combine_bwd":
        rfx.moe_combine_rows_backward(s["dy"], s["rows"], s["pos"], s["w"], s["dys"], s["dw"])
        return {"dys": s["dys"], "dw": s["dw"]}
    rfx.moe_router_topk_backward(s["idx"], s["w"], s["dw"], s["dlogits"])
    return s["dlogits"]


def work(case):
    c = case
    op = c["op"]
    if op in ("gemv_g4", "experts_g4"):
        mats = 1 if op == "gemv_g4" else c["hit"] * (2 if c["kind"] == "gate_up" else 1)
        per = c["N"] * (c["K"] // 2 + c["K"] // c["G"] * (3 if c["zeros"] else 2))
        n = c["q"] if op == "gemv_g4" else c["R"]
        products = 2 if c.get("kind") == "gate_up" else 1
        return {"bytes": mats * per + n * (c["K"] * BYTES[c["dtype"]] + c["N"] * 4)
                + (4 * (c["E"] + 1) if op == "experts_g4" else 0), "flops": 2 * n * c["N"] * c["K"] * products}
    T, k, E = c["T"], c["k"], c["E"]
    R = T * k
    if op == "router_bwd":
        return {"bytes": R * 12 + T * E * 4, "flops": 4 * R}
    H, b = c["H"], BYTES[c["dtype"]]
    if op == "group":
        return {"bytes": T * H * b + R * H * b + R * 12 + 4 * (E + 1), "flops": R}
    if op == "group_bwd":
        return {"bytes": R * H * b + T * H * b + R * 4, "flops": R * H}
    if op == "combine":
        return {"bytes": R * H * b + T * H * BYTES[c["out"]] * (2 if c["base"] else 1) + R * 8, "flops": 2 * R * H}
    return {"bytes": 2 * R * H * b + T * H * BYTES[c["out"]] + R * 12, "flops": 3 * R * H}


# ------------------------------------------------------------------ exact ---

def _product64(w, G, x, rows, block=4096):
    """x [n][K] times the matrix of rows `rows` (a slice), in 64 bits, a block of rows at a time."""
    b, s, z = w
    lo, hi, _ = rows.indices(b.shape[0])
    x = x.double()
    even, odd = x[:, 0::2], x[:, 1::2]
    per = G // 2
    out = []
    for a in range(lo, hi, block):
        e = min(a + block, hi)
        scale = s[a:e].double().repeat_interleave(per, dim=1)
        zero = 8.0 if z is None else z[a:e].double().repeat_interleave(per, dim=1)
        first = ((b[a:e] % 16).double() - zero) * scale
        second = ((b[a:e] // 16).double() - zero) * scale
        out.append(even @ first.t() + odd @ second.t())
    return torch.cat(out, dim=1)


def exact(case, seed):
    c = case
    op = c["op"]
    s = _inputs(c, seed)
    if op == "gemv_g4":
        return _product64(s["w0"], c["G"], s["x"], slice(None))
    if op == "experts_g4":
        off = s["offsets"].tolist()
        out = torch.zeros((c["R"], c["N"]), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            rows = slice(e * c["N"], (e + 1) * c["N"])
            a = _product64(s["w0"], c["G"], s["x"][lo:hi], rows)
            if c["kind"] == "gate_up":
                a = a * torch.special.expit(a) * _product64(s["w1"], c["G"], s["x"][lo:hi], rows)
            out[lo:hi] = a
        return out
    T, k, E = c["T"], c["k"], c["E"]
    if op == "group":
        flat = s["idx"].reshape(-1)
        rows = torch.cat([torch.nonzero(flat == e).reshape(-1) for e in range(E)])
        pos = torch.zeros(T * k, dtype=torch.int32, device=DEV)
        pos[rows] = torch.arange(T * k, dtype=torch.int32, device=DEV)
        offsets = torch.tensor([0] + [int(v) for v in torch.bincount(flat, minlength=E).cumsum(0).tolist()],
                               dtype=torch.int32, device=DEV)
        return {"xs": s["x"].double().index_select(0, torch.div(rows, k, rounding_mode="floor")),
                "pos": pos.reshape(T, k), "rows": rows.to(torch.int32), "offsets": offsets}
    w = s["w"].double()
    if op == "router_bwd":
        # the softmax's Jacobian diag(w) - w w^T on the selected logits
        jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        d = torch.einsum("tij,tj->ti", jac, s["dw"].double())
        out = torch.zeros((T, E), dtype=torch.float64, device=DEV)
        out[torch.arange(T, device=DEV)[:, None], s["idx"].long()] = d
        return out
    rows = s["rows"].double()
    pos = s["pos"].long()
    if op in ("group_bwd", "combine"):
        out = s["base"].double().clone() if s.get("base") is not None else \
            torch.zeros((T, c["H"]), dtype=torch.float64, device=DEV)
        for j in range(k):
            part = rows.index_select(0, pos[:, j])
            out += part if op == "group_bwd" else part * w[:, j:j + 1]
        return out
    dy = s["dy"].double()
    dys = torch.zeros_like(rows)
    dw = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        dys.index_copy_(0, pos[:, j], dy * w[:, j:j + 1])
        dw[:, j] = torch.einsum("th,th->t", dy, rows.index_select(0, pos[:, j]))
    return {"dys": dys, "dw": dw}
