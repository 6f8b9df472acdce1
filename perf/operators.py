"""Block-scaled formats next to the 2-bit codes: what is measured.

Two formats share one scale rule (a block is 32 consecutive elements of a row,
its scale the smallest power of two s with max |x| <= top * s):

  mx4  e2m1 elements, top = 6.  Byte i of a row holds element 2 i in its low
       nibble and element 2 i + 1 in its high one (bit 3 the sign).
  mx8  sign and 7-bit magnitude, top = 127.  In each group of four elements the
       bytes hold elements 0, 2, 1, 3.

A scale is the byte log2(s) + 127 (255: the block held a value that is not
finite).  The scales of 128 rows x 128 columns are 512 consecutive bytes: row r,
block b of them at 16 (r % 32) + 4 (r / 32) + b; such tiles lie row of tiles after
row of tiles, bytes outside the matrix are zero.

The operators:

  mx_round      pack a matrix (activations, weights), and the values it stands for
  mx4_linear    Y = Xq Wq^T for weights held in mx4: pack the tokens, multiply
  ckpt_forward  Y = X W~ of a 2-bit layer, and X kept for the backward in mx8
  ckpt_backward dX, dA, dB and dWp of that layer from the X kept in mx8
"""

import math

import torch

own = False

TOP = {"mx4": 6.0, "mx8": 127.0}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token's activations, rounded to 4 bits in front of a layer
        {"name": "round_mx4_token", "op": "mx_round", "fmt": "mx4", "rows": 1, "cols": 4096, "ld": 4096, "dtype": "bf16"},
        # a weight matrix that goes from fp32 to 4 bits once
        {"name": "round_mx4_weights", "op": "mx_round", "fmt": "mx4", "rows": 11008, "cols": 4096, "ld": 4096, "dtype": "fp32"},
        # a slice of a wider activation buffer, an odd number of tokens
        {"name": "round_mx8_strided", "op": "mx_round", "fmt": "mx8", "rows": 333, "cols": 1088, "ld": 1600, "dtype": "bf16"},
        # single-token decoding through a square projection
        {"name": "mx4_token", "op": "mx4_linear", "M": 1, "d_in": 4096, "d_out": 4096, "dtype": "bf16"},
        # a decoding batch through an up-projection
        {"name": "mx4_batch16", "op": "mx4_linear", "M": 16, "d_in": 4096, "d_out": 11008, "dtype": "bf16"},
        # odd token count, sizes that end inside a tile, fp32 in and out
        {"name": "mx4_ragged", "op": "mx4_linear", "M": 77, "d_in": 1088, "d_out": 520, "dtype": "fp32"},
        # the prompt's pass through an up-projection
        {"name": "mx4_prefill", "op": "mx4_linear", "M": 2048, "d_in": 4096, "d_out": 11008, "dtype": "bf16"},
        # a small layer in fp32, a few tokens
        {"name": "ckpt_forward_layer", "op": "ckpt_forward", "M": 16, "d_in": 512, "d_out": 512, "d": 4, "dtype": "fp32"},
        # the training step's forward of a down-projection
        {"name": "ckpt_forward_qat", "op": "ckpt_forward", "M": 8192, "d_in": 14336, "d_out": 4096, "d": 8, "dtype": "bf16"},
        # the small layer's backward
        {"name": "ckpt_backward_layer", "op": "ckpt_backward", "M": 16, "d_in": 512, "d_out": 512, "d": 4, "dtype": "fp32"},
        # an odd number of tokens, sizes that end inside a tile
        {"name": "ckpt_backward_ragged", "op": "ckpt_backward", "M": 333, "d_in": 1088, "d_out": 520, "d": 4, "dtype": "bf16"},
        # the training step's backward of a down-projection
        {"name": "ckpt_backward_qat", "op": "ckpt_backward", "M": 8192, "d_in": 14336, "d_out": 4096, "d": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    return max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step


def draw(rng):
    op = rng.choice(["mx_round", "mx4_linear", "ckpt_forward", "ckpt_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "mx_round":
        cols = _log(rng, 32, 14336, 32)
        return {"op": op, "fmt": rng.choice(["mx4", "mx8"]), "rows": _log(rng, 1, 8192), "cols": cols,
                "ld": cols + rng.choice([0, 0, 8, 512]), "dtype": dtype}
    case = {"op": op, "M": _log(rng, 1, 8192), "d_in": _log(rng, 64, 14336, 64), "d_out": _log(rng, 8, 11008, 8), "dtype": dtype}
    if op != "mx4_linear":
        case["d"] = rng.choice([1, 2, 4, 8])
        if dtype == "fp32":  # full precision is for small layers and checks
            case |= {"M": _log(rng, 1, 512), "d_in": _log(rng, 64, 4096, 64), "d_out": _log(rng, 8, 4096, 8)}
    return case


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "mx_round":
        return {"bytes": 2 * case["rows"] * case["cols"] * size, "flops": case["rows"] * case["cols"]}
    m, k, n = case["M"], case["d_in"], case["d_out"]
    if case["op"] == "mx4_linear":
        return {"bytes": size * (m * k + m * n) + n * k * 17 // 32, "flops": 2 * m * n * k}
    if case["op"] == "ckpt_forward":  # X read; codes read; Y and the values kept for the backward written
        return {"bytes": size * (2 * m * k + m * n) + n * k // 4, "flops": 2 * m * n * k}
    return {"bytes": m * k * 33 // 32 + size * (m * n + m * k) + n * k // 4 + n * k // 8 + 4 * n * k, "flops": 4 * m * n * k}


# ---------------------------------------------------------------- inputs
def _activations(g, rows, cols, dtype, ld=None):
    """N(0, 1) with one channel in a hundred twenty times as large."""
    x = torch.randn(rows, cols if ld is None else ld, generator=g, device="cuda")
    loud = torch.rand(x.shape[1], generator=g, device="cuda") < 0.01
    return torch.where(loud, 20 * x, x).to(DTYPE[dtype])[:, :cols]


def _tiles(e):
    """Scale bytes [rows][blocks] in the order of the 512-byte tiles (zeros outside)."""
    r, b = e.shape
    rt, bt = -(-r // 128), -(-b // 4)
    full = torch.zeros(rt * 128, bt * 4, dtype=torch.uint8, device=e.device)
    full[:r, :b] = e
    return full.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _bytes4(code):
    """Nibbles [rows][cols], two in a byte."""
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _bytes8(code):
    """Sign-and-magnitude bytes in the order 0, 2, 1, 3 of every four."""
    r, c = code.shape
    return code.view(r, c // 4, 2, 2).transpose(2, 3).contiguous().view(r, c)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "mx_round":
        state["X"] = _activations(g, case["rows"], case["cols"], case["dtype"], case["ld"])
        return state
    m, k, n = case["M"], case["d_in"], case["d_out"]
    X = _activations(g, m, k, case["dtype"])
    if case["op"] == "mx4_linear":
        code, e, _ = _quantise(0.02 * torch.randn(n, k, generator=g, device="cuda"), "mx4")
        return state | {"X": X, "Wq": _bytes4(code), "Ws": _tiles(e)}
    d = case["d"]
    eye = torch.eye(d, device="cuda")
    A = 0.02 * eye * (1 + 0.2 * torch.randn(d, d, generator=g, device="cuda")).abs()
    A = A + 0.002 * (1 - eye) * torch.randn(d, d, generator=g, device="cuda")
    state |= {"A": A, "B": -1.5 * A.sum(1)}
    Wp = 1.5 + torch.randn(n, k, generator=g, device="cuda")  # 13% of the weights outside [0, 3]
    z = Wp.round().clamp(0, 3).to(torch.uint8).view(n, k // 4, 4)
    state["packed"] = z[..., 0] | (z[..., 1] << 2) | (z[..., 2] << 4) | (z[..., 3] << 6)
    if case["op"] == "ckpt_forward":
        state["X"] = X
        return state
    inside = ((Wp >= 0) & (Wp <= 3)).view(n, k // 8, 8)
    state["mask"] = (inside.to(torch.int32) << torch.arange(8, device="cuda", dtype=torch.int32)).sum(-1).to(torch.uint8)
    code, e, _ = _quantise(X.float(), "mx8")
    state["Xq"], state["Xs"] = _bytes8(code), _tiles(e)
    state["dY"] = (0.1 * torch.randn(m, n, generator=g, device="cuda")).to(DTYPE[case["dtype"]])
    return state


# ---------------------------------------------------------------- the plain forms
def _quantise(x, fmt):
    """fp32 [rows][cols] -> element codes, scale bytes, values (fp32)."""
    r, c = x.shape
    b = x.view(r, c // 32, 32)
    most = b.abs().amax(-1, keepdim=True)
    frac, ex = torch.frexp(most)  # most = 2 frac * 2^(ex - 1)
    drop, edge = (2, 1.5) if fmt == "mx4" else (6, 127 / 64)
    e = (ex - 1 - drop + (2 * frac > edge)).clamp(min=-127)
    e = torch.where(most > 0, e, torch.full_like(e, -127))
    scale = torch.ldexp(torch.ones_like(most), e)
    v = b / scale
    a = v.abs()
    if fmt == "mx4":  # nearest of the grid, ties to the even code
        mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).to(torch.uint8)
        value = torch.tensor(GRID, device=x.device)[mag.long()]
        code = mag | ((v < 0).to(torch.uint8) << 3)
    else:
        value = a.round()
        code = value.to(torch.uint8) | ((v < 0).to(torch.uint8) << 7)
    value = torch.where(v < 0, -value, value) * scale
    return code.view(r, c), (e + 127).to(torch.uint8).view(r, c // 32), value.view(r, c)


def _scales(tiles, r, c):
    """The 512-byte tiles -> fp32 scales [rows][blocks]."""
    rt, bt = -(-r // 128), -(-c // 128)
    e = tiles.view(rt, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)[:r, : c // 32]
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e.to(torch.int32) - 127)


def _values4(q, tiles):
    r, c = q.shape[0], 2 * q.shape[1]
    code = torch.stack((q & 15, q >> 4), -1).view(r, c)
    v = torch.tensor(GRID, device=q.device)[(code & 7).long()]
    v = torch.where(code > 7, -v, v)
    return (v.view(r, c // 32, 32) * _scales(tiles, r, c)[..., None]).view(r, c)


def _values8(q, tiles):
    r, c = q.shape
    code = q.view(r, c // 4, 2, 2).transpose(2, 3).reshape(r, c)
    v = (code & 127).float()
    v = torch.where(code > 127, -v, v)
    return (v.view(r, c // 32, 32) * _scales(tiles, r, c)[..., None]).view(r, c)


def _codes(packed):
    n, kb = packed.shape
    return torch.stack((packed & 3, (packed >> 2) & 3, (packed >> 4) & 3, packed >> 6), -1).view(n, 4 * kb)


def _weights(packed, A, B):
    """W~ = A z + B of every vector of codes."""
    z = _codes(packed).to(A.dtype)
    d = A.shape[0]
    return (z.view(-1, d) @ A.T + B).view(z.shape)


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    out = DTYPE[case["dtype"]]
    if case["op"] == "mx_round":
        return _quantise(state["X"].float(), case["fmt"])[2].to(out)
    if case["op"] == "mx4_linear":
        X = _quantise(state["X"].float(), "mx4")[2]
        return (X @ _values4(state["Wq"], state["Ws"]).T).to(out)
    if case["op"] == "ckpt_forward":
        X = state["X"].float()
        return {"Y": (X @ _weights(state["packed"], state["A"], state["B"]).T).to(out), "kept": _quantise(X, "mx8")[2].to(out)}
    d = case["d"]
    dY = state["dY"].float()
    dX = dY @ _weights(state["packed"], state["A"], state["B"])
    G = (dY.T @ _values8(state["Xq"], state["Xs"])).view(-1, d)
    z = _codes(state["packed"]).view(-1, d)
    G64 = G.double()  # the sums over every vector of the matrix
    n, kb = state["mask"].shape
    bits = (state["mask"][..., None] >> torch.arange(8, device=G.device, dtype=torch.uint8)) & 1
    return {"dX": dX.to(out), "dA": (G64.T @ z.double()).float(), "dB": G64.sum(0).float(),
            "dWp": (G @ state["A"]).view(n, 8 * kb) * bits.view(n, 8 * kb)}


def _run_own(case, state):
    from bit_weight_only_lcvq_b200 import lcvq

    k = case.get("d_in")
    if case["op"] == "mx_round":
        q, s = lcvq.mx_pack(state["X"], case["fmt"])
        return lcvq.mx_decode(q, s, case["cols"], case["fmt"], dtype=state["X"].dtype)
    if case["op"] == "mx4_linear":
        q, s = lcvq.mx_pack(state["X"], "mx4")
        if "ws" not in state:
            state["ws"] = lcvq.new_workspace(lcvq.workspace_size(lcvq.OP_MX4_GEMM, state["X"].dtype, case["M"], case["d_out"], k, 8))
        return lcvq.mx4_gemm(q, s, state["Wq"], state["Ws"], dtype=state["X"].dtype, workspace=state["ws"])
    if case["op"] == "ckpt_forward":
        if "ws" not in state:
            state["ws"] = lcvq.new_workspace(lcvq.workspace_size(lcvq.OP_GEMM_CKPT, state["X"].dtype, case["M"], case["d_out"], k, case["d"]))
        Y, kept = lcvq.gemm_ckpt(state["X"], state["packed"], k, state["A"], state["B"], case["d"], workspace=state["ws"])
        return {"Y": Y, "kept": lcvq.mx_decode(*kept, k, "mx8", dtype=state["X"].dtype)}
    if "ws" not in state:
        state["ws"] = lcvq.new_workspace(lcvq.workspace_size(lcvq.OP_GEMM_BACKWARD_CKPT, state["dY"].dtype, case["M"], case["d_out"], k, case["d"]))
    g = lcvq.gemm_backward_ckpt((state["Xq"], state["Xs"]), state["dY"], state["packed"], state["mask"], k, state["A"], state["B"], case["d"], workspace=state["ws"])
    return {"dX": g["dX"], "dA": g["dA"], "dB": g["dB"], "dWp": g["dWp"]}


# ---------------------------------------------------------------- in 64 bits
def _near(x, fmt):
    """x as the format holds it, by searching the scale and the neighbours on the grid."""
    r, c = x.shape
    b = x.double().view(r, -1, 32)
    most = b.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(most / TOP[fmt])).clamp(-127, 127))
    s = torch.where(s * TOP[fmt] < most, 2 * s, s)
    s = torch.where((s / 2 * TOP[fmt] >= most) & (s > 2.0**-127), s / 2, s)
    v = b / s
    if fmt == "mx8":
        return (torch.round(v) * s).view(r, c)
    grid = torch.tensor(GRID, device=x.device, dtype=torch.float64)
    lo = (torch.searchsorted(grid, v.abs().contiguous(), right=True) - 1).clamp(0, 6)
    under, over = v.abs() - grid[lo], grid[lo + 1] - v.abs()
    up = (over < under) | ((over == under) & (lo % 2 == 1))
    return (torch.sign(v) * grid[lo + up] * s).view(r, c)


def _unpack64(q, tiles, fmt):
    """Values of packed bytes: each element's byte and scale looked up by their positions."""
    r = q.shape[0]
    c = q.shape[1] * (2 if fmt == "mx4" else 1)
    row, col = torch.arange(r, device=q.device)[:, None], torch.arange(c, device=q.device)[None]
    blk = torch.arange(c // 32, device=q.device)[None]
    at = (row // 128 * -(-c // 128) + blk // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + blk % 4
    s = torch.exp2(tiles[at].double() - 127).repeat_interleave(32, 1)
    if fmt == "mx4":
        code = (q.repeat_interleave(2, 1) >> (col % 2 * 4).to(torch.uint8)) & 15
        mag, neg = torch.tensor(GRID, device=q.device, dtype=torch.float64)[(code & 7).long()], code >> 3
    else:
        code = q[:, (col // 4 * 4 + torch.tensor([0, 2, 1, 3], device=q.device)[col % 4])[0]]
        mag, neg = (code & 127).double(), code >> 7
    return mag * (1 - 2 * neg.double()) * s


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "mx_round":
        return _near(state["X"], case["fmt"])
    if case["op"] == "mx4_linear":
        return _near(state["X"], "mx4") @ _unpack64(state["Wq"], state["Ws"], "mx4").T
    n, k, d = case["d_out"], case["d_in"], case["d"]
    z = ((state["packed"].repeat_interleave(4, 1) >> (torch.arange(k, device="cuda") % 4 * 2).to(torch.uint8)) & 3).double().view(n, k // d, d)
    A = state["A"].double()
    W = (torch.einsum("ij,ngj->ngi", A, z) + state["B"].double()).reshape(n, k)
    if case["op"] == "ckpt_forward":
        return {"Y": state["X"].double() @ W.T, "kept": _near(state["X"], "mx8")}
    dY = state["dY"].double()
    dX = dY @ W
    G = (dY.T @ _unpack64(state["Xq"], state["Xs"], "mx8")).view(n, k // d, d)
    inside = (state["mask"].repeat_interleave(8, 1) >> (torch.arange(k, device="cuda") % 8).to(torch.uint8)) & 1
    return {"dX": dX, "dA": torch.einsum("ngi,ngj->ij", G, z), "dB": G.sum((0, 1)),
            "dWp": torch.einsum("ij,ngi->ngj", A, G).reshape(n, k) * inside}
