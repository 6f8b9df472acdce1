"""Block-scaled formats on the GPU: packing, decoding, the mx4 product, and the
training step that keeps X in 8 bits, against their fp64 definitions."""

import numpy as np
import pytest
import torch

from bit_weight_only_lcvq_b200 import lcvq, synth
from oracle import lcvq_oracle as O
from oracle import mx_oracle as MX
from tests.gpu_util import dev, guard_intact, guarded, to_dev, to_np

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def bf16_np(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(BF16).float().numpy()


def matrix(seed, rows, cols, dtype, wild=False):
    """N(0, 1) with loud channels; wild: blocks of every magnitude, zeros, signed
    zeros, subnormals and non-finite values too."""
    g = rng(seed)
    x = g.standard_normal((rows, cols)).astype(np.float32)
    x[:, g.random(cols) < 0.02] *= 20
    if wild:
        e = g.integers(-140, 126, (rows, cols // 32))
        with np.errstate(over="ignore"):
            x = np.ldexp(x, np.repeat(e, 32, 1)).astype(np.float32)
        b = x.reshape(rows, -1, 32)
        hit = g.random((rows, cols // 32))
        b[hit < 0.05] = 0
        b[(hit >= 0.05) & (hit < 0.1), 0] = -0.0
        b[(hit >= 0.1) & (hit < 0.15), 7] = np.nan
        b[(hit >= 0.15) & (hit < 0.2), 31] = -np.inf
        b[(hit >= 0.2) & (hit < 0.25), 3] = np.finfo(np.float32).max
        x[np.isfinite(x) & (np.abs(x) > 3.3e38)] = 3.3e38
    return bf16_np(x) if dtype == BF16 else x


def grid_values(seed, rows, cols):
    """Exact halves around every rounding border of both formats, scale 1 and 2."""
    g = rng(seed)
    x = (g.integers(-12, 13, (rows, cols)) / 4).astype(np.float32)
    x.reshape(rows, -1, 32)[:, :, 0] = 6
    x.reshape(rows, -1, 32)[:, 1::2, 1] = 7
    return x


def same_values(a, b):
    return np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])


# ---------------------------------------------------------------- packing
@pytest.mark.parametrize("fmt", ["mx4", "mx8"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols,wild", [(1, 32, False), (1, 4096, False), (3, 96, True), (129, 160, True),
                                            (77, 1088, False), (300, 2080, True), (2500, 8320, False)])
def test_pack_bytes_and_values(fmt, dtype, rows, cols, wild):
    x = matrix(rows + cols, rows, cols, dtype, wild)
    X = to_dev(x, dtype)
    nb = lcvq.mx_scale_bytes(rows, cols)
    q, qbuf = guarded((rows, cols // 2 if fmt == "mx4" else cols), torch.uint8)
    s, sbuf = guarded((nb,), torch.uint8)
    lcvq.mx_pack(X, fmt, q=q, scales=s)
    want, byte = MX.pack(x, fmt)
    tiles = s.cpu().numpy()
    assert np.array_equal(MX.untile_scales(tiles, rows, cols), byte)
    assert np.array_equal(q.cpu().numpy(), want)
    assert guard_intact(q, qbuf) and guard_intact(s, sbuf)
    # bytes of the last tile's columns beyond the last: 0 in the rows there are
    if cols % 128:
        t = tiles.reshape(-1, -(-cols // 128), 32, 4, 4)[:, -1].transpose(0, 2, 1, 3).reshape(-1, 4)
        assert not t[:rows, (cols % 128) // 32:].any()
    for odt in (BF16, F32):
        out, obuf = guarded((rows, cols), odt)
        lcvq.mx_decode(q, s, cols, fmt, out=out)
        assert guard_intact(out, obuf)
        assert same_values(to_np(out), MX.unpack(want, byte, fmt))


@pytest.mark.parametrize("fmt", ["mx4", "mx8"])
def test_pack_rounds_ties_to_even(fmt):
    x = grid_values(5, 64, 256)
    if fmt == "mx8":
        x = x * 10.5  # max 63 and 73.5: scale 1/2 and 1, quarters and halves
    q, s = lcvq.mx_pack(to_dev(x, F32), fmt)
    assert np.array_equal(q.cpu().numpy(), MX.pack(x, fmt)[0])
    assert np.array_equal(to_np(lcvq.mx_decode(q, s, 256, fmt, dtype=F32)), MX.values(x, fmt))


@pytest.mark.parametrize("dtype,ld", [(BF16, 1096), (BF16, 1600), (F32, 1092)])
def test_pack_takes_strided_rows(dtype, ld):
    x = matrix(8, 131, 1088, dtype)
    wide = torch.full((131, ld), 1e30, dtype=dtype, device=dev())
    wide[:, :1088] = to_dev(x, dtype)
    for fmt in ("mx4", "mx8"):
        q, s = lcvq.mx_pack(wide[:, :1088], fmt)
        assert np.array_equal(q.cpu().numpy(), MX.pack(x, fmt)[0])
    with pytest.raises(ValueError):
        lcvq.mx_pack(wide.t(), "mx4")
    with pytest.raises(lcvq.LcvqError):
        lcvq.mx_pack(wide[:, 1:1089], "mx4")  # rows start off a 16-byte boundary


def test_pack_of_nothing():
    for shape in ((0, 64), (3, 0)):
        q, s = lcvq.mx_pack(torch.empty(shape, dtype=BF16, device=dev()), "mx8")
        assert q.shape == shape and lcvq.mx_decode(q, s, shape[1], "mx8").shape == shape


# ---------------------------------------------------------------- mx4 product
def product_tolerance(K, dtype, y, D):
    """The products of a block are exact.  Their sums meet in fp32: one rounding
    per block of 32 and, at the end, up to 16 parts; a tensor core may truncate
    instead of rounding, so 2^-23 of the sum of magnitudes for each.  Then the
    output's own rounding, half a step."""
    return (K / 32 + 16) * 2.0 ** -23 * D + torch.finfo(dtype).eps / 2 * np.abs(y)


def mx4_operands(seed, M, N, K):
    x, w = matrix(seed, M, K, BF16), 0.02 * matrix(seed + 1, N, K, F32)
    xq, xs = lcvq.mx_pack(to_dev(x, BF16), "mx4")
    wq, ws = lcvq.mx_pack(to_dev(w, F32), "mx4")
    return xq, xs, wq, ws, MX.values(x, "mx4"), MX.values(w, "mx4")


SHAPES = [(1, 8, 64), (1, 4096, 4096), (2, 520, 192), (7, 136, 1088), (8, 128, 128), (9, 264, 320),
          (16, 1000, 4096), (17, 192, 576), (32, 512, 960), (33, 200, 448), (64, 256, 2048), (77, 520, 1088),
          (128, 192, 256), (129, 384, 704), (200, 1544, 1216), (256, 2048, 512), (513, 776, 1472),
          (1024, 1600, 64), (200, 8, 64), (129, 16, 128), (128, 8, 320)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_mx4_gemm(M, N, K, dtype):
    xq, xs, wq, ws, xv, wv = mx4_operands(M + N + K, M, N, K)
    out, buf = guarded((M, N), dtype)
    lcvq.mx4_gemm(xq, xs, wq, ws, out=out)
    y, D = MX.gemm(xv, wv)
    assert guard_intact(out, buf)
    assert (np.abs(to_np(out) - y) <= product_tolerance(K, dtype, y, D)).all()


def whole_operands(seed, rows, cols):
    """mx4 bytes whose products sum exactly in fp32: integer elements, scales 1 and 2."""
    g = rng(seed)
    x = g.integers(-6, 7, (rows, cols)).astype(np.float32)
    x[np.abs(x) == 5] = 4
    b = x.reshape(rows, -1, 32)
    b[:, :, 0] = 6
    b *= g.integers(1, 3, (rows, cols // 32, 1))
    return x


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_mx4_gemm_exact_on_whole_numbers(M, N, K):
    x, w = whole_operands(1, M, K), whole_operands(2, N, K)
    xq, xs = lcvq.mx_pack(to_dev(x, F32), "mx4")
    wq, ws = lcvq.mx_pack(to_dev(w, F32), "mx4")
    y = lcvq.mx4_gemm(xq, xs, wq, ws, dtype=F32)
    assert np.array_equal(to_np(y), x.astype(np.float64) @ w.T.astype(np.float64))


@pytest.mark.parametrize("M", [1, 5, 16, 32, 100, 300])
def test_mx4_gemm_scales_far_apart_and_nan(M):
    """Blocks of very different size next to one another, zero blocks, and blocks
    that stand for NaN: their row or column is NaN, nothing else is."""
    g = rng(M)
    N, K = 264, 448
    x, w = matrix(M, M, K, F32), matrix(M + 1, N, K, F32)
    x = np.ldexp(x, np.repeat(g.integers(-20, 20, (M, K // 32)), 32, 1)).astype(np.float32)
    w = np.ldexp(w, np.repeat(g.integers(-20, 20, (N, K // 32)), 32, 1)).astype(np.float32)
    x[:, 32:64] = 0
    w[5] = 0
    clean_rows = M > 1
    if clean_rows:
        x[M // 2, 40] = np.inf
    w[77, 447] = np.nan
    xq, xs = lcvq.mx_pack(to_dev(x, F32), "mx4")
    wq, ws = lcvq.mx_pack(to_dev(w, F32), "mx4")
    y = to_np(lcvq.mx4_gemm(xq, xs, wq, ws, dtype=F32))
    xv, wv = MX.values(x, "mx4"), MX.values(w, "mx4")
    bad = np.zeros((M, N), bool)
    if clean_rows:
        bad[M // 2] = True
    bad[:, 77] = True
    assert np.array_equal(np.isnan(y), bad)
    ref, D = MX.gemm(np.nan_to_num(xv), np.nan_to_num(wv))
    tol = product_tolerance(K, F32, ref, D)
    assert (np.abs(y - ref)[~bad] <= tol[~bad]).all()


@pytest.mark.parametrize("M", [3, 200])
def test_mx4_gemm_extreme_scales(M):
    """Activations near 1e-37 times weights near 1e30, and the other way round."""
    for a, b in ((-120, 100), (100, -120)):
        x, w = np.ldexp(whole_operands(3, M, 256), a), np.ldexp(whole_operands(4, 136, 256), b)
        xq, xs = lcvq.mx_pack(to_dev(x, F32), "mx4")
        wq, ws = lcvq.mx_pack(to_dev(w, F32), "mx4")
        y = lcvq.mx4_gemm(xq, xs, wq, ws, dtype=F32)
        assert np.array_equal(to_np(y), x.astype(np.float64) @ w.T.astype(np.float64))


def test_mx4_gemm_empty_and_repeatable():
    e = torch.empty((0, 32), dtype=torch.uint8, device=dev())
    xq, xs, wq, ws, _, _ = mx4_operands(3, 40, 136, 320)
    assert lcvq.mx4_gemm(xq[:0].contiguous(), xs[:0].contiguous(), wq, ws).shape == (0, 136)
    assert e.shape[0] == 0
    k0 = torch.empty((4, 0), dtype=torch.uint8, device=dev())
    n0 = torch.empty((8, 0), dtype=torch.uint8, device=dev())
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    assert not lcvq.mx4_gemm(k0, none, n0, none, dtype=F32).any()
    a = lcvq.mx4_gemm(xq, xs, wq, ws, dtype=F32)
    assert torch.equal(a, lcvq.mx4_gemm(xq, xs, wq, ws, dtype=F32))


@pytest.mark.parametrize("M", [1, 16, 130])
def test_mx4_linear_replays_in_a_graph_and_on_another_stream(M):
    K, N = 1088, 520
    x = to_dev(matrix(1, M, K, BF16), BF16)
    wq, ws = lcvq.mx_pack(to_dev(0.02 * matrix(2, N, K, F32), F32), "mx4")
    work = lcvq.new_workspace(lcvq.workspace_size(lcvq.OP_MX4_GEMM, BF16, M, N, K, 8))

    def linear():
        return lcvq.mx4_gemm(*lcvq.mx_pack(x, "mx4"), wq, ws, workspace=work)
    first = linear()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = linear()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = linear()
    x.copy_(to_dev(matrix(9, M, K, BF16), BF16))
    for _ in range(3):
        graph.replay()
    assert torch.equal(y, linear())
    assert not torch.equal(y, first)
    assert lcvq.check_device_error(work) == 0


def test_calls_on_a_given_stream():
    """A `stream` argument takes the whole call there, its allocations too; a stream
    that is kept busy shows that nothing ran ahead of it."""
    M, K, N, d = 130, 512, 264, 8
    Wp, A, B, x, dy = layer(2, M, K, N, d, BF16)
    packed, mask = lcvq.assign_pack(to_dev(Wp, F32), d)
    At, Bt, dY = to_dev(A, F32), to_dev(B, F32), to_dev(dy, BF16)
    X, late = to_dev(np.zeros_like(x), BF16), to_dev(x, BF16)
    wq, ws = lcvq.mx_pack(to_dev(matrix(3, 72, K, F32), F32), "mx4")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        X.copy_(late)
    q = lcvq.mx_pack(X, "mx4", stream=side)
    y4 = lcvq.mx4_gemm(*q, wq, ws, stream=side)
    Y, kept = lcvq.gemm_ckpt(X, packed, K, At, Bt, d, stream=side)
    g = lcvq.gemm_backward_ckpt(kept, dY, packed, mask, K, At, Bt, d, stream=side)
    v = lcvq.mx_decode(*kept, K, "mx8", stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y4, lcvq.mx4_gemm(*lcvq.mx_pack(late, "mx4"), wq, ws))
    Y1, kept1 = lcvq.gemm_ckpt(late, packed, K, At, Bt, d)
    g1 = lcvq.gemm_backward_ckpt(kept1, dY, packed, mask, K, At, Bt, d)
    assert torch.equal(Y, Y1) and all(torch.equal(g[k], g1[k]) for k in g1)
    assert torch.equal(v, lcvq.mx_decode(*kept1, K, "mx8"))


def test_two_products_at_once():
    """Calls on two streams, each with its own workspace, few and many tokens."""
    work = [mx4_operands(40 + i, M, 1544, 2048)[:4] for i, M in enumerate((700, 16, 100, 300))]
    want = [lcvq.mx4_gemm(*w) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    got = [[lcvq.mx4_gemm(*w, stream=s) for w, s in zip(work, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, z) for ys in got for y, z in zip(ys, want))


# ---------------------------------------------------------------- X kept in 8 bits
def layer(seed, M, K, N, d, dtype):
    w = synth.workload(4, M=M, d_in=K, d_out=N) if d == 8 else None
    g = rng(seed)
    Wp = (w["Wp"] if w else 1.5 + g.standard_normal((N, K))).astype(np.float32)
    A = (np.diag(0.02 * np.abs(1 + 0.2 * g.standard_normal(d))) + 0.002 * g.standard_normal((d, d))).astype(np.float32)
    B = (-1.5 * A.sum(1)).astype(np.float32)
    X = matrix(seed + 1, M, K, dtype)
    dY = (0.1 * g.standard_normal((M, N))).astype(np.float32)
    return Wp, A, B, X, bf16_np(dY) if dtype == BF16 else dY


CKPT = [(1, 64, 8, 8, BF16), (16, 512, 512, 4, F32), (3, 192, 136, 1, BF16), (16, 512, 512, 8, BF16),
        (33, 448, 200, 2, BF16), (77, 192, 72, 2, F32), (130, 1088, 520, 4, BF16), (333, 1088, 520, 8, BF16),
        (700, 576, 264, 1, BF16), (64, 320, 264, 8, F32), (40, 4160, 72, 8, BF16), (330, 8320, 280, 4, BF16),
        (130, 2112, 264, 2, BF16)]


@pytest.mark.parametrize("M,K,N,d,dtype", CKPT)
def test_forward_keeps_x(M, K, N, d, dtype):
    Wp, A, B, x, _ = layer(M, M, K, N, d, dtype)
    packed, _ = lcvq.assign_pack(to_dev(Wp, F32), d)
    X, At, Bt = to_dev(x, dtype), to_dev(A, F32), to_dev(B, F32)
    q, qbuf = guarded((M, K), torch.uint8)
    s, sbuf = guarded((lcvq.mx_scale_bytes(M, K),), torch.uint8)
    out, obuf = guarded((M, N), dtype)
    lcvq.gemm_ckpt(X, packed, K, At, Bt, d, out=out, kept=(q, s))
    assert guard_intact(q, qbuf) and guard_intact(s, sbuf) and guard_intact(out, obuf)
    if dtype == F32 or M <= 32:
        assert torch.equal(out, lcvq.gemm(X, packed, K, At, Bt, d))
    else:
        # X' and Y are rounded to bf16 (2^-9 of each), the codes are within 3/2 of
        # their mean; fp32 sums of terms up to 67 |X'|, truncated: 2^-23 per 16
        z, _ = O.assign(Wp)
        y, _ = O.forward(x, z, A, B)
        xp = np.abs(x.reshape(M, K // d, d).astype(np.float64) @ A.astype(np.float64)).sum((1, 2))
        tol = (1.5 * 2.0 ** -9 + 67 * (K / 16 + 8) * 2.0 ** -23) * xp[:, None] + 2.0 ** -8 * np.abs(y)
        assert (np.abs(to_np(out) - y) <= tol).all()
    want, byte = MX.pack(x, "mx8")
    assert np.array_equal(q.cpu().numpy(), want)
    assert np.array_equal(MX.untile_scales(s.cpu().numpy(), M, K), byte)


def test_forward_keeps_x_one_workspace_for_all_batches():
    """A workspace of exactly the size for the largest batch, its scratch full of
    NaN bytes, gives every smaller batch (other splits of K) the bits of a fresh one."""
    Wp, A, B, x, _ = layer(5, 400, 8320, 280, 4, BF16)
    packed, _ = lcvq.assign_pack(to_dev(Wp, F32), 4)
    X, At, Bt = to_dev(x, BF16), to_dev(A, F32), to_dev(B, F32)
    n = lcvq.workspace_size(lcvq.OP_GEMM_CKPT, BF16, 400, 280, 8320, 4)
    ws, buf = guarded((n,), torch.uint8)
    ws[:256] = 0
    ws[256:] = 0xFF
    for M in (400, 40, 256, 130, 33, 5):
        Y, _ = lcvq.gemm_ckpt(X[:M], packed, 8320, At, Bt, 4, workspace=ws)
        want, _ = lcvq.gemm_ckpt(X[:M], packed, 8320, At, Bt, 4)
        assert torch.equal(Y, want)
    assert guard_intact(ws, buf)
    assert lcvq.check_device_error(ws) == 0


def grad_tolerance(dtype, M, terms):
    """fp32 sums: dWp's over M tokens (16 of them per tensor-core step, truncated:
    2^-23 each) and the d products with A; dA's and dB's also over the matrix,
    `terms` fp32 additions per thread before the fp64 join.  All relative to the
    sum of magnitudes.  fp32 activations take one rounding (2^-24) per token."""
    steps = M / 16 if dtype == BF16 else M / 2
    return (steps + 24 + terms) * 2.0 ** -23


@pytest.mark.parametrize("M,K,N,d,dtype", CKPT)
def test_backward_from_kept_x(M, K, N, d, dtype):
    Wp, A, B, x, dy = layer(M, M, K, N, d, dtype)
    packed, mask = lcvq.assign_pack(to_dev(Wp, F32), d)
    At, Bt = to_dev(A, F32), to_dev(B, F32)
    kept = lcvq.mx_pack(to_dev(x, dtype), "mx8")
    work = lcvq.new_workspace(lcvq.workspace_size(lcvq.OP_GEMM_BACKWARD_CKPT, dtype, M, N, K, d))
    outs, bufs = {}, {}
    for k, shape, dt in (("dX", (M, K), dtype), ("dA", (d, d), F32), ("dB", (d,), F32), ("dWp", (N, K), F32)):
        outs[k], bufs[k] = guarded(shape, dt)
    g = lcvq.gemm_backward_ckpt(kept, to_dev(dy, dtype), packed, mask, K, At, Bt, d, workspace=work, outs=outs)
    z, m = O.assign(Wp)
    ref = O.backward(MX.values(x, "mx8"), dy, z, m, A, B)
    for k in outs:
        assert guard_intact(outs[k], bufs[k]), k
    tol = grad_tolerance(dtype, M, 0)
    assert O.rel_err(to_np(g["dWp"]), ref["dWp"], ref["D_dWp"]) <= tol
    tol = grad_tolerance(dtype, M, 512)
    for k in ("dA", "dB"):
        assert O.rel_err(to_np(g[k]), ref[k], ref["D_" + k]) <= tol, k
    # dX is the plain backward's: it does not depend on X
    plain = lcvq.gemm_backward(to_dev(x, dtype), to_dev(dy, dtype), packed, mask, K, At, Bt, d)
    assert torch.equal(g["dX"], plain["dX"])
    assert lcvq.check_device_error(work) == 0
    # parts that are not wanted, and the same bits again
    part = lcvq.gemm_backward_ckpt(kept, to_dev(dy, dtype), packed, None, K, At, Bt, d, want_dx=False,
                                   want_dwp=False, workspace=work)
    assert part["dX"] is None and part["dWp"] is None
    assert torch.equal(part["dA"], g["dA"]) and torch.equal(part["dB"], g["dB"])


@pytest.mark.parametrize("d", [1, 2, 4, 8])
@pytest.mark.parametrize("K,N", [(512, 512), (192, 72), (1088, 136)])
def test_fp32_rows_do_not_depend_on_their_number(K, N, d):
    """Few fp32 tokens take smaller tiles; the sums are the same ones in the same
    order, so every row has the bits it has among thousands."""
    M = 5000
    Wp, A, B, x, dy = layer(17, M, K, N, d, F32)
    packed, mask = lcvq.assign_pack(to_dev(Wp, F32), d)
    At, Bt, X, dY = to_dev(A, F32), to_dev(B, F32), to_dev(x, F32), to_dev(dy, F32)
    Y = lcvq.gemm(X, packed, K, At, Bt, d)
    dX = lcvq.gemm_backward(X, dY, packed, mask, K, At, Bt, d)["dX"]
    for m in (1, 16, 37, 190, 330):
        assert torch.equal(lcvq.gemm(X[:m].contiguous(), packed, K, At, Bt, d), Y[:m])
        g = lcvq.gemm_backward(X[:m].contiguous(), dY[:m].contiguous(), packed, mask, K, At, Bt, d)
        assert torch.equal(g["dX"], dX[:m])


def test_gradient_by_differences():
    """L = sum dY * Y is linear in A and B: (L(A + h E) - L(A - h E)) / 2 h is dA,
    with the kept values as X."""
    M, K, N, d = 40, 128, 24, 4
    Wp, A, B, x, dy = layer(11, M, K, N, d, F32)
    packed, mask = lcvq.assign_pack(to_dev(Wp, F32), d)
    kept = lcvq.mx_pack(to_dev(x, F32), "mx8")
    g = lcvq.gemm_backward_ckpt(kept, to_dev(dy, F32), packed, mask, K, to_dev(A, F32), to_dev(B, F32), d)
    xv = to_np(lcvq.mx_decode(*kept, K, "mx8", dtype=F32))
    z, _ = O.assign(Wp)

    def loss(A, B):
        return float((dy * O.forward(xv, z, A, B)[0]).sum())
    A64, B64, h = A.astype(np.float64), B.astype(np.float64), 2.0 ** -6
    D = np.abs(dy).sum() * np.abs(xv).max() * 3
    for i in range(d):
        for j in range(d):
            E = np.zeros((d, d)); E[i, j] = h
            diff = (loss(A64 + E, B64) - loss(A64 - E, B64)) / (2 * h)
            assert abs(diff - float(g["dA"][i, j])) <= 1e-5 * D
        e = np.zeros(d); e[i] = h
        diff = (loss(A64, B64 + e) - loss(A64, B64 - e)) / (2 * h)
        assert abs(diff - float(g["dB"][i])) <= 1e-5 * D


def test_kept_x_with_a_non_finite_block():
    """A block with an infinity makes the gradients of its 32 channels NaN, and no
    other channel's dWp."""
    M, K, N, d = 70, 192, 136, 8
    Wp, A, B, x, dy = layer(5, M, K, N, d, BF16)
    x[7, 70] = np.inf
    packed, mask = lcvq.assign_pack(to_dev(Wp, F32), d)
    kept = lcvq.mx_pack(to_dev(x, BF16), "mx8")
    g = lcvq.gemm_backward_ckpt(kept, to_dev(dy, BF16), packed, mask, K, to_dev(A, F32), to_dev(B, F32), d)
    bad = np.isnan(to_np(g["dWp"]))
    inside = O.assign(Wp)[1].astype(bool)
    assert np.array_equal(bad[:, 64:96], inside[:, 64:96])
    assert not bad[:, :64].any() and not bad[:, 96:].any()


@pytest.mark.parametrize("M", [16, 300])
def test_a_training_step_in_a_graph(M):
    """Forward with X kept, a frozen 4-bit layer behind it, and the backward, as
    one captured step; replayed on other inputs it gives their results."""
    K, N, d = 512, 264, 8
    Wp, A, B, x, dy = layer(2, M, K, N, d, BF16)
    packed, mask = lcvq.assign_pack(to_dev(Wp, F32), d)
    At, Bt, X, dY = to_dev(A, F32), to_dev(B, F32), to_dev(x, BF16), to_dev(dy, BF16)
    hq, hs = lcvq.mx_pack(to_dev(matrix(3, 72, 256, F32), F32), "mx4")
    ws = [lcvq.new_workspace(lcvq.workspace_size(op, BF16, M, N, K, d))
          for op in (lcvq.OP_GEMM_CKPT, lcvq.OP_GEMM_BACKWARD_CKPT, lcvq.OP_MX4_GEMM)]

    def step():
        Y, kept = lcvq.gemm_ckpt(X, packed, K, At, Bt, d, workspace=ws[0])
        head = lcvq.mx4_gemm(*lcvq.mx_pack(Y[:, :256], "mx4"), hq, hs, workspace=ws[2])
        g = lcvq.gemm_backward_ckpt(kept, dY, packed, mask, K, At, Bt, d, workspace=ws[1])
        return [Y, head, g["dX"], g["dA"], g["dB"], g["dWp"]]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    X.copy_(to_dev(matrix(31, M, K, BF16), BF16))
    for _ in range(3):
        graph.replay()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
    for w in ws:
        assert lcvq.check_device_error(w) == 0


# ---------------------------------------------------------------- bounded waits
@pytest.mark.parametrize("M,N,K,sites", [(300, 520, 4096, range(31, 38)), (700, 2000, 256, range(31, 38)),
                                         (16, 520, 4096, range(41, 44)), (5, 264, 256, range(41, 44)),
                                         (100, 2000, 2048, range(41, 44))])
def test_mx4_gemm_wait_gives_up_and_recovers(M, N, K, sites):
    """With a wait limit far below one copy's round trip the kernel winds down and
    says so; the next call on the same workspace is right."""
    x, w = whole_operands(1, M, K), whole_operands(2, N, K)
    xq, xs = lcvq.mx_pack(to_dev(x, F32), "mx4")
    wq, ws = lcvq.mx_pack(to_dev(w, F32), "mx4")
    work = lcvq.new_workspace(lcvq.workspace_size(lcvq.OP_MX4_GEMM, F32, M, N, K, 8))
    lcvq.set_wait_limit(work, 64)
    for _ in range(3):
        lcvq.mx4_gemm(xq, xs, wq, ws, dtype=F32, workspace=work)
    torch.cuda.synchronize()
    err, site = work[:8].view(torch.int32).cpu().tolist()
    assert err == 6 and site in sites, (err, site)
    assert lcvq.check_device_error(work) == 6
    lcvq.set_wait_limit(work, 0)
    y = lcvq.mx4_gemm(xq, xs, wq, ws, dtype=F32, workspace=work)
    assert lcvq.check_device_error(work) == 0
    assert np.array_equal(to_np(y), x.astype(np.float64) @ w.T.astype(np.float64))


def test_gemm_ckpt_wait_gives_up_and_recovers():
    M, K, N, d = 200, 512, 520, 8
    Wp, A, B, x, _ = layer(1, M, K, N, d, BF16)
    packed, _ = lcvq.assign_pack(to_dev(Wp, F32), d)
    X, At, Bt = to_dev(x, BF16), to_dev(A, F32), to_dev(B, F32)
    want, _ = lcvq.gemm_ckpt(X, packed, K, At, Bt, d)
    work = lcvq.new_workspace(lcvq.workspace_size(lcvq.OP_GEMM_CKPT, BF16, M, N, K, d))
    lcvq.set_wait_limit(work, 64)
    lcvq.gemm_ckpt(X, packed, K, At, Bt, d, workspace=work)
    assert lcvq.check_device_error(work) == 6
    lcvq.set_wait_limit(work, 0)
    y, _ = lcvq.gemm_ckpt(X, packed, K, At, Bt, d, workspace=work)
    assert lcvq.check_device_error(work) == 0 and torch.equal(y, want)
