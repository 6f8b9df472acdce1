"""Block-scaled formats on the CPU: the oracle against the formats' definition,
and the calls' refusals (all before any device call)."""

import numpy as np
import pytest
import torch

from bit_weight_only_lcvq_b200 import lcvq
from oracle import mx_oracle as X


def test_grid_and_ties_mx4():
    # one block with max 6 (scale 1): every midpoint goes to the even code
    x = np.zeros((1, 32))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -2.5]
    v = X.values(x, "mx4")[0]
    assert v[:9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -2]


def test_ties_mx8():
    x = np.zeros((1, 32))
    x[0, :5] = [127, 0.5, 1.5, -2.5, 126.5]
    assert X.values(x, "mx8")[0, :5].tolist() == [127, 0, 2, -2, 126]


@pytest.mark.parametrize("fmt,top", [("mx4", 6.0), ("mx8", 127.0)])
def test_scale_is_the_smallest_that_fits(fmt, top):
    g = np.random.Generator(np.random.PCG64(3))
    x = g.standard_normal((64, 128)) * 2.0 ** g.integers(-60, 60, (64, 1))
    byte = X.quantise(x, fmt)[2]
    most = np.abs(x.reshape(64, 4, 32)).max(-1)
    s = 2.0 ** (byte.astype(float) - 127)
    assert (most <= top * s).all() and (most > top * s / 2).all()
    # within half a step of the grid: 1 for mx8, up to 1 (between 4 and 6) for mx4
    step = 0.5 if fmt == "mx8" else 1.0
    assert (np.abs(X.values(x, fmt) - x).reshape(64, 4, 32) <= step * s[..., None]).all()
    # values that the format holds stay
    v = X.values(x, fmt)
    assert np.array_equal(X.values(v, fmt), v)


@pytest.mark.parametrize("fmt", ["mx4", "mx8"])
def test_bytes_round_trip(fmt):
    g = np.random.Generator(np.random.PCG64(4))
    x = g.standard_normal((131, 160)).astype(np.float32)
    q, byte = X.pack(x, fmt)
    assert np.array_equal(X.unpack(q, byte, fmt), X.values(x, fmt))
    assert np.array_equal(X.untile_scales(X.tile_scales(byte), 131, 160), byte)


def test_stored_order_by_hand():
    x = np.zeros((1, 32))
    x[0, :4] = [1, -2, 3, 6]
    q, byte = X.pack(x, "mx4")
    assert byte[0, 0] == 127 and q[0, 0] == (2 | (8 + 4) << 4) and q[0, 1] == (5 | 7 << 4)
    x[0, 0] = 127
    q, byte = X.pack(x, "mx8")
    assert byte[0, 0] == 127 and q[0, :4].tolist() == [127, 3, 128 + 2, 6]
    t = X.tile_scales(np.arange(200 * 5, dtype=np.int64).reshape(200, 5).astype(np.uint8))
    assert len(t) == 2 * 2 * 512
    r, b = 170, 4  # second tile of rows, second of columns
    assert t[(1 * 2 + 1) * 512 + (42 % 32) * 16 + 1 * 4 + 0] == (r * 5 + b) % 256


def test_non_finite_and_extreme_blocks():
    x = np.zeros((4, 32), np.float32)
    x[0, 3], x[1, 3] = np.nan, -np.inf
    x[2, 0] = np.finfo(np.float32).max
    x[3, 0] = 1e-45
    for fmt in ("mx4", "mx8"):
        v = X.values(x, fmt)
        assert np.isnan(v[:2]).all()
        assert np.isfinite(v[2:]).all() and v[2, 0] < 2.0 ** 128
        assert X.quantise(x, fmt)[2][:, 0].tolist()[:2] == [255, 255]
        assert X.quantise(x, fmt)[2][3, 0] == 0


def test_scale_bytes():
    assert lcvq.mx_scale_bytes(1, 32) == 512
    assert lcvq.mx_scale_bytes(129, 160) == 4 * 512
    assert lcvq.mx_scale_bytes(0, 160) == 0
    assert lcvq.mx_scale_bytes(8, 33) == 0 and lcvq.mx_scale_bytes(-1, 32) == 0


def test_pack_and_decode_refusals():
    L = lcvq.lib()
    pack = L.lcvq_mx_pack
    assert pack(16, 1, 4, 48, 48, 0, 16, 16, None) == 1        # cols % 32
    assert pack(16, 1, -1, 64, 64, 0, 16, 16, None) == 1
    assert pack(16, 1, 4, 64, 32, 0, 16, 16, None) == 1        # ld < cols
    assert pack(16, 1, 4, 64, 64, 2, 16, 16, None) == 1        # format
    assert pack(16, 3, 4, 64, 64, 0, 16, 16, None) == 1        # dtype
    assert pack(None, 1, 4, 64, 64, 0, 16, 16, None) == 1
    assert pack(16, 1, 4, 64, 64, 0, None, 16, None) == 1
    assert pack(16, 1, 4, 64, 64, 0, 16, None, None) == 1
    assert pack(8, 1, 4, 64, 64, 0, 16, 16, None) == 3
    assert pack(16, 1, 4, 64, 68, 0, 16, 16, None) == 3        # rows not 16-byte aligned (bf16)
    assert pack(16, 0, 4, 64, 66, 0, 16, 16, None) == 3        # (fp32)
    assert pack(16, 1, 1 << 30, 1 << 14, 1 << 14, 0, 16, 16, None) == 1  # too many pieces
    assert pack(None, 1, 0, 64, 64, 0, None, None, None) == 0  # empty
    assert pack(None, 1, 4, 0, 0, 0, None, None, None) == 0
    dec = L.lcvq_mx_decode
    assert dec(16, 16, 4, 40, 1, 16, 1, None) == 1
    assert dec(16, 16, 4, 64, 5, 16, 1, None) == 1
    assert dec(16, 16, 4, 64, 1, 16, 2, None) == 1
    assert dec(None, 16, 4, 64, 1, 16, 1, None) == 1
    assert dec(16, 16, 4, 64, 1, 24, 1, None) == 3
    assert dec(None, None, 0, 64, 1, None, 1, None) == 0


def test_mx4_gemm_refusals():
    L = lcvq.lib()
    need = L.lcvq_workspace_size(lcvq.OP_MX4_GEMM, 1, 4, 64, 64, 8)
    assert need >= 256

    def call(M=4, n=64, k=64, x=256, sx=256, w=256, sw=256, y=256, dt=1, ws=256, nb=need):
        return L.lcvq_mx4_gemm(x, sx, M, w, sw, n, k, y, dt, ws, nb, None)
    assert call(k=96) == 1 and call(n=12) == 1 and call(M=-1) == 1 and call(dt=4) == 1
    for name in ("x", "sx", "w", "sw", "y", "ws"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: 264}) == 3, name
    assert call(nb=need - 1) == 4
    assert call(M=0) == 0 and call(n=0) == 0


@pytest.mark.parametrize("d_out,d_in", [(72, 4160), (264, 2112), (11008, 4096), (4096, 11008), (520, 1088)])
def test_ckpt_workspace_serves_smaller_batches(d_out, d_in):
    # what the largest batch asks for is enough for every smaller one
    sizes = [lcvq.workspace_size(lcvq.OP_GEMM_CKPT, torch.bfloat16, M, d_out, d_in, 8)
             for M in (0, 1, 16, 32, 33, 40, 127, 128, 129, 256, 300, 640, 1024, 2048, 8192, 20000)]
    assert sizes == sorted(sizes)


def test_ckpt_refusals():
    L = lcvq.lib()
    need = L.lcvq_workspace_size(lcvq.OP_GEMM_CKPT, 1, 4, 64, 64, 8)

    def fwd(dt=1, M=4, n=64, k=64, d=8, x=256, p=256, A=256, B=256, y=256, x8=256, s8=256, ws=256, nb=need):
        return L.lcvq_gemm_ckpt(x, dt, M, p, n, k, d, A, B, y, x8, s8, ws, nb, None)
    assert fwd(k=96) == 1 and fwd(n=12) == 1 and fwd(d=3) == 1 and fwd(dt=2) == 1
    for name in ("x", "p", "A", "B", "y", "x8", "s8", "ws"):
        assert fwd(**{name: None}) == 1, name
        assert fwd(**{name: 264}) == 3, name
    assert fwd(nb=need - 1) == 4
    assert fwd(M=0) == 0
    need = L.lcvq_workspace_size(lcvq.OP_GEMM_BACKWARD_CKPT, 1, 4, 64, 64, 8)
    assert need >= L.lcvq_workspace_size(lcvq.OP_GEMM_BACKWARD, 1, 4, 64, 64, 8)

    def bwd(dt=1, M=4, n=64, k=64, d=8, x8=256, s8=256, dy=256, p=256, mask=256, A=256, B=256, dx=256,
            dA=256, dB=256, dw=256, ws=256, nb=need):
        return L.lcvq_gemm_backward_ckpt(x8, s8, dy, dt, M, p, mask, n, k, d, A, B, dx, dA, dB, dw, ws,
                                         nb, None)
    assert bwd(k=96) == 1 and bwd(n=12) == 1 and bwd(d=5) == 1 and bwd(dt=2) == 1
    for name in ("x8", "s8", "dy", "p", "mask", "A", "B", "dA", "dB", "ws"):
        assert bwd(**{name: None}) == 1, name
    for name in ("x8", "s8", "dy", "p", "mask", "A", "B", "dx", "dA", "dB", "dw", "ws"):
        assert bwd(**{name: 264}) == 3, name
    assert bwd(nb=need - 1) == 4


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        lcvq.mx_pack(x, "mx4")                                   # host memory
    with pytest.raises(ValueError):
        lcvq.mx_pack(torch.zeros(4, 64, dtype=torch.float16), "mx4")
    with pytest.raises(ValueError):
        lcvq.mx_pack(torch.zeros(4), "mx4")
    q = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        lcvq.mx_decode(q, q, 64, "mx4")
    with pytest.raises(ValueError):
        lcvq.mx4_gemm(q, q, q, q)
    with pytest.raises(ValueError):
        lcvq.gemm_ckpt(x, q, 64, x, x, 8)
    with pytest.raises(ValueError):
        lcvq.gemm_backward_ckpt((q, q), x, q, None, 64, x, x, 8)
