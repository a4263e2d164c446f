"""The 8-bit product's CTA-pair kernel where a pair walks over several tiles: every tile width,
both accumulators in turn, the ring of K stages carried from tile to tile, scales and residual
read a tile ahead, rows and columns that end inside a tile, two unequal bands of row tiles. All
outputs, against the product in float64 (elementary torch operations).

The kernel's tiles are 256 rows by 64 to 256 columns, of the width whose waves over 74 pairs of SMs
take least; with one column tile that is the narrowest that holds N, so M > 3 * 74 * 256 rows give
each pair three tiles at least. K of 1168 is nine stages and a part, more than the ring holds, and
57 to 74 MB of activations, past what one band takes (40 MB).

U = 2^-24 is half a float32 step."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests.test_gpu_w8a8 import BF, E4, F32, TYPES, U, bq, draw, half_step, inside, operands, outer_is  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def act64(z, kind):
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def product64(a, sa, w, sw, bias):
    """(z, its error): the bound of test_gpu_w8a8.product_bound, on the GPU in float64."""
    A, W, s = a.double(), w.double(), sa.double()[:, None] * sw.double()
    b = 0.0 if bias is None else bias.double()
    z, mag = (A @ W.t()) * s + b, (A.abs() @ W.abs().t()) * s + (0.0 if bias is None else b.abs())
    return z, mag * ((a.shape[1] / 32 + 16) * 2.0 ** -22 + 4 * U)


def act_bound64(z, ez, kind):
    """test_gpu_w8a8.act_bound: slopes below 1.13, the evaluation 64 U of the value."""
    if kind is None:
        return z, ez
    v = act64(z, kind)
    return v, 1.13 * ez + 64 * U * v.abs() + 1e-15


def agrees(y, want, e):
    err, e = (y.double() - want).abs(), e * 1.01 + (half_step(y.dtype) + 2 * U) * (want.abs() + e)
    bad = ~(err <= e)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), bad.nonzero()[-4:].tolist())


# M, N, K, bias, act, residual; the width that N leaves: 64, 96, 128, 160, 192, 224, 256 columns
ONE_COLUMN_TILE = [(57_100, 48, 1168, True, None, True), (58_000, 80, 1168, True, "gelu", True),
                   (63_489, 112, 1040, False, None, True), (57_000, 144, 1168, True, "silu", True),
                   (59_001, 176, 1168, True, None, False), (60_000, 208, 1168, False, "gelu", True),
                   (57_345, 240, 1296, True, None, True)]
# several column tiles: 192, 224 and 256 wide, fewer stages than the ring holds and more, one band and two
MANY = [(1100, 7696, 272, True, "gelu", True), (2601, 3856, 1168, True, None, True),
        (3000, 4112, 1040, False, "silu", False), (2700, 4112, 16400, True, None, True)]


@TYPES
@pytest.mark.parametrize("M,N,K,bias,act,residual", ONE_COLUMN_TILE + MANY)
def test_linear_over_many_tiles(bq, M, N, K, bias, act, residual, dtype):  # noqa: F811
    a, sa, w, sw = operands(bq, M, N, K, M + N)
    b = draw(5, N, dtype=BF, std=0.1) if bias else None
    r = draw(6, M, N, dtype=dtype) if residual else None
    z, ez = product64(a, sa, w, sw, b)
    want, e = act_bound64(z, ez, act)
    if residual:
        want = want + r.double()
        e = e + U * want.abs()
    y = bq.w8a8_linear(a, sa, w, sw, b, residual=r, activation=act, out_dtype=dtype)
    agrees(y, want, e)
    # inside wider rows, whose other columns stay; the residual strided, and in place
    yv, whole = inside(torch.zeros_like(y), 16, 5.0)
    if residual:
        yv.copy_(r)
    bq.w8a8_linear(a, sa, w, sw, b, residual=yv if residual else None, activation=act, out_dtype=dtype, Y=yv)
    assert torch.equal(yv, y) and outer_is(whole, 16, 5.0)
    assert bq.svdq_check_device_status() == 0


# M, F, K, bias, act: 64, 128, 192, 256 accumulator columns, half of them gate and half up
@TYPES
@pytest.mark.parametrize("M,F,K,bias,act", [
    (57_100, 32, 1168, True, "silu"), (58_001, 48, 1168, False, "gelu"), (57_345, 80, 1296, True, "silu"),
    (60_000, 112, 1168, False, "silu"), (777, 5136, 1040, True, "gelu"), (513, 7696, 272, False, "silu"),
    (2700, 2320, 16400, True, "silu")])
def test_gated_linear_over_many_tiles(bq, M, F, K, bias, act, dtype):  # noqa: F811
    a, sa, w, sw = operands(bq, M, 2 * F, K, M + F)
    b = draw(5, 2 * F, dtype=BF, std=0.1) if bias else None
    z, ez = product64(a, sa, w, sw, b)
    gate, eg = act_bound64(z[:, :F], ez[:, :F], act)
    up, eu = z[:, F:], ez[:, F:]
    want, e = gate * up, gate.abs() * eu + up.abs() * eg + eg * eu
    y = bq.w8a8_gated_linear(a, sa, w, sw, b, activation=act, out_dtype=dtype)
    agrees(y, want, e)
    yv, whole = inside(torch.zeros_like(y), 8, 5.0)
    bq.w8a8_gated_linear(a, sa, w, sw, b, activation=act, out_dtype=dtype, Y=yv)
    assert torch.equal(yv, y) and outer_is(whole, 8, 5.0)
    assert bq.svdq_check_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(200, 4112, 80), (384, 2064, 80), (600, 4112, 208), (57_100, 144, 1168),
                                   (2601, 3856, 1168), (3000, 4112, 656)])
def test_many_tiles_are_exact_on_whole_numbers(bq, M, N, K):  # noqa: F811
    """Small whole numbers and scales of powers of two: every sum is exact in float32, in any
    order. The first three are one tile to a pair at most, of 64 and 192 columns."""
    g = torch.Generator(device="cuda").manual_seed(M)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda").float()

    a, w = whole(-8, 9, M, K), whole(-8, 9, N, K)
    sa, sw = 2.0 ** whole(-3, 4, M), 2.0 ** whole(-3, 4, N)
    b, r = whole(-9, 10, N).to(BF), whole(-9, 10, M, N)
    y = bq.w8a8_linear(a.to(E4), sa, w.to(E4), sw, b, residual=r, out_dtype=F32)
    want = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double() + b.double() + r.double()
    assert torch.equal(y.double(), want)
