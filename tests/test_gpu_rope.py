"""Rotary positions on the GPU against the float64 oracle: both pair layouts, part of the head,
several position axes, far and negative positions, strided and in-place heads, and the tables
in both orders, the fused QKV projection's among them.

Bounds: an angle is off by 2^-51 of itself (both sides' products) and its cosine by 2^-22 + 2 U: the
rest of a quarter turn in float32 (2.5 U of it), the power series (2 U) and the scale (U), each of a
value below 1; a turned value adds three float32 roundings and the output type's."""

import math

import numpy as np
import pytest

from oracle import w8a8 as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_quantized_diffusion_b200 as bq
    return bq


def f64(t):
    return t.detach().double().cpu().numpy()


def positions(seed, M, axes, far, dtype=torch.int32, negative=False):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-far if negative else 0, far, (M, axes), generator=g).to(dtype).cuda()


def tables(pos, freq, axis, scale):
    p, f = pos.cpu().numpy(), f64(freq)
    a = None if axis is None else axis.cpu().numpy()
    c, s = O.cos_sin(p, f, a, scale)
    angle = np.abs(p[:, np.zeros(len(f), int) if a is None else a] * f)
    return c, s, abs(scale) * (2.0 ** -22 + 2 * U + angle * 2.0 ** -51)


def check(y, x, pos, freq, axis, scale, interleaved):
    c, s, e = tables(pos, freq, axis, scale)
    want = O.rope(f64(x), c, s, interleaved)
    both = O.rope(np.abs(f64(x)), np.abs(c), -np.abs(s), interleaved)   # |a c| + |b s| in the first of a pair
    P = c.shape[1]
    xa = np.abs(f64(x))
    mag = np.array(xa)
    first, second = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    mag[..., first] = mag[..., second] = xa[..., first] + xa[..., second]
    bound = np.zeros_like(mag)
    bound[..., first] = mag[..., first] * (e[:, None] + 3 * U * abs(scale))
    bound[..., second] = bound[..., first]
    half = torch.finfo(y.dtype).eps / 2
    assert np.all(np.abs(f64(y) - want) <= bound + half * (np.abs(want) + bound)), both.shape
    assert np.array_equal(f64(y)[..., 2 * P:], f64(x)[..., 2 * P:])


CASES = [  # M, heads, D, rotary columns, axes, far
    (1, 1, 2, 2, 1, 10), (1, 60, 128, 128, 1, 1000000), (3, 2, 64, 64, 1, 5000), (5, 7, 80, 32, 2, 1000),
    (2, 3, 96, 20, 1, 300), (17, 5, 256, 256, 3, 128), (64, 4, 128, 64, 1, 2 ** 31 - 1), (9, 2, 34, 6, 3, 50),
    (300, 12, 64, 16, 2, 4096), (4, 1, 1024, 1024, 1, 9999), (33, 24, 32, 32, 1, 131072)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [True, False], ids=["adjacent", "halves"])
@pytest.mark.parametrize("M,H,D,rot,axes,far", CASES)
def test_rope(bq, M, H, D, rot, axes, far, interleaved, dtype):
    from bit_quantized_diffusion_b200.prep import rope_frequencies
    share = [2 * (rot // 2 // axes + (a < rot // 2 % axes)) for a in range(axes)]
    freq, axis, _ = rope_frequencies(tuple(share))
    freq, axis = freq.cuda(), axis.cuda() if axes > 1 else None
    pos = positions(M + D, M, axes, far, torch.int64 if M % 2 else torch.int32, negative=M % 3 == 0)
    scale = 1.0 if H % 2 else 1.25
    g = torch.Generator().manual_seed(1)
    # the heads inside a wider row: Q and K before V
    row = torch.randn(M, H + 2, D, generator=g).to(dtype).cuda()
    x = row[:, :H]
    y = bq.svdq_rope(x, pos, freq, axis=axis, scale=scale, interleaved=interleaved)
    check(y, x, pos, freq, axis, scale, interleaved)
    packed = bq.svdq_rope(x.contiguous(), pos, freq, axis=axis, scale=scale, interleaved=interleaved)
    assert torch.equal(packed, y)
    # heads outside, rows inside
    outer = torch.empty(H, M, D, dtype=dtype, device="cuda").transpose(0, 1)
    bq.svdq_rope(x, pos, freq, axis=axis, scale=scale, interleaved=interleaved, Y=outer)
    assert torch.equal(outer, y)
    # in place: the other heads of the row stay
    rest = row[:, H:].clone()
    assert bq.svdq_rope(x, pos, freq, axis=axis, scale=scale, interleaved=interleaved, Y=x) is x
    assert torch.equal(x, y) and torch.equal(row[:, H:], rest)


def test_rope_odd_pairs_and_strides(bq):
    """Pair counts and strides that no wide vector fits."""
    for D, P, pad in ((6, 1, 0), (10, 5, 2), (22, 7, 4), (14, 7, 6)):
        freq = torch.linspace(1.0, 0.01, P, dtype=torch.float64).cuda()
        pos = positions(D, 11, 1, 1000)
        for dtype in (BF, F32):
            for inter in (True, False):
                base = torch.randn(11, 3 * (D + pad) + pad, generator=torch.Generator().manual_seed(P)).to(dtype).cuda()
                x = base.as_strided((11, 3, D), (base.shape[1], D + pad, 1)) if base.shape[1] % 2 == 0 else None
                if x is None:
                    base = base[:, :-1].contiguous()
                    x = base.as_strided((11, 3, D), (base.shape[1], D, 1))
                y = bq.svdq_rope(x, pos[:, 0], freq, interleaved=inter)
                check(y, x, pos, freq, None, 1.0, inter)


def test_rope_keeps_odd_values_in_their_pairs(bq):
    """NaN and infinity stay in their pair; an axis that is not there gives NaN in its pairs alone."""
    x = torch.ones(2, 2, 16, device="cuda")
    x[0, 1, 3] = float("nan")
    x[1, 0, 6] = float("inf")
    pos = torch.tensor([[3, 4], [5, 6]], dtype=torch.int32, device="cuda")
    freq = torch.full((4,), 0.1, dtype=torch.float64, device="cuda")
    axis = torch.tensor([0, 1, 1, 0], dtype=torch.int32, device="cuda")
    y = bq.svdq_rope(x, pos, freq, axis=axis, interleaved=True)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 1, 2:4] = True
    want[1, 0, 6:8] = True
    assert torch.equal(bad, want)
    x = torch.ones(2, 2, 16, device="cuda")
    for wrong in (2, -1):
        axis[2] = wrong
        y = bq.svdq_rope(x, pos, freq, axis=axis, interleaved=True)
        want = torch.zeros_like(bad)
        want[:, :, 4:6] = True
        assert torch.equal(torch.isnan(y), want)
        cos, _ = bq.svdq_rope_table(pos, freq, axis=axis)
        assert torch.equal(torch.isnan(cos), torch.tensor([[False, False, True, False]] * 2, device="cuda"))


@pytest.mark.parametrize("angle_major", [False, True], ids=["rows", "angle-major"])
@pytest.mark.parametrize("M,P,axes,far,dtype", [
    (1, 1, 1, 5, torch.int32), (1, 64, 1, 10 ** 6, torch.int64), (7, 10, 3, 100, torch.int32), (1000, 64, 3, 128, torch.int32),
    (513, 48, 2, 2 ** 31 - 1, torch.int64), (4099, 8, 1, 10 ** 6, torch.int32), (30, 512, 1, 70000, torch.int32)])
def test_tables(bq, M, P, axes, far, dtype, angle_major):
    g = torch.Generator().manual_seed(P)
    freq = torch.cat([torch.ones(1, dtype=torch.float64), torch.rand(P - 1, generator=g, dtype=torch.float64)]).cuda()
    axis = torch.randint(0, axes, (P,), generator=g, dtype=torch.int32).cuda() if axes > 1 else None
    pos = positions(M, M, axes, far, dtype, negative=True)
    cos, sin = bq.svdq_rope_table(pos, freq, axis=axis, scale=0.75, angle_major=angle_major)
    c, s, e = tables(pos, freq, axis, 0.75)
    assert cos.shape == ((P, M) if angle_major else (M, P))
    for got, want in ((cos, c), (sin, s)):
        got = f64(got.t() if angle_major else got)
        assert np.all(np.abs(got - want) <= e)


def test_whole_turns_are_exact_however_far(bq):
    """A quarter turn a position: the fraction is exact up to freq's own rounding, so cosines of
    positions up to 2^40 keep 2^-22 besides 2^-52 of the angle."""
    freq = torch.tensor([math.pi / 2], dtype=torch.float64, device="cuda")
    pos = torch.tensor([0, 1, 2, 3, 4, 2 ** 20, 2 ** 20 + 1, -1, -(2 ** 24) + 3], dtype=torch.int64, device="cuda")
    cos, sin = bq.svdq_rope_table(pos, freq)
    q = pos.cpu().numpy() % 4
    e = 2.0 ** -22 + np.abs(pos.cpu().numpy()) * 2.0 ** -50
    assert np.all(np.abs(f64(cos)[:, 0] - np.array([1, 0, -1, 0])[q]) <= e)
    assert np.all(np.abs(f64(sin)[:, 0] - np.array([0, 1, 0, -1])[q]) <= e)


def test_layer_rotates_and_feeds_the_fused_projection(bq):
    """RotaryEmbedding.forward agrees with its own tables through the fused QKV projection: the plain
    projection's heads turned, against the heads turned in the GEMM's epilogue (no head norm
    there: weight and mean square are applied to both by hand)."""
    from bit_quantized_diffusion_b200.layers import RotaryEmbedding, SvdqQkvNormRope
    M, K, H = 150, 256, 2
    g = torch.Generator().manual_seed(0)
    w = (torch.randn(3 * H * 128, K, generator=g) * 0.05).to(BF).cuda()
    x = torch.randn(M, K, generator=g).to(BF).cuda()
    rot = RotaryEmbedding((16, 56, 56), interleaved=True)
    pos = positions(3, M, 3, 64)
    layer = SvdqQkvNormRope.from_linear(w, None, x.float().abs().amax(0), 16, max_tokens=M)
    plain = layer(x).view(M, 3 * H, 128)
    turned = layer(x, rotary=rot, positions=pos).view(M, 3 * H, 128)
    again = rot(plain[:, : 2 * H], pos)
    # plain holds the normalised heads in bf16 (half a step 2^-8), the fused call rounds once, at the end
    size = plain[:, : 2 * H].float().unflatten(-1, (64, 2)).abs().sum(-1).repeat_interleave(2, -1)
    err = (again.float() - turned[:, : 2 * H].float()).abs()
    assert torch.all(err <= size * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -8))
    assert torch.equal(turned[:, 2 * H:], plain[:, 2 * H:])
    # captured: positions change between replays
    y = torch.empty_like(again)
    rot(plain[:, : 2 * H], pos, y=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rot(plain[:, : 2 * H], pos, y=y)
    pos.add_(5)
    graph.replay()
    assert torch.equal(y, rot(plain[:, : 2 * H], pos)) and not torch.equal(y, again)
    assert bq.svdq_check_device_status() == 0


def test_offsets_beyond_32_bits(bq):
    """Heads whose elements number over 2^32, in place: the last rows agree with a call on them alone."""
    M, H, D = 70_000, 64, 1024
    x = torch.empty(M, H, D, dtype=BF, device="cuda")
    x[-2:] = torch.randn(2, H, D, generator=torch.Generator().manual_seed(0)).to(BF).cuda()
    pos = torch.arange(M, dtype=torch.int64, device="cuda")
    freq = torch.logspace(0, -3, 512, dtype=torch.float64).cuda()
    want = bq.svdq_rope(x[-2:], pos[-2:], freq)
    bq.svdq_rope(x, pos, freq, Y=x)
    assert torch.equal(x[-2:], want)
    del x
    M, P = 8_400_000, 512
    cos, sin = bq.svdq_rope_table(torch.arange(M, dtype=torch.int32, device="cuda"), freq)
    c, s = bq.svdq_rope_table(torch.arange(M - 3, M, dtype=torch.int32, device="cuda"), freq)
    assert torch.equal(cos[-3:], c) and torch.equal(sin[-3:], s)


def test_one_row_of_heads_far_apart(bq):
    """One token of a [heads, length, D] cache: its heads lie further apart than 2^31 / heads."""
    H, L, D = 6, 3_400_000, 128
    cache = torch.empty(H, L, D, dtype=BF, device="cuda")
    cache[:, 1:4].zero_()
    row = cache[:, 2:3].transpose(0, 1)
    x = torch.randn(1, H, D, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    assert row.stride(1) * H > 2 ** 31
    pos, freq = torch.tensor([2], dtype=torch.int64, device="cuda"), torch.logspace(0, -3, 64, dtype=torch.float64).cuda()
    want = bq.svdq_rope(x, pos, freq)
    bq.svdq_rope(x, pos, freq, Y=row)
    assert torch.equal(row, want) and not cache[:, 1].any() and not cache[:, 3].any()
    row.copy_(x)
    bq.svdq_rope(row, pos, freq, Y=row)
    assert torch.equal(row, want)


def test_frequencies_that_are_not_finite(bq):
    """NaN in their own pairs, the other pairs as without them: the rotation and both tables."""
    freq = torch.logspace(0, -3, 16, dtype=torch.float64)
    odd = freq.clone()
    odd[2], odd[7], odd[13] = math.inf, math.nan, -math.inf
    lost = torch.zeros(16, dtype=torch.bool)
    lost[[2, 7, 13]] = True
    freq, odd, lost = freq.cuda(), odd.cuda(), lost.cuda()
    pos = torch.tensor([0, 5, -9], dtype=torch.int32, device="cuda")
    x = torch.randn(3, 2, 40, generator=torch.Generator().manual_seed(4)).cuda()
    for interleaved in (False, True):
        want, got = (bq.svdq_rope(x, pos, f, interleaved=interleaved) for f in (freq, odd))
        turned = lost.repeat_interleave(2) if interleaved else lost.repeat(2)
        columns = torch.cat([turned, torch.zeros(8, dtype=torch.bool, device="cuda")])
        assert got[..., columns].isnan().all() and torch.equal(got[..., ~columns], want[..., ~columns])
    for angle_major in (False, True):
        for want, got in zip(bq.svdq_rope_table(pos, freq, angle_major=angle_major),
                             bq.svdq_rope_table(pos, odd, angle_major=angle_major)):
            want, got = (t.t() if angle_major else t for t in (want, got))
            assert got[:, lost].isnan().all() and torch.equal(got[:, ~lost], want[:, ~lost])


@pytest.mark.parametrize("M,P", [(9, 1), (700, 4), (700, 6)])
@pytest.mark.parametrize("angle_major", [False, True], ids=["rows", "angle-major"])
def test_positions_past_32_bits(bq, M, P, angle_major):
    """int64 positions up to 2^40 either way, whose upper half counts. The fraction of a turn carries
    freq's 53 bits and is cut at 2^-64: an angle is off by 2^-52 of itself and 2^-64 turns (2^-61
    radians) a position."""
    freq = torch.full((P,), math.pi / 2, dtype=torch.float64)
    freq[P // 2:] = torch.linspace(1.0, 1e-9, P - P // 2, dtype=torch.float64)
    far = torch.tensor([2 ** 33, -2 ** 33, 2 ** 33 + 1, 2 ** 40, 2 ** 40 + 3, -2 ** 40 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 2])
    g = torch.Generator().manual_seed(M)
    pos = torch.cat([far, torch.randint(-2 ** 40, 2 ** 40, (M - 9,), generator=g)]).cuda()
    cos, sin = bq.svdq_rope_table(pos, freq.cuda(), angle_major=angle_major)
    cos, sin = (f64(t.t() if angle_major else t) for t in (cos, sin))
    p = pos.cpu().numpy()[:, None]
    angle = p * freq.numpy()                                   # rounded once: 2^-53 of itself
    e = 2.0 ** -22 + np.abs(angle) * (2.0 ** -52 + 2.0 ** -53) + np.abs(p) * 2.0 ** -61
    assert np.all(np.abs(cos - np.cos(angle)) <= e) and np.all(np.abs(sin - np.sin(angle)) <= e)
    # a whole number of quarter turns, whatever the bits of pi that float64 lacks add up to
    if P > 1:
        quarter = p[:, 0] % 4
        q = 2.0 ** -22 + np.abs(p[:, 0]) * 2.0 ** -50
        assert np.all(np.abs(cos[:, 0] - np.array([1, 0, -1, 0])[quarter]) <= q)
        assert np.all(np.abs(sin[:, 0] - np.array([0, 1, 0, -1])[quarter]) <= q)


@pytest.mark.parametrize("dtype,D,pairs,pad", [(F32, 2064, 512, 0), (F32, 2064, 500, 2), (BF, 1040, 512, 2), (BF, 4112, 512, 0),
                                               (BF, 1300, 321, 2)])
@pytest.mark.parametrize("interleaved", [True, False], ids=["adjacent", "halves"])
def test_heads_of_more_vectors_than_a_block(bq, dtype, D, pairs, pad, interleaved):
    """Heads that a block's 256 threads walk over more than once, with copied columns behind the
    pairs: packed, in place, and beside heads that stay."""
    freq = torch.logspace(0, -3, pairs, dtype=torch.float64).cuda()
    pos = positions(D, 5, 1, 10000)
    for H in (1, 9):
        base = torch.randn(5, H + 1, D + pad, generator=torch.Generator().manual_seed(H)).to(dtype).cuda()
        x, last = base[:, :H, :D], base[:, H].clone()
        y = bq.svdq_rope(x, pos, freq, scale=1.25, interleaved=interleaved)
        check(y, x, pos, freq, None, 1.25, interleaved)
        assert bq.svdq_rope(x, pos, freq, scale=1.25, interleaved=interleaved, Y=x) is x
        assert torch.equal(x, y) and torch.equal(base[:, H], last)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["int32", "int64"])
@pytest.mark.parametrize("M,P", [(997, 64), (997, 33), (40_000, 8)])
@pytest.mark.parametrize("angle_major", [False, True], ids=["rows", "angle-major"])
def test_small_angles_keep_their_precision(bq, M, P, angle_major, dtype):
    """Cosines and sines are float32 of their own size, not of a turn: slow pairs at near positions,
    whose sines are far below 1, and angles beside a quarter turn. The rest of a quarter turn is off
    by 2.5 U of itself, its series by 2 U, the scale by U: below 8 U = 2^-21 of the value, and the
    angle's own 2^-52 (and the comparison's 2^-53) and 2^-64 turns a position."""
    freq = torch.logspace(-1, -9, P, dtype=torch.float64)
    freq[0], freq[1] = math.pi / 2, math.pi / 2 + 1e-6
    pos = torch.arange(-9, M - 9, dtype=dtype)
    for scale in (1.0, 1.2079):
        cos, sin = bq.svdq_rope_table(pos.cuda(), freq.cuda(), scale=scale, angle_major=angle_major)
        angle = pos.double().numpy()[:, None] * freq.numpy()
        scale = float(np.float32(scale))
        e = scale * (np.abs(angle) * (2.0 ** -52 + 2.0 ** -53) + np.abs(pos.numpy()[:, None]) * 2.0 ** -61)
        for got, want in ((cos, scale * np.cos(angle)), (sin, scale * np.sin(angle))):
            got = f64(got.t() if angle_major else got)
            assert np.all(np.abs(got - want) <= 2.0 ** -21 * np.abs(want) + e)
    # and the rotation's: a unit vector's first coordinates
    x = torch.zeros(M, 1, 2 * P)
    x[..., :P] = 1.0
    y = f64(bq.svdq_rope(x.cuda(), pos.cuda(), freq.cuda()))[:, 0]
    e = np.abs(angle) * (2.0 ** -52 + 2.0 ** -53) + np.abs(pos.numpy()[:, None]) * 2.0 ** -61
    assert np.all(np.abs(y[:, P:] - np.sin(angle)) <= 2.0 ** -21 * np.abs(np.sin(angle)) + e)
