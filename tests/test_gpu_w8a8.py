"""The 8-bit linear path on the GPU against the float64 oracle: the row quantizer bit for bit,
the norm in front of it, the product and its epilogue, the gated product, and a block of
them together. Each bound counts the roundings of the arithmetic it covers.

U = 2^-24 is half a float32 step, H the output type's half step (finfo.eps / 2)."""

import numpy as np
import pytest

from oracle import w8a8 as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module")
def bq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_quantized_diffusion_b200 as bq
    return bq


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def draw(seed, *shape, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def inside(t, cols, fill):
    """t in the middle columns of a wider tensor full of `fill`: (the view, the whole)."""
    whole = torch.full((t.shape[0], t.shape[1] + 2 * cols), fill, dtype=t.dtype, device=t.device)
    whole[:, cols: cols + t.shape[1]] = t
    return whole[:, cols: cols + t.shape[1]], whole


def outer_is(whole, cols, fill):
    return bool((whole[:, :cols] == fill).all() and (whole[:, whole.shape[1] - cols:] == fill).all())


# ------------------------------------------------------------------ quantizer
@TYPES
@pytest.mark.parametrize("M,K", [(1, 16), (1, 3840), (3, 48), (7, 1040), (130, 512), (33, 4112), (2, 15360), (2, 32768),
                                 (9999, 64), (5001, 1040), (2300, 3856), (333, 16400)])
def test_quantize_rows_bit_for_bit(bq, M, K, dtype):
    x = draw(M + K, M, K, dtype=dtype)
    x *= torch.logspace(-20, 20, M, device="cuda").to(dtype)[:, None] if M > 1 else 1
    x[:, K // 2] *= 30
    codes, scale = bq.w8a8_quantize_act(x)
    want, want_scale = O.quantize_rows(f64(x))
    assert np.array_equal(f64(scale), want_scale) and np.array_equal(f64(codes), want)


@TYPES
def test_quantize_rows_at_the_edges(bq, dtype):
    x = torch.zeros(9, 64, dtype=dtype)
    x[1, 5] = -0.0
    x[2, 3] = 2.0 ** -126                      # below the floor
    x[3] = torch.linspace(-1, 1, 64) * 2.0 ** -99
    x[4] = torch.linspace(-1, 1, 64) * 3e38
    x[5] = -2.5
    x[6, 7], x[7, 8], x[8, 9] = float("nan"), float("inf"), float("-inf")
    x[6:, 0] = 3.0
    codes, scale = bq.w8a8_quantize_act(x.cuda())
    want, want_scale = O.quantize_rows(f64(x[:6]))
    assert np.array_equal(f64(codes)[:6], want) and np.array_equal(f64(scale)[:6], want_scale)
    assert torch.isnan(scale[6]) and torch.isinf(scale[7]) and torch.isinf(scale[8])
    # a strided input gives the same as a packed one, and codes go where they are told
    view, _ = inside(x.cuda(), 16, float("nan"))
    buf = torch.full((9, 64), 1.0, device="cuda").to(E4)
    c2, s2 = bq.w8a8_quantize_act(view, codes=buf)
    assert c2 is buf and torch.equal(c2.view(torch.uint8), codes.view(torch.uint8))
    assert torch.equal(s2[:6], scale[:6])


# ------------------------------------------------------------------ norm
def norm_bounds(x, w, r, eps, K):
    """h is one rounding; the sum of squares of K values in float32, added by threads in a
    chain of at most 32 and trees of 5 + 5: 42 roundings and one per square; a square root
    halves that, and five more roundings lead to y: in all below 40 U of y."""
    h, y = O.rmsnorm(f64(x), None if w is None else f64(w), None if r is None else f64(r), eps)
    return h, y, 40 * U


def check_norm(codes, scale, y, rel):
    t = np.maximum(np.abs(y).max(1), O.FLOOR)
    s, c = f64(scale), f64(codes)
    assert np.all(np.abs(s - t / 448) <= (rel + 2 * U) * t / 448)
    # half a step of E4M3: 2^-4 of the value, 2^-10 below the smallest normal
    err = np.abs(c * s[:, None] - y)
    assert np.all(err <= np.abs(y) * (2.0 ** -4 + 3 * rel) + s[:, None] * 2.0 ** -10 * (1 + 3 * rel))


@TYPES
@pytest.mark.parametrize("M,K,weight,residual", [
    (1, 16, True, False), (1, 3840, True, True), (5, 48, False, True), (64, 1040, True, True), (3, 15360, True, True),
    (2, 32768, False, False), (300, 512, True, True), (9999, 64, True, True), (5001, 1040, True, False), (1501, 3840, True, True),
    (333, 16400, False, True)])
def test_rmsnorm_quantize(bq, M, K, weight, residual, dtype):
    x, w = draw(1, M, K, dtype=dtype), (1 + draw(2, K, std=0.2)).to(BF) if weight else None
    x[:, 3] *= 40
    r = draw(3, M, K, dtype=dtype, std=3.0) if residual else None
    codes, scale, out = bq.w8a8_rmsnorm_quantize(x, w, r, eps=1e-5)
    h, y, rel = norm_bounds(x, w, r, 1e-5, K)
    check_norm(codes, scale, y, rel)
    if not residual:
        assert out is None
        return
    assert out.dtype == dtype and np.all(np.abs(f64(out) - h) <= half_step(dtype) * np.abs(h) + U * np.abs(h))
    # in place on the residual stream, inside wider rows whose other columns stay
    rv, whole = inside(r, 8, 7.0)
    xv, _ = inside(x, 16, float("nan"))
    c2, s2, o2 = bq.w8a8_rmsnorm_quantize(xv, w, rv, eps=1e-5, residual_out=rv)
    assert o2 is rv and torch.equal(rv, out) and outer_is(whole, 8, 7.0)
    assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scale)


def test_rmsnorm_rows_of_their_own(bq):
    """Zero rows, tiny rows, and rows that are not finite, which touch no other."""
    x = draw(4, 6, 64)
    clean = bq.w8a8_rmsnorm_quantize(x)
    x[1], x[2], x[3, 5], x[4, 6] = 0.0, x[2] * 1e-30, float("nan"), float("inf")
    codes, scale, _ = bq.w8a8_rmsnorm_quantize(x)
    assert torch.isfinite(scale[:3]).all() and not f64(codes)[1].any() and not torch.isfinite(scale[3:5]).any()
    for row in (0, 5):
        assert torch.equal(codes[row].view(torch.uint8), clean[0][row].view(torch.uint8))
        assert scale[row] == clean[1][row]
    y = f64(x)[2:3] / np.sqrt(1e-6)
    check_norm(codes[2:3], scale[2:3], y, 40 * U)


@pytest.mark.parametrize("M", [4, 9999])
def test_rmsnorm_of_zeros_without_eps(bq, M):
    """0 / 0: NaN in the rows of zeros alone, in both kernels."""
    x = draw(1, M, 64, dtype=BF)
    clean = bq.w8a8_rmsnorm_quantize(x, eps=0.0)
    x[2::3] = 0.0
    codes, scale, _ = bq.w8a8_rmsnorm_quantize(x, eps=0.0)
    zero = torch.arange(M, device="cuda") % 3 == 2
    assert scale[zero].isnan().all() and torch.equal(scale[~zero], clean[1][~zero])
    assert torch.equal(codes[~zero].view(torch.uint8), clean[0][~zero].view(torch.uint8))


@TYPES
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("M,K,weight,residual", [
    (7, 64, False, False), (14, 3840, True, True), (9999, 64, True, True), (5001, 1040, False, False), (1501, 3840, True, True),
    (40, 16400, True, False), (333, 16400, False, True)])
def test_rmsnorm_rows_whose_squares_leave_float32(bq, M, K, weight, residual, eps, dtype):
    """Rows whose squares overflow, vanish or are subnormal in float32, up to h near its largest value
    (where h times the weight overflows too) and h subnormal, between rows of the usual size: the
    formula's values, in both kernels, in place too. The same roundings as elsewhere: the row is
    scaled by a power of two."""
    sizes = torch.tensor([1.0, 1e20, 3e-25, 1.5e37, 1e-38, 2e18, 1e-12], device="cuda")[torch.arange(M) % 7]
    x, w = draw(1, M, K).clamp_(-4, 4), (2 + draw(2, K, std=2.0)).to(BF) if weight else None
    x = (x * sizes[:, None]).to(dtype)
    r = (draw(3, M, K).clamp_(-4, 4) * sizes[:, None]).to(dtype) if residual else None
    codes, scale, out = bq.w8a8_rmsnorm_quantize(x, w, r, eps=eps)
    _, y, rel = norm_bounds(x, w, r, float(np.float32(eps)), K)
    check_norm(codes, scale, y, rel)
    usual = torch.arange(M, device="cuda") % 7 == 0
    c1, s1, _ = bq.w8a8_rmsnorm_quantize(x[usual], w, None if r is None else r[usual], eps=eps)
    if usual.sum() < 300 and M < 300:  # (the same kernel: the same order of the sums)
        assert torch.equal(codes[usual].view(torch.uint8), c1.view(torch.uint8)) and torch.equal(scale[usual], s1)
    if residual:
        assert torch.equal(out, (x.float() + r.float()).to(dtype))
        for into in (r, x):
            rv = into.clone()
            c2, s2, _ = bq.w8a8_rmsnorm_quantize(rv if into is x else x, w, rv if into is r else r, eps=eps, residual_out=rv)
            assert torch.equal(rv, out) and torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scale)


# ------------------------------------------------------------------ product
def operands(bq, M, rows, K, seed):
    x = draw(seed, M, K)
    x[:, K // 3] *= 30
    return (*bq.w8a8_quantize_act(x), *bq.w8a8_quantize_act(draw(seed + 1, rows, K, std=0.02)))


def product_bound(a, sa, w, sw, bias, K):
    """(z, its error): a matrix instruction adds 32 products to the running sum; allow each such
    step 2^-22 of the magnitudes' sum (products aligned to the largest, then cut), splits and
    joins of K a few more, and the epilogue four roundings."""
    z, mag = O.product(f64(a), f64(sa), f64(w), f64(sw), None if bias is None else f64(bias))
    return z, mag * ((K / 32 + 16) * 2.0 ** -22 + 4 * U)


def act_bound(z, ez, kind):
    """|gelu'|, |silu'| < 1.13; evaluated through exp(e) and a quotient: exp's relative error is
    its argument's rounding |e| U and a few U of its own, the quotient two, damped by
    exp/(1 + exp) < 1: (|e| + 12) U of the value, |e| <= 40 wherever the value counts."""
    if kind is None:
        return z, ez
    return O.act(z, kind), 1.13 * ez + 64 * U * np.abs(O.act(z, kind)) + 1e-15


CASES = [  # M, N, K, bias, act, residual: every kernel (few tokens of a small weight, of a large one with and
    # without K shared by a cluster, CTA pairs with a tile of 64 columns each), each at ragged sizes; wider
    # tiles, and several to a pair, are in test_gpu_w8a8_tiles.py
    (1, 4752, 272, True, None, True), (3, 272, 4112, True, "silu", True), (8, 4736, 4096, True, None, False),
    (9, 160, 2048, False, None, True), (13, 15360, 144, True, "gelu", True), (16, 80, 2064, True, None, True),
    (340, 64, 12512, True, "gelu", True), (1000, 48, 4112, True, None, True), (130, 272, 4096, False, "silu", True),
    (100, 15376, 80, False, None, True), (128, 272, 3504, True, "silu", False),
    (1, 16, 16, False, None, False), (1, 3840, 512, True, None, True), (2, 48, 4096, True, "silu", True),
    (7, 1040, 784, False, "gelu", False), (16, 272, 3856, True, None, False), (17, 128, 144, True, "gelu", True),
    (33, 528, 1040, True, None, True), (64, 256, 2048, False, "silu", True), (65, 2064, 272, True, None, True),
    (128, 400, 8192, True, "gelu", True), (129, 144, 640, True, None, False), (255, 768, 320, False, None, True),
    (257, 272, 128, True, "silu", True), (300, 1552, 656, True, None, True), (700, 512, 1536, True, "gelu", True),
    (1100, 528, 112, True, None, True)]


@TYPES
@pytest.mark.parametrize("M,N,K,bias,act,residual", CASES)
def test_linear(bq, M, N, K, bias, act, residual, dtype):
    a, sa, w, sw = operands(bq, M, N, K, 10 * M + N)
    b = draw(5, N, dtype=BF, std=0.1) if bias else None
    r = draw(6, M, N, dtype=dtype) if residual else None
    z, ez = product_bound(a, sa, w, sw, b, K)
    want, e = act_bound(z, ez, act)
    if residual:
        want, e = want + f64(r), e + U * np.abs(want)
    y = bq.w8a8_linear(a, sa, w, sw, b, residual=r, activation=act, out_dtype=dtype)
    err = np.abs(f64(y) - want)
    assert np.all(err <= e * 1.01 + (half_step(dtype) + 2 * U) * (np.abs(want) + e)), (err - e).max()
    # inside wider rows, whose other columns stay; the residual strided, and in place
    yv, whole = inside(torch.zeros_like(y), 16, 5.0)
    if residual:
        yv.copy_(r)
    got = bq.w8a8_linear(a, sa, w, sw, b, residual=yv if residual else None, activation=act, out_dtype=dtype, Y=yv)
    assert got is yv and torch.equal(yv, y) and outer_is(whole, 16, 5.0)
    assert bq.svdq_check_device_status() == 0


@pytest.mark.parametrize("M", [1, 5, 16, 40, 128, 200, 384])
def test_linear_is_exact_on_whole_numbers(bq, M):
    """Small whole numbers and scales of powers of two: every sum is exact in float32, in any order."""
    K, N = 2064, 208
    g = torch.Generator().manual_seed(M)
    a = torch.randint(-8, 9, (M, K), generator=g).float()
    w = torch.randint(-8, 9, (N, K), generator=g).float()
    sa, sw = 2.0 ** torch.randint(-3, 4, (M,), generator=g).float(), 2.0 ** torch.randint(-3, 4, (N,), generator=g).float()
    b, r = torch.randint(-9, 10, (N,), generator=g).to(BF), torch.randint(-9, 10, (M, N), generator=g).float()
    y = bq.w8a8_linear(a.to(E4).cuda(), sa.cuda(), w.to(E4).cuda(), sw.cuda(), b.cuda(), residual=r.cuda(), out_dtype=F32)
    want = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double() + b.double() + r.double()
    assert torch.equal(y.cpu().double(), want)


@TYPES
@pytest.mark.parametrize("M,F,K,bias,act", [
    (1, 2384, 272, True, "silu"), (8, 2368, 4096, False, "silu"), (9, 80, 2048, True, "gelu"), (12, 80, 2064, False, "silu"),
    (199, 96, 1680, True, "silu"), (500, 64, 8208, False, "gelu"), (100, 10256, 80, False, "silu"), (1, 16, 16, False, "silu"), (1, 1040, 3840, False, "silu"), (4, 272, 1040, True, "silu"), (16, 64, 4112, True, "gelu"),
    (31, 400, 144, False, "silu"), (64, 528, 2048, True, None), (128, 80, 512, False, "gelu"), (130, 272, 656, True, "silu"),
    (300, 464, 384, True, "gelu"), (600, 1040, 256, False, "silu")])
def test_gated_linear(bq, M, F, K, bias, act, dtype):
    a, sa, w, sw = operands(bq, M, 2 * F, K, M + F)
    b = draw(5, 2 * F, dtype=BF, std=0.1) if bias else None
    z, ez = product_bound(a, sa, w, sw, b, K)
    gate, eg = act_bound(z[:, :F], ez[:, :F], act)
    up, eu = z[:, F:], ez[:, F:]
    want, e = gate * up, np.abs(gate) * eu + np.abs(up) * eg + eg * eu
    y = bq.w8a8_gated_linear(a, sa, w, sw, b, activation=act, out_dtype=dtype)
    assert np.all(np.abs(f64(y) - want) <= e * 1.01 + (half_step(dtype) + 2 * U) * (np.abs(want) + e))
    yv, whole = inside(torch.zeros_like(y), 8, 5.0)
    bq.w8a8_gated_linear(a, sa, w, sw, b, activation=act, out_dtype=dtype, Y=yv)
    assert torch.equal(yv, y) and outer_is(whole, 8, 5.0)
    assert bq.svdq_check_device_status() == 0


@TYPES
@pytest.mark.parametrize("M", [17, 33, 47, 64, 77, 97, 128])
def test_few_tokens_of_a_wide_weight(bq, M, dtype):
    """A weight with row tiles enough for the GPU, each summed by one block: token counts about the
    epilogue's groups of 16, columns that end inside a tile, with and without a residual."""
    K = 272 if M % 2 else 1296
    for act, residual in (("gelu", False), (None, True)):
        test_linear(bq, M, 15136, K, M % 4 == 1, act, residual, dtype)
    test_gated_linear(bq, M, 7600, K, M % 4 == 1, "silu", dtype)


@pytest.mark.parametrize("M", [3, 20, 150, 300])
def test_a_row_that_is_not_finite_touches_no_other(bq, M):
    N = K = 160
    a, sa, w, sw = operands(bq, M, N, K, M)
    clean = bq.w8a8_linear(a, sa, w, sw, out_dtype=F32)
    gated = bq.w8a8_gated_linear(a, sa, w, sw, out_dtype=F32)
    sa[1], sw[2] = float("nan"), float("inf")
    a.view(torch.uint8)[2, 5] = 0x7F                        # an E4M3 NaN
    y = bq.w8a8_linear(a, sa, w, sw, out_dtype=F32)
    u = bq.w8a8_gated_linear(a, sa, w, sw, out_dtype=F32)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and not torch.isfinite(y[:, 2]).any()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    assert torch.equal(y[keep][:, 3:], clean[keep][:, 3:]) and torch.equal(u[keep][:, 3:], gated[keep][:, 3:])


def test_activations_far_out(bq):
    """+-inf-sized and far arguments keep the activations' limits."""
    a = torch.full((1, 16), 1.0, device="cuda").to(E4)
    w = torch.zeros(16, 16, device="cuda")
    w[:8, 0] = torch.tensor([448.0, -448.0, 100.0, -100.0, 10.0, -10.0, 0.0, -0.0625])
    sw = torch.ones(16, device="cuda")
    for scale in (1.0, 1e9, 1e30):
        sa = torch.full((1,), scale, device="cuda")
        z = f64(w.to(E4)[:, 0]) * float(sa)
        for act in ("silu", "gelu"):
            y = f64(bq.w8a8_linear(a, sa, w.to(E4), sw, activation=act, out_dtype=F32))[0]
            want = O.act(z, act)
            assert np.all(np.isfinite(y)) and np.all(np.abs(y - want) <= 64 * U * np.abs(want) + 1e-30 * scale)


@pytest.mark.parametrize("M", [1, 20, 130])
def test_activations_to_their_last_bits(bq, M):
    """float32 outputs of z that is exact (one product of ones, times its column's scale), in every kernel.
    exp(e) in 2 + 1.17 |e| units of its last place, 2 U each at most, the sum and the quotient in 6 U:
    (2.4 |e| + 10) U of SiLU, where e is exact; GELU's e has five roundings of its own, 5 |e| U more.
    A quotient by more than 2^126 may be 0."""
    N = 1040
    z = torch.cat([torch.linspace(-30, 12, N - 32), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 80.0, -80.0]).repeat(4)]).cuda()
    a, w = torch.zeros(M, 16, device="cuda"), torch.zeros(N, 16, device="cuda")
    a[:, 0] = w[:, 0] = 1.0
    x = f64(z)
    for act, e, own in (("silu", np.abs(x), 2.4), ("gelu", np.abs(1.5957691216057308 * (x + 0.044715 * x ** 3)), 7.4)):
        y = bq.w8a8_linear(a.to(E4), torch.ones(M, device="cuda"), w.to(E4), z, activation=act, out_dtype=F32)
        # (in the form of the exponential: 1 + tanh cancels far out)
        want = x / (1.0 + np.exp(np.minimum(e, 700.0) * -np.sign(x)))
        assert np.all(np.abs(f64(y) - want) <= (own * e + 10) * U * np.abs(want) + 1e-35)


# ------------------------------------------------------------------ use
@pytest.mark.parametrize("M", [1, 24, 200])
def test_graphs_streams_and_repeats(bq, M):
    """Captured and replayed on other inputs, two graphs in turn, on a stream of its own, and
    twice the same: all the bits of the plain call."""
    N, K = 272, 1040
    x, r = draw(1, M, K, dtype=BF), draw(2, M, K, dtype=BF)
    w, sw = bq.w8a8_quantize_act(draw(3, N, K, std=0.02))
    g, sg = bq.w8a8_quantize_act(draw(4, 2 * N, K, std=0.02))

    def once(x, r):
        codes, scale, h = bq.w8a8_rmsnorm_quantize(x, None, r)
        return h, bq.w8a8_linear(codes, scale, w, sw), bq.w8a8_gated_linear(codes, scale, g, sg)

    want = once(x, r)
    again = once(x, r)
    other = once(x * 2, r)
    for t, u in zip(want, again):
        assert torch.equal(t, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    codes, scale, h = bq.w8a8_rmsnorm_quantize(x, None, r, stream=side)
    y = bq.w8a8_linear(codes, scale, w, sw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    sx, sr = x.clone(), r.clone()
    graphs, outs = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(once(sx, sr))
        graphs.append(graph)
    sx.copy_(x * 2)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        for t, u in zip(out, other):
            assert torch.equal(t, u)
    assert bq.svdq_check_device_status() == 0


@pytest.mark.parametrize("M", [1, 50, 300])
def test_gated_block_together(bq, M):
    """W8A8GatedMlp and W8A8Linear: the block against its parts in float64, the 8-bit
    rounding of the hidden rows included through the kernels' own codes."""
    from bit_quantized_diffusion_b200.layers import W8A8GatedMlp, W8A8Linear
    K, F = 512, 1040
    gate, up = draw(1, F, K, dtype=BF, std=0.04), draw(2, F, K, dtype=BF, std=0.04)
    down, norm = draw(3, K, F, dtype=BF, std=0.03), (1 + draw(4, K, std=0.1)).to(BF)
    x, r = draw(5, M, K, dtype=BF), draw(6, M, K, dtype=BF, std=2.0)
    block = W8A8GatedMlp.from_linears(gate, up, down, norm, max_tokens=M + 3)
    y = block(x, r)
    h, n, _ = norm_bounds(x, norm, r, 1e-6, K)
    check_norm(block.codes[:M], block.scale[0, :M], n, 40 * U)
    z, ez = product_bound(block.codes[:M], block.scale[0, :M], block.up["codes"], block.up["scale"], None, K)
    g, eg = act_bound(z[:, :F], ez[:, :F], "silu")
    hidden, e = g * z[:, F:], np.abs(g) * ez[:, F:] + np.abs(z[:, F:]) * eg
    assert np.all(np.abs(f64(block.hidden[:M]) - hidden) <= 1.01 * e + (2.0 ** -8 + 2 * U) * (np.abs(hidden) + e))
    codes, scale = O.quantize_rows(f64(block.hidden[:M]))
    assert np.array_equal(f64(block.hidden_codes[:M]), codes) and np.array_equal(f64(block.scale[1, :M]), scale)
    z, ez = product_bound(block.hidden_codes[:M], block.scale[1, :M], block.down["codes"], block.down["scale"], None, F)
    # h itself went through bf16 on its way to the second projection
    want, e = z + h, ez + 2.0 ** -8 * np.abs(h)
    assert np.all(np.abs(f64(y) - want) <= 1.01 * e + (2.0 ** -8 + 4 * U) * (np.abs(want) + e))
    # in place on the residual stream, without a residual, and the plain layer with its epilogue
    rr = r.clone()
    assert block(x, rr, y=rr) is rr and torch.equal(rr, y)
    hb = h.astype(np.float32)
    same = block(torch.from_numpy(hb).cuda().to(BF))
    assert torch.allclose(same.float(), y.float(), rtol=0, atol=0.25 * float(y.float().abs().max()))
    lin = W8A8Linear.from_linear(gate, None, max_tokens=M, activation="gelu")
    out = lin(x)
    z, ez = product_bound(lin.codes[:M], lin.scale[:M], lin.w["codes"], lin.w["scale"], None, K)
    want, e = act_bound(z, ez, "gelu")
    assert np.all(np.abs(f64(out) - want) <= 1.01 * e + (2.0 ** -8 + 2 * U) * (np.abs(want) + e))
    assert bq.svdq_check_device_status() == 0


@pytest.mark.parametrize("M", [1, 50, 300])
def test_gated_block_without_a_residual(bq, M):
    """The block on x alone, against its parts in float64 through the kernels' own codes: h is x
    itself, and the projection is added to it, into a new tensor and in place."""
    from bit_quantized_diffusion_b200.layers import W8A8GatedMlp
    K, F = 512, 1040
    gate, up = draw(1, F, K, dtype=BF, std=0.04), draw(2, F, K, dtype=BF, std=0.04)
    down, norm = draw(3, K, F, dtype=BF, std=0.03), (1 + draw(4, K, std=0.1)).to(BF)
    x = draw(5, M, K, dtype=BF, std=2.0)
    block = W8A8GatedMlp.from_linears(gate, up, down, norm, max_tokens=M)
    kept = x.clone()
    y = block(x)
    assert y is not x and torch.equal(x, kept)
    h, n, rel = norm_bounds(x, norm, None, 1e-6, K)
    check_norm(block.codes, block.scale[0], n, rel)
    z, ez = product_bound(block.codes, block.scale[0], block.up["codes"], block.up["scale"], None, K)
    g, eg = act_bound(z[:, :F], ez[:, :F], "silu")
    hidden, e = g * z[:, F:], np.abs(g) * ez[:, F:] + np.abs(z[:, F:]) * eg
    assert np.all(np.abs(f64(block.hidden) - hidden) <= 1.01 * e + (2.0 ** -8 + 2 * U) * (np.abs(hidden) + e))
    codes, scale = O.quantize_rows(f64(block.hidden))
    assert np.array_equal(f64(block.hidden_codes), codes) and np.array_equal(f64(block.scale[1]), scale)
    z, ez = product_bound(block.hidden_codes, block.scale[1], block.down["codes"], block.down["scale"], None, F)
    want = z + h
    assert np.all(np.abs(f64(y) - want) <= 1.01 * ez + (2.0 ** -8 + 2 * U) * (np.abs(want) + ez))
    assert block(x, y=x) is x and torch.equal(x, y)
    assert bq.svdq_check_device_status() == 0


@pytest.mark.parametrize("M", [1, 8, 40, 100, 300, 1500])
def test_chain_on_one_buffer(bq, M):
    """Layer after layer on one residual stream and one set of workspaces, each call reading what
    the one before wrote over the values that the one before that had read: the bits of the same
    chain with a new tensor for every result."""
    from bit_quantized_diffusion_b200.layers import RotaryEmbedding, W8A8GatedMlp, W8A8Linear
    K, F = 512, 656
    blocks = [W8A8GatedMlp.from_linears(draw(i, F, K, dtype=BF, std=0.04), draw(i + 50, F, K, dtype=BF, std=0.04),
                                        draw(i + 100, K, F, dtype=BF, std=0.03), None, max_tokens=M) for i in range(3)]
    lin = W8A8Linear.from_linear(draw(7, K, K, dtype=BF, std=0.03), None, max_tokens=M)
    rot = RotaryEmbedding(64)
    pos = torch.arange(M, device="cuda")
    x = draw(9, M, K, dtype=BF)

    def chain(fresh):
        h = x.clone()
        for step in range(12):
            y = None if fresh else h
            h = blocks[step % 3](h, y=y)
            y = None if fresh else h
            h = rot(h.view(M, 8, 64), pos, y=None if fresh else y.view(M, 8, 64)).view(M, K)
            y = None if fresh else h
            h = lin(h, residual=h, y=y)
        return h

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)
    assert torch.isfinite(want.float()).all() and bq.svdq_check_device_status() == 0


@TYPES
@pytest.mark.parametrize("M", [1, 60, 300])
def test_gated_block_with_biases(bq, M, dtype):
    """Gate, up and down with a bias each, on a stream of either type: the block against its parts in
    float64 through the kernels' own codes, and in place."""
    from bit_quantized_diffusion_b200.layers import W8A8GatedMlp
    K, F = 272, 656
    gate, up, down = (draw(i, *s, dtype=BF, std=0.04) for i, s in ((1, (F, K)), (2, (F, K)), (3, (K, F))))
    bg, bu, bd = (draw(i, n, dtype=BF, std=0.5) for i, n in ((4, F), (5, F), (6, K)))
    x, r = draw(7, M, K, dtype=dtype), draw(8, M, K, dtype=dtype, std=2.0)
    block = W8A8GatedMlp.from_linears(gate, up, down, None, M, "gelu", gate_bias=bg, up_bias=bu, down_bias=bd)
    y = block(x, r)
    assert y.dtype == dtype
    h, n, rel = norm_bounds(x, None, r, 1e-6, K)
    check_norm(block.codes, block.scale[0], n, rel)
    z, ez = product_bound(block.codes, block.scale[0], block.up["codes"], block.up["scale"], torch.cat([bg, bu]), K)
    g, eg = act_bound(z[:, :F], ez[:, :F], "gelu")
    hidden, e = g * z[:, F:], np.abs(g) * ez[:, F:] + np.abs(z[:, F:]) * eg + eg * ez[:, F:]
    assert np.all(np.abs(f64(block.hidden) - hidden) <= 1.01 * e + (2.0 ** -8 + 2 * U) * (np.abs(hidden) + e))
    z, ez = product_bound(block.hidden_codes, block.scale[1], block.down["codes"], block.down["scale"], bd, F)
    # h goes through the stream's type on its way to the second projection
    want, e = z + h, ez + (half_step(dtype) + 2 * U) * np.abs(h)
    assert np.all(np.abs(f64(y) - want) <= 1.01 * e + (half_step(dtype) + 2 * U) * (np.abs(want) + e))
    alone = block(x)
    assert alone.dtype == dtype and block(x, y=x) is x and torch.equal(x, alone)
    with pytest.raises(ValueError, match="both or neither"):
        W8A8GatedMlp.from_linears(gate, up, down, None, M, gate_bias=bg)


@TYPES
@pytest.mark.parametrize("M", [1, 60, 300])
def test_linear_layer_on_a_stream_of_either_type(bq, M, dtype):
    """W8A8Linear onto a residual stream of its output's type, new and in place: the calls under it, bit for bit."""
    from bit_quantized_diffusion_b200.layers import W8A8Linear
    K, N = 272, 528
    w, b = draw(1, N, K, dtype=BF, std=0.04), draw(2, N, dtype=BF, std=0.1)
    x, r = draw(3, M, K, dtype=dtype), draw(4, M, N, dtype=dtype)
    lin = W8A8Linear.from_linear(w, b, max_tokens=M, out_dtype=dtype)
    y = lin(x, residual=r)
    assert y.dtype == dtype
    assert torch.equal(y, bq.w8a8_linear(*bq.w8a8_quantize_act(x), *bq.w8a8_quantize_act(w), b, residual=r, out_dtype=dtype))
    assert lin(x, residual=r, y=r) is r and torch.equal(r, y)


@pytest.mark.parametrize("M", [4, 300, 1500])
def test_one_layer_on_several_streams_at_once(bq, M):
    """One block and one linear layer called from two threads and on two streams in turn, and captured
    into two graphs that are replayed side by side: each call's bits are those of the call alone."""
    import threading
    from bit_quantized_diffusion_b200.layers import W8A8GatedMlp, W8A8Linear
    K, F = 512, 1040
    block = W8A8GatedMlp.from_linears(draw(1, F, K, dtype=BF, std=0.04), draw(2, F, K, dtype=BF, std=0.04),
                                      draw(3, K, F, dtype=BF, std=0.03), None, max_tokens=M)
    lin = W8A8Linear.from_linear(draw(4, K, K, dtype=BF, std=0.04), None, max_tokens=M)
    x = [draw(10 + i, M, K, dtype=BF) for i in range(2)]
    r = [draw(20 + i, M, K, dtype=BF) for i in range(2)]

    def once(i, stream=None):
        return lin(block(x[i], r[i], stream=stream), residual=r[i], stream=stream)

    want = [once(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(30):
        for i in range(2):
            got[i].append(once(i, streams[i]))
        got[0].append(once(0))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])
    out, errors = [None, None], []

    def run(i):
        try:
            for _ in range(30):  # both threads on the default stream
                out[i] = once(i)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors and all(torch.equal(out[i], want[i]) for i in range(2))
    graphs, out = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out.append(once(i))
        graphs.append(graph)
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        once(0)
    torch.cuda.synchronize()
    assert all(torch.equal(out[i], want[i]) for i in range(2))
    assert bq.svdq_check_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(1, 1040, 2064), (16, 272, 1040), (40, 528, 1040), (300, 528, 656)])
def test_both_operands_made_just_before(bq, M, N, K):
    """Weight and tokens quantized into the same buffers again and again, each product right behind: the
    bits of operands that nothing writes to."""
    ws, xs = [draw(i, N, K, dtype=BF, std=0.04) for i in range(5)], [draw(9 + i, M, K, dtype=BF) for i in range(5)]
    want = [bq.w8a8_linear(*bq.w8a8_quantize_act(x), *bq.w8a8_quantize_act(w)) for x, w in zip(xs, ws)]
    codes, scale = bq.w8a8_quantize_act(xs[0])
    w_codes, w_scale = bq.w8a8_quantize_act(ws[0])
    torch.cuda.synchronize()
    got = []
    for step in range(100):
        bq.w8a8_quantize_act(xs[step % 5], codes=codes, scale=scale)
        bq.w8a8_quantize_act(ws[step % 5], codes=w_codes, scale=w_scale)
        got.append(bq.w8a8_linear(codes, scale, w_codes, w_scale))
    for step, y in enumerate(got):
        assert torch.equal(y, want[step % 5]), step


def test_offsets_beyond_32_bits(bq):
    """Rows, outputs and residuals whose elements number over 2^32: the last rows and one in the
    middle agree with calls on those rows alone."""
    def rows_of(M):
        return [0, M // 2 + 1, M - 2, M - 1]

    M, K = 262_300, 16_384
    x = torch.empty(M, K, dtype=BF, device="cuda")
    pattern = draw(1, 4, K, dtype=BF)
    for i, row in enumerate(rows_of(M)):
        x[row] = pattern[i]
    codes, scale = bq.w8a8_quantize_act(x)
    want, want_scale = bq.w8a8_quantize_act(pattern)
    assert torch.equal(codes[rows_of(M)].view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(scale[rows_of(M)], want_scale)
    del x, codes
    M, N, K = 1_050_000, 4112, 32
    w, sw = bq.w8a8_quantize_act(draw(2, N, K))
    a = torch.zeros(M, K, device="cuda").to(E4)
    few = draw(3, 4, K).to(E4)
    y = torch.zeros(M, N, dtype=BF, device="cuda")
    r = draw(4, 4, N, dtype=BF)
    for i, row in enumerate(rows_of(M)):
        a.view(torch.uint8)[row] = few.view(torch.uint8)[i]
        y[row] = r[i]
    sa = torch.ones(M, device="cuda")
    bq.w8a8_linear(a, sa, w, sw, residual=y, Y=y)
    want = bq.w8a8_linear(few, sa[:4], w, sw, residual=r)
    # one sum of 32 products, in one matrix instruction or another: the same to bf16's half step
    assert torch.allclose(y[rows_of(M)].float(), want.float(), rtol=2.0 ** -8 + 2.0 ** -20, atol=1e-5)
    assert bq.svdq_check_device_status() == 0


def test_threads_and_stream_handles(bq):
    """Calls from several threads on streams of their own, outputs allocated by the calls, the
    stream given as an object or as its handle."""
    import threading
    K, N = 1040, 272
    w, sw = bq.w8a8_quantize_act(draw(1, N, K, std=0.02))
    x = [draw(10 + i, 30 + 50 * i, K, dtype=BF) for i in range(4)]
    want = [bq.w8a8_linear(*bq.w8a8_quantize_act(t), w, sw) for t in x]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def run(i):
        try:
            s = torch.cuda.Stream()
            handle = s if i % 2 else s.cuda_stream
            for _ in range(20):
                codes, scale = bq.w8a8_quantize_act(x[i], stream=handle)
                y = bq.w8a8_linear(codes, scale, w, sw, stream=handle)
            s.synchronize()
            got[i] = y
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_other_device_is_refused(bq):
    if torch.cuda.device_count() < 2:
        x = torch.zeros(4, 64, dtype=BF)
        with pytest.raises(ValueError, match="CUDA"):
            bq.w8a8_quantize_act(x, codes=torch.zeros(4, 64, device="cuda").to(E4))
        return
    with pytest.raises(ValueError, match="current device"):
        bq.w8a8_quantize_act(torch.zeros(4, 64, dtype=BF, device="cuda:1"))
