"""The 8-bit linear path and rotary positions without a GPU: argument errors of the
C ABI and of the binding (no call here reaches a launch), the frequency scalings in
closed form, the oracle's own pins, and the layers' routing over fake calls."""

import ctypes
import math

import numpy as np
import pytest

from oracle import w8a8 as O

torch = pytest.importorskip("torch")
import bit_quantized_diffusion_b200 as bq  # noqa: E402
import bit_quantized_diffusion_b200.layers as L  # noqa: E402
from bit_quantized_diffusion_b200 import prep  # noqa: E402

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
P = ctypes.c_void_p
GOOD, ODD8, ODD2, ODD1 = P(0x10000), P(0x10008), P(0x10002), P(0x10001)
ARG, ALIGN = 1, 2


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_diffusion_b200 import _native, build
    build.build()
    return _native.load()


def test_quantizer_argument_errors(lib):
    def q(M=4, K=64, X=GOOD, ldx=64, dtype=0, codes=GOOD, scale=GOOD):
        return lib.w8a8_quantize_act(M, K, X, ldx, dtype, codes, scale, None)

    assert q(M=0) == ARG and q(M=-1) == ARG
    assert q(K=0, ldx=0) == ARG and q(K=72, ldx=72) == ARG and q(K=32784, ldx=32784) == ARG
    assert q(ldx=56) == ARG and q(dtype=2) == ARG
    assert q(X=None) == ARG and q(codes=None) == ARG and q(scale=None) == ARG
    assert q(X=ODD8) == ALIGN and q(codes=ODD8) == ALIGN and q(scale=ODD2) == ALIGN
    assert q(ldx=68) == ALIGN and q(ldx=66, dtype=1) == ALIGN

    def n(X=GOOD, ldx=64, r=None, ldr=0, w=None, eps=1e-6, ro=None, ldo=0, dtype=0):
        return lib.w8a8_rmsnorm_quantize(4, 64, X, ldx, r, ldr, w, ctypes.c_float(eps), ro, ldo, dtype, GOOD,
                                         GOOD, None)

    assert n(r=GOOD, ldr=64) == ARG and n(ro=GOOD, ldo=64) == ARG       # both or neither
    assert n(r=GOOD, ldr=56, ro=GOOD, ldo=64) == ARG and n(r=GOOD, ldr=64, ro=GOOD, ldo=0) == ARG
    assert n(eps=-1.0) == ARG and n(eps=math.inf) == ARG and n(eps=math.nan) == ARG
    assert n(w=ODD8) == ALIGN and n(r=ODD8, ldr=64, ro=GOOD, ldo=64) == ALIGN
    assert n(r=GOOD, ldr=64, ro=GOOD, ldo=68) == ALIGN


def test_linear_argument_errors(lib):
    def g(M=4, N=32, K=32, a=GOOD, sa=GOOD, w=GOOD, sw=GOOD, bias=None, act=0, res=None, ldr=0, Y=GOOD, ldy=32,
          out=0):
        return lib.w8a8_linear(M, N, K, a, sa, w, sw, bias, act, res, ldr, Y, ldy, out, None)

    assert g(M=0) == ARG and g(N=0) == ARG and g(N=40, ldy=40) == ARG and g(K=0) == ARG and g(K=24) == ARG
    assert g(act=3) == ARG and g(act=-1) == ARG and g(out=2) == ARG
    for name in ("a", "sa", "w", "sw", "Y"):
        assert g(**{name: None}) == ARG, name
    assert g(ldy=16) == ARG and g(res=GOOD, ldr=16) == ARG
    assert g(a=ODD8) == ALIGN and g(w=ODD8) == ALIGN and g(Y=ODD8) == ALIGN and g(ldy=36) == ALIGN
    assert g(sa=ODD2) == ALIGN and g(sw=ODD2) == ALIGN and g(bias=ODD1) == ALIGN
    assert g(res=ODD8, ldr=32) == ALIGN and g(res=GOOD, ldr=36) == ALIGN

    def d(F=32, act=2, ldy=32, out=0, Y=GOOD):
        return lib.w8a8_gated_linear(4, F, 32, GOOD, GOOD, GOOD, GOOD, None, act, Y, ldy, out, None)

    assert d(F=24) == ARG and d(act=5) == ARG and d(ldy=31) == ARG and d(Y=None) == ARG
    assert d(F=2 ** 30, ldy=2 ** 30) == ARG and d(Y=ODD8) == ALIGN
    assert g(M=2 ** 30 + 1) == 3 and g(K=2 ** 30 + 16) == 3 and g(N=2 ** 30 + 16, ldy=2 ** 30 + 16) == 3


def test_rope_argument_errors(lib):
    def r(M=4, H=2, D=64, pairs=16, axes=1, pos=GOOD, nb=4, freq=GOOD, axis=None, scale=1.0, dtype=0, X=GOOD,
          ldx=128, ldhx=64, Y=GOOD, ldy=128, ldhy=64):
        return lib.svdq_rope(M, H, D, pairs, axes, pos, nb, freq, axis, ctypes.c_float(scale), 0, dtype, X, ldx,
                             ldhx, Y, ldy, ldhy, None)

    assert r(M=0) == ARG and r(H=0) == ARG and r(D=63) == ARG and r(pairs=33) == ARG and r(pairs=0) == ARG
    assert r(D=2048, pairs=513, ldx=4096, ldhx=2048, ldy=4096, ldhy=2048) == ARG
    assert r(axes=0) == ARG and r(pos=None) == ARG and r(freq=None) == ARG and r(X=None) == ARG and r(Y=None) == ARG
    assert r(nb=2) == ARG and r(scale=math.nan) == ARG and r(scale=math.inf) == ARG and r(dtype=2) == ARG
    assert r(ldx=127) == ARG and r(ldhy=65, ldy=200) == ARG and r(ldx=-128) == ARG
    assert r(ldy=64) == ARG and r(ldhy=32) == ARG and r(ldy=126) == ARG   # rows or heads of Y meet
    assert r(H=2 ** 20, D=2048, ldhx=2048, ldhy=2048, ldy=2 ** 31 - 2) == 3
    assert r(X=ODD8) == ALIGN and r(Y=ODD8) == ALIGN and r(pos=ODD2) == ALIGN and r(freq=P(0x10004)) == ALIGN
    assert r(pos=P(0x10004), nb=8) == ALIGN and r(axis=ODD2) == ALIGN

    def t(M=4, pairs=16, axes=1, cos=GOOD, sin=GOOD):
        return lib.svdq_rope_table(M, pairs, axes, GOOD, 4, GOOD, None, ctypes.c_float(1.0), 0, cos, sin, None)

    assert t(M=0) == ARG and t(pairs=513) == ARG and t(axes=0) == ARG and t(cos=None) == ARG
    assert t(sin=ODD2) == ALIGN


def test_binding_refuses_what_does_not_fit():
    z = torch.zeros
    for bad in (z(4, 64), z(4, 64, dtype=BF)):          # right but for the device
        with pytest.raises(ValueError, match="CUDA"):
            bq.w8a8_quantize_act(bad)
    for bad in (z(4, 72, dtype=BF), z(0, 64, dtype=BF), z(64, dtype=BF), z(4, 64, dtype=torch.float16),
                z(4, 32784, dtype=BF), z(64, 4, dtype=BF).t()):
        with pytest.raises(ValueError):
            bq.w8a8_quantize_act(bad)
    a, sa, w, sw = z(4, 32).to(E4), z(4), z(48, 32).to(E4), z(48)
    for kw in (dict(), dict(activation="relu"), dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bq.w8a8_linear(a, sa, w, sw, **kw)
    with pytest.raises(ValueError):
        bq.w8a8_gated_linear(a, sa, w, sw)              # 48 rows: gate and up of 24
    x, pos, freq = z(4, 2, 64), z(4, dtype=torch.int32), z(16, dtype=torch.float64)
    for args in ((x, pos, freq), (x, pos.float(), freq), (x, z(3, dtype=torch.int64), freq), (x[0], pos, freq),
                 (x, pos, z(33, dtype=torch.float64)), (x, pos, freq.float())):
        with pytest.raises(ValueError):
            bq.svdq_rope(*args)
    with pytest.raises(ValueError):
        bq.svdq_rope_table(pos, freq.reshape(4, 4))


def test_frequencies_in_closed_form():
    f, axis, scale = prep.rope_frequencies(8, base=16.0)
    assert f.dtype == torch.float64 and axis.dtype == torch.int32 and scale == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.5, 0.25, 0.125], dtype=torch.float64), rtol=1e-15)
    f3, axis, _ = prep.rope_frequencies((4, 8, 8), base=16.0)
    assert axis.tolist() == [0, 0] + [1] * 4 + [2] * 4
    assert torch.equal(f3[2:6], f) and torch.equal(f3[6:], f)
    assert torch.equal(prep.rope_frequencies(8, 16.0, "linear", 4.0)[0], f / 4.0)
    ntk = prep.rope_frequencies(8, 16.0, "ntk", 4.0)[0]
    assert ntk[0] == 1.0 and float(ntk[-1]) == pytest.approx(0.125 / 4.0, rel=1e-14)
    # yarn: pairs that turn more than 32 times within the length stay, those that turn less
    # than once are divided; the rest lie between, falling
    d, base, length, factor = 128, 10000.0, 4096, 8.0
    plain = prep.rope_frequencies(d, base)[0]
    y, _, scale = prep.rope_frequencies(d, base, "yarn", factor, length)
    turns = length * plain / (2 * math.pi)
    low = math.floor(d * math.log(length / (32 * 2 * math.pi)) / (2 * math.log(base)))
    high = math.ceil(d * math.log(length / (2 * math.pi)) / (2 * math.log(base)))
    ratio = y / plain
    assert torch.equal(y[: low + 1], plain[: low + 1]) and torch.all(turns[:low] > 32)
    assert torch.allclose(ratio[high:], torch.full_like(ratio[high:], 1 / factor)) and torch.all(turns[high:] < 1)
    assert torch.all(ratio[low + 1: high + 1] < ratio[low: high]) and scale == pytest.approx(0.1 * math.log(8) + 1)
    for bad in (dict(dims=7), dict(dims=()), dict(dims=(4, 0)), dict(dims=8, scaling="other"),
                dict(dims=8, scaling="linear", factor=0.5), dict(dims=8, scaling="yarn", factor=2.0),
                dict(dims=(2, 8), scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            prep.rope_frequencies(**bad)


def test_oracle_pins():
    rng = np.random.default_rng(3)
    v = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-4, 2.6, 4000), [0.0, 448.0, 1000.0, -449.0]])
    v32 = v.astype(np.float32)
    want = torch.from_numpy(np.clip(v32, -448, 448)).to(E4).float().numpy()
    assert np.array_equal(O.e4m3(v32.astype(np.float64)), want)
    codes, scale = O.quantize_rows(np.array([[0.0, 0.0], [448.0, 7.0], [-3.5, 1.75]]))
    assert np.array_equal(codes, [[0, 0], [448, 7], [-448, 224]]) and scale[1] == 1.0 and scale[2] == 3.5 / 448
    h, y = O.rmsnorm(np.array([[3.0, 4.0]]), eps=0.0)
    assert np.allclose(y, np.array([[3.0, 4.0]]) / math.sqrt(12.5))
    # a quarter turn, both layouts, the rest untouched
    c, s = O.cos_sin(np.array([[1]]), np.array([math.pi / 2, math.pi]))
    x = np.arange(1.0, 6.0).reshape(1, 1, 5)
    assert np.allclose(O.rope(x, c, s, True), [[[-2, 1, -3, -4, 5]]])
    assert np.allclose(O.rope(x, c, s, False), [[[-3, -2, 1, -4, 5]]])
    assert O.act(np.array([0.0]), "gelu") == 0 and O.act(np.array([30.0]), "silu") == pytest.approx(30.0)


def test_layers_route_workspaces(monkeypatch):
    calls = []

    def norm(x, weight=None, residual=None, eps=1e-6, codes=None, scale=None, residual_out=None, stream=None):
        calls.append(("norm", x, residual, residual_out, codes.shape))
        if residual is not None and residual_out is None:
            residual_out = torch.zeros_like(x)
        return codes, scale, residual_out

    def quant(x, codes=None, scale=None, stream=None):
        calls.append(("quantize", x, codes.shape, scale.shape))
        return codes, scale

    def gated(c, s, w, ws, bias=None, activation="silu", out_dtype=BF, Y=None, stream=None):
        calls.append(("gated", c, activation, Y))
        return Y

    def linear(c, s, w, ws, bias=None, residual=None, activation=None, out_dtype=BF, Y=None, stream=None):
        calls.append(("linear", c, bias, residual, activation, Y))
        return Y

    for name, fn in (("w8a8_rmsnorm_quantize", norm), ("w8a8_quantize_act", quant), ("w8a8_gated_linear", gated),
                     ("w8a8_linear", linear)):
        monkeypatch.setattr(L, name, fn)
    K, F = 32, 64

    def weights(n, k):
        return {"codes": torch.zeros(n, k).to(E4), "scale": torch.ones(n), "N": n, "K": k}

    bias = torch.zeros(F, dtype=BF)
    lin = L.W8A8Linear(weights(F, K), bias, max_tokens=8, activation="gelu")
    x, y, r = (torch.zeros(5, n, dtype=BF) for n in (K, F, F))
    assert lin(x, residual=r, y=y) is y
    assert calls[0][0] == "quantize" and calls[0][1] is x and calls[0][2:] == ((5, K), (5,))
    assert calls[1][0] == "linear" and calls[1][2] is bias and calls[1][3] is r and calls[1][4] == "gelu"
    with pytest.raises(ValueError):
        lin(torch.zeros(9, K, dtype=BF))
    mlp = L.W8A8GatedMlp(weights(2 * F, K), weights(K, F), None, max_tokens=8)
    for residual, out in ((None, torch.zeros_like(x)), (torch.zeros_like(x), torch.zeros_like(x)), (None, x)):
        calls.clear()
        assert mlp(x, residual, y=out) is out
        assert [c[0] for c in calls] == ["norm", "gated", "quantize", "linear"]
        assert calls[0][3] is (None if residual is None else out)       # h goes where the result will
        assert calls[3][3] is (x if residual is None else out)          # and is added to the projection
        assert calls[1][1].data_ptr() == mlp.codes.data_ptr() and calls[3][1].data_ptr() == mlp.hidden_codes.data_ptr()
    with pytest.raises(ValueError):
        L.W8A8GatedMlp(weights(2 * F, K), weights(K, F + 16), None, max_tokens=8)
    with pytest.raises(ValueError):
        mlp(torch.zeros(9, K, dtype=BF))


def test_qkv_layer_makes_its_tables_of_positions(monkeypatch):
    from tests.test_layers_host import Recorder, weights
    rec = Recorder(monkeypatch)
    layer = L.SvdqQkvNormRope(weights(384, 512, 0), None, max_tokens=16)
    rot = L.RotaryEmbedding((16, 56, 56), interleaved=True, device="cpu")
    made = {}

    def table(pos, freq, axis=None, scale=1.0, angle_major=False, cos=None, sin=None, stream=None):
        made.update(pos=pos, freq=freq, axis=axis, angle_major=angle_major)
        return "cos", "sin"

    monkeypatch.setattr(L, "svdq_rope_table", table)
    x, pos = torch.zeros(8, 512, dtype=BF), torch.zeros(8, 3, dtype=torch.int32)
    layer(x, rotary=rot, positions=pos)
    assert made["pos"] is pos and made["freq"] is rot.freq and made["axis"] is rot.axis and made["angle_major"]
    assert rec.calls[-1][6:8] == ("cos", "sin")
    for kw in (dict(rotary=rot), dict(positions=pos), dict(rotary=rot, positions=pos, rope_cos="c", rope_sin="s"),
               dict(rotary=L.RotaryEmbedding(128, device="cpu"), positions=pos),
               dict(rotary=L.RotaryEmbedding(64, interleaved=True, device="cpu"), positions=pos)):
        with pytest.raises(ValueError):
            layer(x, **kw)


def test_rotary_layer_wants_a_position_per_axis(monkeypatch):
    monkeypatch.setattr(L, "svdq_rope_table", lambda pos, *a, **k: "tables")
    monkeypatch.setattr(L, "svdq_rope", lambda x, *a, **k: "turned")
    three, one, tuple_of_one = (L.RotaryEmbedding(d, device="cpu") for d in ((16, 24, 24), 64, (64,)))
    x = torch.zeros(5, 2, 64, dtype=BF)
    for rot, shape in ((three, (5, 3)), (one, (5,)), (one, (5, 1)), (tuple_of_one, (5,))):
        pos = torch.zeros(shape, dtype=torch.int32)
        assert rot.tables(pos) == "tables" and rot(x, pos) == "turned"
    for rot, shape in ((three, (5,)), (three, (5, 2)), (three, (5, 4)), (one, (5, 3)), (tuple_of_one, (5, 2))):
        pos = torch.zeros(shape, dtype=torch.int32)
        with pytest.raises(ValueError, match="positions"):
            rot.tables(pos)
        with pytest.raises(ValueError, match="positions"):
            rot(x, pos)


def test_current_stream_with_and_without_torchs_short_cut(monkeypatch):
    """The older calls' stream: the handle alone where torch gives it, else the public Stream's."""
    from types import SimpleNamespace
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(bq, "_raw_stream", lambda device: 50 + device)
    assert bq._stream(None) == 53
    monkeypatch.setattr(bq, "_raw_stream", None)
    assert bq._stream(None) == 77
    assert bq._stream(SimpleNamespace(cuda_stream=5)) == 5 and bq._stream(9) == 9


def test_binding_is_rebuilt_for_another_torch(lib, tmp_path, monkeypatch):
    """A binding newer than its sources but compiled for another torch is not up to date; this tree's is,
    and says what it was built for."""
    import os
    from bit_quantized_diffusion_b200 import _native, build
    assert build.binding_up_to_date() and _native.binding().built_for == build.built_for()
    source, out = tmp_path / "binding.cpp", tmp_path / "_binding.so"
    source.write_text("")
    out.write_bytes(b"\x7fELF" + build.built_for().encode() + b"\0")
    os.utime(source, (1, 1))
    assert build.binding_up_to_date(str(out), [str(source)])
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")     # one text begins with the other
    assert not build.binding_up_to_date(str(out), [str(source)])
    monkeypatch.undo()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert not build.binding_up_to_date(str(out), [str(source)])
    monkeypatch.undo()
    os.utime(out, (0, 0))
    assert not build.binding_up_to_date(str(out), [str(source)])


def test_binding_that_does_not_load_says_what_to_do(lib, monkeypatch):
    import importlib
    from bit_quantized_diffusion_b200 import _native

    def fails(name):
        raise ImportError("undefined symbol")

    monkeypatch.setattr(_native, "_binding", None)
    monkeypatch.setattr(importlib, "import_module", fails)
    with pytest.raises(RuntimeError, match="build it again"):
        _native.binding()


def test_layers_share_no_buffers_across_streams_threads_and_captures(monkeypatch):
    """A layer's buffers serve the thread and stream that made it; a call on another stream, from another
    thread or in a capture takes none of them."""
    import threading
    given, state = [], {"current": 5, "capturing": False}

    def fresh(*shape, dtype=E4):
        return torch.zeros(shape, dtype=dtype)

    def quant(x, codes=None, scale=None, stream=None):
        given.extend((codes, scale))
        return (fresh(*x.shape) if codes is None else codes), (fresh(x.shape[0], dtype=F32) if scale is None else scale)

    def norm(x, weight=None, residual=None, eps=1e-6, codes=None, scale=None, residual_out=None, stream=None):
        return (*quant(x, codes, scale), residual_out)

    def gated(c, s, w, ws, bias=None, activation="silu", out_dtype=BF, Y=None, stream=None):
        given.append(Y)
        return fresh(c.shape[0], w.shape[0] // 2, dtype=BF) if Y is None else Y

    def linear(c, s, w, ws, bias=None, residual=None, activation=None, out_dtype=BF, Y=None, stream=None):
        return fresh(c.shape[0], w.shape[0], dtype=BF) if Y is None else Y

    for name, fn in (("w8a8_rmsnorm_quantize", norm), ("w8a8_quantize_act", quant), ("w8a8_gated_linear", gated),
                     ("w8a8_linear", linear)):
        monkeypatch.setattr(L, name, fn)
    monkeypatch.setattr(L, "_stream", lambda s: state["current"] if s is None else s, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    K, F = 32, 64
    w = {"codes": torch.zeros(2 * F, K).to(E4), "scale": torch.ones(2 * F), "N": 2 * F, "K": K}
    down = {"codes": torch.zeros(K, F).to(E4), "scale": torch.ones(K), "N": K, "K": F}
    for layer, count in ((L.W8A8Linear(w, None, max_tokens=8), 2), (L.W8A8GatedMlp(w, down, None, max_tokens=8), 5)):
        layer._home = threading.get_ident(), 5
        own = {t.untyped_storage().data_ptr() for t in vars(layer).values() if isinstance(t, torch.Tensor)}

        def shared(run):
            given.clear()
            run()
            assert len(given) == count
            return [t is not None and t.untyped_storage().data_ptr() in own for t in given]

        x = torch.zeros(5, K, dtype=BF)
        assert all(shared(lambda: layer(x))) and all(shared(lambda: layer(x, stream=5)))
        assert not any(shared(lambda: layer(x, stream=6)))

        def elsewhere():
            t = threading.Thread(target=layer, args=(x,))
            t.start()
            t.join()

        assert not any(shared(elsewhere))
        for key, value in (("current", 6), ("capturing", True)):
            before = state[key]
            state[key] = value
            assert not any(shared(lambda: layer(x)))
            state[key] = before
