"""Cases of the 8-bit linear path and of rotary positions, for measuring them.

Operators:
  norm     w8a8_rmsnorm_quantize / w8a8_quantize_act: the residual's addition, RMS norm and rows of E4M3 codes with a
           float32 scale each
  linear   w8a8_linear: the product of E4M3 rows with bias, activation and residual in its epilogue
  gated    w8a8_gated_linear: act(gate) * up of one [2F, K] weight
  rope     svdq_rope: rotary positions on the heads of a row-strided Q | K | V
  table    svdq_rope_table: the cos / sin tables of those positions, row-major or angle-major (the fused QKV call's)

`run` computes a case in elementary float32 torch operations, or, with `own` set, through the package's calls.
"""

import math

import torch

own = False

E4M3_MAX = 448.0          # the largest E4M3 value
TINY = 2.0 ** -100        # a row's maximum counts as at least this


def listed():
    return [
        # one token of a stream through a block's pre-norm: launch latency
        dict(name="norm_token", op="norm", M=1, K=3840, dtype="bf16", norm=True, residual=True),
        # a 1024 x 1024 image's tokens with its text through the same pre-norm
        dict(name="norm_image", op="norm", M=4608, K=3840, dtype="bf16", norm=True, residual=True),
        # an MLP's hidden activation into 8 bits before the second projection
        dict(name="quantize_hidden", op="norm", M=4096, K=15360, dtype="bf16", norm=False, residual=False),
        # one token through the attention's output projection: streaming the weight
        dict(name="linear_token", op="linear", M=1, K=3840, N=3840, bias=True, act="none", residual=True, out="bf16"),
        # a prompt of odd length through an MLP's first projection
        dict(name="linear_prompt", op="linear", M=77, K=3840, N=15360, bias=True, act="gelu", residual=False, out="bf16"),
        # an image's tokens through an MLP's second projection, onto the residual stream
        dict(name="linear_image", op="linear", M=4096, K=15360, N=3840, bias=True, act="none", residual=True, out="bf16"),
        # four streams decoding through a gated block's first half
        dict(name="gated_tokens", op="gated", M=4, K=3840, F=10240, bias=False, act="silu", out="bf16"),
        # an image's tokens through it
        dict(name="gated_image", op="gated", M=4608, K=3840, F=10240, bias=False, act="silu", out="bf16"),
        # 64 streams, one token each, far into a scaled context; half layout, the whole head
        dict(name="rope_tokens", op="rope", M=64, heads=60, D=128, rot=128, axes=1, interleaved=False, far=1000000,
             factor=8.0, dtype="bf16"),
        # an image's Q and K inside the Q | K | V row, three position axes, adjacent pairs
        dict(name="rope_image", op="rope", M=4608, heads=60, D=128, rot=128, axes=3, interleaved=True, far=128,
             factor=1.0, dtype="bf16"),
        # the same image's tables for the fused QKV call
        dict(name="table_image", op="table", M=4608, P=64, axes=3, far=128, factor=1.0, angle_major=True),
        # a long context's tables
        dict(name="table_long", op="table", M=131072, P=64, axes=1, far=1000000, factor=8.0, angle_major=False),
    ]


def _log(rng, lo, hi, step=1):
    """A whole number of [lo, hi], spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "gated", "rope", "table"])
    if op == "norm":
        norm = rng.random() < 0.7
        return dict(op=op, M=_log(rng, 1, 4608), K=_log(rng, 64, 15360, 16), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    norm=norm, residual=norm and rng.random() < 0.7)
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 4096), K=_log(rng, 64, 15360, 16), N=_log(rng, 64, 15360, 16),
                    bias=rng.random() < 0.7, act=rng.choice(["none", "gelu", "silu"]), residual=rng.random() < 0.5,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "gated":
        return dict(op=op, M=_log(rng, 1, 4608), K=_log(rng, 64, 3840, 16), F=_log(rng, 64, 10240, 16),
                    bias=rng.random() < 0.3, act=rng.choice(["silu", "silu", "gelu"]), out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "rope":
        D = rng.choice([32, 64, 80, 96, 128, 256])
        axes = rng.choice([1, 1, 2, 3])
        return dict(op=op, M=_log(rng, 1, 4608), heads=_log(rng, 1, 60 * 128 // D), D=D,
                    rot=rng.choice([r for r in (16, 20, 32, 64, 96, 128, 256) if r <= D]), axes=axes,
                    interleaved=rng.random() < 0.5, far=_log(rng, 64, 1000000), factor=rng.choice([1.0, 4.0, 8.0, 32.0]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    return dict(op=op, M=_log(rng, 1, 131072), P=rng.choice([8, 10, 16, 32, 48, 64]), axes=rng.choice([1, 1, 2, 3]),
                far=_log(rng, 64, 1000000), factor=rng.choice([1.0, 4.0, 8.0, 32.0]), angle_major=rng.random() < 0.5)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows_to_e4m3(w):
    """A weight's or an activation's rows as E4M3 codes and float32 scales."""
    top = w.abs().amax(1).clamp_min(TINY)
    return (w * (E4M3_MAX / top)[:, None]).to(torch.float8_e4m3fn), top / E4M3_MAX


def _activations(g, M, K):
    """N(0, 1) with a few outlier channels 30 times as large, as the layers' inputs have."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 256)]] *= 30.0
    return x


def _angles(case, g, P):
    """Positions [M, axes] and what a program keeps of the frequencies: float64 [P] and each pair's axis."""
    axes, M = case["axes"], case["M"]
    positions = torch.randint(0, case["far"], (M, axes), generator=g, device="cuda", dtype=torch.int32)
    share = [P // axes + (a < P % axes) for a in range(axes)]
    freq = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in share]) / case["factor"]
    axis = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in enumerate(share)])
    # a longer context's attention is sharpened a little through the tables
    scale = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
    return dict(positions=positions, freq=freq.cuda(), axis=axis.cuda(), scale=scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M = case["op"], case["M"]
    s = dict(case=case)
    if op == "norm":
        K, t = case["K"], _TYPES[case["dtype"]]
        s["x"] = _activations(g, M, K).to(t)
        s["residual"] = (3.0 * torch.randn(M, K, generator=g, device="cuda")).to(t) if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * torch.randn(K, generator=g, device="cuda")).bfloat16() if case["norm"] else None
        s["codes"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["scale"] = torch.empty(M, device="cuda")
        s["sum"] = torch.empty(M, K, dtype=t, device="cuda") if case["residual"] else None
    elif op in ("linear", "gated"):
        K, N = case["K"], case["N"] if op == "linear" else case["F"]
        rows = N if op == "linear" else 2 * N
        s["a"], s["a_scale"] = _rows_to_e4m3(_activations(g, M, K))
        s["w"], s["w_scale"] = _rows_to_e4m3(0.02 * torch.randn(rows, K, generator=g, device="cuda"))
        s["bias"] = (0.1 * torch.randn(rows, generator=g, device="cuda")).bfloat16() if case["bias"] else None
        s["residual"] = (torch.randn(M, N, generator=g, device="cuda").to(_TYPES[case["out"]])
                         if case.get("residual") else None)
        s["y"] = torch.empty(M, N, dtype=_TYPES[case["out"]], device="cuda")
    elif op == "rope":
        H, D = case["heads"], case["D"]
        s.update(_angles(case, g, case["rot"] // 2))
        # Q and K heads of a row that holds half as many V heads behind them
        qkv = torch.randn(M, (H + (H + 1) // 2) * D, generator=g, device="cuda").to(_TYPES[case["dtype"]])
        s["x"] = qkv.view(M, -1, D)[:, :H]
        s["y"] = torch.empty(M, H, D, dtype=qkv.dtype, device="cuda")
    else:
        s.update(_angles(case, g, case["P"]))
        shape = (case["P"], M) if case["angle_major"] else (M, case["P"])
        s["cos"], s["sin"] = torch.empty(shape, device="cuda"), torch.empty(shape, device="cuda")
    return s


def _act(y, kind):
    if kind == "silu":
        return y / (1.0 + torch.exp(-y))
    if kind == "gelu":
        return 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def _cos_sin(s):
    """cos and sin of every row's angles, times the tables' scale: the angles in 64 bits, since positions are far."""
    a = s["positions"].double()[:, s["axis"].long()] * s["freq"]
    return (torch.cos(a) * s["scale"]).float(), (torch.sin(a) * s["scale"]).float()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = s["x"].float()
        out = {}
        if case["residual"]:
            h = h + s["residual"].float()
            out["sum"] = h.to(s["x"].dtype)
        if case["norm"]:
            h = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
        top = h.abs().amax(1).clamp_min(TINY)
        out["codes"] = (h * (E4M3_MAX / top)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        out["scale"] = top / E4M3_MAX
        return out
    if op in ("linear", "gated"):
        y = (s["a"].float() @ s["w"].float().t()) * s["a_scale"][:, None] * s["w_scale"]
        if s["bias"] is not None:
            y = y + s["bias"].float()
        if op == "gated":
            y = _act(y[:, : case["F"]], case["act"]) * y[:, case["F"]:]
        else:
            y = _act(y, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(_TYPES[case["out"]])
    cos, sin = _cos_sin(s)
    if op == "table":
        return {"cos": cos.t().contiguous(), "sin": sin.t().contiguous()} if case["angle_major"] else {"cos": cos, "sin": sin}
    x, R = s["x"].float(), case["rot"]
    r = x.clone()
    cos, sin = cos[:, None], sin[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        r[..., 0:R:2], r[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        r[..., : R // 2], r[..., R // 2: R] = a * cos - b * sin, b * cos + a * sin
    return r.to(s["x"].dtype)


def _calls(s):
    import bit_quantized_diffusion_b200 as bq

    case = s["case"]
    op = case["op"]
    act = None if case.get("act") == "none" else case.get("act")
    if op == "norm" and not case["norm"]:
        codes, scale = bq.w8a8_quantize_act(s["x"], codes=s["codes"], scale=s["scale"])
        return {"codes": codes, "scale": scale}
    if op == "norm":
        codes, scale, total = bq.w8a8_rmsnorm_quantize(s["x"], s["weight"], s["residual"], eps=1e-6, codes=s["codes"],
                                                       scale=s["scale"], residual_out=s["sum"])
        out = {"codes": codes, "scale": scale}
        return {**out, "sum": total} if case["residual"] else out
    if op == "linear":
        return bq.w8a8_linear(s["a"], s["a_scale"], s["w"], s["w_scale"], s["bias"], residual=s["residual"],
                              activation=act, out_dtype=s["y"].dtype, Y=s["y"])
    if op == "gated":
        return bq.w8a8_gated_linear(s["a"], s["a_scale"], s["w"], s["w_scale"], s["bias"], activation=act,
                                    out_dtype=s["y"].dtype, Y=s["y"])
    if op == "rope":
        return bq.svdq_rope(s["x"], s["positions"], s["freq"], axis=s["axis"], scale=s["scale"],
                            interleaved=case["interleaved"], Y=s["y"])
    cos, sin = bq.svdq_rope_table(s["positions"], s["freq"], axis=s["axis"], scale=s["scale"],
                                  angle_major=case["angle_major"], cos=s["cos"], sin=s["sin"])
    return {"cos": cos, "sin": sin}


def run(state):
    return _calls(state) if own else _plain(state)


def exact(case, seed):
    """The definition in 64 bits, no value rounded: of the E4M3 codes, what they round."""
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op == "norm":
        h = s["x"].to(d)
        out = {}
        if s["residual"] is not None:
            h += s["residual"].to(d)
            out["sum"] = h.clone()
        if s["weight"] is not None:
            h /= ((h ** 2).sum(1, keepdim=True) / case["K"] + 1e-6).sqrt()
            h *= s["weight"].to(d)
        top = torch.maximum(h.max(1).values, -h.min(1).values).clamp_min(TINY)
        return {**out, "codes": h / (top / 448)[:, None], "scale": top / 448}
    if op in ("linear", "gated"):
        def product(lo, hi):
            y = torch.einsum("mk,nk->mn", s["a"].to(d), s["w"][lo:hi].to(d))
            y *= torch.outer(s["a_scale"].to(d), s["w_scale"][lo:hi].to(d))
            return y if s["bias"] is None else y + s["bias"][lo:hi].to(d)

        def act(y):
            if case["act"] == "gelu":
                return y * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3))
            return y * torch.sigmoid(y) if case["act"] == "silu" else y

        if op == "gated":
            return act(product(0, case["F"])) * product(case["F"], 2 * case["F"])
        y = act(product(0, case["N"]))
        return y if s["residual"] is None else y + s["residual"].to(d)
    # turn pairs as complex numbers
    turn = torch.polar(torch.full((1, 1), s["scale"], dtype=d, device="cuda"),
                       torch.gather(s["positions"].to(d), 1, s["axis"].long().expand(case["M"], -1)) * s["freq"])
    if op == "table":
        turn = turn.transpose(0, 1) if case["angle_major"] else turn
        return {"cos": turn.real.contiguous(), "sin": turn.imag.contiguous()}
    R, x = case["rot"], s["x"].to(d)
    head, rest = x[..., :R], x[..., R:]
    if case["interleaved"]:
        z = torch.view_as_complex(head.unflatten(-1, (R // 2, 2)).contiguous()) * turn[:, None]
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(*head.unflatten(-1, (2, R // 2)).unbind(-2)) * turn[:, None]
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, rest], -1)


def work(case):
    """Each input read once, each output written once."""
    op, M = case["op"], case["M"]
    if op == "norm":
        K, b = case["K"], 2 if case["dtype"] == "bf16" else 4
        n = M * K
        return {"bytes": n * (b * (3 if case["residual"] else 1) + 1) + 4 * M + (2 * K if case["norm"] else 0),
                "flops": n * (7 if case["norm"] else 3)}
    if op in ("linear", "gated"):
        K, N = case["K"], case["N"] if op == "linear" else case["F"]
        rows = N if op == "linear" else 2 * N
        b = 2 if case["out"] == "bf16" else 4
        return {"bytes": M * K + rows * K + 4 * (M + rows) + (2 * rows if case["bias"] else 0)
                + b * M * N * (2 if case.get("residual") else 1), "flops": 2 * M * rows * K}
    if op == "rope":
        n, P = M * case["heads"] * case["D"], case["rot"] // 2
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * M * case["axes"] + 12 * P,
                "flops": 6 * M * case["heads"] * P}
    return {"bytes": 8 * M * case["P"] + 4 * M * case["axes"] + 12 * case["P"], "flops": 4 * M * case["P"]}
