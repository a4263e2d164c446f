"""User-facing layers over the C ABI: the SVDQ W4A4 linear and the AWQ W4A16
linear (the ``SVDQW4A4Linear`` / ``AWQW4A16Linear`` runtime layers of the
Diffusers blog, "quantization_config"), with preallocated workspaces so a
forward call is two (or one) library calls and no allocation (one forward of an
instance at a time); the 8-bit linear and gated feed-forward block for layers
that lose too much in four bits; and rotary positions."""

from __future__ import annotations

import threading

import torch

from . import prep
from . import (_stream, awq_w4a16_linear, svdq_codes_bytes, svdq_quantize_act, svdq_quantize_act_two_level, svdq_rope,
               svdq_rope_table, svdq_scales_bytes, svdq_tensor_scale, svdq_w4a4_linear, svdq_w4a4_linear_qkv_norm_rope,
               svdq_w4a4_linear_two_level, svdq_xl1_splits, w8a8_gated_linear, w8a8_linear, w8a8_quantize_act,
               w8a8_rmsnorm_quantize)


class SvdqW4A4Linear:
    """Y = Q(X_hat) Q(R)^T + (X_hat L1) L2 + bias on prepared weights.

    Weights prepared with a per-tensor scale (``w_tscale``) make the layer two-level
    NVFP4: the activation's scale pair is ``act_scale`` (float32 [2], calibrated) or,
    when that is None, computed on the device for every call."""

    def __init__(self, weights: dict, bias: torch.Tensor | None, max_tokens: int,
                 act_scale: torch.Tensor | None = None):
        self.w = weights
        self.bias = bias
        self.two_level = weights.get("w_tscale") is not None
        self.act_scale = act_scale
        self._a_scale = (torch.empty(2, dtype=torch.float32, device=weights["w_codes"].device)
                         if self.two_level else None)
        self.fmt = weights["fmt"]
        self.N, self.K, self.r = weights["N"], weights["K"], weights["r"]
        dev = weights["w_codes"].device
        self.max_tokens = max_tokens
        self.codes = torch.empty(svdq_codes_bytes(self.fmt, max_tokens, self.K), dtype=torch.uint8,
                                 device=dev)
        self.scales = torch.empty(svdq_scales_bytes(self.fmt, max_tokens, self.K), dtype=torch.uint8,
                                  device=dev)
        # the down-projection's partial sums: at most 8 splits of max_tokens rows
        self.xl1 = (torch.empty(8 * max_tokens * self.r, dtype=torch.float32, device=dev)
                    if self.r else None)

    @classmethod
    def from_linear(cls, weight: torch.Tensor, bias: torch.Tensor | None, x_absmax: torch.Tensor,
                    rank: int, max_tokens: int, fmt: str = "nvfp4", two_level: bool = False,
                    act_scale: torch.Tensor | None = None):
        """From an nn.Linear's weight [N, K] bf16 (and bias [N] bf16 or None) and the
        calibration activations' per-channel max |X| [K]: smoothing, SVD split and the
        residual quantized by the library (prep.prepare_svdq_weights)."""
        w = prep.prepare_svdq_weights(weight, x_absmax, rank, fmt, two_level=two_level)
        return cls(w, bias, max_tokens, act_scale=act_scale)

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        M = x.shape[0]
        if M > self.max_tokens:
            raise ValueError(f"{M} tokens > workspace for {self.max_tokens}")
        xl1 = self.xl1[:svdq_xl1_splits(M, self.K, self.r) * M * self.r] if self.r else None
        if self.two_level:
            a_scale = self.act_scale
            if a_scale is None:
                a_scale = svdq_tensor_scale(x, self.w["smooth_inv"], self._a_scale, stream=stream)
            codes, scales, xl1 = svdq_quantize_act_two_level(
                x, a_scale, self.w["L1s"], self.w["smooth_inv"], codes=self.codes, scales=self.scales,
                xl1=xl1, stream=stream)
            return svdq_w4a4_linear_two_level(codes, scales, a_scale, xl1, self.w["w_codes"],
                                              self.w["w_scales"], self.w["w_tscale"], self.w["L2"],
                                              self.bias, M, self.N, self.K, Y=y, stream=stream)
        codes, scales, xl1 = svdq_quantize_act(x, self.w["L1s"], self.w["smooth_inv"], fmt=self.fmt,
                                               codes=self.codes, scales=self.scales, xl1=xl1,
                                               stream=stream)
        return svdq_w4a4_linear(codes, scales, xl1, self.w["w_codes"], self.w["w_scales"], self.w["L2"],
                                self.bias, M, self.N, self.K, fmt=self.fmt, Y=y, stream=stream)

    __call__ = forward


class SvdqQkvNormRope(SvdqW4A4Linear):
    """The fused QKV projection of an attention block (Diffusers blog, the fused QKV
    section: to_q, to_k, to_v joined into one SVDQ linear, followed by norm_q / norm_k
    per head and the rotary embedding in one fused call). Weights prepared for the
    joined [3 H 128, K] projection, NVFP4, one-level; norm_q, norm_k bf16 [128] or None.
    forward(x, rope_cos, rope_sin) takes the rows' angle tables, float32 [64, M] each,
    angle-major (or None: no rotation), and returns Q | K | V [M, 3 H 128], Q and K
    normalised and rotated."""

    def __init__(self, weights: dict, bias: torch.Tensor | None, max_tokens: int,
                 norm_q: torch.Tensor | None = None, norm_k: torch.Tensor | None = None,
                 eps: float = 1e-6):
        if weights["fmt"] != "nvfp4" or weights.get("w_tscale") is not None:
            raise ValueError("the fused QKV projection takes one-level NVFP4 weights")
        if weights["N"] % 384:
            raise ValueError(f"N = {weights['N']} is not Q, K, V of whole 128-column heads")
        super().__init__(weights, bias, max_tokens)
        self.norm_q, self.norm_k, self.eps = norm_q, norm_k, float(eps)
        self.heads = weights["N"] // 384

    @classmethod
    def from_linears(cls, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     biases: tuple | None, x_absmax: torch.Tensor, rank: int, max_tokens: int,
                     norm_q: torch.Tensor | None = None, norm_k: torch.Tensor | None = None,
                     eps: float = 1e-6):
        """From the to_q, to_k, to_v weights [H 128, K] bf16 (biases: three [H 128] bf16
        tensors or None each, or None): the three are joined along the output dimension
        in the order Q, K, V into one [3 H 128, K] projection, which is prepared once
        (smoothing from x_absmax, SVD split, quantized residual)."""
        if not (q.shape == k.shape == v.shape) or q.dim() != 2 or q.shape[0] % 128:
            raise ValueError("to_q, to_k, to_v must be equal [H 128, K] weights")
        w = torch.cat([q, k, v], dim=0)
        bias = None
        if biases is not None and any(b is not None for b in biases):
            bias = torch.cat([b if b is not None else torch.zeros(q.shape[0], dtype=q.dtype, device=q.device)
                              for b in biases])
        return cls.from_linear(w, bias, x_absmax, rank, max_tokens, norm_q=norm_q, norm_k=norm_k, eps=eps)

    @classmethod
    def from_linear(cls, weight: torch.Tensor, bias: torch.Tensor | None, x_absmax: torch.Tensor,
                    rank: int, max_tokens: int, norm_q: torch.Tensor | None = None,
                    norm_k: torch.Tensor | None = None, eps: float = 1e-6):
        """From an already joined to_qkv weight [3 H 128, K] bf16 (rows Q, then K, then V)."""
        weights = prep.prepare_svdq_weights(weight, x_absmax, rank, "nvfp4")
        return cls(weights, bias, max_tokens, norm_q=norm_q, norm_k=norm_k, eps=eps)

    def forward(self, x: torch.Tensor, rope_cos: torch.Tensor | None = None,
                rope_sin: torch.Tensor | None = None, y: torch.Tensor | None = None,
                stream=None, rotary: "RotaryEmbedding | None" = None,
                positions: torch.Tensor | None = None) -> torch.Tensor:
        """The angle tables, or a rotary embedding and the rows' positions to make them of."""
        M = x.shape[0]
        if rotary is not None or positions is not None:
            if rope_cos is not None or rope_sin is not None or rotary is None or positions is None:
                raise ValueError("give the tables, or a rotary embedding and positions")
            if not rotary.interleaved or rotary.rot_dim != 128:
                raise ValueError("the fused QKV projection turns adjacent pairs of whole 128-column heads")
            rope_cos, rope_sin = rotary.tables(positions, angle_major=True, stream=stream)
        if M > self.max_tokens:
            raise ValueError(f"{M} tokens > workspace for {self.max_tokens}")
        xl1 = self.xl1[:svdq_xl1_splits(M, self.K, self.r) * M * self.r] if self.r else None
        codes, scales, xl1 = svdq_quantize_act(x, self.w["L1s"], self.w["smooth_inv"], fmt="nvfp4",
                                               codes=self.codes, scales=self.scales, xl1=xl1,
                                               stream=stream)
        return svdq_w4a4_linear_qkv_norm_rope(codes, scales, xl1, self.w["w_codes"], self.w["w_scales"],
                                              self.w["L2"], self.bias, self.norm_q, self.norm_k,
                                              rope_cos, rope_sin, M, self.N, self.K, eps=self.eps, Y=y,
                                              stream=stream)

    __call__ = forward


class AwqW4A16Linear:
    def __init__(self, weights: dict, bias: torch.Tensor | None):
        self.w = weights
        self.bias = bias

    @classmethod
    def from_linear(cls, weight: torch.Tensor, bias: torch.Tensor | None):
        """From an nn.Linear's weight [N, K] bf16: asymmetric int4, group 64, packed
        (prep.prepare_awq_weights)."""
        return cls(prep.prepare_awq_weights(weight), bias)

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        return awq_w4a16_linear(x, self.w["qweight"], self.w["sz"], self.bias, self.w["N"], Y=y,
                                stream=stream)

    __call__ = forward


class RotaryEmbedding:
    """Rotary positions of heads: frequencies once (prep.rope_frequencies), then any rows'
    heads turned, or the tables of their angles. ``dims`` is the number of rotary columns,
    or one number per position axis (positions are then [M, axes]; with one axis also [M]);
    ``interleaved`` pairs adjacent columns, otherwise column i pairs with column
    i + (rotary columns) / 2."""

    def __init__(self, dims, base: float = 10000.0, interleaved: bool = False, scaling: str | None = None,
                 factor: float = 1.0, original_length: int | None = None, device="cuda"):
        freq, axis, self.scale = prep.rope_frequencies(dims, base, scaling, factor, original_length)
        self.rot_dim = 2 * freq.numel()
        self.axes = int(axis.max()) + 1
        self.interleaved = bool(interleaved)
        self.freq = freq.to(device)
        self.axis = axis.to(device) if self.axes > 1 else None  # one axis: the library's default

    def _check(self, positions: torch.Tensor):
        # the library gives NaN on an axis that the positions do not have
        if (positions.shape[1] if positions.dim() == 2 else 1) != self.axes:
            raise ValueError(f"positions must be [M, {self.axes}]" + (" or [M]" if self.axes == 1 else "")
                             + f", not {list(positions.shape)}")

    def tables(self, positions: torch.Tensor, angle_major: bool = False, cos=None, sin=None, stream=None):
        """(cos, sin) float32 [M, pairs], or [pairs, M] with angle_major (SvdqQkvNormRope's)."""
        self._check(positions)
        return svdq_rope_table(positions, self.freq, axis=self.axis, scale=self.scale, angle_major=angle_major,
                               cos=cos, sin=sin, stream=stream)

    def forward(self, x: torch.Tensor, positions: torch.Tensor, y: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """x [M, heads, D] turned; y may be x."""
        self._check(positions)
        return svdq_rope(x, positions, self.freq, axis=self.axis, scale=self.scale, interleaved=self.interleaved,
                         Y=y, stream=stream)

    __call__ = forward


class _Buffers:
    """What an 8-bit layer holds between its calls, made once. It serves the thread and stream that made the
    layer: there one forward's calls follow another's. A forward on another stream or thread, or in a
    capture, whose replays may meet either, gets buffers of its own from its stream's (a graph's own)
    pool, so that any number of them may run at once."""

    def _own(self, device: torch.device) -> None:
        self._home = None
        if device.type == "cuda":
            with torch.cuda.device(device):
                self._home = threading.get_ident(), _stream(None)

    def _at_home(self, stream) -> bool:
        if self._home is None:
            return True
        thread, home = self._home
        return (_stream(stream) == home and threading.get_ident() == thread
                and (home == 0 or not torch.cuda.is_current_stream_capturing()))  # (the default stream cannot capture)


class W8A8Linear(_Buffers):
    """Y = act(X W^T + bias) + residual with E4M3 rows of X and W (w8a8_quantize_act,
    w8a8_linear). Y, and so the residual, is bf16 or float32 (out_dtype). One instance may be called on
    several streams and threads at once."""

    def __init__(self, weights: dict, bias: torch.Tensor | None, max_tokens: int, activation: str | None = None,
                 out_dtype: torch.dtype = torch.bfloat16):
        self.w, self.bias, self.activation, self.out_dtype = weights, bias, activation, out_dtype
        dev = weights["codes"].device
        self.max_tokens = max_tokens
        self.codes = torch.empty((max_tokens, weights["K"]), dtype=torch.float8_e4m3fn, device=dev)
        self.scale = torch.empty(max_tokens, dtype=torch.float32, device=dev)
        self._own(dev)

    @classmethod
    def from_linear(cls, weight: torch.Tensor, bias: torch.Tensor | None, max_tokens: int,
                    activation: str | None = None, out_dtype: torch.dtype = torch.bfloat16):
        """From an nn.Linear's weight [N, K] bf16 and bias [N] bf16 or None."""
        return cls(prep.prepare_w8a8_weights(weight), bias, max_tokens, activation, out_dtype)

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, y: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        M = x.shape[0]
        if M > self.max_tokens:
            raise ValueError(f"{M} tokens > workspace for {self.max_tokens}")
        kept = (self.codes[:M], self.scale[:M]) if self._at_home(stream) else (None, None)
        codes, scale = w8a8_quantize_act(x, codes=kept[0], scale=kept[1], stream=stream)
        return self.forward_quantized(codes, scale, residual, y, stream)

    def forward_quantized(self, codes: torch.Tensor, scale: torch.Tensor, residual: torch.Tensor | None = None,
                          y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The product alone, on rows quantized already (by a norm that feeds several layers, say)."""
        return w8a8_linear(codes, scale, self.w["codes"], self.w["scale"], self.bias, residual=residual,
                           activation=self.activation, out_dtype=self.out_dtype, Y=y, stream=stream)

    __call__ = forward


class W8A8GatedMlp(_Buffers):
    """A pre-norm gated feed-forward block in 8 bits, on the residual stream:
    h = x (+ residual);  out = h + down(act(gate(norm(h))) * up(norm(h))), four calls:
    norm into E4M3, the gated product, its rows into E4M3, the second projection with h added in its
    epilogue. ``up`` holds the F gate rows and then the F up rows [2F, K]; ``down`` [K, F].
    The hidden rows pass through bf16 on their way into E4M3 (their scale needs the whole
    row, which no tile of the product holds): 2^-8 of a value beside E4M3's 2^-4. ``up_bias`` [2F] and
    ``down_bias`` [K] are bf16 or None. The stream is bf16 or float32, out of its type. One instance may
    be called on several streams and threads at once."""

    def __init__(self, up: dict, down: dict, norm: torch.Tensor | None, max_tokens: int, activation: str = "silu",
                 eps: float = 1e-6, up_bias: torch.Tensor | None = None, down_bias: torch.Tensor | None = None):
        if up["N"] != 2 * down["K"] or up["K"] != down["N"]:
            raise ValueError("up must be [2F, K] and down [K, F]")
        self.up, self.down, self.norm = up, down, norm
        self.up_bias, self.down_bias = up_bias, down_bias
        self.activation, self.eps = activation, float(eps)
        dev = up["codes"].device
        K, F = up["K"], down["K"]
        self.max_tokens = max_tokens
        self.codes = torch.empty((max_tokens, K), dtype=torch.float8_e4m3fn, device=dev)
        self.hidden = torch.empty((max_tokens, F), dtype=torch.bfloat16, device=dev)
        self.hidden_codes = torch.empty((max_tokens, F), dtype=torch.float8_e4m3fn, device=dev)
        self.scale = torch.empty((2, max_tokens), dtype=torch.float32, device=dev)
        self._own(dev)

    @classmethod
    def from_linears(cls, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, norm: torch.Tensor | None,
                     max_tokens: int, activation: str = "silu", eps: float = 1e-6,
                     gate_bias: torch.Tensor | None = None, up_bias: torch.Tensor | None = None,
                     down_bias: torch.Tensor | None = None):
        """From the gate, up [F, K] and down [K, F] weights, bf16; norm [K] bf16 or None; biases bf16 or
        None, of gate and up both or neither."""
        if gate.shape != up.shape:
            raise ValueError("gate and up must be equal [F, K] weights")
        if (gate_bias is None) != (up_bias is None):
            raise ValueError("gate and up have a bias both or neither")
        return cls(prep.prepare_w8a8_weights(torch.cat([gate, up])), prep.prepare_w8a8_weights(down), norm,
                   max_tokens, activation, eps, None if gate_bias is None else torch.cat([gate_bias, up_bias]), down_bias)

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, y: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """x (and residual) [M, K] bf16 or float32 -> [M, K] of its type; with a residual, y (or a new tensor)
        also holds h between the calls. y may be x or residual."""
        M = x.shape[0]
        if M > self.max_tokens:
            raise ValueError(f"{M} tokens > workspace for {self.max_tokens}")
        if self._at_home(stream):
            codes, scale, hidden = self.codes[:M], self.scale[:, :M], self.hidden[:M]
            hidden_codes = self.hidden_codes[:M]
        else:
            codes, scale, hidden, hidden_codes = None, (None, None), None, None
        codes, s, h = w8a8_rmsnorm_quantize(x, self.norm, residual, eps=self.eps, codes=codes, scale=scale[0],
                                            residual_out=None if residual is None else y, stream=stream)
        hidden = w8a8_gated_linear(codes, s, self.up["codes"], self.up["scale"], self.up_bias,
                                   activation=self.activation, Y=hidden, stream=stream)
        codes, s = w8a8_quantize_act(hidden, codes=hidden_codes, scale=scale[1], stream=stream)
        h = x if h is None else h
        return w8a8_linear(codes, s, self.down["codes"], self.down["scale"], self.down_bias, residual=h,
                           out_dtype=x.dtype, Y=h if residual is not None else y, stream=stream)

    __call__ = forward
