"""The operators around the layer: binding of their C entry points.

Residual-stream norms (``moe_block_norm``) and the router's per-sequence balance
loss (``moe_balance_loss``), each with its backward, and microscaled 4-bit
numbers with the experts' grouped product (``moe_mx4_*``).  As in the
package's root, every function mirrors the C entry point of the same name and
the classes own the output buffers and workspaces of one configuration.  What a
call with ``stream`` allocates belongs to that stream: another stream that uses it
waits for that one first, and tells the allocator (``record_stream``) before it is
dropped.
"""
from __future__ import annotations

import ctypes

import torch

import top_routing_expert_moe_gb300 as _moe
from .mx8 import MX8Tensor

__all__ = ["GATE_NONE", "GATE_CHANNEL", "GATE_TOKEN", "GATE_FULL", "NormConfig",
           "check_norm_config", "norm_workspace_size", "moe_block_norm", "moe_block_norm_mx8",
           "moe_block_norm_backward", "BlockNorm", "BalanceConfig", "check_balance_config",
           "balance_workspace_size", "moe_balance_loss", "moe_balance_loss_backward",
           "BalanceLoss", "MX4_ACT_NONE", "MX4_ACT_SILU", "MX4_ACT_SWIGLU", "MX4Tensor",
           "mx4_scale_bytes", "moe_mx4_quantize", "moe_mx4_quantize_weight", "moe_mx4_dequantize",
           "mx4_quantize", "mx4_quantize_weight", "MX4ProductConfig", "check_mx4_product_config",
           "moe_mx4_grouped_product", "MX4Product", "MX4Experts", "MoEBlock"]

GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3

_p, _s, _on, _call = _moe._p, _moe._s, _moe._on, _moe._call


def _checked(t, shape, dtype, name):
    """The tensor, after a check of its shape and type (None passes)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    return t


# ----------------------------------------------------------------- residual stream
class NormConfig(ctypes.Structure):
    """Mirror of ``moe_norm_config`` (include/moe.h)."""
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("leave", ctypes.c_int32), ("post_norm", ctypes.c_int32),
                ("enter", ctypes.c_int32), ("gate", ctypes.c_int32), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float), ("out_scale", ctypes.c_float)]

    def __init__(self, T, d, dtype=_moe.BF16, leave=1, post_norm=0, enter=1, gate=GATE_NONE,
                 eps=1e-6, res_scale=1.0, out_scale=1.0):
        super().__init__(T, d, dtype, int(leave), int(post_norm), int(enter), gate, eps, res_scale,
                         out_scale)

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == _moe.BF16 else torch.float32

    @property
    def gate_shape(self):
        """(shape, dtype) of the gate, or None."""
        return {GATE_NONE: None, GATE_CHANNEL: ((self.d,), torch.float32),
                GATE_TOKEN: ((self.T,), torch.float32),
                GATE_FULL: ((self.T, self.d), self.torch_dtype)}[self.gate]


def check_norm_config(cfg: NormConfig) -> int:
    return _moe.load_library().moe_check_norm_config(ctypes.byref(cfg))


def norm_workspace_size(cfg: NormConfig) -> int:
    v = ctypes.c_size_t()
    _call("moe_norm_workspace_size", ctypes.byref(cfg), ctypes.byref(v))
    return v.value


def moe_block_norm(cfg, x, u, w_post, gate, w_pre, x_out, z, stream=None):
    _call("moe_block_norm", ctypes.byref(cfg), _p(x), _p(u), _p(w_post), _p(gate), _p(w_pre),
          _p(x_out), _p(z), _s(stream))


def moe_block_norm_mx8(cfg, x, u, w_post, gate, w_pre, x_out, z, codes, scales, stream=None):
    _call("moe_block_norm_mx8", ctypes.byref(cfg), _p(x), _p(u), _p(w_post), _p(gate), _p(w_pre),
          _p(x_out), _p(z), _p(codes), _p(scales), _s(stream))


def moe_block_norm_backward(cfg, x_out, u, w_post, gate, w_pre, dx_out, dz, dx, du, dw_post, dgate,
                            dw_pre, ws, stream=None):
    _call("moe_block_norm_backward", ctypes.byref(cfg), _p(x_out), _p(u), _p(w_post), _p(gate),
          _p(w_pre), _p(dx_out), _p(dz), _p(dx), _p(du), _p(dw_post), _p(dgate), _p(dw_pre),
          _p(ws), _s(stream))


class BlockNorm:
    """One place on the residual stream: leaving a block (normalise its output
    u, gate it, scale it, add it to the stream x), entering the next (the
    normalised copy z), or both in one pass.  Owns its outputs and workspace."""

    def __init__(self, cfg: NormConfig, device="cuda"):
        rc = check_norm_config(cfg)
        if rc != 0:
            raise _moe.MoEError(rc, "moe_check_norm_config")
        self.cfg = c = cfg
        self.device = torch.device(device)
        self._rows, self._vec, self._dt = (c.T, c.d), (c.d,), c.torch_dtype
        self._gate, self._leave = c.gate_shape, bool(c.leave)
        e = lambda on, *s, dtype=c.torch_dtype: (  # noqa: E731
            torch.empty(*s, dtype=dtype, device=self.device) if on else None)
        self.x_out = e(c.leave, c.T, c.d)
        self.z = e(c.enter, c.T, c.d)
        self.z8 = self._grads = self._ws = None

    def _check(self, rows, w_pre, w_post, gate):
        for n, t in rows:
            _checked(t, self._rows, self._dt, n)
        _checked(w_pre, self._vec, torch.float32, "w_pre")
        _checked(w_post, self._vec, torch.float32, "w_post")
        if self._gate is not None:
            _checked(gate, *self._gate, "gate")
        elif gate is not None:
            raise ValueError("gate given, but the configuration has none")

    def forward(self, x, u=None, w_pre=None, w_post=None, gate=None, stream=None):
        """(x_out, z): the stream after the block (x itself without ``leave``)
        and its normalised copy (None without ``enter``)."""
        self._check((("x", x), ("u", u)), w_pre, w_post, gate)
        moe_block_norm(self.cfg, x, u, w_post, gate, w_pre, self.x_out, self.z, stream)
        return (self.x_out if self._leave else x), self.z

    def forward_mx8(self, x, u=None, w_pre=None, w_post=None, gate=None, keep_z=True, stream=None):
        """(x_out, z8, z): forward() with the normalised copy in 8 bits, an MX8Tensor, and
        beside it z itself (None unless ``keep_z``).  Needs ``enter`` and a width of whole
        32s; the backward is that of the unquantised z."""
        c = self.cfg
        if not c.enter:
            raise ValueError("forward_mx8 needs a configuration that enters a block")
        self._check((("x", x), ("u", u)), w_pre, w_post, gate)
        if self.z8 is None:
            with _on(stream):
                self.z8 = MX8Tensor((c.T, c.d), self.device)
        z = self.z if keep_z else None
        _call("moe_block_norm_mx8", ctypes.byref(c), _p(x), _p(u), _p(w_post), _p(gate), _p(w_pre),
              _p(self.x_out), _p(z), *self.z8.ptrs, _s(stream))
        return (self.x_out if self._leave else x), self.z8, z

    def grads(self):
        if self._grads is None:
            c = self.cfg
            e = lambda on, *s, dtype=c.torch_dtype: (  # noqa: E731
                torch.empty(*s, dtype=dtype, device=self.device) if on else None)
            f32 = torch.float32
            self._grads = dict(dx=e(1, c.T, c.d), du=e(c.leave, c.T, c.d),
                               dw_pre=e(c.enter, c.d, dtype=f32),
                               dw_post=e(c.post_norm, c.d, dtype=f32),
                               dgate=(e(1, *c.gate_shape[0], dtype=c.gate_shape[1])
                                      if c.gate != GATE_NONE else None))
            self._ws = torch.empty(max(norm_workspace_size(c), 256), dtype=torch.uint8,
                                   device=self.device)
        return self._grads

    def backward(self, x_out, dx_out=None, dz=None, u=None, w_pre=None, w_post=None, gate=None,
                 stream=None):
        """Gradients dx, du, dw_pre, dw_post, dgate (None where absent) at the
        stored stream x_out (x where the configuration does not leave a block),
        given those of x_out along the stream (None: zero) and of z."""
        self._check((("x_out", x_out), ("dx_out", dx_out), ("dz", dz), ("u", u)), w_pre, w_post, gate)
        with _on(stream):
            g = self.grads()
        moe_block_norm_backward(self.cfg, x_out, u, w_post, gate, w_pre, dx_out, dz, g["dx"],
                                g["du"], g["dw_post"], g["dgate"], g["dw_pre"], self._ws, stream)
        return g


# ----------------------------------------------------------------- balance loss
class BalanceConfig(ctypes.Structure):
    """Mirror of ``moe_balance_config`` (include/moe.h)."""
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("S", ctypes.c_int32), ("balance_coef", ctypes.c_float),
                ("z_coef", ctypes.c_float), ("temperature", ctypes.c_float)]

    def __init__(self, T, E, k, S=1, balance_coef=0.01, z_coef=0.0, temperature=1.0):
        super().__init__(T, E, k, S, balance_coef, z_coef, temperature)


def check_balance_config(cfg: BalanceConfig) -> int:
    return _moe.load_library().moe_check_balance_config(ctypes.byref(cfg))


def balance_workspace_size(cfg: BalanceConfig) -> int:
    v = ctypes.c_size_t()
    _call("moe_balance_workspace_size", ctypes.byref(cfg), ctypes.byref(v))
    return v.value


def moe_balance_loss(cfg, logits, topk_idx, seq_offsets, loss, counts, pbar, grad_w, ws, stream=None):
    _call("moe_balance_loss", ctypes.byref(cfg), _p(logits), _p(topk_idx), _p(seq_offsets),
          _p(loss), _p(counts), _p(pbar), _p(grad_w), _p(ws), _s(stream))


def moe_balance_loss_backward(cfg, logits, topk_idx, seq_offsets, grad_w, dloss, dlogits, stream=None):
    _call("moe_balance_loss_backward", ctypes.byref(cfg), _p(logits), _p(topk_idx),
          _p(seq_offsets), _p(grad_w), _p(dloss), _p(dlogits), _s(stream))


class BalanceLoss:
    """The router's balance and z losses over sequences.  ``forward`` returns
    loss [3] (their sum, balance, z) and fills ``counts`` and ``pbar`` [S, E];
    ``backward`` returns the gradient on the logits, for
    ``MoELayer.backward(dout, dlogits_aux=...)``."""

    def __init__(self, cfg: BalanceConfig, device="cuda"):
        rc = check_balance_config(cfg)
        if rc != 0:
            raise _moe.MoEError(rc, "moe_check_balance_config")
        self.cfg, dev = cfg, torch.device(device)
        self._logits, self._topk, self._offsets = (cfg.T, cfg.E), (cfg.T, cfg.k), (cfg.S + 1,)
        e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        self.loss = e(3)
        self.counts = e(cfg.S, cfg.E, dtype=torch.int32)
        self.pbar = e(cfg.S, cfg.E)
        self.grad_w = e(cfg.S, cfg.E + 2)
        self.dlogits = e(cfg.T, cfg.E)
        self.ws = e(max(balance_workspace_size(cfg), 256), dtype=torch.uint8)
        self._inputs = None

    def forward(self, logits, topk_idx, seq_offsets=None, stream=None):
        c = self.cfg
        _checked(logits, self._logits, torch.float32, "logits")
        _checked(topk_idx, self._topk, torch.int32, "topk_idx")
        _checked(seq_offsets, self._offsets, torch.int32, "seq_offsets")
        moe_balance_loss(c, logits, topk_idx, seq_offsets, self.loss, self.counts, self.pbar,
                         self.grad_w, self.ws, stream)
        self._inputs = (logits, topk_idx, seq_offsets)
        return self.loss

    def backward(self, dloss=None, stream=None):
        """dlogits [T, E] of the last forward, times ``dloss`` (one fp32 on the
        device; None: 1)."""
        if self._inputs is None:
            raise RuntimeError("backward() needs a forward() first")
        if dloss is not None and (dloss.numel() != 1 or dloss.dtype != torch.float32):
            raise ValueError("dloss must be one fp32")
        logits, topk_idx, seq_offsets = self._inputs
        moe_balance_loss_backward(self.cfg, logits, topk_idx, seq_offsets, self.grad_w, dloss,
                                  self.dlogits, stream)
        return self.dlogits


# ----------------------------------------------------------------- microscaled 4-bit numbers
MX4_ACT_NONE, MX4_ACT_SILU, MX4_ACT_SWIGLU = 0, 1, 2


def mx4_scale_bytes(rows: int, K: int) -> int:
    v = ctypes.c_size_t()
    _call("moe_mx4_scale_bytes", rows, K, ctypes.byref(v))
    return v.value


def moe_mx4_quantize(dtype, rows, K, x, rows_used, codes, scales, stream=None):
    _call("moe_mx4_quantize", dtype, rows, K, _p(x), _p(rows_used), _p(codes), _p(scales), _s(stream))


def moe_mx4_quantize_weight(dtype, E, K, N, W, codes, scales, stream=None):
    _call("moe_mx4_quantize_weight", dtype, E, K, N, _p(W), _p(codes), _p(scales), _s(stream))


def moe_mx4_dequantize(dtype, sets, rows, K, codes, scales, out, stream=None):
    _call("moe_mx4_dequantize", dtype, sets, rows, K, _p(codes), _p(scales), _p(out), _s(stream))


_MX4_DTYPES = {torch.bfloat16: _moe.BF16, torch.float32: _moe.F32}


def _mx4_dtype(dtype) -> int:
    code = _MX4_DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"expected bfloat16 or float32, got {dtype}")
    return code


class MX4Tensor:
    """4-bit numbers [rows, K] or, for expert weights, [E, rows, K]: ``codes``
    (two to a byte) and ``scales`` (tiles, see include/moe.h)."""

    def __init__(self, shape, device="cuda"):
        shape = tuple(shape)
        if len(shape) not in (2, 3):
            raise ValueError("expected [rows, K] or [E, rows, K]")
        sets, (rows, K) = (shape[0] if len(shape) == 3 else 1), shape[-2:]
        if rows < 1 or K < 1 or K % 32:
            mx4_scale_bytes(rows, K)                 # raises
        self.shape = shape
        # moe_mx4_scale_bytes, without the call
        n = sets * ((rows + 127) // 128) * ((K + 127) // 128) * 512
        self.codes = torch.empty((*shape[:-1], K // 2), dtype=torch.uint8, device=device)
        self.scales = torch.empty(n, dtype=torch.uint8, device=device)

    def dequantize(self, dtype=torch.bfloat16, stream=None):
        code = _mx4_dtype(dtype)
        with _on(stream):
            out = torch.empty(self.shape, dtype=dtype, device=self.codes.device)
        sets = self.shape[0] if len(self.shape) == 3 else 1
        moe_mx4_dequantize(code, sets, self.shape[-2], self.shape[-1], self.codes, self.scales, out,
                           stream)
        return out


def mx4_quantize(x, rows_used=None, out=None, stream=None) -> MX4Tensor:
    """Quantise rows x [rows, K] along K (K a multiple of 32) into ``out`` or a new
    tensor.  ``rows_used``: one int32 on the device, rows from it on are left out."""
    if x.dim() != 2:
        raise ValueError("x: expected [rows, K]")
    code = _mx4_dtype(x.dtype)
    if out is None:
        with _on(stream):
            out = MX4Tensor(x.shape, x.device)
    elif out.shape != x.shape:
        raise ValueError(f"out: expected {tuple(x.shape)}, got {out.shape}")
    if rows_used is not None and (rows_used.numel() != 1 or rows_used.dtype != torch.int32):
        raise ValueError("rows_used must be one int32")
    moe_mx4_quantize(code, x.shape[0], x.shape[1], x, rows_used, out.codes, out.scales, stream)
    return out


def _quantize_segments(x, offsets, E, out, stream):
    """mx4_quantize of the rows below offsets[E] (a view of it would cost more than the call)."""
    _call("moe_mx4_quantize", _mx4_dtype(x.dtype), x.shape[0], x.shape[1], _p(x), _p(offsets) + 4 * E,
          _p(out.codes), _p(out.scales), _s(stream))


def mx4_quantize_weight(W, stream=None) -> MX4Tensor:
    """Quantise expert weights W [E, K, N] along K: an MX4Tensor [E, N, K]."""
    if W.dim() != 3:
        raise ValueError("W: expected [E, K, N]")
    E, K, N = W.shape
    code = _mx4_dtype(W.dtype)
    with _on(stream):
        out = MX4Tensor((E, N, K), W.device)
    moe_mx4_quantize_weight(code, E, K, N, W, out.codes, out.scales, stream)
    return out


class MX4ProductConfig(ctypes.Structure):
    """Mirror of ``moe_mx4_product_config`` (include/moe.h)."""
    _fields_ = [("rows", ctypes.c_int64), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
                ("E", ctypes.c_int32), ("act", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]

    def __init__(self, rows, K, N, E, act=MX4_ACT_NONE, out_dtype=_moe.BF16):
        super().__init__(rows, K, N, E, act, out_dtype)

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.out_dtype == _moe.BF16 else torch.float32


def check_mx4_product_config(cfg: MX4ProductConfig) -> int:
    return _moe.load_library().moe_check_mx4_product_config(ctypes.byref(cfg))


def moe_mx4_grouped_product(cfg, x_codes, x_scales, offsets, w_codes, w_scales, wg_codes, wg_scales,
                            out, stream=None):
    _call("moe_mx4_grouped_product", ctypes.byref(cfg), _p(x_codes), _p(x_scales), _p(offsets),
          _p(w_codes), _p(w_scales), _p(wg_codes), _p(wg_scales), _p(out), _s(stream))


class MX4Product:
    """out = act(Q(x) Q(W_e)) over expert segments: quantises the rows of x and
    multiplies them with weights from ``mx4_quantize_weight``.  Owns the 4-bit
    rows and the output."""

    def __init__(self, cfg: MX4ProductConfig, device="cuda"):
        rc = check_mx4_product_config(cfg)
        if rc != 0:
            raise _moe.MoEError(rc, "moe_check_mx4_product_config")
        self.cfg = cfg
        self._x, self._offsets, self._w = (cfg.rows, cfg.K), (cfg.E + 1,), (cfg.E, cfg.N, cfg.K)
        self._dual = cfg.act == MX4_ACT_SWIGLU
        self.xq = MX4Tensor(self._x, device)
        self.out = torch.empty(cfg.rows, cfg.N, dtype=cfg.torch_dtype, device=device)

    def forward(self, x, offsets, w: MX4Tensor, wg: MX4Tensor | None = None, stream=None):
        """out [rows, N] (rows from offsets[E] on are not written); x [rows, K] bf16
        or fp32, offsets [E + 1] int32 as from moe_permute, w (and the gate wg for
        SwiGLU) [E, N, K]."""
        c = self.cfg
        if x.shape != self._x:
            raise ValueError(f"x: expected {self._x}, got {tuple(x.shape)}")
        _checked(offsets, self._offsets, torch.int32, "offsets")
        if (wg is not None) != self._dual:
            raise ValueError("wg is required iff act is MX4_ACT_SWIGLU")
        for t, n in ((w, "w"), (wg, "wg")):
            if t is not None and t.shape != self._w:
                raise ValueError(f"{n}: expected {self._w}, got {t.shape}")
        _quantize_segments(x, offsets, c.E, self.xq, stream)
        moe_mx4_grouped_product(c, self.xq.codes, self.xq.scales, offsets, w.codes, w.scales,
                                wg.codes if wg else None, wg.scales if wg else None, self.out, stream)
        return self.out


class MX4Experts:
    """A layer's expert weights in 4 bits, for ``MoELayer.forward_mx4``: quantised
    once from W_up, W_gate (SwiGLU) [E, d, f] and W_down [E, f, d]."""

    def __init__(self, W_up, W_down, W_gate=None, stream=None):
        self.up = mx4_quantize_weight(W_up, stream)
        self.down = mx4_quantize_weight(W_down, stream)
        self.gate = mx4_quantize_weight(W_gate, stream) if W_gate is not None else None


# ----------------------------------------------------------------- the block
class MoEBlock:
    """The layer in its place on the residual stream:

        z = w_in x / rms(x);  u = MoE(z);  n = w_out u / rms(u)  (or u)
        x' = res_scale x + out_scale g n,   and the router's balance loss

    ``weights`` of forward(): w_in [d] fp32, W_r, W_up, W_down and, where the
    configuration has them, W_gate, bias, w_out [d] fp32, gate (see NormConfig),
    shared (as MoELayer.forward takes it).  backward() returns the gradients by
    the same names with a "d" before (dx too).  x may be the block's own last
    output (weights shared along the depth): x' then goes to a second buffer, and
    backward() is that of the last forward(), as always."""

    def __init__(self, cfg, post_norm=0, gate=GATE_NONE, eps=1e-6, res_scale=1.0, out_scale=1.0,
                 sequences=1, balance_coef=0.01, z_coef=0.0, device="cuda"):
        c = cfg
        self.layer = _moe.MoELayer(cfg, device)
        self.enter = BlockNorm(NormConfig(c.T, c.d, c.dtype, leave=0, eps=eps), device)
        self.leave = BlockNorm(NormConfig(c.T, c.d, c.dtype, post_norm=post_norm, enter=0, gate=gate,
                                          eps=eps, res_scale=res_scale, out_scale=out_scale), device)
        self.balance = BalanceLoss(BalanceConfig(c.T, c.E, c.k, sequences, balance_coef, z_coef,
                                                 c.temperature), device)
        self._saved = self._other = None

    def forward(self, x, weights, seq_offsets=None, noise=None, token_mask=None, stream=None):
        """(x', loss [3]): the stream after the block and the router's losses."""
        w = weights
        self._saved = None            # the layer's buffers are this forward's from here on
        z = self.enter.forward(x, w_pre=w["w_in"], stream=stream)[1]
        u = self.layer.forward(z, w["W_r"], w["W_up"], w["W_down"], w.get("W_gate"), w.get("bias"),
                               noise, token_mask, stream, shared=w.get("shared"))
        if x.data_ptr() == self.leave.x_out.data_ptr():
            # backward() reads x, so x' may not be written over it
            if self._other is None:
                with _on(stream):
                    self._other = torch.empty_like(x)
            self.leave.x_out, self._other = self._other, self.leave.x_out
        x_out = self.leave.forward(x, u=u, w_post=w.get("w_out"), gate=w.get("gate"), stream=stream)[0]
        loss = self.balance.forward(self.layer.logits, self.layer.topk_idx, seq_offsets, stream)
        self._saved = (x, u, w)
        return x_out, loss

    def forward_mx4(self, x, weights, experts: MX4Experts, token_mask=None, stream=None):
        """x' with the experts in 4 bits (serving: no loss, no backward)."""
        w = weights
        self._saved = None
        z = self.enter.forward(x, w_pre=w["w_in"], stream=stream)[1]
        u = self.layer.forward_mx4(z, w["W_r"], experts, w.get("bias"), token_mask=token_mask, stream=stream)
        return self.leave.forward(x, u=u, w_post=w.get("w_out"), gate=w.get("gate"), stream=stream)[0]

    def forward_mx8(self, x, weights, experts, token_mask=None, stream=None):
        """x' with the experts in 8 bits, an MX8Experts (serving: no loss, no backward): the
        norm writes their rows in 8 bits beside the router's in 16."""
        w = weights
        self._saved = None
        z8, z = self.enter.forward_mx8(x, w_pre=w["w_in"], stream=stream)[1:]
        u = self.layer.forward_mx8(z, w["W_r"], experts, w.get("bias"), token_mask=token_mask, stream=stream, x8=z8)
        return self.leave.forward(x, u=u, w_post=w.get("w_out"), gate=w.get("gate"), stream=stream)[0]

    def backward(self, dx_out, dloss=None, stream=None):
        """Gradients of <dx_out, x'> + dloss (balance + z) (dloss None: 1)."""
        if self._saved is None:
            raise RuntimeError("backward() needs a forward() first")
        x, u, w = self._saved
        # the leave norm's gradients do not depend on x': it is not normalised there
        gl = self.leave.backward(self.leave.x_out, dx_out=dx_out, u=u, w_post=w.get("w_out"),
                                 gate=w.get("gate"), stream=stream)
        g = dict(self.layer.backward(gl["du"], stream, dlogits_aux=self.balance.backward(dloss, stream)))
        ge = self.enter.backward(x, dx_out=gl["dx"], dz=g["dx"], w_pre=w["w_in"], stream=stream)
        g.update(dx=ge["dx"], dw_in=ge["dw_pre"], dw_out=gl["dw_post"], dgate=gl["dgate"])
        return g
