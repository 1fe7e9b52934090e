"""The experts in 8 bits: binding of their C entry points.

Microscaled 8-bit numbers, the permutation of rows held in them
(``moe_permute_mx8``), the experts' grouped product over segments of any length
(``moe_mx8_grouped_product``), and the experts' forward and backward with their
activations kept in 8 bits (``moe_grouped_ffn_mx8``).  As in the package's root, every function mirrors the C entry
point of the same name and the classes own the output buffers and workspaces of one
configuration.  What a call with ``stream`` allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes

import torch

import top_routing_expert_moe_gb300 as _moe

__all__ = ["MX8Tensor", "MX8Weight", "mx8_weight_bytes", "moe_mx8_dequantize_weight", "mx8_scale_pitch", "moe_mx8_quantize", "moe_mx8_quantize_weight",
           "moe_mx8_dequantize", "mx8_quantize", "mx8_quantize_weight", "mx8_rows_capacity",
           "permute_mx8_workspace_size", "moe_permute_mx8", "MX8Dispatch", "MX8", "MX8_ACT_NONE",
           "MX8_ACT_SILU", "MX8_ACT_SWIGLU", "MX8ProductConfig", "check_mx8_product_config",
           "moe_mx8_grouped_product", "MX8Product", "MX8Experts", "moe_grouped_ffn_mx8",
           "moe_grouped_ffn_backward_mx8", "moe_backward_mx8", "MoECheckpoint"]

MX8 = 2                                              # an output type beside F32 and BF16
MX8_ACT_NONE, MX8_ACT_SILU, MX8_ACT_SWIGLU = 0, 1, 2

_p, _s, _on, _call = _moe._p, _moe._s, _moe._on, _moe._call
_current_device = torch.cuda.current_device


def _checked(t, shape, dtype, name):
    """The tensor, after a check of its shape and type."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    return t


def _checked8(t, shape, name, kind=None):
    kind = kind or MX8Tensor
    if not isinstance(t, kind):
        raise TypeError(f"{name}: expected an {kind.__name__}")
    if t.shape != tuple(shape):
        raise ValueError(f"{name}: expected {tuple(shape)}, got {t.shape}")
    return t


_NONE = (None, None)
_DTYPES = {torch.bfloat16: _moe.BF16, torch.float32: _moe.F32}


def _dtype(dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"expected bfloat16 or float32, got {dtype}")
    return code


def mx8_scale_pitch(K: int) -> int:
    v = ctypes.c_int32()
    _call("moe_mx8_scale_pitch", K, ctypes.byref(v))
    return v.value


def moe_mx8_quantize(dtype, rows, K, x, rows_used, codes, scales, stream=None):
    _call("moe_mx8_quantize", dtype, rows, K, _p(x), _p(rows_used), _p(codes), _p(scales), _s(stream))


def moe_mx8_quantize_weight(dtype, E, K, N, W, codes, scales, stream=None):
    _call("moe_mx8_quantize_weight", dtype, E, K, N, _p(W), _p(codes), _p(scales), _s(stream))


def moe_mx8_dequantize(dtype, rows, K, codes, scales, out, stream=None):
    _call("moe_mx8_dequantize", dtype, rows, K, _p(codes), _p(scales), _p(out), _s(stream))


def mx8_weight_bytes(E: int, K: int, N: int):
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    _call("moe_mx8_weight_bytes", E, K, N, ctypes.byref(c), ctypes.byref(s))
    return c.value, s.value


def moe_mx8_dequantize_weight(dtype, E, K, N, codes, scales, out, stream=None):
    _call("moe_mx8_dequantize_weight", dtype, E, K, N, _p(codes), _p(scales), _p(out), _s(stream))


class _Numbers:
    """``codes`` and ``scales`` of a set of 8-bit numbers: buffers that it holds for good, so that
    their addresses are looked up once."""

    def _hold(self, codes, scales):
        self._codes, self._scales = codes, scales
        self._device = codes.device
        self._ptrs = (codes.data_ptr(), scales.data_ptr()) if codes.is_cuda else None

    @property
    def codes(self):
        return self._codes

    @property
    def scales(self):
        return self._scales

    @property
    def ptrs(self):
        """Addresses of the codes and scales, for a call on the current device."""
        if self._ptrs is None:
            _p(self._codes)                          # raises: not on a GPU
        if self._device.index != _current_device():
            raise ValueError(f"the numbers are on {self._device}, which is not the current device")
        return self._ptrs


class MX8Tensor(_Numbers):
    """Rows of 8-bit numbers, [rows, K] or sets of them [sets, rows, K]: ``codes`` (e4m3, as
    bytes) of that shape and ``scales`` [..., pitch], one byte for 32 codes."""

    def __init__(self, shape, device="cuda"):
        shape = tuple(shape)
        if len(shape) not in (2, 3):
            raise ValueError("expected [rows, K] or [sets, rows, K]")
        K = shape[-1]
        if min(shape) < 1 or K % 32:
            mx8_scale_pitch(K)                       # raises for the width
            raise ValueError(f"expected sizes of 1 or more, got {shape}")
        self.shape = shape
        self._rows = shape[0] if len(shape) == 2 else shape[0] * shape[1]
        # moe_mx8_scale_pitch, without the call
        self._hold(torch.empty(shape, dtype=torch.uint8, device=device),
                   torch.empty((*shape[:-1], (K // 32 + 15) // 16 * 16), dtype=torch.uint8, device=device))

    def dequantize(self, dtype=torch.bfloat16, stream=None):
        code = _dtype(dtype)
        c, s = self.ptrs
        with _on(stream):
            out = torch.empty(self.shape, dtype=dtype, device=self._device)
        _call("moe_mx8_dequantize", code, self._rows, self.shape[-1], c, s, out.data_ptr(), _s(stream))
        return out


class MX8Weight(_Numbers):
    """Expert weights [E, N, K] in 8 bits (each expert's matrix transposed): ``codes`` and
    ``scales`` in blocks of 128 x 128, see include/moe.h."""

    def __init__(self, shape, device="cuda"):
        E, N, K = shape
        codes, scales = mx8_weight_bytes(E, K, N)
        self.shape = (E, N, K)
        self._hold(torch.empty(codes, dtype=torch.uint8, device=device),
                   torch.empty(scales, dtype=torch.uint8, device=device))

    def dequantize(self, dtype=torch.bfloat16, stream=None):
        E, N, K = self.shape
        code = _dtype(dtype)
        c, s = self.ptrs
        with _on(stream):
            out = torch.empty(self.shape, dtype=dtype, device=self._device)
        _call("moe_mx8_dequantize_weight", code, E, K, N, c, s, out.data_ptr(), _s(stream))
        return out


def mx8_quantize(x, rows_used=None, out=None, stream=None) -> MX8Tensor:
    """Quantise rows x [rows, K] along K (K a multiple of 32) into ``out`` or a new
    tensor.  ``rows_used``: one int32 on the device, rows from it on are left out."""
    if x.dim() != 2:
        raise ValueError("x: expected [rows, K]")
    code = _dtype(x.dtype)
    if out is None:
        with _on(stream):
            out = MX8Tensor(x.shape, x.device)
    else:
        _checked8(out, x.shape, "out")
    if rows_used is not None and (rows_used.numel() != 1 or rows_used.dtype != torch.int32):
        raise ValueError("rows_used must be one int32")
    _call("moe_mx8_quantize", code, x.shape[0], x.shape[1], _p(x), _p(rows_used), *out.ptrs, _s(stream))
    return out


def mx8_quantize_weight(W, stream=None) -> MX8Weight:
    """Quantise expert weights W [E, K, N] along K: an MX8Weight [E, N, K]."""
    if W.dim() != 3:
        raise ValueError("W: expected [E, K, N]")
    E, K, N = W.shape
    code = _dtype(W.dtype)
    with _on(stream):
        out = MX8Weight((E, N, K), W.device)
    _call("moe_mx8_quantize_weight", code, E, K, N, _p(W), *out.ptrs, _s(stream))
    return out


# ----------------------------------------------------------------- permutation
def mx8_rows_capacity(cfg) -> int:
    v = ctypes.c_int64()
    _call("moe_mx8_rows_capacity", ctypes.byref(cfg), ctypes.byref(v))
    return v.value


def permute_mx8_workspace_size(cfg) -> int:
    v = ctypes.c_size_t()
    _call("moe_permute_mx8_workspace_size", ctypes.byref(cfg), ctypes.byref(v))
    return v.value


def moe_permute_mx8(cfg, codes, scales, topk_idx, codes_perm, scales_perm, perm_token, slot_of, kept,
                    offsets, stats, ws, stream=None):
    _call("moe_permute_mx8", ctypes.byref(cfg), _p(codes), _p(scales), _p(topk_idx), _p(codes_perm),
          _p(scales_perm), _p(perm_token), _p(slot_of), _p(kept), _p(offsets), _p(stats), _p(ws),
          _s(stream))


class MX8Dispatch:
    """Rows in 8 bits to the experts that they go to: segments without padding,
    ``offsets`` [E + 1], for ``MX8Product``.  Owns the permuted rows, ``perm_token``
    (the token of each row), ``slot_of`` [T, k] (the row of each choice, -1 if dropped)
    and ``kept`` [E]."""

    def __init__(self, cfg, device="cuda"):
        ws = permute_mx8_workspace_size(cfg)          # raises for a bad configuration
        self.cfg, self.rows_cap = cfg, mx8_rows_capacity(cfg)
        e = lambda *s, dtype=torch.int32: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        self.rows = MX8Tensor((self.rows_cap, cfg.d), device)
        self.perm_token, self.slot_of = e(self.rows_cap), e(cfg.T, cfg.k)
        self.kept, self.offsets = e(cfg.E), e(cfg.E + 1)
        self.ws = e(max(ws, 256), dtype=torch.uint8)

    def forward(self, x: MX8Tensor, topk_idx, stats=None, stream=None) -> MX8Tensor:
        """The permuted rows of x [T, d] (those from offsets[E] on are left as they were)
        for topk_idx [T, k] int32, -1 where a token takes part in nothing."""
        c = self.cfg
        _checked8(x, (c.T, c.d), "x")
        if x is self.rows:
            raise ValueError("x: the rows that this dispatch writes")
        _checked(topk_idx, (c.T, c.k), torch.int32, "topk_idx")
        if stats is not None:
            _checked(stats, (9 + c.E,), torch.float32, "stats")
        _call("moe_permute_mx8", ctypes.byref(c), *x.ptrs, _p(topk_idx), *self.rows.ptrs, _p(self.perm_token),
              _p(self.slot_of), _p(self.kept), _p(self.offsets), _p(stats), _p(self.ws), _s(stream))
        return self.rows


# ----------------------------------------------------------------- product
class MX8ProductConfig(ctypes.Structure):
    """Mirror of ``moe_mx8_product_config`` (include/moe.h)."""
    _fields_ = [("rows", ctypes.c_int64), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
                ("E", ctypes.c_int32), ("act", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]

    def __init__(self, rows, K, N, E, act=MX8_ACT_NONE, out_dtype=_moe.BF16):
        super().__init__(rows, K, N, E, act, out_dtype)


def check_mx8_product_config(cfg: MX8ProductConfig) -> int:
    return _moe.load_library().moe_check_mx8_product_config(ctypes.byref(cfg))


def moe_mx8_grouped_product(cfg, x_codes, x_scales, offsets, w_codes, w_scales, wg_codes, wg_scales,
                            out, out_scales, stream=None):
    _call("moe_mx8_grouped_product", ctypes.byref(cfg), _p(x_codes), _p(x_scales), _p(offsets),
          _p(w_codes), _p(w_scales), _p(wg_codes), _p(wg_scales), _p(out), _p(out_scales), _s(stream))


class MX8Product:
    """out = act(x W_e) over expert segments of any length, x and W in 8 bits.  Owns the
    output: a tensor, or an MX8Tensor where ``out_dtype`` is MX8."""

    def __init__(self, cfg: MX8ProductConfig, device="cuda"):
        rc = check_mx8_product_config(cfg)
        if rc != 0:
            raise _moe.MoEError(rc, "moe_check_mx8_product_config")
        self.cfg = c = cfg
        self._x, self._offsets, self._w = (c.rows, c.K), (c.E + 1,), (c.E, c.N, c.K)
        self._dual = c.act == MX8_ACT_SWIGLU
        if c.out_dtype == MX8:
            self.out = MX8Tensor((c.rows, c.N), device)
        else:
            self.out = torch.empty(c.rows, c.N, device=device,
                                   dtype=torch.bfloat16 if c.out_dtype == _moe.BF16 else torch.float32)

    def forward(self, x: MX8Tensor, offsets, w: MX8Weight, wg: MX8Weight | None = None, stream=None):
        """out [rows, N] (rows of no segment are not written); x [rows, K], not this product's
        own out, offsets [E + 1] int32 as from MX8Dispatch, w (and the gate wg for SwiGLU)
        [E, N, K]."""
        _checked8(x, self._x, "x")
        if x is self.out:                            # (tiles are written while others still read x)
            raise ValueError("x: the rows that this product writes")
        _checked(offsets, self._offsets, torch.int32, "offsets")
        if (wg is not None) != self._dual:
            raise ValueError("wg is required iff act is MX8_ACT_SWIGLU")
        _checked8(w, self._w, "w", MX8Weight)
        if wg is not None:
            _checked8(wg, self._w, "wg", MX8Weight)
        out = self.out
        _call("moe_mx8_grouped_product", ctypes.byref(self.cfg), *x.ptrs, _p(offsets), *w.ptrs,
              *(wg.ptrs if wg else _NONE), *(out.ptrs if self.cfg.out_dtype == MX8 else (_p(out), None)), _s(stream))
        return out


class MX8Experts:
    """A layer's expert weights in 8 bits, for ``MoELayer.forward_mx8``: quantised once
    from W_up, W_gate (SwiGLU) [E, d, f] and W_down [E, f, d]."""

    def __init__(self, W_up, W_down, W_gate=None, stream=None):
        self.up = mx8_quantize_weight(W_up, stream)
        self.down = mx8_quantize_weight(W_down, stream)
        self.gate = mx8_quantize_weight(W_gate, stream) if W_gate is not None else None


# ----------------------------------------------------------------- activations kept in 8 bits
def moe_grouped_ffn_mx8(cfg, x_perm, offsets, W_up, W_gate, W_down, h_codes, h_scales, act, y_perm, ws,
                        stream=None):
    _call("moe_grouped_ffn_mx8", ctypes.byref(cfg), _p(x_perm), _p(offsets), _p(W_up), _p(W_gate),
          _p(W_down), _p(h_codes), _p(h_scales), _p(act), _p(y_perm), _p(ws), _s(stream))


def moe_grouped_ffn_backward_mx8(cfg, x_perm, offsets, W_up, W_gate, W_down, h_codes, h_scales, act,
                                 dy_perm, dh, dx_perm, dW_up, dW_gate, dW_down, ws, stream=None):
    _call("moe_grouped_ffn_backward_mx8", ctypes.byref(cfg), _p(x_perm), _p(offsets), _p(W_up),
          _p(W_gate), _p(W_down), _p(h_codes), _p(h_scales), _p(act), _p(dy_perm), _p(dh), _p(dx_perm),
          _p(dW_up), _p(dW_gate), _p(dW_down), _p(ws), _s(stream))


def moe_backward_mx8(cfg, x, W_r, W_up, W_gate, W_down, logits, topk_idx, gate, slot_of, perm_token,
                     offsets, x_perm, h_codes, h_scales, act, y_perm, stats, dlogits_aux, dout, dx, dW_r,
                     dbias, dW_up, dW_gate, dW_down, ws, stream=None):
    _call("moe_backward_mx8", ctypes.byref(cfg), _p(x), _p(W_r), _p(W_up), _p(W_gate), _p(W_down),
          _p(logits), _p(topk_idx), _p(gate), _p(slot_of), _p(perm_token), _p(offsets), _p(x_perm),
          _p(h_codes), _p(h_scales), _p(act), _p(y_perm), _p(stats), _p(dlogits_aux), _p(dout), _p(dx),
          _p(dW_r), _p(dbias), _p(dW_up), _p(dW_gate), _p(dW_down), _p(ws), _s(stream))


class MoECheckpoint:
    """What one forward of a ``MoELayer`` leaves for its backward, the experts' hidden rows
    ``h`` and outputs ``y`` in 8 bits (a third of the 16-bit buffers' bytes, which the
    layer then keeps once for all depths): for ``MoELayer.forward(..., checkpoint=c)`` and
    ``backward(..., checkpoint=c)``.  bf16 layers without shared experts."""

    def __init__(self, cfg, device="cuda"):
        rc = _moe.check_config(cfg)
        if rc != 0:
            raise _moe.MoEError(rc, "moe_check_config")
        c = cfg
        if c.dtype != _moe.BF16 or c.f_shared > 0:
            raise ValueError("a checkpoint needs a bf16 layer without shared experts")
        self.cfg = c
        R = _moe.rows_capacity(c)
        e = lambda *s, dtype=torch.int32: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        f32 = torch.float32
        self.h, self.y = MX8Tensor((c.nh, R, c.f), device), MX8Tensor((R, c.d), device)
        self.logits, self.gate, self.stats = e(c.T, c.E, dtype=f32), e(c.T, c.k, dtype=f32), e(9 + c.E, dtype=f32)
        self.topk_idx, self.slot_of, self.perm_token = e(c.T, c.k), e(c.T, c.k), e(R)
        self.counts, self.kept, self.offsets = e(c.E), e(c.E), e(c.E + 1)
        self.inputs = self.x = None               # (x: a copy, where the forward's x was the layer's own memory)

    def check(self, cfg, device=None):
        if bytes(cfg) != bytes(self.cfg):
            raise ValueError(f"the checkpoint is of another layer: {self.cfg!r}")
        if device is not None and device != self.stats.device:
            raise ValueError(f"the checkpoint is on {self.stats.device}, the layer on {device}")

    def keep_y(self, y_perm, stream=None):
        R, d = self.y.shape
        # the rows below offsets[E] (a view of it would cost more than the call)
        _call("moe_mx8_quantize", _moe.BF16, R, d, _p(y_perm), _p(self.offsets) + 4 * self.cfg.E,
              *self.y.ptrs, _s(stream))

    def y_into(self, y_perm, stream=None):
        R, d = self.y.shape
        _call("moe_mx8_dequantize", _moe.BF16, R, d, *self.y.ptrs, _p(y_perm), _s(stream))
