"""Linear layers on the weights that the casts write: behind a layer norm on MXFP8 weights (``NormLinear``), and
behind an RMS norm in a residual stream on MXFP8 or NVFP4 weights (``RMSNormLinear``, below).

    h = LayerNorm(x),  y = h W^T

The FP32 master weight lives in shards and reaches its MXFP8 copies (rowwise and columnwise)
through ``driver.ShardedCast``; ``refresh`` lays their scales out for the products.  What the
backward pass needs of the activations is kept in 8 bits: the layer's input as a rowwise
checkpoint (layer norm's gradients read it) and the normalised input as a columnwise one
(the weight's gradient contracts over tokens).  The normalised input's rowwise copy, which
the forward product reads, is a buffer of the layer too: 3 bytes per value of the input's
shape in all, and the scales.  A step's calls:

    forward    save(x), layer norm, save(h), y = h W^T
    backward   save(dy), dh = dy W, dW += dy^T h, layer norm's gradients

All buffers are allocated once; every call goes to the current stream.  A kernel that gives up a wait
leaves invalid output and its call has already returned: ``check`` raises for it, at the end of a step or
wherever the program waits for the GPU anyway.

    s = x + residual,  h = RMSNorm(s),  y = h W^T

With MXFP8 weights the norm writes the product's 8-bit operand itself; with NVFP4 weights it writes h and its largest
magnitude, and the quantisation reads both.  A step's calls:

    MXFP8   forward    norm (s, h, 8-bit h), save(h) along its columns, y = h W^T
            backward   save(dy), dh = dy W, dW += dy^T h, the norm's gradients (+ ds)
    NVFP4   forward    norm (s, h, max |h|), quantise(h), y = h W^T
            backward   max |dy|, quantise(dy), dh = dy W, dW += dy^T h, the norm's gradients (+ ds)

A layer that only serves (``training=False``) keeps neither h nor what a backward pass reads.
"""
from __future__ import annotations

import torch

from . import api, driver


def _pitch(n: int) -> int:
    """Row stride of a code buffer: whole 16-byte units, so that TMA can fetch its rows."""
    return (n + 15) // 16 * 16


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _check_input(x: torch.Tensor, name: str, tokens: int, width: int) -> None:
    """An input is tokens x width, or as many values in one dimension: the C entry points take larger buffers, of
    which they read the first rows and columns, and a larger input would be cut without a word."""
    if tuple(x.shape) not in ((tokens, width), (tokens * width,)):
        raise api.MXFP8Error(2, f"{name}: shape {list(x.shape)}, expected [{tokens}, {width}]")


class Checkpoint:
    """Buffers of an activation's 8-bit checkpoint, tokens x width, in one or both directions."""

    def __init__(self, tokens: int, width: int, device, rowwise: bool = True, colwise: bool = True):
        self.tokens, self.width = tokens, width
        u8 = lambda *shape: torch.empty(*shape, dtype=torch.uint8, device=device)  # noqa: E731
        self.codes_r = u8(tokens, _pitch(width)) if rowwise else None
        self.scale_r = u8(api.mxfp8_swizzled_scales_size(tokens, _blocks(width))) if rowwise else None
        self.codes_c = u8(tokens, _pitch(width)) if colwise else None
        self.scale_c = u8(api.mxfp8_swizzled_scales_size(width, _blocks(tokens))) if colwise else None

    def save(self, x: torch.Tensor) -> None:
        _check_input(x, "input", self.tokens, self.width)
        api.mxfp8_checkpoint_save(x, self.codes_r, self.scale_r, self.codes_c, self.scale_c, self.tokens, self.width)

    def restore(self, out: torch.Tensor, colwise: bool = False) -> None:
        codes, scale = (self.codes_c, self.scale_c) if colwise else (self.codes_r, self.scale_r)
        api.mxfp8_checkpoint_restore(codes, scale, out, self.tokens, self.width, colwise=colwise)


class NormLinear:
    """One layer for ``tokens`` tokens per step, weight [outs][ins], master shards cut at
    ``bounds`` of the flat weight (default: one shard)."""

    def __init__(self, tokens: int, ins: int, outs: int, device="cuda", dtype=torch.bfloat16, bounds=None,
                 eps: float = 1e-5):
        self.tokens, self.ins, self.outs, self.eps = tokens, ins, outs, eps
        self.device = dev = torch.device(device)
        self.cast = driver.ShardedCast([driver.WeightSpec(outs, ins, True)], bounds or [0, outs * ins], dev)
        (rr, rc), (cr, cc) = api.block_shapes(outs, ins)
        self._grids = (rr, rc, cr, cc)
        self.w_scale_r = torch.empty(api.mxfp8_swizzled_scales_size(rr, rc), dtype=torch.uint8, device=dev)
        self.w_scale_c = torch.empty(api.mxfp8_swizzled_scales_size(cr, cc, True), dtype=torch.uint8, device=dev)
        # parameters of the norm and the gradients, which accumulate (weight) or are set (norm)
        self.norm_weight, self.norm_bias = torch.ones(ins, device=dev), torch.zeros(ins, device=dev)
        self.grad_weight = torch.zeros(outs, ins, device=dev)
        self.grad_norm_weight, self.grad_norm_bias = torch.empty(ins, device=dev), torch.empty(ins, device=dev)
        # kept from forward to backward: a byte per value of x and the columnwise byte per value of h, and two
        # floats per token; h8's rowwise copy serves the forward product only
        self.x8 = Checkpoint(tokens, ins, dev, colwise=False)
        self.h8 = Checkpoint(tokens, ins, dev)
        self.mean, self.rstd = torch.empty(tokens, device=dev), torch.empty(tokens, device=dev)
        # working buffers of a step
        self.dy8 = Checkpoint(tokens, outs, dev)
        self.h = torch.empty(tokens, ins, dtype=dtype, device=dev)
        self.y = torch.empty(tokens, outs, dtype=dtype, device=dev)
        self.dh = torch.empty(tokens, ins, dtype=dtype, device=dev)
        self.dx = torch.empty(tokens, ins, dtype=dtype, device=dev)
        self.workspace = torch.empty(max(1, api.mxfp8_layer_norm_workspace_size(tokens, ins)), dtype=torch.uint8, device=dev)

    def refresh(self, shards) -> None:
        """New MXFP8 weights from the master shards."""
        self.cast.step(shards)
        rr, rc, cr, cc = self._grids
        sr, sc = self.cast.scales[0]
        api.mxfp8_swizzle_scales(sr, self.w_scale_r, rr, rc)
        api.mxfp8_swizzle_scales(sc, self.w_scale_c, cr, cc, transpose=True)

    def check(self) -> None:
        """Waits for the current stream; raises when a kernel of a layer on this device gave up a wait, so that
        what it wrote is invalid."""
        api.mxfp8_device_status(self.device)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """y of this step's input (tokens x ins); valid until the next call."""
        t, i, o = self.tokens, self.ins, self.outs
        _check_input(x, "x", t, i)
        if x.dtype != self.h.dtype:
            raise api.MXFP8Error(3, f"x: dtype {x.dtype}, the layer's is {self.h.dtype}")
        self.x8.save(x)
        api.mxfp8_layer_norm_forward(x, self.norm_weight, self.norm_bias, self.h, self.mean, self.rstd, t, i, self.eps)
        self.h8.save(self.h)
        api.mxfp8_gemm(self.h8.codes_r, self.h8.scale_r, self.cast.outputs[0][0], self.w_scale_r, None, self.y, t, o, i,
                       b_block=32)
        return self.y

    def backward(self, dy: torch.Tensor) -> torch.Tensor:
        """dx of this step's output gradient; adds to grad_weight, sets the norm's gradients."""
        t, i, o = self.tokens, self.ins, self.outs
        _check_input(dy, "dy", t, o)
        self.dy8.save(dy)
        api.mxfp8_gemm(self.dy8.codes_r, self.dy8.scale_r, self.cast.outputs[0][1], self.w_scale_c, None, self.dh, t, i, o,
                       b_colwise=True, b_block=32)
        api.mxfp8_gemm(self.dy8.codes_c, self.dy8.scale_c, self.h8.codes_c, self.h8.scale_c, self.grad_weight,
                       self.grad_weight, o, i, t, a_colwise=True, b_colwise=True)
        api.mxfp8_layer_norm_backward(self.dh, self.x8.codes_r, self.x8.scale_r, self.norm_weight, self.mean, self.rstd,
                                      self.dx, self.grad_norm_weight, self.grad_norm_bias, self.workspace, t, i)
        return self.dx


class Operands4:
    """Buffers of an activation's NVFP4 operands, tokens x width: along its rows and/or, transposed, along its columns."""

    def __init__(self, tokens: int, width: int, device, rowwise: bool = True, colwise: bool = True):
        self.tokens, self.width = tokens, width
        u8 = lambda *shape: torch.empty(*shape, dtype=torch.uint8, device=device)  # noqa: E731
        codes = lambda r, c: u8(r, _pitch((c + 1) // 2))  # noqa: E731
        scale = lambda r, c: u8(api.mxfp8_swizzled_scales_size(r, (c + 15) // 16))  # noqa: E731
        self.codes_r, self.scale_r = (codes(tokens, width), scale(tokens, width)) if rowwise else (None, None)
        self.codes_c, self.scale_c = (codes(width, tokens), scale(width, tokens)) if colwise else (None, None)
        self.amax = torch.zeros(1, device=device)  # largest magnitude, which every code is relative to

    def measure(self, x: torch.Tensor) -> None:
        """The largest magnitude of x."""
        _check_input(x, "input", self.tokens, self.width)
        api.nvfp4_tensor_amax(x, self.amax, self.tokens, self.width)

    def quantize(self, x: torch.Tensor) -> None:
        """Codes and scales of x, relative to ``amax``."""
        _check_input(x, "input", self.tokens, self.width)
        api.nvfp4_quantize(x, self.amax, self.codes_r, self.scale_r, self.codes_c, self.scale_c, self.tokens, self.width)

    def save(self, x: torch.Tensor) -> None:
        self.measure(x)
        self.quantize(x)

    def restore(self, out: torch.Tensor, colwise: bool = False) -> None:
        """The values of the rowwise operand (tokens x width) or of the columnwise one (width x tokens)."""
        if colwise:
            api.nvfp4_restore(self.codes_c, self.scale_c, self.amax, out, self.width, self.tokens)
        else:
            api.nvfp4_restore(self.codes_r, self.scale_r, self.amax, out, self.tokens, self.width)


class _Weights8:
    """MXFP8 copies of a weight [outs][ins] and the products with them, activations in 8 bits."""

    def __init__(self, tokens, ins, outs, device, bounds, training):
        self.tokens, self.ins, self.outs = tokens, ins, outs
        self.cast = driver.ShardedCast([driver.WeightSpec(outs, ins, training)], bounds or [0, outs * ins], device)
        (rr, rc), (cr, cc) = self._grids = api.block_shapes(outs, ins)
        self.scale_r = torch.empty(api.mxfp8_swizzled_scales_size(rr, rc), dtype=torch.uint8, device=device)
        self.h8 = Checkpoint(tokens, ins, device, colwise=training)
        if training:
            self.scale_c = torch.empty(api.mxfp8_swizzled_scales_size(cr, cc, True), dtype=torch.uint8, device=device)
            self.dy8 = Checkpoint(tokens, outs, device)

    def refresh(self, shards):
        self.cast.step(shards)
        (rr, rc), (cr, cc) = self._grids
        sr, sc = self.cast.scales[0]
        api.mxfp8_swizzle_scales(sr, self.scale_r, rr, rc)
        if sc is not None:
            api.mxfp8_swizzle_scales(sc, self.scale_c, cr, cc, transpose=True)

    def norm(self, x, residual, weight, total, h, rstd, eps):
        t, i = self.tokens, self.ins
        api.mxfp8_rms_norm_forward(x, residual, weight, total, h, self.h8.codes_r, self.h8.scale_r, None, rstd, t, i, eps)
        if self.h8.codes_c is not None:
            api.mxfp8_checkpoint_save(h, None, None, self.h8.codes_c, self.h8.scale_c, t, i)

    def output(self, y):
        api.mxfp8_gemm(self.h8.codes_r, self.h8.scale_r, self.cast.outputs[0][0], self.scale_r, None, y, self.tokens,
                       self.outs, self.ins, b_block=32)

    def gradients(self, dy, dh, grad_weight):
        t, i, o = self.tokens, self.ins, self.outs
        self.dy8.save(dy)
        api.mxfp8_gemm(self.dy8.codes_r, self.dy8.scale_r, self.cast.outputs[0][1], self.scale_c, None, dh, t, i, o,
                       b_colwise=True, b_block=32)
        api.mxfp8_gemm(self.dy8.codes_c, self.dy8.scale_c, self.h8.codes_c, self.h8.scale_c, grad_weight, grad_weight, o,
                       i, t, a_colwise=True, b_colwise=True)


class _Weights4:
    """NVFP4 copies of a weight [outs][ins], ins even, and the products with them, activations in 4 bits."""

    def __init__(self, tokens, ins, outs, device, bounds, training):
        if ins % 2 != 0:
            raise api.MXFP8Error(1, f"ins: {ins}, must be even (two codes share a byte)")
        if bounds is not None and list(bounds) != [0, outs * ins]:
            raise api.MXFP8Error(1, "bounds: an NVFP4 weight comes as one shard")
        self.tokens, self.ins, self.outs, self.training = tokens, ins, outs, training
        u8 = lambda *shape: torch.empty(*shape, dtype=torch.uint8, device=device)  # noqa: E731
        (rr, rc), (cr, cc) = self._grids = api.nvfp4_block_shapes(outs, ins)
        self.amax = torch.zeros(1, device=device)
        self._amax_r, self._grid_r, self._dense_r = torch.empty(rr, rc, device=device), u8(rr, rc), u8(outs, ins // 2)
        self._amax_c = self._grid_c = self._dense_c = None
        self.codes_r = self._dense_r if ins % 32 == 0 else u8(outs, _pitch(ins // 2))
        self.scale_r = u8(api.mxfp8_swizzled_scales_size(rr, rc))
        self.h4 = Operands4(tokens, ins, device, colwise=training)
        if training:
            self._amax_c, self._grid_c, self._dense_c = torch.empty(cr, cc, device=device), u8(cr, cc), u8(outs, ins // 2)
            self.codes_c = u8(ins, _pitch((outs + 1) // 2))
            self.scale_c = u8(api.mxfp8_swizzled_scales_size(cr, cc, True))
            self.dy4 = Operands4(tokens, outs, device)

    def refresh(self, shards):
        if len(shards) != 1:
            raise api.MXFP8Error(1, f"shards: {len(shards)}, an NVFP4 weight comes as one shard")
        o, i, master = self.outs, self.ins, shards[0]
        (rr, rc), (cr, cc) = self._grids
        if master.numel() != o * i:
            raise api.MXFP8Error(2, f"shards: {master.numel()} values, expected {o} x {i}")
        self.amax.zero_()
        api.nvfp4_partial_amax(master, self._amax_r, self._amax_c, self.amax, o, i, 0)
        api.nvfp4_update_scales(self._amax_r, self._amax_c, self.amax, self._grid_r, self._grid_c, o, i)
        dense = lambda q: None if q is None else q.view(-1)  # noqa: E731
        api.nvfp4_partial_cast(master, self._grid_r, self._grid_c, self.amax, dense(self._dense_r), dense(self._dense_c), o, i, 0, 0)
        api.mxfp8_swizzle_scales(self._grid_r, self.scale_r, rr, rc)
        if self.codes_r is not self._dense_r:
            api.nvfp4_lay_out(self._dense_r, self.codes_r, o, i)
        if self.training:
            api.mxfp8_swizzle_scales(self._grid_c, self.scale_c, cr, cc, transpose=True)
            api.nvfp4_lay_out(self._dense_c, self.codes_c, o, i, transpose=True)

    def norm(self, x, residual, weight, total, h, rstd, eps):
        self.h4.amax.zero_()
        api.mxfp8_rms_norm_forward(x, residual, weight, total, h, None, None, self.h4.amax, rstd, self.tokens, self.ins, eps)
        self.h4.quantize(h)

    def output(self, y):
        api.nvfp4_gemm(self.h4.codes_r, self.h4.scale_r, self.h4.amax, self.codes_r, self.scale_r, self.amax, None, y,
                       self.tokens, self.outs, self.ins)

    def gradients(self, dy, dh, grad_weight):
        t, i, o = self.tokens, self.ins, self.outs
        self.dy4.save(dy)
        api.nvfp4_gemm(self.dy4.codes_r, self.dy4.scale_r, self.dy4.amax, self.codes_c, self.scale_c, self.amax, None, dh, t, i, o)
        api.nvfp4_gemm(self.dy4.codes_c, self.dy4.scale_c, self.dy4.amax, self.h4.codes_c, self.h4.scale_c, self.h4.amax,
                       grad_weight, grad_weight, o, i, t)


class RMSNormLinear:
    """A linear layer behind an RMS norm in a residual stream, for ``tokens`` tokens per step, weight [outs][ins] in
    ``weights`` "mxfp8" (master shards cut at ``bounds`` of the flat weight, default one) or "nvfp4" (one shard, ins even)."""

    def __init__(self, tokens: int, ins: int, outs: int, device="cuda", dtype=torch.bfloat16, weights: str = "mxfp8",
                 bounds=None, eps: float = 1e-5, training: bool = True):
        if weights not in ("mxfp8", "nvfp4"):
            raise api.MXFP8Error(1, f'weights: {weights!r}, expected "mxfp8" or "nvfp4"')
        self.tokens, self.ins, self.outs, self.eps, self.training, self.dtype = tokens, ins, outs, eps, training, dtype
        self.device = dev = torch.device(device)
        self.weights = (_Weights8 if weights == "mxfp8" else _Weights4)(tokens, ins, outs, dev, bounds, training)
        self.norm_weight = torch.ones(ins, device=dev)
        self.sum = torch.empty(tokens, ins, dtype=dtype, device=dev)
        self.y = torch.empty(tokens, outs, dtype=dtype, device=dev)
        # the norm's values: what is saved along the columns, or quantised to 4 bits
        self.h = torch.empty(tokens, ins, dtype=dtype, device=dev) if training or weights == "nvfp4" else None
        self.rstd = torch.empty(tokens, device=dev) if training else None
        if training:  # the weight's gradient accumulates, the norm's is set
            self.grad_weight, self.grad_norm_weight = torch.zeros(outs, ins, device=dev), torch.empty(ins, device=dev)
            self.dh, self.dx = (torch.empty(tokens, ins, dtype=dtype, device=dev) for _ in range(2))
            self.workspace = torch.empty(max(1, api.mxfp8_rms_norm_workspace_size(tokens, ins)), dtype=torch.uint8, device=dev)

    def refresh(self, shards) -> None:
        """New 8- or 4-bit weights from the master shards."""
        self.weights.refresh(shards)

    def check(self) -> None:
        """Waits for the current stream; raises when a kernel of a layer on this device gave up a wait, so that
        what it wrote is invalid."""
        api.mxfp8_device_status(self.device)

    def _input(self, x: torch.Tensor, name: str, width: int) -> None:
        _check_input(x, name, self.tokens, width)
        if x.dtype != self.dtype:
            raise api.MXFP8Error(3, f"{name}: dtype {x.dtype}, the layer's is {self.dtype}")

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        """(y, s) of this step's input (tokens x ins) and the residual stream before it (None: none); valid until the
        next call."""
        self._input(x, "x", self.ins)
        if residual is not None:
            self._input(residual, "residual", self.ins)
        self.weights.norm(x, residual, self.norm_weight, self.sum, self.h, self.rstd, self.eps)
        self.weights.output(self.y)
        return self.y, self.sum

    def backward(self, dy: torch.Tensor, ds: torch.Tensor | None = None) -> torch.Tensor:
        """The gradient of s, which is that of x and of the residual, from this step's output gradient and the one that
        reaches s along the residual stream (None: none); adds to grad_weight, sets grad_norm_weight."""
        if not self.training:
            raise api.MXFP8Error(1, "backward: the layer was made for serving (training=False)")
        self._input(dy, "dy", self.outs)
        if ds is not None:
            self._input(ds, "ds", self.ins)
        self.weights.gradients(dy, self.dh, self.grad_weight)
        api.mxfp8_rms_norm_backward(self.dh, ds, self.sum, self.norm_weight, self.rstd, self.dx, self.grad_norm_weight,
                                    self.workspace, self.tokens, self.ins)
        return self.dx
