"""A linear layer behind a layer norm, trained on the MXFP8 weights that the cast writes.

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
