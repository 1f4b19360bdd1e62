"""Plain 64-bit definitions of the training operators, for the tests: block quantisation by the
definition, scale tiles by their index formula, products and layer norm in float64."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 128


def as64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def power_of(v: np.ndarray) -> np.ndarray:
    """floor(log2 |v|) of nonzero finite values, exactly."""
    return np.frexp(np.abs(v))[1] - 1


def e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 value, ties to even, saturating at 448; NaN stays NaN."""
    a = np.minimum(np.abs(v), 448.0)
    with np.errstate(invalid="ignore"):
        quantum = np.ldexp(1.0, np.maximum(np.where(a > 0, power_of(np.where(a > 0, a, 1.0)) - 3, -9), -9))
        return np.copysign(np.rint(a / quantum) * quantum, v)


def quantise(x: np.ndarray, block: int = BLOCK, master: np.ndarray | None = None):
    """(values kept, code values, scale bytes [rows][blocks]) of blocks along the last axis.
    ``master``: the values whose block maxima give the scales, where they are not x's own."""
    m = x if master is None else master
    r, c = x.shape
    nb = -(-c // block)
    kept, codes = np.empty((r, c)), np.empty((r, c))
    byte = np.empty((r, nb), np.uint8)
    for b in range(nb):
        part = x[:, b * block:(b + 1) * block]
        amax = np.abs(m[:, b * block:(b + 1) * block]).max(1)
        bad = ~np.isfinite(amax)
        e = np.where((amax > 0) & ~bad, np.maximum(power_of(np.where((amax > 0) & ~bad, amax, 1.0)) - 8, -127), -127)
        byte[:, b] = np.where(bad, 255, e + 127)
        f = np.where(bad, np.nan, np.ldexp(1.0, e))[:, None]
        q = e4m3(part / f)
        codes[:, b * block:(b + 1) * block] = q
        kept[:, b * block:(b + 1) * block] = q * f
    return kept, codes, byte


def tiles(grid: np.ndarray) -> np.ndarray:
    """A scale grid in 128x4 tiles, by the index formula, zeros where it is padded."""
    r, c = grid.shape
    tr, tcn = -(-r // 128), -(-c // 4)
    out = np.zeros(tr * tcn * 512, np.uint8)
    i, j = np.meshgrid(np.arange(r), np.arange(c), indexing="ij")
    out[((i // 128) * tcn + j // 4) * 512 + (i % 32) * 16 + (i // 32 % 4) * 4 + j % 4] = grid
    return out


def codes_to_values(q: torch.Tensor) -> np.ndarray:
    return as64(q.contiguous().view(torch.float8_e4m3fn).float())


def norm_forward(x, w, b, eps):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return d * rstd[:, None] * w + (0.0 if b is None else b), mean, rstd


def norm_backward(dy, x, w, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
