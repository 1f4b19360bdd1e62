"""Plain definitions of the NVFP4 operands, for the tests: every F32 step of the convention as one numpy operation, the
roundings to E4M3 and E2M1 in float64."""
from __future__ import annotations

import numpy as np
import torch

import linear_ref as ref

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
LARGEST = np.finfo(np.float32).max


def e2m1(v: np.ndarray) -> np.ndarray:
    """Nearest E2M1 value, ties to the even code, saturating at 6."""
    a = np.minimum(np.abs(np.asarray(v, np.float64)), 6.0)
    quantum = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.copysign(np.rint(a / quantum) * quantum, v)


def tensor_scale(top) -> np.float32:
    top = np.float32(top)
    if not np.isfinite(top):
        return np.float32(np.nan)
    with np.errstate(over="ignore"):
        return np.float32(1) if top == 0 else np.minimum(np.float32(2688) / top, LARGEST)


def quantise(x: np.ndarray, top):
    """(E2M1 values, scale values [rows][blocks]) of blocks of 16 along the last axis."""
    x = np.asarray(x, np.float32)
    r, c = x.shape
    S, nb = tensor_scale(top), -(-c // 16)
    q, s = np.zeros((r, c), np.float32), np.zeros((r, nb), np.float32)
    with np.errstate(all="ignore"):
        for b in range(nb):
            part = x[:, 16 * b:16 * b + 16]
            amax = np.abs(part).max(1)
            v = (amax / np.float32(6)) * S
            s[:, b] = np.where(np.isfinite(amax) & ~np.isnan(v), ref.e4m3(v.astype(np.float64)), np.nan)
            mul = np.where((s[:, b] == 0) | np.isnan(s[:, b]), np.float32(0), np.minimum(S / s[:, b], LARGEST))
            q[:, 16 * b:16 * b + 16] = e2m1(part * mul[:, None].astype(np.float32))
    return q, s


def spread(s: np.ndarray, c: int) -> np.ndarray:
    return np.repeat(s, 16, axis=1)[:, :c]


def kept(x, top):
    """F32 values that the codes stand for."""
    q, s = quantise(x, top)
    return (q * spread(s, q.shape[1])) * (np.float32(1) / tensor_scale(top))


def unpack(buf: torch.Tensor, rows: int, cols: int) -> np.ndarray:
    """E2M1 values of packed codes."""
    b = buf[:rows, :(cols + 1) // 2].cpu().numpy()
    code = np.stack((b & 15, b >> 4), 2).reshape(rows, -1)
    if cols % 2:
        assert not np.any(code[:, cols]), "the half byte behind an odd row is not zero"
    code = code[:, :cols]
    return np.where(code & 8, -1.0, 1.0) * LEVELS[code & 7]


def pack(q: np.ndarray, pitch: int) -> np.ndarray:
    r, c = q.shape
    code = np.searchsorted(LEVELS, np.abs(q)).astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 3)
    code = np.pad(code, ((0, 0), (0, c % 2)))
    out = np.zeros((r, pitch), np.uint8)
    out[:, :code.shape[1] // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    return out


def scale_bytes(s: np.ndarray) -> np.ndarray:
    """E4M3 bytes of scale values (0x7F for NaN)."""
    t = torch.from_numpy(np.nan_to_num(s)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return np.where(np.isnan(s), np.uint8(0x7F), t)
