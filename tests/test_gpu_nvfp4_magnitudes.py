"""Products of NVFP4 operands whose largest magnitudes are very large or very small.

Every scale of an operand is the same power of two, so a sum is a whole number of quanta, at most 144 k < 2^24 of them,
and exact in F32.  What remains are two roundings (the sum times 1 / Sa and that times 1 / Sb, or both factors joined and the
sum times them), each 2^-24 of its result or, where it is subnormal, 2^-150: of the first, what the second factor leaves of it,
which is less than all of it.  The addend adds one rounding, a BF16 result half a unit, 2^-8 of the value or 2^-134."""
import numpy as np
import pytest
import torch

import fp4_ref as fp4
import linear_ref as ref
from mxfp8_master_weight_gb300 import api

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LARGEST = float(fp4.LARGEST)
# by shape: the kernel of few rows or few columns; pairs of CTAs
SHAPES = [(1, 300, 64), (40, 200, 100), (200, 7, 64), (130, 140, 64), (300, 264, 100)]
# largest magnitudes and the exponent of the scales: 2^-9, the least; 1; 256
TOPS = [(1e23, 1e23, -9), (1e24, 1e24, -9), (1e19, 1e28, -9), (1e28, 1e19, -9), (1e30, 1e30, -9), (LARGEST, LARGEST, -9),
        (1e30, 1e-30, 0), (1e-30, 1e30, 0), (1e-17, 1e-17, 8), (1e-20, 1e-20, 8), (1e-38, 1e-3, 8), (1e-40, 1e3, 8),
        (1e3, 1e-40, 8), (1e-40, 1e-40, 8)]


def operand(rng, mn, k, power):
    """Codes without a zero but for whole rows of them, every third; their values, the buffers."""
    q = rng.choice(fp4.LEVELS[1:], (mn, k)) * rng.choice([-1.0, 1.0], (mn, k))
    q[2::3] = 0.0
    byte = np.full((mn, -(-k // 16)), 0x01 if power == -9 else (power + 7) << 3, np.uint8)
    buf = fp4.pack(q, -(-((k + 1) // 2) // 16) * 16)
    return q * 2.0 ** power, torch.from_numpy(buf).cuda(), torch.from_numpy(ref.tiles(byte)).cuda()


@pytest.mark.parametrize("ta,tb,power", TOPS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, ta, tb, power):
    rng = np.random.default_rng(m + n + k)
    a, qa, sa = operand(rng, m, k, power)
    b, qb, sb = operand(rng, n, k, power)
    ga, gb = (torch.tensor([t], dtype=torch.float32, device="cuda") for t in (ta, tb))
    ra, rb = (float(np.float32(1) / fp4.tensor_scale(t)) for t in (ta, tb))
    want0 = (a @ b.T) * ra * rb
    c = torch.randn(m, n, device="cuda")
    for dtype, over, add in ((torch.float32, 0, False), (torch.float32, 3, False), (torch.bfloat16, 0, False),
                             (torch.bfloat16, 3, False), (torch.float32, 0, True)):
        out = torch.full((m, n + over), -3.0, dtype=dtype, device="cuda")
        api.nvfp4_gemm(qa, sa, ga, qb, sb, gb, c if add else None, out[:, :n], m, n, k)
        api.mxfp8_device_status()
        got, want = ref.as64(out[:, :n]), want0 + (ref.as64(c) if add else 0.0)
        tol = 2 * U * (1 + U) * np.abs(want0) + 2.0 ** -149
        if add:
            tol = tol + U * (np.abs(want) + tol)
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134
        if not add:
            assert np.all(got[want == 0] == 0)
        # BF16 ends at 3.39e38 and half a unit, F32 at 3.4028e38
        finite, past = np.abs(want) < 3.38e38, np.abs(want) > 3.41e38
        assert np.all(np.abs(got[finite] - want[finite]) <= tol[finite])
        assert np.array_equal(got[past], np.copysign(np.inf, want[past]))
        assert not np.any(np.isnan(got))


def test_activation_with_a_huge_value():
    """An activation that holds 1e24, rows of zeros and rows of small values, and its weight gradient with another such:
    every output is what the operands' values give, none is NaN."""
    t, i, o = 96, 80, 144
    g = torch.Generator(device="cuda").manual_seed(4)
    x, dy = (torch.randn(t, n, generator=g, device="cuda") for n in (i, o))
    x[::5], dy[1::5] = 0.0, 0.0
    x *= 1e20
    dy *= 1e20
    x[3, 7], dy[8, 40] = 1e24, -1e24
    buf = []
    for v, n in ((x, i), (dy, o)):
        top = torch.empty(1, device="cuda")
        api.nvfp4_tensor_amax(v, top, t, n)
        q = torch.empty(n, -(-t // 32) * 16, dtype=torch.uint8, device="cuda")
        s = torch.empty(api.mxfp8_swizzled_scales_size(n, -(-t // 16)), dtype=torch.uint8, device="cuda")
        api.nvfp4_quantize(v, top, None, None, q, s, t, n)
        kept = torch.empty(n, t, device="cuda")
        api.nvfp4_restore(q, s, top, kept, n, t)
        buf.append((q, s, top, ref.as64(kept)))
    (qx, sx, gx, vx), (qd, sd, gd, vd) = buf
    out = torch.full((o, i), -3.0, device="cuda")
    api.nvfp4_gemm(qd, sd, gd, qx, sx, gx, None, out, o, i, t)
    api.mxfp8_device_status()
    got, want = ref.as64(out), vd @ vx.T
    assert not np.any(np.isnan(got))
    # terms exact in F32 (10 bits); 64 join the sum per instruction: t / 16 + 32 roundings or truncations of 2^-23 of the sum of
    # magnitudes, and of the factors and the two restored values four of 2^-24
    tol = (t / 16 + 36) * 2.0 ** -23 * (np.abs(vd) @ np.abs(vx).T)
    finite, past = np.abs(want) + tol < LARGEST, np.abs(want) - tol > LARGEST
    assert np.any(finite & (want != 0)) and np.all(np.abs(got - want)[finite] <= tol[finite])
    assert np.array_equal(got[past], np.copysign(np.inf, want[past]))


# several CTAs add parts of k: of few columns, whose sums are sent; of 64 and of 128, whose sums are read
SPLIT = [(1, 300, 8192), (30, 200, 4096), (200, 60, 8192), (256, 256, 8192)]


@pytest.mark.parametrize("ta,tb,power", TOPS)
@pytest.mark.parametrize("m,n,k", SPLIT)
def test_product_split_over_k(m, n, k, ta, tb, power):
    test_product(m, n, k, ta, tb, power)


@pytest.mark.parametrize("ta,tb", [(1e24, 1e24), (3e21, 1e24), (1e30, 1e30)])
@pytest.mark.parametrize("m,n,k", SPLIT + [(300, 300, 4096)])
def test_parts_that_cancel(m, n, k, ta, tb):
    """Sums over parts of k that leave F32 once the tensor scales are in them, and whose total does not: 0, or two terms."""
    q, p = np.full((m, k), 6.0), np.full((n, k), 6.0)
    q[:, k // 2:] = -6.0
    q[1::2, 0] = 4.0
    a, b = q * 2.0 ** -9, p * 2.0 ** -9
    codes = lambda v: torch.from_numpy(fp4.pack(v, k // 2)).cuda()  # noqa: E731
    scales = lambda r: torch.from_numpy(ref.tiles(np.full((r, k // 16), 0x01, np.uint8))).cuda()  # noqa: E731
    ga, gb = (torch.tensor([t], dtype=torch.float32, device="cuda") for t in (ta, tb))
    ra, rb = (float(np.float32(1) / fp4.tensor_scale(t)) for t in (ta, tb))
    want = (a @ b.T) * ra * rb
    out = torch.full((m, n), -3.0, device="cuda")
    api.nvfp4_gemm(codes(q), scales(m), ga, codes(p), scales(n), gb, None, out, m, n, k)
    api.mxfp8_device_status()
    got = ref.as64(out)
    assert not np.any(np.isnan(got))
    fits = np.abs(want) < 3.38e38
    assert np.all(np.abs(got - want)[fits] <= 2 * U * (1 + U) * np.abs(want)[fits])
    assert np.array_equal(got[~fits], np.copysign(np.inf, want[~fits]))
