"""NVFP4 operands against the convention: codes, scales and restored values are equal, every step of theirs being one
rounding; products against float64.  A product's terms q_a q_b s_a s_b are exact in F32 (10 bits), 64 of them join the sum
per instruction: at most (k / 16 + 32) roundings or truncations of 2^-23 of the running magnitude, bounded by
sum |a b|, and four of the tensor scales and the addend; a BF16 result adds half a unit, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import fp4_ref as fp4
import linear_ref as ref
from mxfp8_master_weight_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def u8(*shape, fill=0xA5):
    return torch.full(shape, fill, dtype=torch.uint8, device="cuda")


def pitch(n):
    return -(-n // 16) * 16


def scales(rows, cols):
    return u8(api.mxfp8_swizzled_scales_size(rows, -(-cols // 16)))


def values(rows, cols, dtype, seed=0):
    """Normal values over many magnitudes, with whole blocks of zeros and lone values among them."""
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-12, 5, (rows, 1), generator=g, device="cuda").float())
    x[:, (torch.arange(cols, device="cuda") // 16) % 5 == 3] = 0.0
    x[(torch.arange(rows, device="cuda") // 16) % 3 == 1] *= 2.0 ** -14
    return x.to(DT[dtype])


def amax(x, rows, cols, before=None):
    top = torch.full((1,), 0.0 if before is None else before, device="cuda")
    api.nvfp4_tensor_amax(x, top, rows, cols, accumulate=before is not None)
    return top


SHAPES = [(1, 1), (1, 16), (1, 17), (2, 15), (3, 4096), (16, 16), (31, 33), (128, 128), (129, 130), (160, 96), (257, 1023),
          (1000, 31), (5, 6143)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantise_and_restore(rows, cols, dtype):
    x = values(rows, cols, dtype)
    x32 = x.float().cpu().numpy()
    top = amax(x, rows, cols)
    assert float(top) == np.abs(x32).max()
    q_r, s_r, q_c, s_c = u8(rows, pitch((cols + 1) // 2)), scales(rows, cols), u8(cols, pitch((rows + 1) // 2)), scales(cols, rows)
    api.nvfp4_quantize(x, top, q_r, s_r, q_c, s_c, rows, cols)
    for q, s, v in ((q_r, s_r, x32), (q_c, s_c, x32.T)):
        r, c = v.shape
        want, sv = fp4.quantise(v, float(top))
        assert np.array_equal(fp4.unpack(q, r, c), want)
        assert np.array_equal(s.cpu().numpy(), ref.tiles(fp4.scale_bytes(sv)))
        assert bool((q[:, (c + 1) // 2:] == 0xA5).all())
        for dt in (torch.float32, torch.bfloat16):
            out = torch.full((r, c + 3), -3.0, dtype=dt, device="cuda")
            api.nvfp4_restore(q, s, top, out[:, :c], r, c)
            assert torch.equal(out[:, :c].cpu(), torch.from_numpy(fp4.kept(v, float(top))).to(dt))
            assert bool((out[:, c:] == -3.0).all())
    # one direction alone writes the same
    for row in (True, False):
        q2, s2 = torch.full_like(q_r if row else q_c, 0xA5), torch.full_like(s_r if row else s_c, 0xA5)
        api.nvfp4_quantize(x, top, q2 if row else None, s2 if row else None, None if row else q2, None if row else s2, rows, cols)
        assert torch.equal(q2, q_r if row else q_c) and torch.equal(s2, s_r if row else s_c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_views_and_odd_strides(dtype):
    rows, cols = 70, 149
    wide = values(rows, cols + 60, dtype)
    for start in (0, 1, 8):
        x = wide[:, start:start + cols]
        x32 = x.float().cpu().numpy()
        top = amax(x, rows, cols)
        assert float(top) == np.abs(x32).max()
        q_r, q_c = u8(rows, 77)[:, 1:76], u8(cols, 41)[:, 3:38]
        s_r, s_c = scales(rows, cols), scales(cols, rows)
        api.nvfp4_quantize(x, top, q_r, s_r, q_c, s_c, rows, cols)
        for q, s, v in ((q_r, s_r, x32), (q_c, s_c, x32.T)):
            want, sv = fp4.quantise(v, float(top))
            assert np.array_equal(fp4.unpack(q, *v.shape), want)
            assert np.array_equal(s.cpu().numpy(), ref.tiles(fp4.scale_bytes(sv)))
            out = torch.zeros(v.shape[0], v.shape[1] + 5, device="cuda")[:, 1:1 + v.shape[1]]
            api.nvfp4_restore(q, s, top, out, *v.shape)
            assert np.array_equal(out.cpu().numpy(), fp4.kept(v, float(top)))


@pytest.mark.parametrize("top", [0.0, 1e-38, 3e-36, 1e-3, 0.37, 2688.0, 1e30])
def test_given_maximum(top):
    """A maximum from elsewhere: larger than the values', smaller (saturates), tiny (S at its largest)."""
    rows, cols = 33, 64
    x = values(rows, cols, "f32") * max(top, 1e-38)
    t = torch.tensor([top], device="cuda")
    q, s = u8(rows, 32), scales(rows, cols)
    api.nvfp4_quantize(x, t, q, s, None, None, rows, cols)
    want, sv = fp4.quantise(x.cpu().numpy(), top)
    assert np.array_equal(fp4.unpack(q, rows, cols), want)
    assert np.array_equal(s.cpu().numpy(), ref.tiles(fp4.scale_bytes(sv)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_not_finite(dtype):
    rows, cols = 48, 80
    x = values(rows, cols, dtype)
    x[3, 20], x[17, 5], x[40, 79] = float("nan"), float("inf"), -float("inf")
    top = torch.full((1,), float(x[torch.isfinite(x)].abs().max()), device="cuda")
    q, s = u8(rows, 48), scales(rows, cols)
    out = torch.empty(rows, cols, device="cuda")
    api.nvfp4_quantize(x, top, q, s, None, None, rows, cols)
    api.nvfp4_restore(q, s, top, out, rows, cols)
    want = torch.zeros(rows, cols, dtype=torch.bool)
    for r, c in ((3, 20), (17, 5), (40, 79)):
        want[r, c // 16 * 16:c // 16 * 16 + 16] = True
    assert torch.equal(torch.isnan(out).cpu(), want)
    # and through a product: the rows that hold one
    y = torch.empty(rows, rows, device="cuda")
    api.nvfp4_gemm(q, s, top, q, s, top, None, y, rows, rows, cols)
    bad = want.any(1)
    assert torch.equal(torch.isnan(y).cpu(), bad[:, None] | bad[None, :])
    # the maximum itself
    nan = amax(x, rows, cols)
    assert nan.view(torch.int32).item() == 0x7FC00000
    x[3, 20] = 0.0
    assert float(amax(x, rows, cols)) == float("inf")
    for t in (float("nan"), float("inf")):
        api.nvfp4_quantize(x, torch.tensor([t], device="cuda"), q, s, None, None, rows, cols)
        want = np.zeros((rows, 5), np.uint8) + 0x7F
        assert np.array_equal(s.cpu().numpy(), ref.tiles(want))


def test_amax_accumulates():
    x = torch.tensor([[1.0, -5.0], [2.0, 3.0]], device="cuda")
    assert float(amax(x, 2, 2, before=7.0)) == 7.0
    assert float(amax(x, 2, 2, before=4.0)) == 5.0
    assert float(amax(x, 2, 1)) == 5.0 or float(amax(x[:, :1], 2, 1)) == 2.0
    t = torch.full((1,), 9.0, device="cuda")
    api.nvfp4_tensor_amax(x[:0], t, 0, 2)
    assert float(t) == 0.0
    big = torch.zeros(9_000_001, dtype=torch.bfloat16, device="cuda")
    big[-1] = -2.5
    assert float(amax(big, 1, 9_000_001)) == 2.5


@pytest.mark.parametrize("rows,cols", [(1, 2), (7, 16), (16, 30), (128, 128), (130, 66), (333, 514)])
def test_lay_out(rows, cols):
    rng = np.random.default_rng(rows)
    code = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    src = torch.from_numpy(code).cuda()
    out = u8(rows, pitch(cols // 2))
    api.nvfp4_lay_out(src.view(-1), out, rows, cols)
    assert torch.equal(out[:, :cols // 2], src) and bool((out[:, cols // 2:] == 0xA5).all())
    turned = u8(cols, pitch((rows + 1) // 2))
    api.nvfp4_lay_out(src, turned, rows, cols, transpose=True)
    q = fp4.unpack(src, rows, cols)
    got = fp4.unpack(turned, cols, rows)
    assert np.array_equal(got, q.T) and np.array_equal(np.signbit(got), np.signbit(q.T))
    assert bool((turned[:, (rows + 1) // 2:] == 0xA5).all())


# ------------------------------------------------------------------------------ products
def operand(rng, mn, k, extra=0):
    """Random operand: its values before the tensor scale in float64, the buffers, the tensor's maximum."""
    q = fp4.LEVELS[rng.integers(0, 8, (mn, k))] * rng.choice([-1.0, 1.0], (mn, k))
    byte = rng.integers(8, 0x7F, (mn, -(-k // 16)), dtype=np.uint8)
    byte[rng.random(byte.shape) < 0.05] = 0
    s = torch.from_numpy(byte).view(torch.float8_e4m3fn).double().numpy()
    buf = fp4.pack(q, pitch((k + 1) // 2) + extra)
    buf[:, (k + 1) // 2:] = 0x77
    top = float(np.float32(rng.uniform(0.1, 30)))
    return q * fp4.spread(s, k), torch.from_numpy(buf).cuda(), torch.from_numpy(ref.tiles(byte)).cuda(), top


def check(out, a, b, k, ta, tb, c=None):
    f = float(np.float32(1) / fp4.tensor_scale(ta)) * float(np.float32(1) / fp4.tensor_scale(tb))
    want, mag = (a @ b.T) * f, (np.abs(a) @ np.abs(b).T) * f
    if c is not None:
        want, mag = want + c, mag + np.abs(c)
    tol = (k / 16 + 36) * 2.0 ** -23 * mag
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(ref.as64(out) - want)
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


def run(m, n, k, dtype="f32", addend=False, inplace=False, extra=0, over=3, seed=0):
    rng = np.random.default_rng(seed + m * 31 + n * 17 + k)
    a, qa, sa, ta = operand(rng, m, k, extra)
    b, qb, sb, tb = operand(rng, n, k, extra)
    ga, gb = torch.tensor([ta], device="cuda"), torch.tensor([tb], device="cuda")
    out = torch.full((m, n + over), -3.0, dtype=DT[dtype], device="cuda")
    c = torch.randn(m, n, device="cuda") * k if addend else None
    c64 = None if c is None else ref.as64(c)
    if inplace:
        out[:, :n] = c
        c = out[:, :n]
    api.nvfp4_gemm(qa, sa, ga, qb, sb, gb, c, out[:, :n], m, n, k)
    api.mxfp8_device_status()
    check(out[:, :n], a, b, k, ta, tb, c64)
    assert bool((out[:, n:] == -3.0).all())


@pytest.mark.parametrize("m,n,k", [(128, 128, 256), (1, 1, 1), (1, 1, 16), (1, 128, 64), (16, 128, 257), (17, 130, 255),
                                   (64, 64, 1000), (65, 300, 33), (100, 70, 511), (200, 300, 999), (1, 4096, 4096),
                                   (33, 515, 2049), (130, 1, 3001), (256, 256, 512), (257, 513, 1024)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_product(m, n, k, dtype):
    run(m, n, k, dtype)


@pytest.mark.parametrize("m,n,k", [(64, 256, 512), (300, 260, 300), (20, 1111, 999)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("over", [0, 3, 4, 8])
def test_product_with_addend(m, n, k, dtype, over):
    run(m, n, k, dtype, addend=True, over=over)
    if dtype == "f32":
        run(m, n, k, dtype, addend=True, inplace=True, over=over)


@pytest.mark.parametrize("m,n,k,extra", [(200, 300, 1000, 16), (40, 300, 1000, 48)])
def test_product_of_padded_rows(m, n, k, extra):
    run(m, n, k, extra=extra)


@pytest.mark.parametrize("m,n", [(77 * 256, 256), (76 * 256 + 1, 512), (38 * 256, 257)])
def test_product_of_many_tiles(m, n):
    """More tiles than pairs of SMs: both buffers of sums, whole and half tiles, in turn."""
    run(m, n, 520, "bf16")
    run(m, n, 77, "f32", addend=True)


def test_product_without_contraction():
    out = torch.full((5, 7), 3.0, device="cuda")
    api.nvfp4_gemm(None, None, None, None, None, None, None, out, 5, 7, 0)
    assert bool((out == 0).all())
    c = torch.randn(300, 7, device="cuda")
    out = torch.full((300, 7), 3.0, device="cuda")
    api.nvfp4_gemm(None, None, None, None, None, None, c, out, 300, 7, 0)
    assert torch.equal(out, c)


@pytest.mark.parametrize("m,n,k", [(64, 512, 4096), (1, 1024, 2048), (500, 500, 700), (4096, 4096, 512)])
def test_product_does_not_depend_on_the_run(m, n, k):
    rng = np.random.default_rng(5)
    _, qa, sa, ta = operand(rng, m, k)
    _, qb, sb, tb = operand(rng, n, k)
    ga, gb = torch.tensor([ta], device="cuda"), torch.tensor([tb], device="cuda")
    outs = [torch.empty(m, n, device="cuda") for _ in range(3)]
    for o in outs:
        api.nvfp4_gemm(qa, sa, ga, qb, sb, gb, None, o, m, n, k)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_zero_tensors():
    """A maximum of zero: S is 1, every code is zero, and products are zero."""
    x = torch.zeros(130, 64, device="cuda")
    top = amax(x, 130, 64)
    q, s = u8(130, 32), scales(130, 64)
    api.nvfp4_quantize(x, top, q, s, None, None, 130, 64)
    out = torch.full((130, 130), 3.0, device="cuda")
    api.nvfp4_gemm(q, s, top, q, s, top, None, out, 130, 130, 64)
    assert bool((out == 0).all()) and bool((s == 0).all())
