"""Block-scaled products against float64.  Products of E4M3 values are exact, so the error is that
of summing k exact terms in F32: at most (k / 32 + 32) roundings or truncations of 2^-23 of the
running magnitude, bounded by sum |a b|; a BF16 result adds half a unit, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from mxfp8_master_weight_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SPECIAL = (0x7F, 0xFF)


def tiled(byte):
    return torch.from_numpy(ref.tiles(byte)).cuda()


def operand(rng, mn, k, colwise, block, pitch=None, offset=0, spread=6):
    """Random codes of an operand (values [mn][k] in float64), its buffer and scales."""
    code = rng.integers(0, 256, (mn, k), dtype=np.uint8)
    code[np.isin(code, SPECIAL)] = 0x38
    byte = rng.integers(127 - spread, 127 + spread + 1, (mn, -(-k // block)), dtype=np.uint8)
    stored = code.T if colwise else code
    pitch = pitch or stored.shape[1]
    buf = torch.full((stored.shape[0] * pitch + offset,), 0x7F, dtype=torch.uint8, device="cuda")
    view = buf[offset:].view(stored.shape[0], pitch)
    view[:, :stored.shape[1]] = torch.from_numpy(np.ascontiguousarray(stored)).cuda()
    val = torch.from_numpy(code).view(torch.float8_e4m3fn).double().numpy()
    val = val * np.repeat(np.ldexp(1.0, byte.astype(np.int32) - 127), block, axis=1)[:, :k]
    return val, view, tiled(byte)


def check(out, a, b, k, c=None):
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if c is not None:
        want, mag = want + c, mag + np.abs(c)
    tol = (k / 32 + 34) * 2.0 ** -23 * mag
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    got = ref.as64(out)
    err = np.abs(got - want)
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


def run(m, n, k, acol=False, bcol=False, ablk=128, bblk=128, dtype="f32", pitch=16, offset=0, addend=False, seed=0):
    rng = np.random.default_rng(seed + m * 31 + n * 17 + k)
    up = lambda w: -(-w // pitch) * pitch  # noqa: E731
    a, qa, sa = operand(rng, m, k, acol, ablk, up(m if acol else k), offset)
    b, qb, sb = operand(rng, n, k, bcol, bblk, up(n if bcol else k), offset)
    out = torch.full((m, n + 3), -3.0, dtype=DT[dtype], device="cuda")
    c = torch.randn(m, n, device="cuda") * k if addend else None
    api.mxfp8_gemm(qa, sa, qb, sb, c, out[:, :n], m, n, k, acol, bcol, ablk, bblk)
    api.mxfp8_device_status()
    check(out[:, :n], a, b, k, None if c is None else ref.as64(c))
    assert bool((out[:, n:] == -3.0).all())


SHAPES = [(1, 1, 1), (1, 16, 32), (3, 5, 7), (1, 4096, 640), (16, 256, 512), (64, 1000, 2048), (127, 129, 131),
          (128, 128, 128), (256, 256, 512), (257, 255, 1030), (300, 77, 4096), (512, 768, 96), (1000, 16, 1000)]


@pytest.mark.parametrize("acol,bcol", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_layouts(m, n, k, acol, bcol):
    run(m, n, k, acol, bcol)


@pytest.mark.parametrize("ablk,bblk", [(128, 32), (32, 128), (32, 32)])
@pytest.mark.parametrize("m,n,k", [(8, 256, 200), (130, 200, 1111), (300, 520, 1024)])
def test_block_sizes(m, n, k, ablk, bblk):
    run(m, n, k, ablk=ablk, bblk=bblk)
    run(m, n, k, True, True, ablk, bblk, dtype="bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pitch,offset", [(1, 0), (1, 3), (4, 4), (2, 2), (16, 8)])
def test_unaligned_operands(pitch, offset, dtype):
    """Rows and bases off 16 bytes, down to single bytes, each layout."""
    for acol, bcol in ((False, False), (False, True), (True, True)):
        run(131, 203, 259, acol, bcol, dtype=dtype, pitch=pitch, offset=offset)
        run(5, 333, 515, acol, bcol, dtype=dtype, pitch=pitch, offset=offset)


@pytest.mark.parametrize("m,n,k", [(5, 9, 100), (256, 512, 384), (200, 300, 4096), (2048, 2048, 256), (1024, 256, 8192)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_addend(m, n, k, dtype):
    run(m, n, k, True, True, dtype=dtype, addend=True)


@pytest.mark.parametrize("m,n,k", [(1024, 2048, 1536), (2560, 1280, 768), (4096, 300, 640), (777, 4097, 272)])
def test_many_tiles(m, n, k):
    run(m, n, k, dtype="bf16", bblk=32)
    run(m, n, k, False, True)


def test_addend_in_place_and_repeatable():
    """Gradient accumulation: out += product; equal calls give equal bits."""
    rng = np.random.default_rng(3)
    a, qa, sa = operand(rng, 384, 2048, True, 128)
    b, qb, sb = operand(rng, 512, 2048, True, 128)
    outs = []
    for _ in range(3):
        out = torch.ones(384, 512, device="cuda")
        api.mxfp8_gemm(qa, sa, qb, sb, out, out, 384, 512, 2048, True, True)
        outs.append(out)
    check(outs[0], a, b, 2048, np.ones((384, 512)))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("m,n", [(1, 1), (40, 70), (300, 260)])
def test_no_contraction(m, n):
    """k = 0: the empty sum."""
    out = torch.full((m, n), 5.0, device="cuda")
    api.mxfp8_gemm(None, None, None, None, None, out, m, n, 0)
    assert bool((out == 0).all())
    c = torch.randn(m, n, device="cuda")
    api.mxfp8_gemm(None, None, None, None, c, out, m, n, 0)
    assert torch.equal(out, c)
    api.mxfp8_gemm(None, None, None, None, None, None, 0, n, 64)


@pytest.mark.parametrize("m,n,k", [(7, 200, 300), (300, 400, 640)])
def test_nan_stays_in_its_row_and_column(m, n, k):
    """A NaN code, and a block with the NaN scale, reach exactly the outputs that read them."""
    rng = np.random.default_rng(0)
    a, qa, sa = operand(rng, m, k, False, 128)
    b, qb, sb = operand(rng, n, k, False, 128)
    qa[3, 129], qb[150, 1] = 0x7F, 0xFF
    byte = np.full((n, -(-k // 128)), 127, np.uint8)
    byte[60, 1] = 255
    sb = tiled(byte)
    out = torch.zeros(m, n, device="cuda")
    api.mxfp8_gemm(qa, sa, qb, sb, None, out, m, n, k)
    want = torch.zeros(m, n, dtype=torch.bool)
    want[3], want[:, 150], want[:, 60] = True, True, True
    assert torch.equal(torch.isnan(out).cpu(), want)


def test_extreme_scales():
    """The smallest and largest scale bytes: products that underflow and that nearly overflow."""
    k = 128
    qa = torch.full((32, k), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    qb = torch.full((64, k), 0x38, dtype=torch.uint8, device="cuda")
    for ea, eb, want in ((0, 0, 0.0), (0, 254, 128.0), (254, 0, 128.0), (240, 130, 128.0 * 2.0 ** 116), (100, 60, 128.0 * 2.0 ** -94)):
        sa, sb = tiled(np.full((32, 1), ea, np.uint8)), tiled(np.full((64, 1), eb, np.uint8))
        out = torch.ones(32, 64, device="cuda")
        api.mxfp8_gemm(qa, sa, qb, sb, None, out, 32, 64, k)
        assert bool((out.double() == want).all()), (ea, eb, out[0, 0].item())


def test_mxfp8_weights_from_the_cast():
    """The product of a checkpoint and a weight that the master-weight cast wrote, forward and
    towards the input, from the cast's own grids through mxfp8_swizzle_scales."""
    outs, ins, tokens = 320, 416, 200
    w = torch.randn(outs, ins, device="cuda") * 0.02
    (rr, rc), (cr, cc) = api.block_shapes(outs, ins)
    sr, sc = torch.empty(rr, rc, dtype=torch.uint8, device="cuda"), torch.empty(cr, cc, dtype=torch.uint8, device="cuda")
    qr, qc = (torch.empty(outs * ins, dtype=torch.uint8, device="cuda") for _ in range(2))
    api.mxfp8_quantize_whole_blocks(w, None, None, sr, sc, qr, qc, outs, ins, 0)
    tr = torch.empty(api.mxfp8_swizzled_scales_size(rr, rc), dtype=torch.uint8, device="cuda")
    tcw = torch.empty(api.mxfp8_swizzled_scales_size(cr, cc, True), dtype=torch.uint8, device="cuda")
    api.mxfp8_swizzle_scales(sr, tr, rr, rc)
    api.mxfp8_swizzle_scales(sc, tcw, cr, cc, transpose=True)
    # the cast takes block maxima of the master values and codes of their BF16 roundings
    w64, w16 = ref.as64(w), ref.as64(w.bfloat16())
    wr, wc = ref.quantise(w16, 32, w64)[0], ref.quantise(w16.T, 32, w64.T)[0].T
    for width, q, s, colwise, val in ((ins, qr, tr, False, wr), (outs, qc, tcw, True, wc.T)):
        x = torch.randn(tokens, width, device="cuda")
        qx = torch.empty(tokens, width, dtype=torch.uint8, device="cuda")
        sx = torch.empty(api.mxfp8_swizzled_scales_size(tokens, -(-width // 128)), dtype=torch.uint8, device="cuda")
        api.mxfp8_checkpoint_save(x, qx, sx, None, None, tokens, width)
        other = val.shape[0]
        y = torch.empty(tokens, other, device="cuda")
        api.mxfp8_gemm(qx, sx, q, s, None, y, tokens, other, width, b_colwise=colwise, b_block=32)
        check(y, ref.quantise(ref.as64(x))[0], val, width)


def test_streams_and_graph():
    rng = np.random.default_rng(5)
    a, qa, sa = operand(rng, 300, 1024, False, 128)
    b, qb, sb = operand(rng, 520, 1024, False, 128)
    outs = [torch.zeros(300, 520, device="cuda") for _ in range(3)]
    sts = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for o, st in zip(outs, sts):
        with torch.cuda.stream(st):
            api.mxfp8_gemm(qa, sa, qb, sb, None, o, 300, 520, 1024)
    torch.cuda.synchronize()
    call = api.prepare_gemm(qa, sa, qb, sb, None, outs[0], 300, 520, 1024)
    g = torch.cuda.CUDAGraph()
    outs[0].zero_()
    with torch.cuda.graph(g):
        call.call()
        call.call()
    g.replay()
    torch.cuda.synchronize()
    for o in outs:
        check(o, a, b, 1024)


def test_refusals():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    q, s, out = u8(64, 128), u8(512), torch.zeros(64, 64, device="cuda")

    def status(*a, **kw):
        with pytest.raises(api.MXFP8Error) as e:
            api.mxfp8_gemm(*a, **kw)
        return e.value.status

    assert status(q, s, q, s, None, None, 64, 64, 128) == 4
    assert status(None, s, q, s, None, out, 64, 64, 128) == 4
    assert status(q, None, q, s, None, out, 64, 64, 128) == 4
    assert status(q, s, q, s, None, out, 64, 64, 129) == 2
    assert status(q, s, q, s, None, out, 64, 65, 128) == 2
    assert status(q, s[:511], q, s, None, out, 64, 64, 128) == 2
    assert status(q, u8(528)[1:], q, s, None, out, 64, 64, 128) == 1
    assert status(q, s, q, s, None, out, 64, 64, 128, a_block=64) == 1
    assert status(q, s, q, s, None, out, -1, 64, 128) == 1
    assert status(q, s, q, s, None, out.half(), 64, 64, 128) == 3
    assert status(out, s, q, s, None, out, 64, 64, 64) == 3
    assert status(q, s, q, s, out.bfloat16(), out, 64, 64, 128) == 3
    big = torch.zeros(64 * 64 + 16, device="cuda")
    assert status(q, s, q, s, big[16:].view(64, 64), big[:4096].view(64, 64), 64, 64, 128) == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("m,n,k", [(1, 300, 256), (300, 1, 512), (16, 1000, 1024), (13, 130, 4096), (1030, 29, 2048),
                                   (50, 516, 640), (516, 64, 1100), (64, 2052, 4096), (96, 130, 2304), (515, 500, 4096)])
def test_few_tiles(m, n, k, pad, dtype):
    """One to eight CTAs per tile, either operand on the tile's lanes; output rows on 16 bytes, whole or
    with a ragged end, and off them; lines of the tile past the output."""
    rng = np.random.default_rng(m + n + k)
    a, qa, sa = operand(rng, m, k, False, 128, -(-k // 16) * 16)
    b, qb, sb = operand(rng, n, k, False, 32, -(-k // 16) * 16)
    pitch = -(-n // 8) * 8 + 8 + pad
    buf = torch.full((m, pitch), -3.0, dtype=DT[dtype], device="cuda")
    c = torch.randn(m, pitch, device="cuda") * k
    for addend in (None, c[:, :n]):
        api.mxfp8_gemm(qa, sa, qb, sb, addend, buf[:, :n], m, n, k, b_block=32)
        api.mxfp8_device_status()
        check(buf[:, :n], a, b, k, None if addend is None else ref.as64(addend))
        assert bool((buf[:, n:] == -3.0).all())


def test_one_row_many_times():
    """Launches that follow one another, most lines of their tiles empty: equal bits every time."""
    rng = np.random.default_rng(8)
    a, qa, sa = operand(rng, 1, 4096, False, 128)
    b, qb, sb = operand(rng, 2048, 4096, False, 32)
    outs = torch.empty(64, 1, 2048, device="cuda")
    for o in outs:
        api.mxfp8_gemm(qa, sa, qb, sb, None, o, 1, 2048, 4096, b_block=32)
    api.mxfp8_device_status()
    check(outs[0], a, b, 4096)
    assert bool((outs == outs[:1]).all())
