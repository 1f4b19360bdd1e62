"""Products of more tiles than the GPU has pairs of SMs: a pair's second and later tiles, whole tiles followed by
halves, every way an operand can lie, operands that are realigned; against float64 on the GPU with the
bound of test_gpu_gemm: (k / 32 + 34) roundings of 2^-23 of sum |a b|, and half a unit of BF16."""
import pytest
import torch

from mxfp8_master_weight_gb300 import api

pytestmark = pytest.mark.gpu


def operand(g, mn, k, colwise, block, pitch, offset):
    """Values [mn][k] in float64, the stored codes in rows of `pitch` from byte `offset`, scales."""
    rows, cols = (k, mn) if colwise else (mn, k)
    code = torch.randint(0, 256, (rows, cols), generator=g, device="cuda", dtype=torch.uint8)
    code[(code & 0x7F) == 0x7F] = 0x38
    buf = torch.full((rows * pitch + offset,), 0x7F, dtype=torch.uint8, device="cuda")
    view = buf[offset:].view(rows, pitch)
    view[:, :cols] = code
    nb = -(-k // block)
    byte = torch.randint(121, 134, (mn, nb), generator=g, device="cuda", dtype=torch.uint8)
    val = code.view(torch.float8_e4m3fn).double()
    val = (val.t() if colwise else val) * torch.exp2(byte.double() - 127).repeat_interleave(block, 1)[:, :k]
    r, c = -(-mn // 128), -(-nb // 4)
    grid = torch.nn.functional.pad(byte, (0, 4 * c - nb, 0, 128 * r - mn))
    return val, view, grid.view(r, 4, 32, c, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def run(m, n, k, acol=False, bcol=False, ablk=128, bblk=128, dtype=torch.float32, addend=False, apitch=16, bpitch=16, offset=(0, 0)):
    g = torch.Generator(device="cuda").manual_seed(m * 31 + n * 17 + k)
    up = lambda w, p: -(-w // p) * p  # noqa: E731
    a, qa, sa = operand(g, m, k, acol, ablk, up(m if acol else k, apitch), offset[0])
    b, qb, sb = operand(g, n, k, bcol, bblk, up(n if bcol else k, bpitch), offset[1])
    out = torch.full((m, n + 3), -3.0, dtype=dtype, device="cuda")
    c = torch.randn(m, n, generator=g, device="cuda") * k if addend else None
    api.mxfp8_gemm(qa, sa, qb, sb, c, out[:, :n], m, n, k, acol, bcol, ablk, bblk)
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    if addend:
        want, mag = want + c, mag + c.abs()
    tol = (k / 32 + 34) * 2.0 ** -23 * mag
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    worst = ((out[:, :n].double() - want).abs() / tol.clamp(min=1e-300)).max().item()
    assert worst <= 1.0, f"worst {worst:.3g} of the tolerance"
    assert bool((out[:, n:] == -3.0).all())
    api.mxfp8_device_status()


# with 76 pairs: 90 tiles (76 whole, 28 halves); 121 (all whole, 45 of them second); 289 (four rounds); 256 (three
# rounds, then halves); 79 (3 tiles left: 6 halves behind whole ones)
SHAPES = [(2560, 2304, 640), (2816, 2816, 384), (4352, 4352, 256), (4096, 4096, 200), (256, 20224, 512)]
LAYOUTS = [(False, False), (False, True), (True, False), (True, True)]


@pytest.mark.parametrize("acol,bcol", LAYOUTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_later_tiles(m, n, k, acol, bcol):
    run(m, n, k, acol, bcol)
    run(m, n, k, acol, bcol, dtype=torch.bfloat16, bblk=32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(2560, 2304, 1152), (2801, 2789, 130), (2048, 8192, 256)])
def test_later_tiles_with_addend(m, n, k, dtype):
    run(m, n, k, True, True, dtype=dtype, addend=True)
    run(m, n, k, dtype=dtype, addend=True, ablk=32, bblk=32)


@pytest.mark.parametrize("m,n,k", [(2561, 2303, 1), (2817, 2800, 129), (4099, 4090, 33)])
def test_ragged_later_tiles(m, n, k):
    for acol, bcol in LAYOUTS:
        run(m, n, k, acol, bcol, dtype=torch.bfloat16)


@pytest.mark.parametrize("offset", [(0, 3), (5, 0), (7, 9)])
@pytest.mark.parametrize("acol,bcol", LAYOUTS)
@pytest.mark.parametrize("m,n,k", [(2561, 2303, 645), (2817, 2811, 1029), (2305, 4609, 259)])
def test_realigned_whole_tiles(m, n, k, acol, bcol, offset):
    """Either operand off 16 bytes, and both: boxes of whole and of half tiles, many stages through three raw boxes."""
    run(m, n, k, acol, bcol, apitch=1 if offset[0] else 16, bpitch=1 if offset[1] else 16, offset=offset)
    run(m, n, k, acol, bcol, apitch=1, bpitch=1, offset=offset, dtype=torch.bfloat16, bblk=32)


def test_equal_bits_every_time():
    g = torch.Generator(device="cuda").manual_seed(0)
    m, n, k = 2560, 2304, 640
    _, qa, sa = operand(g, m, k, False, 128, k, 0)
    _, qb, sb = operand(g, n, k, False, 32, k, 0)
    outs = torch.empty(5, m, n, device="cuda")
    for o in outs:
        api.mxfp8_gemm(qa, sa, qb, sb, None, o, m, n, k, b_block=32)
    api.mxfp8_device_status()
    assert bool((outs == outs[:1]).all())
