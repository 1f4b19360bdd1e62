"""8-bit activation checkpoints against their definition in 64 bits: codes, scales and restored
values are exact (one rounding, powers of two), so every comparison is for equality."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from mxfp8_master_weight_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def u8(*shape, fill=0xA5):
    return torch.full(shape, fill, dtype=torch.uint8, device="cuda")


def scales(rows, cols, block=128):
    return u8(api.mxfp8_swizzled_scales_size(rows, -(-cols // block)), fill=0xEE)


def equal(a, b):
    return np.array_equal(a, b, equal_nan=True)


def save_and_check(x, row=True, col=True, pad=0, offset=0):
    """Saves x; checks codes, scales, what must stay untouched, and both restored types."""
    rows, cols = x.shape
    buf = [u8(rows * (cols + pad) + offset)[offset:].view(rows, cols + pad) if d else None for d in (row, col)]
    sr, sc = scales(rows, cols) if row else None, scales(cols, rows) if col else None
    api.mxfp8_checkpoint_save(x, buf[0], sr, buf[1], sc, rows, cols)
    x64 = ref.as64(x)
    for q, s, colwise in ((buf[0], sr, False), (buf[1], sc, True)):
        if q is None:
            continue
        kept, codes, byte = ref.quantise(x64.T if colwise else x64)
        if colwise:
            kept, codes = kept.T, codes.T
        assert equal(ref.codes_to_values(q[:, :cols]), codes)
        assert np.all(q[:, cols:].cpu().numpy() == 0xA5)
        assert np.array_equal(s.cpu().numpy(), ref.tiles(byte))
        for dt in DT.values():
            out = torch.full((rows, cols + pad), 7.0, dtype=dt, device="cuda")
            api.mxfp8_checkpoint_restore(q, s, out, rows, cols, colwise=colwise)
            want = torch.from_numpy(kept).to(torch.float32).to(dt)
            assert equal(ref.as64(out[:, :cols]), ref.as64(want))
            assert bool((out[:, cols:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 5), (2, 4096), (127, 129), (128, 128), (129, 257),
                                       (160, 96), (1000, 333), (513, 640)])
def test_save_and_restore(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(4 * torch.randn(rows, 1, generator=g, device="cuda"))
    save_and_check(x.to(DT[dtype]))


@pytest.mark.parametrize("row,col", [(True, False), (False, True)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_direction(row, col, dtype):
    x = torch.randn(150, 300, device="cuda").to(DT[dtype])
    save_and_check(x, row, col)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_special_values(dtype):
    """Zero blocks, NaN and infinities (their whole blocks become NaN), subnormals, the largest
    values, signed zeros, ties and the saturating band [448, 512)."""
    x = torch.randn(300, 520, device="cuda")
    x[:40] = 0.0
    x[:, 130:270] *= 1e-38
    x[128:, 256:384] = 0.0
    x[5, 400], x[70, 3], x[299, 519] = float("nan"), float("inf"), float("-inf")
    x[200, :64] = torch.linspace(440, 511.9, 64)
    x[201, :64] = torch.arange(64) / 16 + 16.5
    x[202, 0], x[203, 0] = 3.0e38, -3.0e38
    x[204, 384:512] = -0.0
    x[205, 384:512] = 1e-44
    save_and_check(x.to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift,pad", [(1, 3), (2, 16), (0, 8)])
def test_strides_and_offsets(dtype, shift, pad):
    """A slice of a wider buffer, off 16-byte alignment; codes in padded or unaligned rows."""
    wide = torch.randn(200, 300 + shift + 5, device="cuda").to(DT[dtype])
    save_and_check(wide[:, shift:shift + 300], pad=pad, offset=shift)


def test_large_offsets():
    """Rows whose byte offsets pass 2^32 in the input and 2^31 in the codes."""
    rows, cols, stride = 9, 200, 1 << 28
    x = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda").view(rows, stride)[:, :cols]
    x.copy_(torch.randn(rows, cols, device="cuda"))
    q = torch.empty(rows * stride, dtype=torch.uint8, device="cuda").view(rows, stride)
    s = scales(rows, cols)
    api.mxfp8_checkpoint_save(x, q, s, None, None, rows, cols)
    kept, codes, byte = ref.quantise(ref.as64(x))
    assert equal(ref.codes_to_values(q[:, :cols]), codes)
    out = torch.empty(rows, cols, device="cuda")
    api.mxfp8_checkpoint_restore(q, s, out, rows, cols)
    assert equal(ref.as64(out), kept)


def test_other_stream_and_graph():
    x = torch.randn(256, 512, device="cuda")
    q, s = u8(256, 512), scales(256, 512)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call = api.prepare_checkpoint_save(x, q, s, None, None, 256, 512)
        call.call()
    st.synchronize()
    first = q.clone()
    g = torch.cuda.CUDAGraph()
    q.zero_()
    with torch.cuda.graph(g):
        call.call()
    x.mul_(-1.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q ^ 0x80, first)


def test_empty():
    e = torch.empty(0, 64, device="cuda")
    api.mxfp8_checkpoint_save(e, None, None, None, None, 0, 64)
    api.mxfp8_checkpoint_restore(None, None, e, 0, 64)


def test_refusals():
    x, q, s = torch.zeros(64, 64, device="cuda"), u8(64, 64), scales(64, 64)

    def status(*a, fn=api.mxfp8_checkpoint_save, **kw):
        with pytest.raises(api.MXFP8Error) as e:
            fn(*a, **kw)
        return e.value.status

    assert status(x, None, None, None, None, 64, 64) == 4
    assert status(None, q, s, None, None, 64, 64) == 4
    assert status(x, q, None, None, None, 64, 64) == 4
    assert status(x, q, s, None, None, 65, 64) == 2
    assert status(x, q, s[:-1], None, None, 64, 64) == 2
    assert status(x, q[:, :60], s, None, None, 64, 64) == 2
    assert status(x, x, s, None, None, 64, 64) == 3
    assert status(x.to(torch.uint8), q, s, None, None, 64, 64) == 3
    assert status(x, q, u8(4096)[1:], None, None, 64, 64) == 1
    assert status(x, q, s, None, None, -1, 64) == 1
    assert status(x.t()[:, :32], q, s, None, None, 32, 32) == 5
    assert status(q, s, x, 64, 65, fn=api.mxfp8_checkpoint_restore) == 2
    assert status(q, s, q, 64, 64, fn=api.mxfp8_checkpoint_restore) == 3
