"""Addend and output as column ranges of one buffer: fine where they share no element, refused where they do."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from mxfp8_master_weight_gb300 import api
from test_gpu_gemm import check, operand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,gap", [(33, 40, 200, 0), (300, 260, 384, 0), (5, 7, 64, 1), (130, 129, 640, 3), (1, 50, 64, 0)])
def test_column_ranges_of_one_buffer(m, n, k, gap):
    rng = np.random.default_rng(m + n)
    a, qa, sa = operand(rng, m, k, False, 128)
    b, qb, sb = operand(rng, n, k, False, 128)
    first, last = slice(0, n), slice(n + gap, 2 * n + gap)
    for add, to in ((first, last), (last, first)):
        buf = torch.randn(m, 2 * n + gap, device="cuda") * k
        keep, c = buf.clone(), ref.as64(buf[:, add])
        api.mxfp8_gemm(qa, sa, qb, sb, buf[:, add], buf[:, to], m, n, k)
        check(buf[:, to], a, b, k, c)
        buf[:, to] = keep[:, to]
        assert torch.equal(buf, keep)
    api.mxfp8_device_status()


def test_shared_elements_are_refused():
    m, n, k = 20, 30, 64
    q, s = torch.zeros(64, k, dtype=torch.uint8, device="cuda"), torch.full((512,), 127, dtype=torch.uint8, device="cuda")
    buf = torch.zeros(m + 1, 3 * n, device="cuda")

    def status(addend, out):
        try:
            api.mxfp8_gemm(q, s, q, s, addend, out, m, n, k)
        except api.MXFP8Error as e:
            return e.status
        return 0

    part = lambda c, r=0: buf[r:r + m, c:c + n]  # noqa: E731
    for c in (1, n - 1):
        assert status(part(0), part(c)) == 1 and status(part(c), part(0)) == 1  # ranges that share columns
    assert status(part(0), part(0, 1)) == 1 and status(part(0, 1), part(0)) == 1  # the same columns, a row apart
    assert status(part(n), part(0, 1)) == 0 and status(part(0, 1), part(2 * n)) == 0
    # a row of the addend that runs on into the output's next row
    flat = buf.view(-1)
    wrapped = flat[2 * n + 1:2 * n + 1 + (m - 1) * 3 * n + n].as_strided((m, n), (3 * n, 1))
    assert status(wrapped, part(0)) == 1 and status(part(0), wrapped) == 1
    assert status(part(0), buf[:, :].view(-1)[n:n + m * n].view(m, n)) == 1         # another row stride
    assert status(buf[:1, :n].expand(1, n), part(0)) != 0                            # one row is no m x n addend
    assert status(part(0), part(0)) == 0                                             # the same matrix
    torch.cuda.synchronize()
