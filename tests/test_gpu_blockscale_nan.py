"""fp8_gemm_blockscale keeps a NaN to the row of A or of W that holds it, in
every kernel and wherever the row ends: the other outputs have the bits that
they have without it."""
import pytest
import torch

from tests.test_gpu_gemm_blockscale import _operands, _run

pytestmark = pytest.mark.gpu

# waves that split K; 128 x 128 tiles; 256 x 256 tiles without and with a tail
# of 128 x 128 ones
SHAPES = [(4, 260, 2368), (40, 260, 144), (600, 4104, 2368), (2816, 4480, 1040), (4090, 4099, 2064)]


def _same_but(one, two, rows=(), cols=()):
    bad = torch.zeros(one.shape, dtype=torch.bool, device=one.device)
    for r in rows:
        bad[r] = True
    for c in cols:
        bad[:, c] = True
    assert torch.isnan(two[bad]).all()
    assert torch.equal(one.view(torch.int16)[~bad], two.view(torch.int16)[~bad])


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_nan_codes_stay_in_their_row_of_w(m, n, k):
    a, sa, w, sw = _operands(m, n, k, 31)
    one = _run(a, sa, w, sw)
    assert torch.isfinite(one).all()
    cols = (0, 17, n // 2, n - 1)
    for c in cols:
        w[c] = 0x7F
    _same_but(one, _run(a, sa, w, sw), cols=cols)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_nan_codes_and_scales_stay_in_their_row_of_a(m, n, k):
    a, sa, w, sw = _operands(m, n, k, 32)
    one = _run(a, sa, w, sw)
    rows = (0, m // 2, m - 1)
    for r in rows[:2]:
        a[r] = 0xFF
    sa[m - 1] = float("nan")
    _same_but(one, _run(a, sa, w, sw), rows=rows)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_nan_scales_stay_in_their_block_of_w(m, n, k):
    a, sa, w, sw = _operands(m, n, k, 33)
    one = _run(a, sa, w, sw)
    sw[1, -1] = float("nan")
    _same_but(one, _run(a, sa, w, sw), cols=range(128, min(256, n)))
