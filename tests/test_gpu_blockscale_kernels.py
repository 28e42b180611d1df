"""Every kernel of fp8_gemm_blockscale against the product in 64 bits
(tolerance: layer_ref.assert_gemm), on the shapes of tests/blockscale_shapes."""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import layer_ref as ref
from tests.blockscale_shapes import ALL, KSPLIT, TILES
from tests.test_gpu_gemm_blockscale import DEV, _check, _operands, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel,shape", ALL)
def test_matches_the_product_in_64_bits(kernel, shape):
    assert qp.fp8_gemm_blockscale_kernel(*shape) == kernel
    _check(*shape, seed=11)


# a shape of every tile kernel, ragged and whole K, and a few with K split
SOME = [shapes[i] for shapes in TILES.values() for i in (-2, -1)] + [shapes[0] for shapes in KSPLIT.values()][::4]


@pytest.mark.parametrize("shape", SOME)
def test_same_bits_twice_and_on_a_stream(shape):
    m, n, _ = shape
    a, sa, w, sw = _operands(*shape, 12)
    one = _run(a, sa, w, sw)
    st = torch.cuda.Stream()
    room = torch.full((m * n + 64,), 3.0, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    qp.fp8_gemm_blockscale(a, sa, w, sw, room[:m * n].view(m, n), stream=st)
    st.synchronize()
    assert torch.equal(one.view(torch.int16), room[:m * n].view(m, n).view(torch.int16))
    assert torch.all(room[m * n:] == 3.0)


@pytest.mark.parametrize("shape", SOME)
def test_scales_reach_their_own_rows_and_blocks(shape):
    """Each output is one scaled block's sum: the row's other blocks are switched
    off by a zero scale."""
    m, n, k = shape
    kb = -(-k // 128)
    a, _, w, _ = _operands(m, n, k, 13)
    sa = torch.zeros((m, kb), device=DEV)
    rows = torch.arange(m, device=DEV)
    sa[rows, rows % kb] = 2.0 ** ((rows % 23).float() - 11)
    sw = 2.0 ** (torch.arange(-(-n // 128) * kb, device=DEV).reshape(-1, kb) % 19 - 9).float()
    ref.assert_gemm(_run(a, sa, w, sw), ref.gemm_blockscale(a, sa, w, sw), 128)
