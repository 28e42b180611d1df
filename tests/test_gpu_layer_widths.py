"""Rows of 12, 23 and 24 blocks of 128, with a whole and a ragged last block:
12 and 24 are multiples of most of what the kernels step by."""
import pytest

import gemv_nvfp4_int8_amd as qp
from tests import layer_ref as ref
from tests.test_gpu_layer_quant import FMTS, REL, _check_norm, _normal, _outputs
from tests.test_gpu_moe import _check, _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [1, 16, 700])
@pytest.mark.parametrize("k", [1472, 2944, 3040])
def test_norm_and_activation(rows, k, fmt):
    _check_norm(_normal((rows, k), 1), _normal((rows, k), 2, 4.0), _normal((k,), 3), fmt)
    gu = _normal((rows, 2 * k), 4, 2.0)
    q, s = _outputs(rows, k, fmt)
    qp.silu_mul_quant(gu, fmt, q, s)
    ref.assert_quantized(q, s, ref.silu_mul(gu), fmt, REL)


# windows of two blocks: 11 and 12 blocks are six of them, 23 and 24 twelve
@pytest.mark.parametrize("t,e,topk", [(1, 12, 4), (3, 12, 4), (16, 12, 2), (16, 5, 3)])
@pytest.mark.parametrize("h,i", [(2944, 384), (384, 1408), (2944, 1408), (384, 2944), (1408, 2944)])
def test_mixture(t, e, topk, h, i):
    _check(_layer(t, e, h, i, seed=h + i), topk, True)
