"""Calls at the ends of the accepted sizes, and the binding's refusal of a
missing scale."""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests.test_gpu_layer_quant import DEV, _normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [qp.QP_ACT_FP8_ROW, qp.QP_ACT_FP8_BLOCK128, qp.QP_ACT_BF16])
def test_norm_of_more_rows_than_one_launch_holds(fmt):
    """2^26 rows of a wave each pass the 2^32 threads of a launch.  A row's bits
    do not depend on its batch, so calls on pieces are the reference."""
    rows, k, piece = (1 << 26) + 3, 16, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((rows, k), dtype=torch.bfloat16, device=DEV)
    for at in range(0, rows, 1 << 22):
        x[at:at + (1 << 22)].normal_(generator=g)
    w, res = _normal((k,), 2), x.flip(0)
    bf16 = fmt == qp.QP_ACT_BF16
    q = torch.full((rows, k), 0x5A, dtype=torch.uint8, device=DEV) if not bf16 else torch.full_like(x, 7.0)
    s = None if bf16 else torch.full((rows, 1), float("nan"), device=DEV)
    out = torch.full_like(x, 7.0)
    qp.rmsnorm_residual_quant(x, res, w, 1e-6, fmt, q, s, out)
    torch.cuda.synchronize()
    for at in (0, (1 << 25) - piece // 2, (1 << 26) - piece // 2, rows - piece):
        part = slice(at, at + piece)
        q1, o1 = torch.zeros_like(q[part]), torch.zeros_like(out[part])
        s1 = None if bf16 else torch.zeros_like(s[part])
        part = slice(at, at + q1.shape[0])
        qp.rmsnorm_residual_quant(x[part], res[part], w, 1e-6, fmt, q1, s1, o1)
        torch.cuda.synchronize()
        assert torch.equal(q1, q[part]) and torch.equal(o1, out[part])
        assert bf16 or torch.equal(s1, s[part])
    assert bf16 or bool(torch.isfinite(s).all())


@pytest.mark.parametrize("fmt", [qp.QP_ACT_FP8_ROW, qp.QP_ACT_FP8_BLOCK128, qp.QP_ACT_INT8_BLOCK32])
def test_a_missing_scale_is_a_type_error(fmt):
    x, w = _normal((2, 256), 3), _normal((256,), 4)
    q = torch.empty((2, 256), dtype=torch.int8 if fmt == qp.QP_ACT_INT8_BLOCK32 else torch.uint8, device=DEV)
    with pytest.raises(TypeError, match="scale"):
        qp.rmsnorm_residual_quant(x, None, w, 1e-6, fmt, q, None)
    with pytest.raises(TypeError, match="scale"):
        qp.silu_mul_quant(_normal((2, 512), 5), fmt, q, None)


def test_rowwise_quantizer_of_more_rows_than_one_launch_holds():
    """quant_rowwise_fp8 gives a row a wave as well."""
    rows, k, piece = (1 << 26) + 3, 16, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.empty((rows, k), dtype=torch.bfloat16, device=DEV)
    for at in range(0, rows, 1 << 22):
        x[at:at + (1 << 22)].normal_(generator=g)
    q, s = torch.full((rows, k), 0x5A, dtype=torch.uint8, device=DEV), torch.full((rows,), float("nan"), device=DEV)
    qp.quant_rowwise_fp8(x, q, s)
    torch.cuda.synchronize()
    for at in (0, (1 << 25) - piece // 2, (1 << 26) - piece // 2, rows - piece):
        part = slice(at, min(at + piece, rows))
        q1, s1 = torch.zeros_like(q[part]), torch.zeros_like(s[part])
        qp.quant_rowwise_fp8(x[part], q1, s1)
        torch.cuda.synchronize()
        assert torch.equal(q1, q[part]) and torch.equal(s1, s[part])
    assert bool(torch.isfinite(s).all())
