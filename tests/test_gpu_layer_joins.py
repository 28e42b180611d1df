"""The per-row E4M3 and the int8 form of the norm and the activation as operands
of the products that they are for, as a layer chains them.

Tolerances, derived from the products' arithmetic: E4M3 as in
layer_ref.assert_gemm, but with all k/8 groups summed in F32 before the scales
come in; int8 block sums are exact, then ceil(k/32) scaled blocks are added in
F32 (one ulp each, one more for each product of scales).
"""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import layer_ref as ref
from tests.test_gpu_layer_quant import DEV, REL, _norm, _normal, _outputs

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -23


def _operand(source, rows, k, fmt):
    """(codes, scales, exact values) of the norm or of the activation."""
    if source == "norm":
        x, r, w = _normal((rows, k), 1), _normal((rows, k), 2, 4.0), _normal((k,), 3)
        q, s, _ = _norm(x, r, w, fmt)
        return q, s, ref.rms_norm(x, r, w, 1e-6)[1]
    gu = _normal((rows, 2 * k), 4, 2.0)
    q, s = _outputs(rows, k, fmt)
    qp.silu_mul_quant(gu, fmt, q, s)
    torch.cuda.synchronize()
    return q, s, ref.silu_mul(gu)


def _near(out, c, y, w):
    """The chain against the unquantized product: 8 bits of each value, 2^-4 of
    it at most, in the 2-norm."""
    want = y @ w.t()
    assert (out.double() - want).norm() <= 2.0 ** -4 * want.norm()
    assert (out.double() - c).norm() <= 2.0 ** -8 * c.norm()


@pytest.mark.parametrize("rows,k", [(1, 512), (37, 2368), (300, 1040)])
@pytest.mark.parametrize("source", ["norm", "activation"])
def test_row_form_into_the_row_scaled_product(source, rows, k):
    n = 520
    q, s, y = _operand(source, rows, k, qp.QP_ACT_FP8_ROW)
    ref.assert_quantized(q, s, y, ref.FMT_ROW, REL)
    g = torch.Generator(device=DEV).manual_seed(5)
    w = (100.0 * torch.randn((n, k), generator=g, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = 1e-3 * (0.5 + torch.rand((n,), generator=g, device=DEV))
    out = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    qp.fp8_gemm_rowscale(q, s.view(rows), w, ws, out)
    torch.cuda.synchronize()
    av, wv = ref.decoded(q) * s.double(), w.double() * ws.double()[:, None]
    top = lambda v: v.abs().view(v.shape[0], -1, 8).amax(dim=2)  # noqa: E731
    c = av @ wv.t()
    ref.assert_rounded(out, c, (k / 8 + 8) * ULP * (av.abs() @ wv.abs().t()) + 7 * 2.0 ** -13 * (top(av) @ top(wv).t()))
    _near(out, c, y, wv)


@pytest.mark.parametrize("rows,k", [(1, 512), (37, 2368), (300, 1056)])
@pytest.mark.parametrize("source", ["norm", "activation"])
def test_int8_form_into_the_block_scaled_product(source, rows, k):
    n = 520
    q, s, y = _operand(source, rows, k, qp.QP_ACT_INT8_BLOCK32)
    ref.assert_quantized(q, s, y, ref.FMT_INT8, REL)
    g = torch.Generator(device=DEV).manual_seed(6)
    w = torch.randint(-127, 128, (n, k), generator=g, device=DEV, dtype=torch.int8)
    ws = 1e-3 * (0.5 + torch.rand((n, k // 32), generator=g, device=DEV))
    out = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    qp.int8_gemm_blockscaled(q, w, s, ws, out)
    torch.cuda.synchronize()
    spread = lambda v: v.double().repeat_interleave(32, dim=1)  # noqa: E731
    av, wv = q.double() * spread(s), w.double() * spread(ws)
    c = av @ wv.t()
    ref.assert_rounded(out, c, (k / 32 + 4) * ULP * (av.abs() @ wv.abs().t()))
    _near(out, c, y, wv)


@pytest.mark.parametrize("source", ["norm", "activation"])
def test_bf16_form_into_the_gemv(source):
    """The row-scaled GEMV takes BF16 rows; its sums are F32 of exact products."""
    rows, k, n = 4, 1024, 520
    y16 = torch.full((rows, k), 7.0, dtype=torch.bfloat16, device=DEV)
    if source == "norm":
        x, w = _normal((rows, k), 1), _normal((k,), 3)
        qp.rmsnorm_residual_quant(x, None, w, 1e-6, qp.QP_ACT_BF16, y16, None)
    else:
        qp.silu_mul_quant(_normal((rows, 2 * k), 4, 2.0), qp.QP_ACT_BF16, y16, None)
    g = torch.Generator(device=DEV).manual_seed(7)
    w = (100.0 * torch.randn((n, k), generator=g, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = 1e-3 * (0.5 + torch.rand((n,), generator=g, device=DEV))
    out = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    qp.fp8_gemv_rowscale(y16, w, ws, out)
    torch.cuda.synchronize()
    av, wv = y16.double(), w.double() * ws.double()[:, None]
    ref.assert_rounded(out, av @ wv.t(), (k + 4) * ULP * (av.abs() @ wv.abs().t()))
