"""The BF16 form of the norm and the activation, the row lengths and counts at
which another kernel of theirs takes over, and the layers of the example.

Tolerances: REL as in test_gpu_layer_quant (the F32 value before its rounding);
a BF16 output has to lie between what values REL away on either side round to.
A layer against its plain form: every BF16 rounding may fall the other way
(2^-8 of a value), so a gated value moves by at most 2^-7 + 2^-8, and an E4M3
code by one step (2^-3 of it) for at most the share of values that near to a
rounding point: a 2-norm of at most sqrt(2^-6 * 2^-3) = 2^-4.5 of the
activation's, before the products average it.  2^-5 is held.
"""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from examples import layer_step
from tests import layer_ref as ref
from tests.test_gpu_layer_quant import DEV, FMTS, REL, _check_norm, _normal, _outputs

pytestmark = pytest.mark.gpu


def _bf16_out(rows, k):
    return torch.full((rows, k), 7.0, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("rows,k", [(1, 16), (3, 48), (1, 5120), (2047, 1376), (2, 8208), (300, 16384),
                                    (2, 24592), (1, 32784), (1, 262144)])
def test_bf16_norm_and_activation(rows, k):
    x, r, w = _normal((rows, k), 1), _normal((rows, k), 2, 4.0), _normal((k,), 3)
    for res in (r, None):
        y, out = _bf16_out(rows, k), None if res is None else torch.empty_like(r)
        qp.rmsnorm_residual_quant(x, res, w, 1e-6, qp.QP_ACT_BF16, y, None, out)
        h, want = ref.rms_norm(x, res, w, 1e-6)
        ref.assert_rounded(y, want, REL * want.abs())
        assert res is None or torch.equal(out.view(torch.int16), h.view(torch.int16))
    gu, y = _normal((rows, 2 * k), 4, 3.0), _bf16_out(rows, k)
    qp.silu_mul_quant(gu, qp.QP_ACT_BF16, y, None)
    want = ref.silu_mul(gu)
    ref.assert_rounded(y, want, REL * want.abs())


def test_bf16_of_zero_and_far_gates():
    gu = torch.zeros((4, 2 * 256), dtype=torch.bfloat16, device=DEV)
    gu[2, :256], gu[2, 256:] = -300.0, 2.0
    gu[3, :256], gu[3, 256:] = 300.0, -2.0
    y = _bf16_out(4, 256)
    qp.silu_mul_quant(gu, qp.QP_ACT_BF16, y, None)
    torch.cuda.synchronize()
    assert torch.all(y[:2] == 0) and torch.all(y[2] == 0) and torch.all(y[3] == -600.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,k", [(512, 1024), (513, 1024), (8192, 512), (8193, 512), (9000, 32), (820, 640),
                                    (2, 8160), (2, 16352), (2, 24576), (2, 24608), (2, 32768)])
def test_each_side_of_every_change_of_kernel(rows, k, fmt):
    x, r, w = _normal((rows, k), 5), _normal((rows, k), 6, 4.0), _normal((k,), 7)
    _check_norm(x, r, w, fmt)
    gu = _normal((rows, 2 * k), 8, 2.0)
    q, s = _outputs(rows, k, fmt)
    qp.silu_mul_quant(gu, fmt, q, s)
    ref.assert_quantized(q, s, ref.silu_mul(gu), fmt, REL)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k", [1024, 8192, 24576])
def test_activation_rows_do_not_depend_on_the_batch(fmt, k):
    rows = 9000 * 512 // k + 1
    gu = _normal((rows, 2 * k), 9)
    q, s = _outputs(rows, k, fmt)
    qp.silu_mul_quant(gu, fmt, q, s)
    for n in (1, 3):
        q1, s1 = _outputs(n, k, fmt)
        qp.silu_mul_quant(gu[-n:].contiguous(), fmt, q1, s1)
        torch.cuda.synchronize()
        assert torch.equal(q1, q[-n:]) and torch.equal(s1, s[-n:])


def test_the_binding_checks_the_bf16_form():
    x, w = _normal((2, 256), 10), _normal((256,), 11)
    with pytest.raises(ValueError, match="has none"):
        qp.rmsnorm_residual_quant(x, None, w, 1e-6, qp.QP_ACT_BF16, _bf16_out(2, 256), torch.ones(2, device=DEV))
    with pytest.raises(TypeError, match="q"):
        qp.rmsnorm_residual_quant(x, None, w, 1e-6, qp.QP_ACT_BF16, torch.empty((2, 256), dtype=torch.uint8, device=DEV),
                                  None)
    with pytest.raises(ValueError, match="q"):
        qp.silu_mul_quant(_normal((2, 512), 12), qp.QP_ACT_BF16, _bf16_out(2, 512), None)


@pytest.mark.parametrize("rows", [1, 4, 37, 300])
def test_dense_layer(rows):
    layer = layer_step.Dense(rows, 512, 1376, torch.device(DEV))
    assert layer_step.check(layer, rows, 512, torch.device(DEV)) <= 2.0 ** -5


@pytest.mark.parametrize("rows", [1, 5, 16])
def test_mixture_layer(rows):
    layer = layer_step.Mixture(rows, 512, 384, 24, 4, torch.device(DEV))
    assert layer_step.check(layer, rows, 512, torch.device(DEV)) <= 2.0 ** -5
