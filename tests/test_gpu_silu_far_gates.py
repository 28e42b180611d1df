"""The activation where 1 + exp(-g) is finite in F32 but its reciprocal is below
the normal numbers: gates from -88.7 to -87.3, of which BF16 holds three.

Tolerance: as in test_gpu_layer_quant (REL); the argument's rounding is at most
88.5 * 2^-24 = 5.3e-6 relative there.
"""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import layer_ref as ref
from tests.test_gpu_layer_quant import DEV, FMTS, REL, _outputs

pytestmark = pytest.mark.gpu

FAR = (-87.0, -87.5, -88.0, -88.5)


def _gate_up(k, smallest):
    """A row for each gate and one of them mixed; up values 10^U(smallest, 38) of both signs."""
    g = torch.Generator(device=DEV).manual_seed(21)
    gate = torch.tensor(FAR, device=DEV)[:, None].expand(-1, k)
    mixed = gate[torch.randint(0, len(FAR), (k,), generator=g, device=DEV), 0]
    gate = torch.cat([gate, mixed[None]])
    up = 10.0 ** (smallest + (38.0 - smallest) * torch.rand(gate.shape, generator=g, device=DEV))
    up *= torch.where(torch.rand(gate.shape, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    return torch.cat([gate, up], dim=1).to(torch.bfloat16)


@pytest.mark.parametrize("k", [16, 1376, 32784])
def test_bf16_of_gates_with_a_subnormal_reciprocal(k):
    gu = _gate_up(k, 4.0)
    y = torch.full((gu.shape[0], k), 7.0, dtype=torch.bfloat16, device=DEV)
    qp.silu_mul_quant(gu, qp.QP_ACT_BF16, y, None)
    want = ref.silu_mul(gu)
    ref.assert_rounded(y, want, REL * want.abs())
    assert torch.all(y != 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k", [32, 1376, 32800])
def test_codes_of_gates_with_a_subnormal_reciprocal(k, fmt):
    """Blocks made of nothing else have scales of their own, and codes."""
    gu = _gate_up(k, 20.0)
    q, s = _outputs(gu.shape[0], k, fmt)
    qp.silu_mul_quant(gu, fmt, q, s)
    torch.cuda.synchronize()
    assert torch.all(s > 0)
    ref.assert_quantized(q, s, ref.silu_mul(gu), fmt, REL)


def test_gates_past_the_exponential_and_the_largest_values():
    """exp(-g) = inf gives 0; gates and ups next to BF16's largest and smallest
    normal numbers pass through unchanged in F32."""
    big, tiny = (2.0 - 2.0 ** -7) * 2.0 ** 127, 2.0 ** -126
    gate = torch.tensor([-89.0, -200.0, -big, big, tiny, -tiny, 1.5 * tiny, big], device=DEV)
    up = torch.tensor([big, 1.0, 1.0, 0.5, 64.0, 64.0, 2.0, tiny], device=DEV)
    gu = torch.cat([gate.repeat(2), up.repeat(2)])[None].to(torch.bfloat16)
    y = torch.full((1, 16), 7.0, dtype=torch.bfloat16, device=DEV)
    qp.silu_mul_quant(gu, qp.QP_ACT_BF16, y, None)
    want = torch.tensor([0, 0, 0, 0.5 * big, 32 * tiny, -32 * tiny, 1.5 * tiny, big * tiny], device=DEV).repeat(2)
    assert torch.equal(y[0].float().abs(), want.abs()) and torch.all(y[0].float() * want >= 0)
