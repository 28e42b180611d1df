"""rmsnorm_residual_quant and silu_mul_quant against plain 64-bit forms.

Tolerance: the F32 norm sums k squares in chains of 8, 4 and at most 32 + 6
additions, so the mean is within about 50 * 2^-24 of exact, its root half of
that, and the products, the maximum and the division add a few roundings more:
4e-6 relative bounds y, the scale, and their quotient twice that.  The
activation's exponential rounds its argument, |g| * 2^-24 for |g| < 90, 6e-6 in
all.  Both are held to REL = 2e-5: a scale may be that far off, a code may lie
anywhere between the codes of the exact quotient moved by that much.
"""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL = 2e-5
FMTS = [qp.QP_ACT_FP8_ROW, qp.QP_ACT_FP8_BLOCK128, qp.QP_ACT_INT8_BLOCK32]


def _normal(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(torch.bfloat16)


def _outputs(rows, k, fmt):
    q = torch.full((rows, k), 0x5A, dtype=torch.int8 if fmt == ref.FMT_INT8 else torch.uint8, device=DEV)
    nb = -(-k // ref.block_of(fmt, k))
    return q, torch.full((rows, nb), float("nan"), device=DEV)


def _norm(x, res, w, fmt, eps=1e-6):
    rows, k = x.shape
    q, s = _outputs(rows, k, fmt)
    out = None if res is None else torch.full_like(x, 7.0)
    qp.rmsnorm_residual_quant(x, res, w, eps, fmt, q, s, out)
    torch.cuda.synchronize()
    return q, s, out


def _check_norm(x, res, w, fmt, eps=1e-6):
    q, s, out = _norm(x, res, w, fmt, eps)
    h, y = ref.rms_norm(x, res, w, eps)
    if res is not None:
        assert torch.equal(out.view(torch.int16), h.view(torch.int16))
    ref.assert_quantized(q, s, y, fmt, REL)


# one chunk pair, a ragged block, whole blocks, both sides of each register
# capacity, rows past every capacity
SIZES = [(1, 32), (3, 96), (5, 160), (1, 5120), (4, 5120), (130, 1376), (1000, 2368), (2, 4096), (2, 4128),
         (7, 8192), (2, 8224), (3, 16384), (2, 16416), (1, 32800), (2, 262144)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,k", SIZES)
def test_norm_matches_the_plain_form(rows, k, fmt):
    x, r = _normal((rows, k), 1), _normal((rows, k), 2, 4.0)
    x[:, ::97] *= 30
    w = (1 + 0.2 * _normal((k,), 3).float()).to(torch.bfloat16)
    _check_norm(x, r, w, fmt)
    _check_norm(x, None, w, fmt)


@pytest.mark.parametrize("k", [16, 48, 4112, 16400])
@pytest.mark.parametrize("fmt", FMTS[:2])
def test_fp8_norm_of_half_blocks(k, fmt):
    """k a multiple of 16 but not of 32 (the int8 format refuses those)."""
    x, r, w = _normal((3, k), 4), _normal((3, k), 5), _normal((k,), 6)
    _check_norm(x, r, w, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_of_zero_tiny_and_large_rows(fmt):
    """A row of zeros (scale 0, codes +0), zero blocks inside a row, a zero
    weight, values whose squares are below and near the ends of F32's range."""
    k = 512
    x = _normal((8, k), 7)
    x[0] = 0
    x[1, 128:256] = 0
    x[2] *= 1e-18
    x[3] *= 1e-30
    x[4] *= 1e15
    x[5, :] = 0
    x[5, 77] = -3.0
    w = _normal((k,), 8)
    w[256:384] = 0
    _check_norm(x, None, w, fmt)
    _check_norm(x, torch.zeros_like(x), w, fmt)
    _check_norm(x, -x, w, fmt)
    _check_norm(x, None, (w.float() * 1e-36).to(torch.bfloat16), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k", [160, 5120, 16384, 20480])
def test_norm_rows_do_not_depend_on_the_batch(fmt, k):
    """Each row alone gives the bits it has among many (the kernels chosen for
    few and for many rows agree)."""
    rows = 4200 if k <= 5120 else 300
    x, r, w = _normal((rows, k), 9), _normal((rows, k), 10), _normal((k,), 11)
    q, s, out = _norm(x, r, w, fmt)
    for n in (1, 2, 33):
        q1, s1, out1 = _norm(x[-n:].contiguous(), r[-n:].contiguous(), w, fmt)
        assert torch.equal(q1, q[-n:]) and torch.equal(s1, s[-n:]) and torch.equal(out1, out[-n:])


@pytest.mark.parametrize("k", [5120, 40000])
def test_residual_updated_in_place(k):
    x, r, w = _normal((9, k), 12), _normal((9, k), 13), _normal((k,), 14)
    q, s, out = _norm(x, r, w, qp.QP_ACT_FP8_BLOCK128)
    q2, s2 = _outputs(9, k, qp.QP_ACT_FP8_BLOCK128)
    stream = r.clone()
    qp.rmsnorm_residual_quant(x, stream, w, 1e-6, qp.QP_ACT_FP8_BLOCK128, q2, s2, stream)
    torch.cuda.synchronize()
    assert torch.equal(stream, out) and torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,k", SIZES)
def test_silu_matches_the_plain_form(rows, k, fmt):
    gu = _normal((rows, 2 * k), 15)
    gu[:, ::89] *= 20
    q, s = _outputs(rows, k, fmt)
    qp.silu_mul_quant(gu, fmt, q, s)
    torch.cuda.synchronize()
    ref.assert_quantized(q, s, ref.silu_mul(gu), fmt, REL)


@pytest.mark.parametrize("fmt", FMTS)
def test_silu_at_the_ends_of_its_range(fmt):
    """Zero rows and blocks, gates so negative that exp(-g) leaves F32, gates
    so large that it vanishes."""
    k = 256
    gu = _normal((6, 2 * k), 16)
    gu[0] = 0
    gu[1, :k] = -200.0
    gu[2, :k] = 150.0
    gu[3, :128] = 0
    gu[4, k:] = 0
    gu[5, :k] = torch.linspace(-85, 85, k, device=DEV).to(torch.bfloat16)
    q, s = _outputs(6, k, fmt)
    qp.silu_mul_quant(gu, fmt, q, s)
    torch.cuda.synchronize()
    ref.assert_quantized(q, s, ref.silu_mul(gu), fmt, REL)


def test_on_a_stream_of_the_callers():
    x, r, w = _normal((64, 5120), 17), _normal((64, 5120), 18), _normal((5120,), 19)
    q, s, out = _norm(x, r, w, qp.QP_ACT_FP8_ROW)
    st = torch.cuda.Stream()
    q2, s2 = _outputs(64, 5120, qp.QP_ACT_FP8_ROW)
    out2 = torch.empty_like(out)
    torch.cuda.synchronize()
    qp.rmsnorm_residual_quant(x, r, w, 1e-6, qp.QP_ACT_FP8_ROW, q2, s2, out2, stream=st)
    st.synchronize()
    assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(out2, out)
