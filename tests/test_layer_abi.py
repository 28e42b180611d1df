"""Argument checks of the entry points of include/qproj_layer.h (no GPU): each
bad call is refused on the host, with its code, and enqueues nothing."""
import os
import re
import subprocess

import pytest

import gemv_nvfp4_int8_amd as qp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = qp.lib()
A, B = 0x10000, 0x20000          # aligned, never dereferenced
BLOCK, ROW, INT8 = qp.QP_ACT_FP8_BLOCK128, qp.QP_ACT_FP8_ROW, qp.QP_ACT_INT8_BLOCK32


def _declared():
    text = open(os.path.join(ROOT, "include", "qproj_layer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^(?:int|uint64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))


# name -> (call(pointers, sizes), number of pointers, sizes that pass)
CALLS = {
    "rmsnorm_residual_quant": (lambda p, n: L.rmsnorm_residual_quant(
        p[0], p[1], p[2], 1e-6, BLOCK, p[3], p[4], p[5], n[0], n[1], None), 6, (4, 256)),
    "silu_mul_quant": (lambda p, n: L.silu_mul_quant(p[0], BLOCK, p[1], p[2], n[0], n[1], None), 3, (4, 256)),
    "fp8_gemm_blockscale": (lambda p, n: L.fp8_gemm_blockscale(
        p[0], p[1], p[2], p[3], p[4], n[0], n[1], n[2], None), 5, (4, 256, 256)),
    "moe_fp8_blockscale": (lambda p, n: L.moe_fp8_blockscale(
        p[0], p[1], p[2], p[3], p[4], p[5], p[6], 1 << 20, p[7], n[0], n[1], n[2], n[3], n[4], 1, None),
        8, (4, 16, 2, 256, 256)),
}


def _pointers(count):
    return [A if i % 2 == 0 else B for i in range(count)]


@pytest.fixture(autouse=True)
def nothing_is_launched():
    before = qp.launch_count()
    yield
    assert qp.launch_count() == before


def test_header_and_library_agree():
    out = subprocess.run(["nm", "-D", "--defined-only", qp.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(_declared()) <= exported
    assert set(CALLS) <= set(_declared())


@pytest.mark.parametrize("name", sorted(CALLS))
def test_every_pointer_is_checked(name):
    call, count, sizes = CALLS[name]
    for i in range(count):
        p = _pointers(count)
        p[i] = 0
        assert call(p, sizes) == qp.QP_ERR_NULL, i
        p = _pointers(count)
        p[i] += 8
        assert call(p, sizes) == qp.QP_ERR_ALIGN, i


@pytest.mark.parametrize("name", sorted(CALLS))
def test_every_empty_extent_is_refused(name):
    call, count, sizes = CALLS[name]
    for i in range(len(sizes)):
        n = list(sizes)
        n[i] = 0
        assert call(_pointers(count), n) in (qp.QP_ERR_SHAPE, qp.QP_ERR_RANGE), i


def _norm(eps=1e-6, fmt=BLOCK, rows=4, k=256):
    return L.rmsnorm_residual_quant(A, None, B, eps, fmt, A, B, None, rows, k, None)


def test_norm_refusals():
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert _norm(eps=eps) == qp.QP_ERR_RANGE
    for fmt in (-1, 3, 99):
        assert _norm(fmt=fmt) == qp.QP_ERR_FORMAT
    for fmt, k in ((BLOCK, 24), (ROW, 8), (INT8, 48), (BLOCK, (1 << 18) + 16)):
        assert _norm(fmt=fmt, k=k) == qp.QP_ERR_SHAPE
    assert _norm(rows=1 << 20, k=1 << 11) == qp.QP_ERR_SHAPE       # 2^31 elements


def test_silu_refusals():
    call = lambda fmt, rows, k: L.silu_mul_quant(A, fmt, B, A, rows, k, None)  # noqa: E731
    assert call(7, 4, 256) == qp.QP_ERR_FORMAT
    for fmt, k in ((BLOCK, 24), (ROW, 8), (INT8, 48), (ROW, (1 << 18) + 16)):
        assert call(fmt, 4, k) == qp.QP_ERR_SHAPE
    assert call(BLOCK, 1 << 20, 1 << 10) == qp.QP_ERR_SHAPE        # gate_up holds 2^31 elements


def test_only_the_bf16_form_has_no_scale():
    for fmt, code in ((qp.QP_ACT_BF16, qp.QP_ERR_SHAPE), (BLOCK, qp.QP_ERR_NULL), (ROW, qp.QP_ERR_NULL),
                      (INT8, qp.QP_ERR_NULL)):
        assert L.rmsnorm_residual_quant(A, None, B, 1e-6, fmt, A, None, None, 4, 8, None) == code
        assert L.silu_mul_quant(A, fmt, B, None, 4, 8, None) == code


def test_gemm_refusals():
    call = lambda m, n, k: L.fp8_gemm_blockscale(A, B, A, B, A, m, n, k, None)  # noqa: E731
    for k in (8, 24, 100):
        assert call(4, 256, k) == qp.QP_ERR_SHAPE
    assert call(1 << 16, 128, 1 << 15) == qp.QP_ERR_SHAPE          # a holds 2^31 elements
    assert call(128, 1 << 16, 1 << 15) == qp.QP_ERR_SHAPE
    assert call(1 << 16, 1 << 15, 128) == qp.QP_ERR_SHAPE


def _moe(t=4, e=16, topk=2, h=256, i=256, work=1 << 20):
    return L.moe_fp8_blockscale(A, B, A, B, A, B, A, work, B, t, e, topk, h, i, 1, None)


def test_moe_refusals():
    for bad in (dict(t=17), dict(topk=17), dict(e=4, topk=5), dict(t=1 << 20)):
        assert _moe(**bad) == qp.QP_ERR_RANGE, bad
    for bad in (dict(e=513), dict(h=192), dict(i=64), dict(h=1 << 16, i=1 << 14)):
        assert _moe(**bad) == qp.QP_ERR_SHAPE, bad
    # the rows between the two launches pass 2^31 bytes before an expert's weight does
    assert _moe(t=16, topk=16, h=128, i=1 << 21, work=1 << 40) == qp.QP_ERR_SHAPE
    need = qp.moe_fp8_blockscale_workspace(4, 2, 256)
    assert 4 * 4 * 2 * 256 < need <= 4 * 4 * 2 * 256 + 65536
    assert _moe(work=need - 1) == qp.QP_ERR_SCRATCH
    assert _moe(work=0) == qp.QP_ERR_SCRATCH


def test_binding_refuses_what_the_kernels_would_overrun():
    import torch
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        qp.silu_mul_quant(x, BLOCK, x, x)
    with pytest.raises(TypeError, match="dtype"):
        qp.silu_mul_quant(x.float(), BLOCK, x, x)
