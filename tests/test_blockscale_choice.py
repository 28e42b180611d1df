"""Which kernel of fp8_gemm_blockscale serves which shape (no GPU; on 256
compute units), so that a change of the choice cannot leave a kernel untested
unnoticed: test_gpu_blockscale_kernels runs the same shapes."""
import os
import random
import re

import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests.blockscale_shapes import ALL, KSPLIT, TILES

pytestmark = pytest.mark.skipif(
    torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256,
    reason="the choice is for another number of compute units")


@pytest.mark.parametrize("kernel,shape", ALL)
def test_shape_takes_its_kernel(kernel, shape):
    assert qp.fp8_gemm_blockscale_kernel(*shape) == kernel


def test_every_kernel_that_a_shape_can_take_is_listed():
    rng = random.Random(0)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())  # noqa: E731
    seen = set()
    for _ in range(60000):
        m, n, k = log(1, rng.choice([64, 20000])), log(1, 200000), 16 * log(1, 8192)
        if max(m * n, m * k, n * k) < 1 << 31:
            seen.add(qp.fp8_gemm_blockscale_kernel(m, n, k))
    assert len(seen) > 20 and seen <= set(TILES) | set(KSPLIT)


def test_a_prefill_takes_the_large_tiles():
    for shape in ((4096, 5120, 17408), (8192, 12288, 5120), (8192, 5120, 17408)):
        assert qp.fp8_gemm_blockscale_kernel(*shape) in (qp.QP_BLOCKSCALE_TILES_256,
                                                         qp.QP_BLOCKSCALE_TILES_256_QUARTERS)


def test_refusals():
    for shape in ((0, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, 24), (1 << 16, 1 << 15, 128)):
        with pytest.raises(qp.QProjError) as e:
            qp.fp8_gemm_blockscale_kernel(*shape)
        assert e.value.status == qp.QP_ERR_SHAPE


def test_values_agree_with_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "qproj_layer.h")).read()
    declared = dict(re.findall(r"(QP_BLOCKSCALE_\w+) = (\d+)", text))
    assert len(declared) == 4
    for name, value in declared.items():
        assert getattr(qp, name) == int(value)
