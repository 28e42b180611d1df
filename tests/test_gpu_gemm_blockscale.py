"""fp8_gemm_blockscale against the product in 64 bits (tolerance: layer_ref.assert_gemm)."""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _codes(shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = (64.0 * torch.randn(shape, generator=g, device=DEV)).clamp(-448, 448)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(shape, seed):
    """10^U(-4, -2)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return 10.0 ** (-4.0 + 2.0 * torch.rand(shape, generator=g, device=DEV))


def _operands(m, n, k, seed=0):
    kb = -(-k // 128)
    return (_codes((m, k), seed + 1), _scales((m, kb), seed + 2), _codes((n, k), seed + 3),
            _scales((-(-n // 128), kb), seed + 4))


def _run(a, sa, w, sw):
    out = torch.full((a.shape[0], w.shape[0]), float("nan"), dtype=torch.bfloat16, device=DEV)
    qp.fp8_gemm_blockscale(a, sa, w, sw, out)
    torch.cuda.synchronize()
    return out


def _check(m, n, k, seed=0):
    a, sa, w, sw = _operands(m, n, k, seed)
    csg = ref.gemm_blockscale(a, sa, w, sw)
    ref.assert_gemm(_run(a, sa, w, sw), csg, k)


# single rows and columns, the sides of every tile size, half and quarter
# blocks at the end of K, odd N (whose rows start at 2-byte addresses)
SHAPES = [(1, 1, 16), (1, 128, 128), (1, 5120, 1024), (2, 130, 144), (4, 17408, 512), (5, 97, 2368),
          (15, 640, 3200), (16, 2048, 1280), (17, 4104, 1040), (31, 129, 256), (33, 257, 384),
          (37, 5120, 1536 + 16), (63, 512, 8192), (64, 768, 640), (65, 1000, 896), (100, 4100, 2048),
          (127, 127, 127 * 16), (128, 128, 128), (129, 385, 272), (255, 256, 512), (256, 256, 128),
          (256, 256, 256), (256, 512, 384), (257, 511, 1296), (300, 1031, 640), (512, 768, 2176),
          (600, 4104, 2368), (1000, 2048, 1152), (1024, 1280, 5120)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matches_the_product_in_64_bits(m, n, k):
    _check(m, n, k)


@pytest.mark.parametrize("m,n,k", [(4100, 4352, 256), (2048, 12288, 640), (8192, 2304, 1280)])
def test_many_tiles(m, n, k):
    _check(m, n, k)


@pytest.mark.parametrize("m", [3, 40, 300, 520])
def test_scales_reach_their_own_rows_and_blocks(m):
    """Each output is one scaled block's sum: scales that are powers of two of
    their place, all other blocks of the row switched off by a zero scale."""
    n, k = 520, 1088
    kb = -(-k // 128)
    a, _, w, _ = _operands(m, n, k, 9)
    sa = torch.zeros((m, kb), device=DEV)
    rows = torch.arange(m, device=DEV)
    sa[rows, rows % kb] = 2.0 ** ((rows % 23).float() - 11)
    sw = 2.0 ** (torch.arange(-(-n // 128) * kb, device=DEV).reshape(-1, kb) % 19 - 9).float()
    csg = ref.gemm_blockscale(a, sa, w, sw)
    ref.assert_gemm(_run(a, sa, w, sw), csg, 128)


@pytest.mark.parametrize("m", [2, 48, 700])
def test_every_code_and_extreme_scales(m):
    n, k = 384, 512
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    pick = lambda shape: codes[torch.randint(0, 254, shape, generator=g, device=DEV)]  # noqa: E731
    a, w = pick((m, k)), pick((n, k))
    sa = 2.0 ** torch.randint(-30, 11, (m, 4), generator=g, device=DEV).float()
    sw = 2.0 ** torch.randint(-30, 11, (3, 4), generator=g, device=DEV).float()
    sa[0] = 0
    sw[1, 2] = 0
    csg = ref.gemm_blockscale(a, sa, w, sw)
    out = _run(a, sa, w, sw)
    ref.assert_gemm(out, csg, k)
    assert torch.all(out[0] == 0)


@pytest.mark.parametrize("m", [1, 20, 150, 600])
def test_same_bits_twice_and_on_a_stream(m):
    a, sa, w, sw = _operands(m, 1160, 1408, 5)
    one = _run(a, sa, w, sw)
    st = torch.cuda.Stream()
    two = torch.empty_like(one)
    torch.cuda.synchronize()
    qp.fp8_gemm_blockscale(a, sa, w, sw, two, stream=st)
    st.synchronize()
    assert torch.equal(one.view(torch.int16), two.view(torch.int16))


def test_agrees_with_the_blockscaled_gemv():
    """Activations whose BF16 values are E4M3 codes times a power of two give
    both products the same operands."""
    m, n, k = 8, 512, 1024
    a, _, w, sw = _operands(m, n, k, 7)
    sa = torch.full((m, k // 128), 0.25, device=DEV)
    x = (ref.e4m3(a) * 0.25).to(torch.bfloat16)
    y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    qp.fp8_gemv_blockscale(x, w, sw, y)
    csg = ref.gemm_blockscale(a, sa, w, sw)
    ref.assert_gemm(_run(a, sa, w, sw), csg, k)
    torch.cuda.synchronize()
    ref.assert_gemm(y, csg, k)


@pytest.mark.parametrize("m,n,k", [(2, 8208, 8192), (16, 131072, 528), (20, 16416, 16384), (64, 65600, 4112)])
def test_weights_larger_than_the_caches(m, n, k):
    _check(m, n, k)


@pytest.mark.parametrize("nb", [1, 2, 3, 4, 5, 7, 8, 9, 31, 32, 33, 36, 63])
@pytest.mark.parametrize("m", [2, 40])
def test_every_remainder_of_the_k_blocks(m, nb):
    """A wave takes runs of K blocks: none, some or all of a run may exist."""
    _check(m, 160, 128 * nb, seed=nb)
    _check(m, 160, 128 * nb - 48, seed=nb)


@pytest.mark.parametrize("m,n,k", [(4200, 4353, 144), (7000, 1276, 128), (2100, 2091, 272), (700, 1030, 1040),
                                   (284, 223, 2048), (989, 100, 1536), (500, 12, 4096), (70, 5000, 640)])
def test_rows_at_any_alignment(m, n, k):
    """N of every remainder by 8; nothing is written past the last row."""
    a, sa, w, sw = _operands(m, n, k, seed=7)
    room = torch.full((m * n + 64,), 3.0, dtype=torch.bfloat16, device=DEV)
    out = room[:m * n].view(m, n)
    out.fill_(float("nan"))
    qp.fp8_gemm_blockscale(a, sa, w, sw, out)
    torch.cuda.synchronize()
    ref.assert_gemm(out, ref.gemm_blockscale(a, sa, w, sw), k)
    assert torch.all(room[m * n:] == 3.0)
