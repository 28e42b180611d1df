"""moe_fp8_blockscale against the layer in 64 bits (tolerance: layer_ref.moe and assert_rounded)."""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")


def _codes(g, shape):
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    for part in out.view(shape[0], -1):
        part.copy_((112.0 * torch.randn(part.shape, generator=g, device=DEV)).clamp_(-448, 448))
    return out.view(torch.uint8)


def _layer(t, e, h, i, seed=0):
    g = torch.Generator(device=DEV).manual_seed(100 + seed)
    x = torch.randn((t, h), generator=g, device=DEV).to(torch.bfloat16)
    logits = 1.5 * torch.randn((t, e), generator=g, device=DEV)
    grid = lambda *s: 2e-4 * (0.5 + torch.rand(s, generator=g, device=DEV))  # noqa: E731
    return (x, logits, _codes(g, (e, 2 * i, h)), grid(e, 2 * i // 128, h // 128),
            _codes(g, (e, h, i)), grid(e, h // 128, i // 128))


def _run(layer, topk, renorm, stream=None):
    x = layer[0]
    t, i = x.shape[0], layer[4].shape[2]
    work = torch.full((qp.moe_fp8_blockscale_workspace(t, topk, i),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    qp.moe_fp8_blockscale(*layer, topk, renorm, work, out, stream=stream)
    torch.cuda.synchronize()
    return out


def _check(layer, topk, renorm):
    out = _run(layer, topk, renorm)
    want, tol = ref.moe(*layer, topk, renorm)
    ref.assert_rounded(out, want, tol)
    return out


# one token and sixteen, one expert and 512, K ranges that end inside a window
SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 256, 384), (1, 128, 8, 2048, 768), (2, 16, 16, 384, 128),
          (3, 60, 4, 640, 1408), (4, 64, 6, 1024, 256), (5, 8, 2, 1152, 2048), (7, 256, 8, 512, 512),
          (8, 100, 3, 768, 640), (16, 4, 4, 512, 256), (16, 64, 6, 2560, 384), (16, 512, 16, 256, 128),
          (13, 130, 5, 896, 896)]


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t,e,topk,h,i", SHAPES)
def test_matches_the_layer_in_64_bits(t, e, topk, h, i, renorm):
    _check(_layer(t, e, h, i), topk, renorm)


@pytest.mark.parametrize("t", range(1, 17))
def test_all_tokens_at_one_expert(t):
    """Every count of tokens that an expert can have."""
    layer = _layer(t, 9, 384, 256, t)
    layer[1][:, 5] = 50.0
    _check(layer, 2, True)


@pytest.mark.parametrize("renorm", [False, True])
def test_masked_experts(renorm):
    """Rows that leave fewer experts than topk, one, or none; the lowest
    finite logit is a logit like any other."""
    layer = _layer(6, 40, 256, 256, 50)
    lg = layer[1]
    lg[0] = -INF                              # nothing: a row of zeros
    lg[1, 1:] = -INF
    lg[2, 3:] = -INF
    lg[3, ::2] = -INF
    lg[4] = torch.finfo(torch.float32).min    # all equal: the lowest experts
    lg[5, :30] = torch.finfo(torch.float32).min
    out = _check(layer, 4, renorm)
    assert torch.all(out[0] == 0)
    layer[1][:] = -INF
    assert torch.all(_check(layer, 4, renorm) == 0)


@pytest.mark.parametrize("e", [8, 64, 96, 200, 512])
def test_equal_logits_go_to_the_lowest_experts(e):
    layer = _layer(5, e, 128, 128, e)
    lg = layer[1]
    lg[0] = 0.0
    lg[1] = 0.0
    lg[1, 1::2] = -0.0                         # equal to +0
    lg[2] = (torch.arange(e, device=DEV) // 3).float()
    lg[3] = -(torch.arange(e, device=DEV) // 3).float()
    lg[4] = lg[4].round()
    _check(layer, 7, True)


def test_same_bits_twice_and_on_a_stream():
    layer = _layer(11, 32, 1024, 640, 3)
    one = _run(layer, 4, True)
    assert torch.equal(one.view(torch.int16), _run(layer, 4, True).view(torch.int16))
    assert torch.equal(one.view(torch.int16),
                       _run(layer, 4, True, torch.cuda.Stream()).view(torch.int16))


def test_experts_past_32_bit_offsets():
    """All experts' weights together hold over 2^31 elements; the chosen ones
    lie at both ends."""
    e, h, i = 48, 5120, 4608
    g = torch.Generator(device=DEV).manual_seed(1)
    some = _codes(g, (4, 2 * i, h))
    w13 = some.repeat(e // 4, 1, 1)
    w2 = _codes(g, (4, h, i)).repeat(e // 4, 1, 1)
    assert w13.numel() > 1 << 31
    grid = lambda *s: 2e-4 * (0.5 + torch.rand(s, generator=g, device=DEV))  # noqa: E731
    x = torch.randn((2, h), generator=g, device=DEV).to(torch.bfloat16)
    logits = torch.full((2, e), -INF, device=DEV)
    logits[0, 0], logits[0, 47], logits[1, 46], logits[1, 47] = 1.0, 2.0, 0.5, 0.25
    _check((x, logits, w13, grid(e, 2 * i // 128, h // 128), w2, grid(e, h // 128, i // 128)), 2, True)


# every number of columns a workgroup can own, with one token, few and many
# tokens an expert
@pytest.mark.parametrize("h", [1024, 2048, 2560, 4096, 5120, 6144, 7168, 8192, 8320])
@pytest.mark.parametrize("t,e,topk", [(1, 5, 2), (5, 7, 2), (16, 6, 4), (9, 3, 1)])
def test_every_split_of_the_columns(t, e, topk, h):
    _check(_layer(t, e, h, 128, seed=h), topk, True)


@pytest.mark.parametrize("t,topk", [(2, 3), (4, 3), (5, 2), (8, 1), (9, 3), (13, 2), (16, 3), (16, 1)])
@pytest.mark.parametrize("i", [128, 640])
def test_experts_with_parts_of_every_size(t, topk, i):
    """Few experts: parts of one to eight tokens, whole and ragged groups."""
    for e in (3, 4):
        _check(_layer(t, e, 640, i, seed=t), topk, False)
