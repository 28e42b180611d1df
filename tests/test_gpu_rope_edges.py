"""qk_norm_rope_cache: entries that are not turned, beside infinities, NaN and
zeros of either sign; heads so small that their scale is below F32's normal
numbers."""
import math

import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests.decoder_ref import BF16, F32, I32, U8, DEV, Cache, gen, normal

pytestmark = pytest.mark.gpu


def call(x, heads, kv, d, rot, half, fp8=False, rope_scale=1.0):
    t = len(x)
    cache = Cache(2, kv, 16, d, fp8)
    q = torch.full((t, heads, d), -7.0, dtype=BF16, device=DEV)
    freq = qp.rope_inv_freq(rot, 1e4).to(DEV) if rot else None
    qp.qk_norm_rope_cache(x.to(BF16).contiguous(), None, None, 1e-6, 5 + torch.arange(t, dtype=I32, device=DEV), freq, rope_scale,
                          qp.QP_ROPE_HALF if half else qp.QP_ROPE_INTERLEAVED, torch.arange(t, dtype=I32, device=DEV),
                          qp.KVCache(cache.k, cache.v, cache.ks, cache.vs), q)
    torch.cuda.synchronize()
    return q, cache


@pytest.mark.parametrize("half", [True, False], ids=["half", "pairs"])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 32), (80, 20), (128, 64), (128, 96), (128, 2), (192, 128), (256, 102)])
def test_what_is_not_turned_stays_as_it_is(d, rot, half):
    """No norms, a BF16 cache: the bits of these entries, and the turned ones those
    of a call where the others are zeros."""
    t, heads, kv = 6, 5, 2
    x = normal(gen(d + rot), t, heads + 2 * kv, d).to(BF16)
    odd = torch.randint(0, 6, x.shape, generator=gen(1), device=DEV)
    for n, bad in enumerate((math.inf, -math.inf, math.nan, 0.0, -0.0)):
        x[..., rot:] = torch.where(odd[..., rot:] == n, bad, x[..., rot:])
    clean = x.clone()
    clean[..., rot:] = 0.0
    got, want = (call(v.view(t, -1), heads, kv, d, rot, half) for v in (x, clean))
    bits = lambda v: v.contiguous().view(torch.int16)  # noqa: E731
    for a, b, given in ((got[0], want[0], x[:, :heads]), (got[1].k[0].transpose(0, 1)[:t], want[1].k[0].transpose(0, 1)[:t],
                                                         x[:, heads:heads + kv])):
        assert torch.equal(bits(a[..., :rot]), bits(b[..., :rot]))
        nan = torch.isnan(given[..., rot:])
        assert torch.isnan(a[..., rot:][nan]).all()
        assert torch.equal(bits(a[..., rot:])[~nan], bits(given[..., rot:])[~nan])


def test_scales_below_the_normal_numbers():
    """Heads of F32 values around 1e-42 (a rope_scale that small): their scale has a
    few bits left and a value over it may be far above 448, which is then the code's
    largest, not NaN."""
    t, heads, kv, d = 16, 4, 2, 64
    x = normal(gen(4), t, heads + 2 * kv, d).to(BF16)
    for rope_scale in (1e-39, 2e-41, 1e-42, 2e-43, 1e-44):
        _, cache = call(x.view(t, -1), heads, kv, d, d, True, fp8=True, rope_scale=rope_scale)
        codes, scale = cache.k[0, :, :t], cache.ks[0, :, :t]
        assert not ((codes & 0x7F) == 0x7F).any(), rope_scale
        assert not codes[scale == 0].any()
        # the largest value of a head over amax / 448 is 448 or (a rounded scale) more
        assert torch.all((codes & 0x7F).amax(dim=2)[scale > 0] >= 0x70)
