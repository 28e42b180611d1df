"""qk_norm_rope_cache against the 64-bit form: layouts, parts of the head, norms,
cache forms, head sizes and counts, far positions, padding and bad slots."""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import decoder_ref as ref
from tests.decoder_ref import BF16, F32, I32, U8, DEV, Cache, gen, normal

pytestmark = pytest.mark.gpu
EPS = 1e-6


def run(t, heads, kv, d, rot, half=True, norm=True, fp8=False, page=16, seed=0, far=50000, rope_scale=1.0,
        slots=None, x=None):
    g = gen(seed)
    qkv = (normal(g, t, (heads + 2 * kv) * d) if x is None else x).to(BF16)
    qw, kw = ((1.0 + 0.3 * normal(g, d)).to(BF16) if norm else None for _ in range(2))
    pos = torch.randint(0, far, (t,), generator=g, device=DEV, dtype=I32)
    freq = qp.rope_inv_freq(rot, 1e6).to(DEV) if rot else None
    pages = t // page + 2
    cache = Cache(pages, kv, page, d, fp8)
    before = [c.clone() for c in cache.tensors()]
    if slots is None:
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:t].to(I32)
    q = torch.full((t, heads, d), -777.0, dtype=BF16, device=DEV)
    qp.qk_norm_rope_cache(qkv, qw, kw, EPS, pos, freq, rope_scale, qp.QP_ROPE_HALF if half else qp.QP_ROPE_INTERLEAVED,
                          slots, qp.KVCache(cache.k, cache.v, cache.ks, cache.vs), q)
    torch.cuda.synchronize()
    parts = qkv.view(t, heads + 2 * kv, d).float().split([heads, kv, kv], dim=1)
    want = [ref.rope(parts[0], qw, EPS, pos, freq, rope_scale, half),
            ref.rope(parts[1], kw, EPS, pos, freq, rope_scale, half)]
    return qkv, slots, cache, before, q, parts[2], want


def check(result, where=None):
    qkv, slots, cache, before, q, v, ((yq, tq), (yk, tk)) = result
    ref.assert_rounded(q, yq, tq)
    kept = (slots >= 0) & (slots < cache.pages * cache.page)
    s = slots[kept].long()
    at, off = s // cache.page, s % cache.page
    if cache.fp8:
        ref.assert_row_codes(cache.k[at, :, off], cache.ks[at, :, off], yk[kept], tk[kept])
        # F32 quotients, correctly rounded (in F32 torch multiplies by a constant's reciprocal)
        scale = (v[kept].abs().amax(dim=2).double() / 448.0).float()
        assert torch.equal(cache.vs[at, :, off], scale)
        codes = (v[kept].double() / torch.where(scale > 0, scale, 1.0)[..., None].double()).float().to(torch.float8_e4m3fn)
        codes = torch.where(scale[..., None] > 0, codes.view(U8), 0)
        assert torch.equal(cache.v[at, :, off], codes)
    else:
        ref.assert_rounded(cache.k[at, :, off], yk[kept], tk[kept])
        assert torch.equal(cache.v[at, :, off].float(), v[kept])
    # nothing else was written
    for now, was in zip(cache.tensors(), before):
        now, was = (c.view(torch.int16 if c.dtype == BF16 else torch.int32 if c.dtype == F32 else U8).clone() for c in (now, was))
        now[at, :, off] = 0
        was[at, :, off] = 0
        assert torch.equal(now, was)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("half", [True, False], ids=["half", "pairs"])
@pytest.mark.parametrize("d,rot", [(16, 16), (32, 6), (64, 64), (80, 80), (80, 20), (96, 48), (128, 128), (128, 64),
                                   (128, 2), (128, 0), (192, 128), (256, 256), (256, 102)])
def test_head_sizes_and_rotated_parts(d, rot, half, fp8):
    check(run(5, 6, 2, d, rot, half=half, fp8=fp8, seed=d + rot))


@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("t,heads,kv", [(1, 1, 1), (1, 32, 8), (2, 1, 1), (7, 3, 1), (33, 10, 5), (300, 40, 4), (17, 5, 3)])
def test_rows_and_head_counts(t, heads, kv, norm):
    for fp8 in (False, True):
        check(run(t, heads, kv, 128, 128, norm=norm, fp8=fp8, page=64, seed=t))


def test_one_large_call():
    check(run(4099, 32, 8, 128, 128, page=32, seed=3))


@pytest.mark.parametrize("half", [True, False], ids=["half", "pairs"])
def test_far_positions_and_a_scale(half):
    check(run(64, 4, 2, 128, 128, half=half, far=(1 << 31) - 1, rope_scale=1.3689, seed=5))


def test_slots_outside_the_cache_write_nothing():
    for fp8 in (False, True):
        pages = 9 // 16 + 2
        bad = torch.tensor([3, -1, pages * 16, 31, -(1 << 31), (1 << 31) - 1, 0, -16, 17], dtype=I32, device=DEV)
        check(run(9, 4, 2, 64, 64, fp8=fp8, slots=bad))


def test_zero_and_large_heads():
    """A head of zeros: the norm gives zeros, the cache a zero scale and +0 codes."""
    g = gen(1)
    x = normal(g, 6, 8 * 64)
    x[1] = 0.0
    x[2] = 0.0
    x[2, 5] = -1.0
    x[3] *= 1e18                       # squares beyond F32's half range, sums below its largest
    x[4] *= 1e-18
    for fp8 in (False, True):
        for norm in (True, False):
            r = run(6, 4, 2, 64, 64, fp8=fp8, norm=norm, x=x)
            check(r)
            if fp8:
                c = r[2]
                s = r[1][1].item()
                assert not c.k[s // 16, :, s % 16].any() and not c.ks[s // 16, :, s % 16].any()


def test_a_token_does_not_depend_on_its_batch():
    for fp8 in (False, True):
        whole = run(37, 12, 4, 128, 96, fp8=fp8, seed=9)
        qkv, slots, cache, q = whole[0], whole[1], whole[2], whole[4]
        g = gen(9)
        normal(g, 37, 20 * 128)
        qw, kw = ((1.0 + 0.3 * normal(g, 128)).to(BF16) for _ in range(2))
        pos = torch.randint(0, 50000, (37,), generator=g, device=DEV, dtype=I32)
        for r in (0, 19, 36):
            one = Cache(cache.pages, 4, 16, 128, fp8)
            q1 = torch.empty((1, 12, 128), dtype=BF16, device=DEV)
            qp.qk_norm_rope_cache(qkv[r:r + 1], qw, kw, EPS, pos[r:r + 1].clone(), qp.rope_inv_freq(96, 1e6).to(DEV), 1.0,
                                  qp.QP_ROPE_HALF, slots[r:r + 1].clone(), qp.KVCache(one.k, one.v, one.ks, one.vs), q1)
            assert torch.equal(q1[0], q[r])
            s = slots[r].item()
            for a, b in zip(one.tensors(), cache.tensors()):
                assert torch.equal(a[s // 16, :, s % 16], b[s // 16, :, s % 16])
