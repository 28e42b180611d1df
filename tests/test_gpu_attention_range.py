"""paged_attention with scores of any finite size, infinities in K, and the bits
of rows beside keys that they do not see."""
import math

import pytest
import torch

from tests import decoder_ref as ref
from tests.decoder_ref import DEV, gen
from tests.test_gpu_attention import FORMS, Batch

pytestmark = pytest.mark.gpu


def slots_of(b, i):
    at = torch.arange(b.seqs[i][1], device=DEV)
    return b.table[i].long()[at // b.cache.page] * b.cache.page + at % b.cache.page


@FORMS
@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("n,length", [(1, 700), (5, 300), (150, 400), (1, 5000)])
def test_scores_of_any_size(n, length, d, fp8):
    """One entry a head, so that a score is one product: size * (1 + i / 128) of a
    random i.  From 2^20 on scores of different i are more than 2^12 apart and the
    softmax is even over the visible keys of the largest.  Equal scores have equal
    probabilities, rounded to BF16 over the line alone: 2^-8 of the mean |v| and
    the output's own rounding."""
    b = Batch([(n, length)], 8, 2, d, fp8, seed=n, scale=0.75)
    i = torch.randint(0, 128, (length,), generator=gen(d), device=DEV)
    v = b.v[0]
    pos = length - n + torch.arange(n, device=DEV)[:, None]
    seen = torch.arange(length, device=DEV)[None] <= pos
    for sign in (1.0, -1.0):
        best = torch.where(seen, sign * i, -math.inf).amax(dim=1, keepdim=True)
        w = (seen & (sign * i == best)).double()
        w /= w.sum(dim=1, keepdim=True)
        want, mag = ((w @ x.reshape(length, -1)).view(n, 2, d).repeat_interleave(4, dim=1) for x in (v, v.abs()))
        for size in (20, 26, 29, 31, 33, 40, 64, 100, 120):
            k = torch.zeros((length, 2, d), device=DEV)
            k[..., d // 3] = (sign * 2.0 ** (size // 2) * (1.0 + i / 128.0))[:, None]
            b.cache.put("k", slots_of(b, 0), k)
            b.q.zero_()
            b.q[..., d // 3] = 2.0 ** (size - size // 2)
            ref.assert_rounded(b.call(), want, 2.0 ** -8 * mag + 1e-30)


@pytest.mark.parametrize("d", [16, 48, 80, 96, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("n", [1, 6, 90])
def test_scores_of_minus_infinity(n, d):
    """-inf in one entry of K that every query multiplies with something positive:
    the position's probability is 0, wherever in the head it stands."""
    b = Batch([(n, 200), (n, 90 + n)], 8, 2, d, seed=d + n)
    for element in (0, 5, d // 2, d - 1):
        c = Batch([(n, 200), (n, 90 + n)], 8, 2, d, seed=d + n)
        c.q[..., element] = c.q[..., element].abs() + 0.5
        for s, (_, length) in enumerate(c.seqs):
            hidden = torch.arange(length, device=DEV) % 7 == 3
            slots = slots_of(c, s)[hidden]
            c.cache.k[slots // c.cache.page, :, slots % c.cache.page, element] = -math.inf
            # (what the 64-bit form leaves out as it does a hole's positions)
            c.hole[s] |= hidden
        c.check()
    b.check()


@FORMS
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 4, 16, 60, 300])
def test_bits_do_not_depend_on_unseen_keys(n, d, fp8):
    """A key that only the last token's rows see, of any score there: the bits of
    the rows before stay the same; and one that the window hides from all but the
    first rows.  Scores rise along the keys, some units of base 2 a tile, so that
    every tile brings every row a new maximum."""
    for window in (0, 64):
        b = Batch([(n, n + 537)], 8, 2, d, fp8, window=window, seed=n)
        slots = slots_of(b, 0)
        b.q.copy_(b.q.abs())
        rise = 0.05 * d ** -0.5 * torch.arange(n + 537, device=DEV)[:, None, None]
        b.cache.put("k", slots, rise + 0.2 * torch.randn((n + 537, 2, d), generator=gen(n), device=DEV))
        want = b.call().clone()
        last, old = n + 536, 537 - 63
        for at, rows, seen_by in ((last, slice(0, n - 1), n - 1), (old, slice(1, n), 0)):
            if at == old and not window:
                continue
            for size in (1.0, 3.0, 30.0, 1000.0):
                kept = [x.clone() for x in b.cache.tensors()]
                q = b.q[seen_by].float().view(2, 4, d).mean(dim=1)
                b.cache.put("k", slots[at:at + 1], size * q[None])
                out = b.call()
                assert not torch.equal(out[seen_by], want[seen_by])
                assert torch.equal(out[rows], want[rows]), (window, at, size)
                for x, was in zip(b.cache.tensors(), kept):
                    x.copy_(was)


@pytest.mark.parametrize("d,heads,n,length", [(128, 8, 1, 700), (128, 8, 8, 300), (128, 16, 1, 3000), (64, 8, 16, 500), (64, 12, 3, 900),
                                              (80, 8, 4, 400), (256, 8, 4, 600), (192, 16, 2, 333)])
def test_few_rows_over_a_bf16_cache_round_the_output_alone(d, heads, n, length):
    """Probabilities meet V in two parts, to 2^-16: the 64-bit form's bound less what
    it has for their rounding to BF16, 2^-8 of sum p |v|."""
    b = Batch([(n, length), (n, n + 5)], heads, 2, d, seed=d + n)
    out = b.check()
    for i, (_, m) in enumerate(b.seqs):
        rows = slice(b.starts[i], b.starts[i] + n)
        args = b.q[rows], b.k[i], ref.visible(n, m, 0), b.scale
        want, tol = ref.attention(args[0], args[1], b.v[i], *args[2:])
        mag, _ = ref.attention(args[0], args[1], b.v[i].abs(), *args[2:])
        ref.assert_rounded(out[rows], want, tol - (2.0 ** -8 - 2.0 ** -16) * mag)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n,length,d", [(1, 700, 128), (5, 5000, 64), (100, 900, 128), (300, 700, 256), (40, 4000, 80)])
def test_infinities_in_v(n, length, d, bad):
    """Early in the cache, where all rows see whole tiles, among the chunk's own
    positions, and where its window begins: NaN or an infinity for the rows that see
    the position, in that element; all other numbers keep their bits."""
    for window in (0, length - n - 70):
        b = Batch([(n, length)], 8, 2, d, window=window, seed=n)
        want = b.call().clone()
        slots = slots_of(b, 0)
        pos = length - n + torch.arange(n, device=DEV)
        first = length - n - window + 1 if window else 0
        for at in (3, 130, first + n // 2, length - n, length - 1):
            where = slots[at] // b.cache.page, 1, slots[at] % b.cache.page, d // 3
            kept = b.cache.v[where].clone()
            b.cache.v[where] = bad
            out = b.call()
            hit = torch.zeros_like(out, dtype=torch.bool)
            hit[(at <= pos) & ((pos - at < window) if window else True), 4:, d // 3] = True
            assert not torch.isfinite(out[hit].float()).any(), (window, at)
            assert torch.equal(out[~hit], want[~hit]), (window, at)
            b.cache.v[where] = kept
