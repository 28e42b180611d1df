"""paged_attention with infinities in K."""
import math

import pytest
import torch

from tests.decoder_ref import DEV
from tests.test_gpu_attention import Batch

pytestmark = pytest.mark.gpu


def slots_of(b, i):
    at = torch.arange(b.seqs[i][1], device=DEV)
    return b.table[i].long()[at // b.cache.page] * b.cache.page + at % b.cache.page


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
