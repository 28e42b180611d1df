"""paged_attention where one kernel ends and another begins: rows of a sequence
(times heads of a kv head) around 16, 32, 64 and 128, for every padded head size
and both cache forms, over few keys and over so many that they are split; what a
row does not see, at every head size; and rows joined from few and many parts."""
import math

import pytest
import torch

from tests import decoder_ref as ref
from tests.test_gpu_attention import FORMS, Batch

pytestmark = pytest.mark.gpu


@FORMS
@pytest.mark.parametrize("d", [32, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("heads,n", [(15, 1), (16, 1), (17, 1), (8, 4), (11, 3), (33, 1), (16, 4), (13, 5), (65, 1), (32, 4),
                                     (43, 3)])
def test_around_the_boundaries(heads, n, d, fp8):
    Batch([(n, 333), (n, n), (max(n - 1, 0), 40)], heads, 1, d, fp8, seed=heads).check()
    Batch([(n, 5003)], heads, 1, d, fp8, seed=heads).check()


@FORMS
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,n", [(1, 1), (3, 1), (8, 1), (5, 4), (60, 1), (8, 50)])
def test_joins_of_few_and_many_parts(heads, n, d, fp8):
    Batch([(n, 40000)], heads, 1, d, fp8, page=64, seed=n).check()
    Batch([(n, 2100 + 700 * (i % 3)) for i in range(60)], heads, 1, d, fp8, page=64, seed=n).check()


@FORMS
@pytest.mark.parametrize("d", [48, 64, 192, 256])
@pytest.mark.parametrize("heads,n", [(2, 1), (2, 3), (24, 2), (4, 40), (2, 150)])
def test_what_a_row_does_not_see_at_every_head_size(heads, n, d, fp8):
    """A NaN in one element of V: it reaches the rows that see its position, in
    that element alone, and no other row."""
    b = Batch([(n, n + 37), (n, 2 * n + 3)], heads, 2, d, fp8, seed=n)
    want = b.check()
    for element in (0, 1, 15, 16, d // 2 - 1, d // 2, d - 9, d - 1):
        for back in (0, n // 2):
            pos = n + 37 - 1 - back
            at = b.table[0, pos // 16], 1, pos % 16, element
            kept = b.cache.v[at].clone()
            b.cache.v[at] = ref.NAN_CODE if fp8 else math.nan
            out = b.call()
            hit = torch.zeros_like(out, dtype=torch.bool)
            hit[n - 1 - back:n, heads // 2:, element] = True
            assert torch.isnan(out[hit].float()).all(), (element, back)
            assert torch.equal(out[~hit], want[~hit]), (element, back)
            b.cache.v[at] = kept


@FORMS
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows_and_holes_over_split_keys(d, fp8):
    for heads, n in ((4, 1), (4, 7), (4, 40), (2, 300)):
        for window in (0, 1500):
            Batch([(n, 6000), (n, 900 + n)], heads, 2, d, fp8, page=32, window=window, seed=n,
                  holes=[(0, 0, -1), (0, 130, 1 << 29), (0, 187, -5), (1, 3, -1)]).check()


@FORMS
def test_windows_larger_than_any_length(fp8):
    """The largest windows are the call without one."""
    for n in (1, 5, 90):
        b = Batch([(n, 700), (n, 95 + n)], 8, 2, 128, fp8, seed=n)
        want = b.check().clone()
        for window in (701, (1 << 27) - 1, 1 << 27, (1 << 31) - 1, 1 << 31, (1 << 32) - 1):
            b.window = window
            assert torch.equal(b.call(), want), window


@FORMS
def test_rows_of_another_sequence_and_shared_pages(fp8):
    """Sequences that share a prefix's pages read the same keys."""
    b = Batch([(1, 640), (3, 643), (70, 710), (1, 640)], 8, 2, 128, fp8, page=64, seed=3)
    pages = b.table[0, :10].clone()
    for i in (1, 2, 3):
        b.table[i, :10] = pages
        b.k[i][:640], b.v[i][:640] = b.k[0], b.v[0]
    b.check()


@FORMS
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("n", [255, 256, 257, 700])
def test_small_heads_in_units_of_either_size(n, d, fp8):
    for window in (0, 150):
        Batch([(n, n), (3, 90), (n - 9, 2 * n), (1, 1), (64, 3000)], 8, 2, d, fp8, window=window, seed=n).check()
        Batch([(n, 2 * n)], 14, 2, d, fp8, window=window, seed=n, holes=[(0, 3, -1), (0, 20, 1 << 30)]).check()
