"""token_logprobs over the whole range of finite logits: masks by large finite
values, and logits far from zero.  A shift of all logits changes nothing in the
formula, and the bounds of the 64-bit form have no term in the logits' size."""
import math

import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import decoder_ref as ref
from tests.decoder_ref import BF16, F32, I32, U8, DEV, gen
from tests.test_gpu_logprobs import call, check, logits, some_targets

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
# rows that several workgroups share, and 2048 that have one each
SIZES = pytest.mark.parametrize("rows,vocab", [(14, 152064), (9, 4099), (2048, 5003)])
FILLS = [-1e4, -1e9, -1e10, -1e20, -1e30]


def masked(rows, vocab, dtype, fill):
    """Rows in turn: masked here and there (half, nine in ten, nearly all), in
    front, behind, in the middle, but for one token, and whole; the last ones are
    masked by fills that differ."""
    g = gen(vocab)
    x = logits(vocab, rows, vocab, F32)
    row, col = torch.arange(rows, device=DEV)[:, None] % 9, torch.arange(vocab, device=DEV)[None]
    share = torch.tensor([0.5, 0.9, 0.999], device=DEV)[row.clamp(max=2)]
    hide = torch.where(row < 3, torch.rand((rows, vocab), generator=g, device=DEV) < share, False)
    hide |= (row == 3) & (col < min(3000, vocab - 7))
    hide |= (row == 4) & (col >= vocab // 3)
    hide |= (row == 5) & (col >= 64) & (col < vocab - 64)
    hide |= (row == 6) & (col != vocab // 2)
    hide |= row == 7
    x[hide] = fill
    other = (row == 8) & (torch.rand((rows, vocab), generator=g, device=DEV) < 0.9)
    fills = torch.tensor(FILLS, device=DEV)[torch.randint(0, 5, (rows, vocab), generator=g, device=DEV)]
    return torch.where(other, fills, x).to(dtype)


@TYPES
@SIZES
@pytest.mark.parametrize("fill", FILLS)
def test_finite_masks(rows, vocab, fill, dtype):
    x = masked(rows, vocab, dtype, fill)
    t = some_targets(3, rows, vocab)
    check(x, t, 5)
    # and without the entropy, which another kernel serves: the same numbers
    logprob, _, ids, best = call(x, t, 5)
    a, i, b = torch.empty_like(logprob), torch.empty_like(ids), torch.empty_like(best)
    work = torch.empty(qp.token_logprobs_workspace(rows, vocab, 5), dtype=U8, device=DEV)
    qp.token_logprobs(x, t, a, None, i, b, work)
    assert torch.equal(a, logprob) and torch.equal(i, ids) and torch.equal(b, best)


@TYPES
@SIZES
@pytest.mark.parametrize("offset", [-30.0, 1e2, -1e3, 1e4, -1e5, 1e6, -1e7, 1.6777e7, 1e8, 1e10, -1e20, 1e30])
def test_logits_far_from_zero(rows, vocab, offset, dtype):
    """Where a type's steps are wider than the logits' spread many are equal."""
    x = (logits(vocab, rows, vocab, F32).double() + offset).to(dtype)
    check(x, some_targets(5, rows, vocab), 7)


@TYPES
@SIZES
def test_logits_of_all_sizes_in_a_row(rows, vocab, dtype):
    """Maxima that grow along the row, slowly and by orders of magnitude."""
    n = torch.arange(vocab, device=DEV, dtype=torch.float64) / vocab
    shapes = [2.0 ** 24 + 300.0 * (n - 0.5), -(2.0 ** 24) + 300.0 * (0.5 - n), 10.0 ** (8.0 * n), -(10.0 ** (30.0 * (1.0 - n))),
              1e6 + 40.0 * n, -1e5 + 60.0 * n, 10.0 ** (30.0 * n), 20.0 * n, -2e7 - 80.0 * n]
    x = torch.stack([shapes[r % len(shapes)] for r in range(rows)]).to(dtype)
    check(x, some_targets(7, rows, vocab), 6)


@TYPES
def test_a_shift_changes_nothing(dtype):
    """Logits on a grid that the shifted ones lie on as well: the same numbers, up
    to the sums' roundings."""
    rows, vocab = 4, 20011
    x = torch.randint(-20, 21, (rows, vocab), generator=gen(1), device=DEV).float()
    if dtype == F32:
        x /= 4.0
    t = some_targets(2, rows, vocab)
    want = call(x.to(dtype), t, 3)
    for offset in ((64.0,) if dtype == BF16 else (64.0, -4096.0, 1048576.0, -2097152.0)):
        got = call((x + offset).to(dtype), t, 3)
        assert torch.equal(got[2], want[2])
        rel = torch.full((rows,), 2.0 * ((vocab / 256 + 64) * 2.0 ** -23 + 2.0 ** -20), device=DEV)
        for a, b in zip(got[:2] + got[3:], want[:2] + want[3:]):
            ref.assert_logprobs(a.reshape(rows, -1), b.double().reshape(rows, -1), rel * (1.0 + math.log(vocab)))
