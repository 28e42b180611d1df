"""token_logprobs against the 64-bit form: sizes, types, ties, masks, targets."""
import math

import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import decoder_ref as ref
from tests.decoder_ref import BF16, F32, I32, U8, DEV, gen, normal

pytestmark = pytest.mark.gpu


def call(x, targets, top):
    rows, vocab = x.shape
    new = lambda *s, dtype=F32: torch.full(s, -77, dtype=dtype, device=DEV)  # noqa: E731
    out = new(rows), new(rows), new(rows, top, dtype=I32), new(rows, top)
    work = torch.full((qp.token_logprobs_workspace(rows, vocab, top),), 0xFF, dtype=U8, device=DEV)
    qp.token_logprobs(x, targets, *out, work)
    torch.cuda.synchronize()
    return out


def check(x, targets, top):
    logprob, entropy, ids, best = call(x, targets, top)
    want, ent, order, wbest, rel = ref.logprobs(x, targets, top)
    assert torch.equal(ids.long(), order)
    ref.assert_logprobs(logprob[:, None], want[:, None], rel)
    ref.assert_logprobs(best, wbest, rel)
    # the entropy's parts ln s and sum p y each carry the sums' error
    room = rel * (2.0 + (ent.abs() + math.log(x.shape[1])) * 2.0) + 2.0 ** -22 * ent.abs() + 1e-30
    assert torch.all((entropy.double() - ent).abs() <= room), (entropy.double() - ent).abs().max()


def logits(seed, rows, vocab, dtype, spread=3.0):
    return (spread * normal(gen(seed), rows, vocab)).to(dtype)


def some_targets(seed, rows, vocab):
    return torch.randint(0, vocab, (rows,), generator=gen(seed + 1), device=DEV, dtype=I32)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 7, 5), (5, 33, 32), (4, 255, 4), (3, 257, 20), (2, 2048, 32), (3, 4097, 8),
    (1, 8193, 32), (7, 50257, 20), (1, 129281, 20), (2, 152064, 32), (16, 152064, 5), (1, 262145, 1), (300, 1031, 3),
    (513, 10007, 2), (40, 70001, 7)])
def test_sizes(rows, vocab, top, dtype):
    check(logits(vocab + rows, rows, vocab, dtype), some_targets(rows, rows, vocab), top)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("vocab", [64, 9000, 152064])
def test_ties_go_to_the_lowest_token(vocab, dtype):
    g = gen(vocab)
    top = 32
    same = torch.zeros((1, vocab), device=DEV)
    few = torch.randint(-2, 3, (2, vocab), generator=g, device=DEV).float()
    zeros = torch.where(torch.rand((1, vocab), generator=g, device=DEV) < 0.5, 0.0, -0.0)      # +0 and -0 are equal
    late = torch.full((1, vocab), -1.0, device=DEV)
    late[0, -top:] = 2.0
    rising = torch.arange(vocab, device=DEV)[None].float() / vocab
    for x in (same, few, zeros, late, rising, -rising):
        check(x.to(dtype).contiguous(), some_targets(0, x.shape[0], vocab), min(top, vocab))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("vocab", [50, 9001, 152064])
def test_masked_logits(vocab, dtype):
    x = logits(vocab, 8, vocab, dtype)
    x[0] = -math.inf                                     # nothing is left
    x[1, 1:] = -math.inf                                 # one is left, the first
    x[2, :-1] = -math.inf                                # the last
    x[3, torch.rand(vocab, generator=gen(2), device=DEV) < 0.95] = -math.inf
    x[4, : vocab // 2] = -math.inf
    x[5] = torch.finfo(dtype).min                        # masked by the lowest value, all of it
    x[6, ::2] = torch.finfo(dtype).min
    x[7] = torch.finfo(dtype).max
    t = torch.tensor([0, 0, vocab - 1, 7, vocab - 2, 3, 2, 4], dtype=I32, device=DEV)
    check(x, t, 20)
    logprob, entropy, _, best = call(x, t, 20)
    assert logprob[0] == -math.inf and entropy[0] == 0 and torch.all(best[0] == -math.inf)
    assert logprob[1] == 0 and logprob[2] == 0 and entropy[1] == 0 and entropy[2] == 0


def test_targets_outside_the_vocabulary_give_zero():
    x = logits(4, 5, 999, F32)
    t = torch.tensor([-1, 999, 0, -(1 << 31), (1 << 31) - 1], dtype=I32, device=DEV)
    check(x, t, 3)
    assert call(x, t, 0)[0][[0, 1, 3, 4]].abs().max() == 0


def test_each_output_alone():
    x = logits(6, 9, 20011, BF16)
    t = some_targets(6, 9, 20011)
    work = torch.empty(qp.token_logprobs_workspace(9, 20011, 4), dtype=U8, device=DEV)
    logprob, entropy, ids, best = call(x, t, 4)
    a, b = torch.empty_like(logprob), torch.empty_like(entropy)
    qp.token_logprobs(x, t, a, None, None, None, work)
    qp.token_logprobs(x, None, None, b, None, None, work)
    i, c = torch.empty_like(ids), torch.empty_like(best)
    qp.token_logprobs(x, None, None, None, i, c, work)
    assert torch.equal(a, logprob) and torch.equal(b, entropy) and torch.equal(i, ids) and torch.equal(c, best)


def test_nan_and_infinities_stay_in_their_row():
    x = logits(8, 4, 30001, F32)
    want = call(x[::2].contiguous(), some_targets(8, 4, 30001)[::2].contiguous(), 8)
    y = x.clone()
    y[1, 100:200] = math.nan
    y[3, 5] = math.inf
    logprob, entropy, ids, best = call(y, some_targets(8, 4, 30001), 8)
    assert torch.all((ids >= 0) & (ids < 30001))
    for a, b in zip((logprob, entropy, ids, best), want):
        ref.assert_logprobs(a[::2].double().reshape(2, -1), b.double().reshape(2, -1), torch.full((2,), 130 * 2.0 ** -23, device=DEV))


def test_the_largest_number_of_elements():
    rows, vocab = 14122, 152064                          # 2^31 - 1 elements hold 14122.7 rows
    x = torch.empty((rows, vocab), dtype=BF16, device=DEV)
    for at in range(0, rows, 1024):
        x[at:at + 1024].normal_(generator=gen(at))
    t = some_targets(0, rows, vocab)
    got = call(x, t, 4)
    for r in (0, 7000, rows - 1):
        want = ref.logprobs(x[r:r + 1], t[r:r + 1], 4)
        assert torch.equal(got[2][r:r + 1].long(), want[2])
        ref.assert_logprobs(got[0][r:r + 1, None], want[0][:, None], want[4])
