"""paged_attention against the 64-bit form: lengths, heads, sizes, windows, cache
forms, holes, padding, NaN where nothing may be read."""
import math

import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests import decoder_ref as ref
from tests.decoder_ref import BF16, I32, U8, DEV, Cache, gen, normal

pytestmark = pytest.mark.gpu
CANARY = -12288.0


class Batch:
    """Sequences of (new tokens, cached positions), with random pages."""

    def __init__(self, seqs, heads, kv, d, fp8=False, page=16, window=0, seed=0, before=0, behind=0, holes=(), peaked=1.0,
                 max_q=None, width=None, scale=None):
        g = gen(seed)
        self.seqs, self.window, self.kv, self.heads, self.d = seqs, window, kv, heads, d
        news, lens = [n for n, _ in seqs], [m for _, m in seqs]
        self.t = sum(news) + before + behind
        self.before = before
        each = [-(-m // page) for m in lens]
        pages = max(sum(each) + 3, 4)
        width = width or max(max(each), 1)
        order = torch.randperm(pages, generator=g, device=DEV).to(I32)
        # unused entries name pages that exist (and hold NaN), or none
        self.table = torch.randint(-2, pages + 2, (len(seqs), width), generator=g, device=DEV, dtype=I32)
        self.cache = Cache(pages, kv, page, d, fp8)
        self.k, self.v, self.hole = [], [], []
        at = 0
        for i, m in enumerate(lens):
            ids = order[at:at + each[i]]
            at += each[i]
            self.table[i, :each[i]] = ids
            slots = (ids.long()[torch.arange(m, device=DEV) // page] * page + torch.arange(m, device=DEV) % page)
            if m:
                self.cache.put("k", slots, peaked * normal(g, m, kv, d))
                self.cache.put("v", slots, normal(g, m, kv, d) + 0.5)
            self.k.append(self.cache.get("k", slots))
            self.v.append(self.cache.get("v", slots))
            self.hole.append(torch.zeros(m, dtype=torch.bool, device=DEV))
        for i, block, name in holes:
            self.table[i, block] = name
            self.hole[i][block * page:(block + 1) * page] = True
        self.starts = [before + sum(news[:i]) for i in range(len(seqs) + 1)]
        self.q_start = torch.tensor(self.starts, dtype=I32, device=DEV)
        self.kv_len = torch.tensor(lens, dtype=I32, device=DEV)
        self.q = normal(g, self.t, heads, d).to(BF16)
        self.q[:before] = math.nan
        self.q[self.starts[-1]:] = math.nan
        self.max_q = max_q or max(max(news), 1)
        self.scale = scale or d ** -0.5
        self.handle = qp.KVCache(self.cache.k, self.cache.v, self.cache.ks, self.cache.vs)
        self.work = torch.full((qp.paged_attention_workspace(self.t, len(seqs), self.max_q, heads, kv, d),), 0xFF,
                               dtype=U8, device=DEV)

    def call(self, out=None, stream=None):
        if out is None:
            out = torch.full_like(self.q, CANARY)
        qp.paged_attention(self.q, self.handle, self.table, self.q_start, self.kv_len, self.max_q, self.scale, self.window,
                           self.work, out, stream=stream)
        return out

    def check(self, out=None):
        if out is None:
            out = self.call()
        torch.cuda.synchronize()
        inside = torch.zeros(self.t, dtype=torch.bool, device=DEV)
        for i, (n, m) in enumerate(self.seqs):
            if n == 0:
                continue
            rows = slice(self.starts[i], self.starts[i] + n)
            inside[rows] = True
            seen = ref.visible(n, m, self.window, self.hole[i])
            want, tol = ref.attention(self.q[rows], self.k[i], self.v[i], seen, self.scale)
            ref.assert_rounded(out[rows], want, tol)
            assert (out[rows].double() - want).norm() <= 2.0 ** -8 * want.norm()
            assert not out[rows][~seen.any(dim=1)].any()
        assert torch.all(out[~inside] == CANARY)
        return out


FORMS = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])


@FORMS
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 300, 1000, 4099])
def test_one_token(length, fp8):
    Batch([(1, length)], 8, 2, 128, fp8, seed=length).check()


@FORMS
@pytest.mark.parametrize("heads,kv", [(1, 1), (2, 2), (5, 1), (8, 1), (14, 2), (12, 3), (16, 1), (20, 2), (40, 4), (33, 1),
                                      (64, 1), (96, 2), (300, 1)])
def test_groups_of_heads(heads, kv, fp8):
    Batch([(1, 77), (1, 300), (1, 1)], heads, kv, 64, fp8, page=32, seed=heads).check()
    Batch([(3, 77), (2, 150)], heads, kv, 64, fp8, page=32, seed=heads).check()


@FORMS
@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
def test_head_sizes(d, fp8):
    Batch([(1, 70), (1, 200)], 8, 2, d, fp8, seed=d).check()
    Batch([(40, 70), (9, 200)], 8, 2, d, fp8, seed=d).check()
    Batch([(200, 333)], 4, 2, d, fp8, seed=d).check()


@FORMS
@pytest.mark.parametrize("page", [16, 32, 128, 512, 4096])
def test_page_sizes(page, fp8):
    Batch([(1, 700), (1, 513), (1, 16)], 8, 2, 128, fp8, page=page, seed=page).check()
    Batch([(100, 700), (65, 513), (16, 16)], 8, 2, 128, fp8, page=page, seed=page).check()


@FORMS
@pytest.mark.parametrize("n", [2, 3, 4, 5, 7, 8, 16, 17, 31, 33, 64, 65, 100, 129, 257, 600])
def test_chunks(n, fp8):
    Batch([(n, n)], 8, 2, 128, fp8, seed=n).check()
    Batch([(n, n + 301), (n - 1, 2 * n)], 10, 2, 128, fp8, seed=n).check()


@FORMS
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 129, 400, 5000])
def test_windows(window, fp8):
    Batch([(1, 500), (1, 30), (1, 129)], 8, 2, 128, fp8, window=window, seed=window).check()
    Batch([(5, 500), (4, 30), (2, 129)], 8, 2, 128, fp8, window=window, seed=window).check()
    Batch([(150, 500), (30, 30), (129, 129), (1, 260)], 8, 2, 64, fp8, window=window, seed=window).check()


@FORMS
def test_a_ragged_batch_with_empty_sequences_and_padding(fp8):
    seqs = [(0, 0), (1, 40), (0, 100), (7, 7), (1, 1), (130, 333), (0, 0), (16, 900), (0, 5)]
    Batch(seqs, 12, 4, 128, fp8, before=3, behind=21, seed=1).check()
    Batch([(0, 0), (1, 40), (0, 100), (1, 1), (1, 2000), (0, 0)], 12, 4, 128, fp8, before=1, behind=4, seed=2).check()
    Batch([(0, 0), (0, 7)], 8, 8, 128, fp8, behind=2, seed=2).check()


@FORMS
def test_rows_with_nothing_to_attend_to(fp8):
    """Fewer cached positions than rows: the first rows see nothing and give zeros."""
    Batch([(5, 2), (1, 0), (200, 70), (3, 3)], 8, 2, 128, fp8, seed=4).check()
    Batch([(1, 0), (1, 0), (1, 9)], 8, 2, 128, fp8, seed=5).check()


@FORMS
@pytest.mark.parametrize("n", [1, 6, 90])
def test_holes(n, fp8):
    """Page numbers outside the cache: their positions are as if they were not there."""
    b = Batch([(n, 200), (n, 64 + n), (n, 100)], 8, 2, 128, fp8, page=32, seed=n,
              holes=[(0, 0, -1), (0, 3, 1 << 30), (1, 0, -(1 << 31)), (1, 1, -7)])
    b.table[2, :4] = b.cache.pages                      # nothing but holes
    b.hole[2][:] = True
    b.check()


@FORMS
def test_sequences_whose_numbers_do_not_fit_are_left_out(fp8):
    b = Batch([(2, 40), (3, 50), (1, 30)], 4, 2, 64, fp8, seed=6)
    good = b.check()
    for change in ("len", "negative", "start", "past", "falling"):
        c = Batch([(2, 40), (3, 50), (1, 30)], 4, 2, 64, fp8, seed=6)
        out_rows = slice(2, 5)                          # the middle sequence's rows
        if change == "len":
            c.kv_len[1] = 65                            # 4 pages of 16 in the table
        elif change == "negative":
            c.kv_len[1] = -5
        elif change == "start":
            c.q_start[0], out_rows = -1, slice(0, 2)
        elif change == "past":
            c.q_start[3], out_rows = 7, slice(5, 6)
        else:
            c.q_start[2], out_rows = 1, slice(2, 5)
        out = c.call()
        torch.cuda.synchronize()
        if change == "falling":                         # the last then spans rows 1..5, more than max_q
            assert torch.all(out[2:] == CANARY) and torch.equal(out[:2], good[:2])
            continue
        kept = torch.ones(6, dtype=torch.bool)
        kept[out_rows] = False
        assert torch.all(out[out_rows] == CANARY), change
        assert torch.equal(out[kept.to(DEV)], good[kept.to(DEV)]), change


@FORMS
def test_more_rows_than_max_q_are_left_out(fp8):
    b = Batch([(2, 40), (40, 50), (1, 30)], 4, 2, 64, fp8, seed=7, max_q=2)
    out = b.call()
    torch.cuda.synchronize()
    assert torch.all(out[2:42] == CANARY)
    b.seqs = [(2, 40), (0, 50), (1, 30)]
    b.starts = [0, 42, 42]
    b.check(out)


@FORMS
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n", [3, 40, 300])
def test_what_a_row_does_not_see_has_no_influence(n, bad, fp8):
    """NaN and infinities at a chunk's own later positions: the rows before them
    are as if they were not there, those after them are not finite."""
    if fp8 and not math.isnan(bad):
        pytest.skip("E4M3 has no infinities")
    for window in (0, 50):
        b = Batch([(n, n + 37)], 8, 2, 128, fp8, window=window, seed=n)
        want = b.check()
        for which in (b.cache.k, b.cache.v):
            for back in (0, 1, n // 2):
                pos = n + 37 - 1 - back
                slot = b.table[0, pos // 16], slice(None), pos % 16
                kept = which[slot].clone()
                which[slot] = ref.NAN_CODE if fp8 else bad
                out = b.call()
                row = n - 1 - back
                assert torch.equal(out[:row], want[:row]), (window, back)
                if which is b.cache.v:
                    assert not torch.isfinite(out[row].float()).any()
                which[slot] = kept
        # and one that only the window hides
        if window and n > 60:
            slot = b.table[0, 0], slice(None), 5
            b.cache.v[slot] = ref.NAN_CODE if fp8 else bad
            out = b.call()
            first = 5 + window - 37                      # the first row that no longer sees position 5
            assert torch.equal(out[max(first, 0):], want[max(first, 0):])


@FORMS
def test_sharp_and_large_scores(fp8):
    """Scores far apart: the running maximum moves, small probabilities vanish."""
    for n, length in ((1, 900), (4, 900), (130, 400)):
        for peaked in (8.0, 60.0):
            b = Batch([(n, length)], 8, 2, 128, fp8, seed=n, peaked=peaked)
            b.check()
    # rising along the sequence, so that every step brings a new maximum
    b = Batch([(1, 1000), (70, 900)], 4, 1, 64, False, seed=3)
    for i, (n, m) in enumerate(b.seqs):
        slots = b.table[i].long()[torch.arange(m, device=DEV) // 16] * 16 + torch.arange(m, device=DEV) % 16
        ramp = torch.arange(m, device=DEV)[:, None, None] / 8.0 * torch.ones((m, 1, 64), device=DEV)
        b.cache.put("k", slots, ramp)
        b.k[i] = b.cache.get("k", slots)
    b.q.copy_(b.q.abs())
    b.check()


def test_identical_values_come_back():
    """V the same everywhere: the weights sum to one, whatever they are."""
    for n, length in ((1, 5000), (6, 777), (150, 600)):
        b = Batch([(n, length)], 8, 2, 128, seed=n)
        slots = b.table[0].long()[torch.arange(length, device=DEV) // 16] * 16 + torch.arange(length, device=DEV) % 16
        b.cache.put("v", slots, torch.full((length, 2, 128), 3.0, device=DEV))
        b.v[0] = b.cache.get("v", slots)
        b.check()


@FORMS
def test_many_sequences(fp8):
    seqs = [(1, 1 + (37 * i) % 211) for i in range(700)]
    Batch(seqs, 8, 2, 64, fp8, seed=8).check()
    seqs = [((7 * i) % 23, 23 + (37 * i) % 211) for i in range(300)]
    Batch(seqs, 6, 2, 64, fp8, seed=8).check()


def test_a_long_cache_and_a_wide_table():
    Batch([(1, 60000), (1, 3)], 8, 1, 128, seed=9, width=9000, page=16).check()
    Batch([(40, 30000), (3, 3)], 8, 1, 128, seed=9, width=5000, page=16).check()


def test_the_same_call_gives_the_same_bits():
    for seqs in ([(1, 3000), (1, 100), (1, 5)], [(100, 900), (33, 2000)]):
        b = Batch(seqs, 8, 2, 128, seed=3)
        first = b.call().clone()
        for _ in range(3):
            b.work.fill_(0x7F)
            assert torch.equal(b.call(), first)


@FORMS
def test_a_cache_of_more_than_2_to_the_32_bytes(fp8):
    """Pages beyond 2^32 bytes and 2^31 elements: offsets are 64 bits wide."""
    d, kv, page = 128, 8, 256
    pages = (1 << 33) // (kv * page * d * 2) + 3        # 8.6 GB of BF16, 4.3 GB of E4M3
    shape = (pages, kv, page, d)
    k, v = (torch.zeros(shape, dtype=U8 if fp8 else BF16, device=DEV) for _ in range(2))
    ks, vs = ((torch.zeros(shape[:3], device=DEV) if fp8 else None) for _ in range(2))
    for n in (1, 64):
        b = Batch([(n, 600)], 16, kv, d, fp8, page=page, seed=12)
        ids = torch.tensor([pages - 1, pages // 2 + 1, pages - 2], device=DEV)
        for big, small in ((k, b.cache.k), (v, b.cache.v), (ks, b.cache.ks), (vs, b.cache.vs)):
            if big is not None:
                big[ids] = small[b.table[0].long()]
        b.table[0] = ids.to(I32)
        b.handle = qp.KVCache(k, v, ks, vs)
        b.check()
