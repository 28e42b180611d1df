"""The operators of include/qproj_decoder.h together, as a decoder calls them:
a prompt in chunks and then token by token, a layer and a head against their
plain forms, captured graphs, several streams."""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from examples import layer_step
from tests import decoder_ref as ref
from tests.decoder_ref import BF16, F32, I32, U8, DEV, Cache, gen, normal

pytestmark = pytest.mark.gpu
FORMS = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
HEADS, KV, D, PAGE = 10, 2, 64, 16


@FORMS
def test_a_prompt_in_chunks_and_then_token_by_token(fp8):
    """Two sequences grow by different chunks; after each call the attention's rows
    are those of the 64-bit form over what the cache then holds."""
    g = gen(1)
    cache = Cache(40, KV, PAGE, D, fp8)
    handle = qp.KVCache(cache.k, cache.v, cache.ks, cache.vs)
    table = torch.randperm(40, generator=g, device=DEV).to(I32).view(2, 20)
    weights = [(1.0 + 0.2 * normal(g, D)).to(BF16) for _ in range(2)]
    inv_freq = qp.rope_inv_freq(D, 10000.0).to(DEV)
    have = [0, 0]
    for chunk in ((50, 7), (1, 1), (30, 0), (0, 1), (1, 1), (5, 5), (1, 130), (1, 1)):
        pos = [torch.arange(h, h + n, device=DEV) for h, n in zip(have, chunk)]
        slots = torch.cat([table[s].long()[p // PAGE] * PAGE + p % PAGE for s, p in enumerate(pos)]).to(I32)
        t = sum(chunk)
        qkv = normal(g, t, (HEADS + 2 * KV) * D).to(BF16)
        q, out = (torch.empty((t, HEADS, D), dtype=BF16, device=DEV) for _ in range(2))
        have = [h + n for h, n in zip(have, chunk)]
        qp.qk_norm_rope_cache(qkv, *weights, 1e-6, torch.cat(pos).to(I32), inv_freq, 1.0, qp.QP_ROPE_HALF, slots, handle, q)
        q_start = torch.tensor([0, chunk[0], t], dtype=I32, device=DEV)
        kv_len = torch.tensor(have, dtype=I32, device=DEV)
        work = torch.empty(qp.paged_attention_workspace(t, 2, max(chunk), HEADS, KV, D), dtype=U8, device=DEV)
        qp.paged_attention(q, handle, table, q_start, kv_len, max(chunk), D ** -0.5, 0, work, out)
        torch.cuda.synchronize()
        for s in range(2):
            if not chunk[s]:
                continue
            at = torch.arange(have[s], device=DEV)
            at = table[s].long()[at // PAGE] * PAGE + at % PAGE
            rows = slice(0, chunk[0]) if s == 0 else slice(chunk[0], t)
            want, tol = ref.attention(q[rows], cache.get("k", at), cache.get("v", at), ref.visible(chunk[s], have[s], 0), D ** -0.5)
            ref.assert_rounded(out[rows], want, tol)


@pytest.mark.parametrize("rows,heads,kv,d,cached", [(1, 8, 2, 64, 0), (3, 10, 2, 128, 333), (16, 8, 8, 80, 100)])
def test_a_layer_against_its_plain_form(rows, heads, kv, d, cached):
    """Queries, keys and outputs are BF16 on both sides, the probabilities on one:
    together less than 2^-7 of the attention's output.  Before the output product
    that output is E4M3, whose values are up to 2^-3 apart: a value off by 2^-7
    takes the next code in 2^-7 / 2^-3 of cases and is then off by 2^-3, so that the
    square of the error is 2^-10 of the value's.  The BF16 results are 2^-9 more."""
    layer = layer_step.Attention(rows, 512, heads, kv, d, cached, DEV)
    assert layer_step.check(layer, rows, 512, DEV) <= 2.0 ** -5 + 2.0 ** -9


def test_a_head_against_its_plain_form():
    """Log probabilities, about ln 2003 = 7.6, of F32 sums on both sides: an error of
    the sum is one of the logarithm, and 2003 / 256 + 64 roundings of 2^-23 are 2^-17
    of 7.6, 2^-19.6 on either side; the rest, 2^-22, is far below."""
    layer = layer_step.Head(5, 512, 2003, 7, DEV)
    assert layer_step.check(layer, 5, 512, DEV) <= 2.0 ** -18


class Step:
    """Chunks of prompts and single tokens in two attention calls that share a
    workspace, then the logits of every row; all lengths and slots on the device."""

    def __init__(self, fp8, work=None):
        self.fp8, self.seqs, self.t = fp8, 6, 6 * 40
        g = gen(3)
        self.cache = Cache(6 * 30, KV, PAGE, D, fp8)
        self.handle = qp.KVCache(self.cache.k, self.cache.v, self.cache.ks, self.cache.vs)
        self.table = torch.randperm(180, generator=g, device=DEV).to(I32).view(6, 30)
        new = lambda *s, dtype=I32: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
        self.qkv = new(self.t, (HEADS + 2 * KV) * D, dtype=BF16)
        self.positions, self.slots, self.q_start, self.kv_len = new(self.t), new(self.t), new(7), new(6)
        self.one_start = torch.arange(7, dtype=I32, device=DEV)
        self.q, self.out, self.last = (new(n, HEADS, D, dtype=BF16) for n in (self.t, self.t, 6))
        self.weight = (1.0 + 0.2 * normal(g, D)).to(BF16)
        self.inv_freq = qp.rope_inv_freq(D, 10000.0).to(DEV)
        self.logits, self.targets = new(self.t, 20011, dtype=BF16), new(self.t)
        self.found = new(self.t, dtype=F32), new(self.t, dtype=F32), new(self.t, 5), new(self.t, 5, dtype=F32)
        size = max(qp.paged_attention_workspace(self.t, 6, 40, HEADS, KV, D), qp.paged_attention_workspace(6, 6, 1, HEADS, KV, D),
                   qp.token_logprobs_workspace(self.t, 20011, 5))
        self.work = torch.empty(size, dtype=U8, device=DEV) if work is None else work

    def fill(self, seed):
        g = gen(seed)
        some = lambda lo, hi, n: torch.randint(lo, hi, (n,), generator=g, device=DEV)  # noqa: E731
        for x in self.cache.tensors():
            x.copy_(torch.randint(0, 0x70, x.shape, generator=g, device=DEV) if x.dtype == U8 else normal(g, *x.shape).abs())
        new, old = some(1, 41, 6), some(0, 400, 6)
        self.q_start[1:] = new.cumsum(0)
        self.kv_len.copy_(new + old)
        row = torch.arange(self.t, device=DEV)
        seq = (row[:, None] >= self.q_start[None, 1:]).sum(dim=1).clamp(max=5)
        pos = (old[seq] + row - self.q_start[seq]).clamp(max=479)
        inside = row < self.q_start[6]
        self.positions.copy_(pos)
        self.slots.copy_(torch.where(inside, self.table[seq, pos // PAGE] * PAGE + pos % PAGE, -1))
        self.qkv.copy_(normal(g, *self.qkv.shape))
        self.logits.copy_(3.0 * normal(g, *self.logits.shape))
        self.targets.copy_(some(0, 20011, self.t))
        for x in (self.q, self.out, self.last, *self.found):
            x.fill_(-3)

    def run(self):
        qp.qk_norm_rope_cache(self.qkv, self.weight, self.weight, 1e-6, self.positions, self.inv_freq, 1.0, qp.QP_ROPE_INTERLEAVED,
                              self.slots, self.handle, self.q)
        qp.paged_attention(self.q, self.handle, self.table, self.q_start, self.kv_len, 40, 0.125, 100, self.work, self.out)
        qp.paged_attention(self.q[:6], self.handle, self.table, self.one_start, self.kv_len, 1, 0.125, 0, self.work, self.last)
        qp.token_logprobs(self.logits, self.targets, *self.found, self.work)

    def result(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (*self.cache.tensors(), self.q, self.out, self.last, *self.found)]


def same(a, b):
    return all(torch.equal(x.view(U8), y.view(U8)) for x, y in zip(a, b))


def capture(step):
    step.run()                                        # loads the kernels before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    return graph


@FORMS
def test_replays_equal_the_eager_calls(fp8):
    step = Step(fp8)
    step.fill(0)
    graph = capture(step)
    for seed in range(1, 7):
        step.fill(seed)
        step.run()
        want = step.result()
        step.fill(seed)
        step.work.fill_(0xFF)
        graph.replay()
        assert same(step.result(), want), seed
        # the program's own work on the same buffers between two replays
        step.fill(100 + seed)
        step.run()
        step.out.float().sum().item()


@FORMS
def test_two_graphs_that_share_a_workspace(fp8):
    """One after the other on a stream, in both orders, several times."""
    first = Step(fp8)
    second = Step(fp8, first.work)
    want = []
    for seed, s in ((1, first), (2, second)):
        s.fill(seed)
        s.run()
        want.append(s.result())
    graphs = [capture(first), capture(second)]
    for turn in range(5):
        first.fill(1)
        second.fill(2)
        for g in (graphs if turn % 2 else graphs[::-1]):
            g.replay()
        assert same(first.result(), want[0]) and same(second.result(), want[1]), turn


@FORMS
def test_two_streams_at_once(fp8):
    steps, want = [Step(fp8) for _ in range(2)], []
    for n, s in enumerate(steps):
        s.fill(n)
        s.run()
        want.append(s.result())
    for turn in range(3):
        for n, s in enumerate(steps):
            s.fill(n)
        streams = [torch.cuda.Stream() for _ in steps]
        torch.cuda.synchronize()
        for _ in range(4):
            for s, st in zip(steps, streams):
                with torch.cuda.stream(st):
                    s.run()
        for s, w in zip(steps, want):
            assert same(s.result(), w), turn


@FORMS
def test_a_slot_given_twice(fp8):
    """Which of the two is kept is open; no other slot is touched, and the queries
    are those of the call that names each slot once."""
    a, b = Step(fp8), Step(fp8)
    for s in (a, b):
        s.fill(7)
    assert int(a.slots[4]) >= 0 and int(a.slots[9]) >= 0
    before = [x.clone() for x in b.cache.tensors()]
    b.slots[9] = b.slots[4]
    a.run()
    b.run()
    torch.cuda.synchronize()
    assert torch.equal(a.q, b.q)
    at = lambda x, slot: x[int(slot) // PAGE, :, int(slot) % PAGE]  # noqa: E731
    for x, y, old in zip(a.cache.tensors(), b.cache.tensors(), before):
        at(y, b.slots[4]).copy_(at(x, b.slots[4]))      # open
        at(x, a.slots[9]).copy_(at(old, a.slots[9]))    # not written by b
        assert torch.equal(x, y)


def test_tensors_that_do_not_fit_are_refused():
    s = Step(False)
    s.fill(1)
    s.run()
    want = s.result()
    att = lambda **k: qp.paged_attention(*[k.get(n, v) for n, v in dict(  # noqa: E731
        q=s.q, cache=s.handle, table=s.table, q_start=s.q_start, kv_len=s.kv_len, max_q=40, scale=0.125, window=100, work=s.work,
        out=s.out).items()])
    rope = lambda **k: qp.qk_norm_rope_cache(*[k.get(n, v) for n, v in dict(  # noqa: E731
        qkv=s.qkv, q_norm=s.weight, k_norm=s.weight, eps=1e-6, positions=s.positions, inv_freq=s.inv_freq, rope_scale=1.0,
        layout=qp.QP_ROPE_HALF, slots=s.slots, cache=s.handle, q_out=s.q).items()])
    logp = lambda **k: qp.token_logprobs(*[k.get(n, v) for n, v in dict(  # noqa: E731
        logits=s.logits, targets=s.targets, logprob=s.found[0], entropy=s.found[1], ids=s.found[2], best=s.found[3],
        work=s.work).items()])
    wrong = [
        lambda: att(q=s.q.float()), lambda: att(q=s.q[:, ::2]), lambda: att(out=s.out[:5]), lambda: att(table=s.table.long()),
        lambda: att(table=s.table.t()), lambda: att(q_start=s.q_start[:6]), lambda: att(kv_len=s.kv_len.cpu()),
        lambda: att(work=s.work[:64]), lambda: att(max_q=0), lambda: att(max_q=s.t + 1), lambda: att(scale=0.0),
        lambda: att(scale=float("nan")), lambda: att(work=s.work[1:]), lambda: att(q=s.q[:, :9].contiguous(), out=s.out[:, :9].contiguous()),
        lambda: rope(qkv=s.qkv[:, :-64]), lambda: rope(q_norm=None), lambda: rope(positions=s.positions[:-1]),
        lambda: rope(slots=s.slots.float()), lambda: rope(layout=5), lambda: rope(eps=0.0),
        lambda: rope(inv_freq=torch.ones(33, device=DEV)), lambda: rope(rope_scale=float("inf")),
        lambda: logp(logits=s.logits.half()), lambda: logp(targets=s.targets[:-1]), lambda: logp(work=s.work[:8]),
        lambda: logp(ids=s.found[2][:, :4]), lambda: logp(targets=None), lambda: logp(logits=s.logits[:, 1:]),
        lambda: qp.KVCache(s.cache.k, s.cache.v[:, :1]), lambda: qp.KVCache(s.cache.k, s.cache.v.view(U8)),
        lambda: qp.KVCache(s.cache.k.transpose(1, 2), s.cache.v.transpose(1, 2)),
        lambda: qp.KVCache(s.cache.k, s.cache.v, torch.ones(180, KV, PAGE, device=DEV)),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises((ValueError, TypeError, qp.QProjError)):
            call()
            pytest.fail(f"call {i} was not refused")
    assert same(s.result(), want)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_ties_in_rows_that_are_not_split(dtype):
    """More equal logits than a row's list of candidates holds, a workgroup a row."""
    rows, vocab, top = 3000, 4001, 32
    x = torch.zeros((rows, vocab), device=DEV).to(dtype)
    x[1::2, 1000:] = 1.0
    found = (torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty((rows, top), dtype=I32, device=DEV),
             torch.empty((rows, top), device=DEV))
    work = torch.empty(qp.token_logprobs_workspace(rows, vocab, top), dtype=U8, device=DEV)
    qp.token_logprobs(x, torch.zeros(rows, dtype=I32, device=DEV), *found, work)
    first = torch.where(torch.arange(rows, device=DEV) % 2 == 1, 1000, 0)
    assert torch.equal(found[2], (first[:, None] + torch.arange(top, device=DEV)).to(I32))


# ------------------------------------------------------------------ the largest calls
def test_the_most_rows_of_logits():
    rows, vocab = (1 << 24) - 1, 3
    x = torch.empty((rows, vocab), dtype=BF16, device=DEV).normal_(generator=gen(1))
    targets = torch.randint(0, 3, (rows,), generator=gen(2), device=DEV, dtype=I32)
    found = (torch.full((rows,), 9.0, device=DEV), torch.full((rows,), 9.0, device=DEV),
             torch.full((rows, 2), 9, dtype=I32, device=DEV), torch.full((rows, 2), 9.0, device=DEV))
    work = torch.empty(qp.token_logprobs_workspace(rows, vocab, 2), dtype=U8, device=DEV)
    qp.token_logprobs(x, targets, *found, work)
    for at in range(0, rows, 1 << 22):
        want, _, order, best, rel = ref.logprobs(x[at:at + (1 << 22)], targets[at:at + (1 << 22)], 2)
        got = [f[at:at + (1 << 22)] for f in found]
        assert torch.equal(got[2].long(), order)
        ref.assert_logprobs(got[0][:, None], want[:, None], rel)
        ref.assert_logprobs(got[3], best, rel)


def test_the_most_tokens_of_heads():
    """Nearly 2^31 elements of 17 heads of 16; a token's outputs depend on it alone."""
    heads, d = 15, 16
    t = ((1 << 31) - 1) // ((heads + 2) * d)
    qkv = torch.empty((t, (heads + 2) * d), dtype=BF16, device=DEV)
    for at in range(0, t, 1 << 20):
        qkv[at:at + (1 << 20)].normal_(generator=gen(at))
    some = torch.tensor([0, 1, 4097, t // 2, t - 2, t - 1], device=DEV)
    positions = torch.arange(t, dtype=I32, device=DEV)
    slots = torch.full((t,), -1, dtype=I32, device=DEV)
    slots[some] = torch.arange(1, 7, dtype=I32, device=DEV)
    inv_freq = qp.rope_inv_freq(d, 10000.0).to(DEV)
    out = []
    for rows in (slice(None), some):
        cache = Cache(1, 1, 16, d, False)
        q = torch.full((len(positions[rows]), heads, d), -3.0, dtype=BF16, device=DEV)
        qp.qk_norm_rope_cache(qkv[rows], None, None, 1e-6, positions[rows], inv_freq, 1.0, qp.QP_ROPE_HALF, slots[rows],
                              qp.KVCache(cache.k, cache.v), q)
        out.append([q[some] if isinstance(rows, slice) else q, cache.k, cache.v])
    assert same(*out)
    assert not torch.isnan(out[0][1][0, 0, 1:7].float()).any() and torch.isnan(out[0][1][0, 0, 7:].float()).all()


def test_the_most_sequences():
    """Nearly 2^31 elements of queries, a token each of a million sequences."""
    seqs, heads, kv, d = (1 << 20) - 1, 128, 8, 16
    g = gen(4)
    cache = Cache(40, kv, 16, d, False)
    slots = torch.arange(640, device=DEV)
    cache.put("k", slots, normal(g, 640, kv, d))
    cache.put("v", slots, normal(g, 640, kv, d))
    q = torch.empty((seqs, heads, d), dtype=BF16, device=DEV)
    for at in range(0, seqs, 1 << 17):
        q[at:at + (1 << 17)].normal_(generator=gen(at))
    table = torch.randint(0, 40, (seqs, 1), generator=g, device=DEV, dtype=I32)
    kv_len = torch.randint(0, 17, (seqs,), generator=g, device=DEV, dtype=I32)
    q_start = torch.arange(seqs + 1, dtype=I32, device=DEV)
    out = torch.full_like(q, -3.0)
    work = torch.empty(qp.paged_attention_workspace(seqs, seqs, 1, heads, kv, d), dtype=U8, device=DEV)
    qp.paged_attention(q, qp.KVCache(cache.k, cache.v), table, q_start, kv_len, 1, 0.25, 0, work, out)
    torch.cuda.synchronize()
    for at in range(0, seqs, 1 << 17):
        assert not (out[at:at + (1 << 17)] == -3.0).all(dim=(1, 2)).any()
    for s in (0, 1, 255, 256, 70001, seqs // 2, seqs - 257, seqs - 2, seqs - 1):
        n = int(kv_len[s])
        at = int(table[s]) * 16 + torch.arange(n, device=DEV)
        want, tol = ref.attention(q[s:s + 1], cache.get("k", at), cache.get("v", at), ref.visible(1, n, 0), 0.25)
        ref.assert_rounded(out[s:s + 1], want, tol)
