"""The layers of a decoder in FP8: attention, feed-forward (dense and
mixture-of-experts), and what is reported of the logits.

    python -m examples.layer_step [--rows 4] [--hidden 5120] [--inner 17408]
                                  [--experts 64] [--topk 6] [--expert-inner 1408]
                                  [--heads 32] [--kv-heads 8] [--head-size 128]
                                  [--cached 4000] [--vocab 152064] [--top 8]

Layers on one residual stream:

  attention  norm + residual -> E4M3 per row -> q/k/v product -> norms and
             rotation of the heads, keys and values to the paged cache
             -> attention over the cache -> E4M3 per row -> output product
             (6 calls; here a token each of `rows` sequences)
  dense      norm + residual -> E4M3 per 128 -> gate/up product -> activation
             -> E4M3 per 128 -> down product               (4 calls, any rows)
  mixture    norm + residual -> BF16 -> router -> experts  (2 calls of the
             library and the router's product, up to 16 rows)
  head       norm + residual -> BF16 -> logits -> log probabilities, entropy
             and the most probable tokens (2 calls and the logits' product)

Weights are random; each layer is checked against plain torch operations and
timed.  The layers' buffers are allocated once and reused, as a serving program
would; only the router's product, which is torch's, takes a temporary.
"""
from __future__ import annotations

import argparse

import torch

import gemv_nvfp4_int8_amd as qp

EPS = 1e-6
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def ceil128(v):
    return (v + 127) // 128


def quantize_blocks(w):
    """E4M3 codes and one F32 scale per 128 x 128 block of a weight [..., n, k]."""
    n, k = w.shape[-2:]
    nb, kb = ceil128(n), ceil128(k)
    full = torch.zeros((*w.shape[:-2], nb * 128, kb * 128), dtype=F32, device=w.device)
    full[..., :n, :k] = w.float()
    blocks = full.unflatten(-2, (nb, 128)).unflatten(-1, (kb, 128))
    scale = blocks.abs().amax(dim=(-3, -1)) / 448.0
    safe = torch.where(scale > 0, scale, 1.0)
    codes = (blocks / safe[..., :, None, :, None]).to(torch.float8_e4m3fn)
    codes = codes.view(U8).flatten(-2, -1).flatten(-3, -2)[..., :n, :k]
    return codes.contiguous(), scale.contiguous()


def decode_blocks(codes, scale):
    n, k = codes.shape[-2:]
    s = scale.repeat_interleave(128, dim=-2)[..., :n, :].repeat_interleave(128, dim=-1)[..., :k]
    return codes.view(torch.float8_e4m3fn).float() * s


def quantize_rows(y):
    """Plain form of QP_ACT_FP8_BLOCK128, decoded again: what the product sees."""
    rows, k = y.shape
    kb = ceil128(k)
    full = torch.zeros((rows, kb * 128), dtype=F32, device=y.device)
    full[:, :k] = y
    blocks = full.view(rows, kb, 128)
    scale = blocks.abs().amax(dim=2, keepdim=True) / 448.0
    codes = (blocks / torch.where(scale > 0, scale, 1.0)).to(torch.float8_e4m3fn)
    return (codes.float() * scale).view(rows, -1)[:, :k]


def plain_norm(x, residual, weight):
    h = (x.float() + residual.float()).to(BF16)
    f = h.float()
    return h, f * torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS) * weight.float()


def plain_silu_mul(gate_up):
    g, u = gate_up.float().chunk(2, dim=-1)
    return g / (1.0 + torch.exp(-g)) * u


def quantize_each_row(y):
    """Plain form of E4M3 with a scale per row: codes and scales."""
    scale = y.float().abs().amax(dim=1) / 448.0
    codes = (y.float() / torch.where(scale > 0, scale, 1.0)[:, None]).to(torch.float8_e4m3fn)
    return codes.view(U8), scale


def decode_rows(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale[:, None]


class Attention:
    """norm -> q/k/v -> heads' norms, rotation, cache -> attention -> output, for a
    new token each of `rows` sequences with `cached` positions behind them, in a
    BF16 cache of 16-position pages in no order."""

    PAGE, BASE = 16, 1e6

    def __init__(self, rows, hidden, heads, kv, d, cached, device, seed=3):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=device)  # noqa: E731
        self.heads, self.kv, self.d, self.cached = heads, kv, d, cached
        self.norm, self.q_norm, self.k_norm = ((1.0 + 0.1 * rnd(n)).to(BF16) for n in (hidden, d, d))
        self.wqkv, self.sqkv = quantize_each_row(rnd((heads + 2 * kv) * d, hidden) * hidden ** -0.5)
        self.wo, self.so = quantize_each_row(rnd(hidden, heads * d) * (heads * d) ** -0.5)
        self.inv_freq = qp.rope_inv_freq(d, self.BASE).to(device)
        width = cached // self.PAGE + 1
        self.table = torch.randperm(rows * width, generator=g, device=device).to(I32).view(rows, width)
        self.k, self.v = (rnd(rows * width, kv, self.PAGE, d).to(BF16) for _ in range(2))
        self.cache = qp.KVCache(self.k, self.v)
        self.positions = torch.full((rows,), cached, dtype=I32, device=device)
        self.slots = self.table[:, cached // self.PAGE] * self.PAGE + cached % self.PAGE
        self.q_start = torch.arange(rows + 1, dtype=I32, device=device)
        self.kv_len = self.positions + 1
        self.x8, self.xs = new(rows, hidden, dtype=U8), new(rows, dtype=F32)
        self.qkv, self.q, self.o = new(rows, (heads + 2 * kv) * d), new(rows, heads, d), new(rows, heads, d)
        self.o8, self.os = new(rows, heads * d, dtype=U8), new(rows, dtype=F32)
        self.work = new(qp.paged_attention_workspace(rows, rows, 1, heads, kv, d), dtype=U8)

    def __call__(self, x, residual, out):
        qp.rmsnorm_residual_quant(x, residual, self.norm, EPS, qp.QP_ACT_FP8_ROW, self.x8, self.xs, residual)
        qp.fp8_gemm_rowscale(self.x8, self.xs, self.wqkv, self.sqkv, self.qkv)
        qp.qk_norm_rope_cache(self.qkv, self.q_norm, self.k_norm, EPS, self.positions, self.inv_freq, 1.0,
                              qp.QP_ROPE_HALF, self.slots, self.cache, self.q)
        qp.paged_attention(self.q, self.cache, self.table, self.q_start, self.kv_len, 1, self.d ** -0.5, 0,
                           self.work, self.o)
        qp.quant_rowwise_fp8(self.o.view(len(x), -1), self.o8, self.os)
        qp.fp8_gemm_rowscale(self.o8, self.os, self.wo, self.so, out)
        return out

    def plain(self, x, residual):
        rows, heads, kv, d = len(x), self.heads, self.kv, self.d
        h, y = plain_norm(x, residual, self.norm)
        y8 = decode_rows(*quantize_each_row(y))
        qkv = (y8 @ decode_rows(self.wqkv, self.sqkv).t()).to(BF16).float().view(rows, heads + 2 * kv, d)
        angle = self.positions.double()[:, None, None] * self.inv_freq.double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

        def turned(t, weight):
            t = t * torch.rsqrt((t * t).mean(dim=2, keepdim=True) + EPS) * weight.float()
            a, b = t.chunk(2, dim=2)
            return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2).to(BF16).float()

        q, k = turned(qkv[:, :heads], self.q_norm), turned(qkv[:, heads:heads + kv], self.k_norm)
        v = qkv[:, heads + kv:]
        o = torch.empty((rows, heads, d), device=x.device)
        for i in range(rows):
            # [kv, positions, d] of the sequence's pages, and the new token's at the end
            ks, vs = (torch.cat([c[self.table[i].long()].transpose(0, 1).reshape(kv, -1, d)[:, :self.cached].float(),
                                 new[i][:, None]], dim=1) for c, new in ((self.k, k), (self.v, v)))
            p = torch.softmax((q[i].view(kv, -1, 1, d) * ks[:, None]).sum(dim=3) * d ** -0.5, dim=2)
            o[i] = (p[..., None] * vs[:, None]).sum(dim=2).view(heads, d)
        o8 = decode_rows(*quantize_each_row(o.view(rows, -1).to(BF16)))
        return h, o8 @ decode_rows(self.wo, self.so).t()


class Head:
    """norm -> logits -> log probabilities of the targets, entropy, `top` tokens."""

    def __init__(self, rows, hidden, vocab, top, device, seed=4):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        new = lambda *s, dtype=F32: torch.empty(s, dtype=dtype, device=device)  # noqa: E731
        self.norm = (1.0 + 0.1 * rnd(hidden)).to(BF16)
        self.w = (rnd(vocab, hidden) * hidden ** -0.5).to(BF16)
        self.targets = torch.randint(0, vocab, (rows,), generator=g, device=device, dtype=I32)
        self.y, self.logits = new(rows, hidden, dtype=BF16), new(rows, vocab, dtype=BF16)
        self.logprob, self.entropy = new(rows), new(rows)
        self.ids, self.top_logprobs = new(rows, top, dtype=I32), new(rows, top)
        self.work = new(qp.token_logprobs_workspace(rows, vocab, top), dtype=U8)

    def __call__(self, x, residual, out=None):
        qp.rmsnorm_residual_quant(x, residual, self.norm, EPS, qp.QP_ACT_BF16, self.y, None, residual)
        torch.matmul(self.y, self.w.t(), out=self.logits)
        qp.token_logprobs(self.logits, self.targets, self.logprob, self.entropy, self.ids, self.top_logprobs, self.work)
        return self.logprob

    def plain(self, x, residual):
        """Of the logits of the last call: (h, log probabilities of the targets)."""
        p = torch.log_softmax(self.logits.float(), dim=1)
        assert torch.equal(p.gather(1, self.ids.long()), p.topk(self.ids.shape[1], dim=1).values)
        return plain_norm(x, residual, self.norm)[0], p.gather(1, self.targets.long()[:, None])[:, 0]


class Dense:
    """norm -> gate/up -> activation -> down, with its buffers for up to `rows` rows."""

    def __init__(self, rows, hidden, inner, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.norm = (1.0 + 0.1 * rnd(hidden)).to(BF16)
        self.w13, self.s13 = quantize_blocks(rnd(2 * inner, hidden) * hidden ** -0.5)
        self.w2, self.s2 = quantize_blocks(rnd(hidden, inner) * inner ** -0.5)
        new = lambda *s, dtype: torch.empty(s, dtype=dtype, device=device)  # noqa: E731
        self.q, self.qs = new(rows, hidden, dtype=U8), new(rows, ceil128(hidden), dtype=F32)
        self.gate_up = new(rows, 2 * inner, dtype=BF16)
        self.a, self.as_ = new(rows, inner, dtype=U8), new(rows, ceil128(inner), dtype=F32)

    def __call__(self, x, residual, out):
        """residual += x (in place); out = the layer's output, to be added next."""
        r = x.shape[0]
        q, qs, gu, a, as_ = self.q[:r], self.qs[:r], self.gate_up[:r], self.a[:r], self.as_[:r]
        qp.rmsnorm_residual_quant(x, residual, self.norm, EPS, qp.QP_ACT_FP8_BLOCK128, q, qs, residual)
        qp.fp8_gemm_blockscale(q, qs, self.w13, self.s13, gu)
        qp.silu_mul_quant(gu, qp.QP_ACT_FP8_BLOCK128, a, as_)
        qp.fp8_gemm_blockscale(a, as_, self.w2, self.s2, out)
        return out

    def plain(self, x, residual):
        h, y = plain_norm(x, residual, self.norm)
        gu = (quantize_rows(y) @ decode_blocks(self.w13, self.s13).t()).to(BF16)
        return h, quantize_rows(plain_silu_mul(gu)) @ decode_blocks(self.w2, self.s2).t()


class Mixture:
    """norm -> router -> the topk experts of each row, with its buffers."""

    def __init__(self, rows, hidden, inner, experts, topk, device, seed=1):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.topk = topk
        self.norm = (1.0 + 0.1 * rnd(hidden)).to(BF16)
        self.router = rnd(experts, hidden) * hidden ** -0.5
        each = [(quantize_blocks(rnd(2 * inner, hidden) * hidden ** -0.5),
                 quantize_blocks(rnd(hidden, inner) * inner ** -0.5)) for _ in range(experts)]
        self.w13, self.s13 = (torch.stack([e[0][i] for e in each]) for i in (0, 1))
        self.w2, self.s2 = (torch.stack([e[1][i] for e in each]) for i in (0, 1))
        self.y = torch.empty((rows, hidden), dtype=BF16, device=device)
        self.logits = torch.empty((rows, experts), dtype=F32, device=device)
        self.work = torch.empty(qp.moe_fp8_blockscale_workspace(rows, topk, inner), dtype=U8, device=device)

    def __call__(self, x, residual, out):
        r = x.shape[0]
        y, logits = self.y[:r], self.logits[:r]
        qp.rmsnorm_residual_quant(x, residual, self.norm, EPS, qp.QP_ACT_BF16, y, None, residual)
        torch.matmul(y.float(), self.router.t(), out=logits)
        qp.moe_fp8_blockscale(y, logits, self.w13, self.s13, self.w2, self.s2, self.topk, True, self.work, out)
        return out

    def plain(self, x, residual):
        """Routed by the logits of the last call (the choice of experts is not
        continuous), so call it after the layer itself."""
        h, y = plain_norm(x, residual, self.norm)
        y = y.to(BF16).float()
        p, chosen = torch.softmax(self.logits[:x.shape[0]], dim=1).topk(self.topk, dim=1)
        p = p / p.sum(dim=1, keepdim=True)
        out = torch.zeros_like(y)
        for row in range(y.shape[0]):
            for weight, e in zip(p[row], chosen[row].tolist()):
                inner = plain_silu_mul(y[row] @ decode_blocks(self.w13[e], self.s13[e]).t())
                out[row] += weight * (inner @ decode_blocks(self.w2[e], self.s2[e]).t())
        return h, out


def relative(got, want):
    return ((got.float() - want).norm() / want.norm()).item()


def check(layer, rows, hidden, device, seed=2):
    """2-norm error of one step of `layer` against its plain form; the residual
    stream has to be the same bits."""
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn((rows, hidden), generator=g, device=device).to(BF16)
    residual = (2.0 * torch.randn((rows, hidden), generator=g, device=device)).to(BF16)
    kept, out = residual.clone(), torch.empty_like(x)
    out = layer(x, residual, out)
    h, want = layer.plain(x, kept)
    assert torch.equal(h.view(torch.int16), residual.view(torch.int16))
    return relative(out, want)


def timed(layer, rows, hidden, device, steps=50):
    x = torch.randn((rows, hidden), device=device).to(BF16)
    residual, out = torch.zeros_like(x), torch.empty_like(x)
    for _ in range(5):
        layer(x, residual, out)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        layer(x, residual, out)
    end.record()
    end.synchronize()
    return begin.elapsed_time(end) / steps * 1e3


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--rows", type=int, default=4)
    p.add_argument("--hidden", type=int, default=5120)
    p.add_argument("--inner", type=int, default=17408)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--topk", type=int, default=6)
    p.add_argument("--expert-inner", type=int, default=1408)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--head-size", type=int, default=128)
    p.add_argument("--cached", type=int, default=4000)
    p.add_argument("--vocab", type=int, default=152064)
    p.add_argument("--top", type=int, default=8)
    a = p.parse_args()
    dev = torch.device("cuda:0")
    layers = [("dense", Dense(a.rows, a.hidden, a.inner, dev))]
    if a.rows <= 16:
        layers.append(("mixture", Mixture(a.rows, a.hidden, a.expert_inner, a.experts, a.topk, dev)))
    if a.rows <= 256:
        layers.append(("attention", Attention(a.rows, a.hidden, a.heads, a.kv_heads, a.head_size, a.cached, dev)))
    layers.append(("head", Head(a.rows, a.hidden, a.vocab, a.top, dev)))
    for name, layer in layers:
        err = check(layer, a.rows, a.hidden, dev)
        print(f"{name}: {a.rows} rows, error {err:.1e} of the plain form's 2-norm, "
              f"{timed(layer, a.rows, a.hidden, dev):.1f} us a step", flush=True)


if __name__ == "__main__":
    main()
