"""The feed-forward half of a decoder, dense and mixture-of-experts, in FP8.

    python -m examples.layer_step [--rows 4] [--hidden 5120] [--inner 17408]
                                  [--experts 64] [--topk 6] [--expert-inner 1408]

Two layers on one residual stream:

  dense    norm + residual -> E4M3 per 128 -> gate/up product -> activation
           -> E4M3 per 128 -> down product               (4 calls, any rows)
  mixture  norm + residual -> BF16 -> router -> experts  (2 calls of the
           library and the router's product, up to 16 rows)

Weights are random; each layer is checked against plain torch operations and
timed.  The layers' buffers are allocated once and reused, as a serving program
would; only the router's product, which is torch's, takes a temporary.
"""
from __future__ import annotations

import argparse

import torch

import gemv_nvfp4_int8_amd as qp

EPS = 1e-6
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


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
    layer(x, residual, out)
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
    a = p.parse_args()
    dev = torch.device("cuda:0")
    layers = [("dense", Dense(a.rows, a.hidden, a.inner, dev))]
    if a.rows <= 16:
        layers.append(("mixture", Mixture(a.rows, a.hidden, a.expert_inner, a.experts, a.topk, dev)))
    for name, layer in layers:
        err = check(layer, a.rows, a.hidden, dev)
        print(f"{name}: {a.rows} rows, error {err:.1e} of the plain form's 2-norm, "
              f"{timed(layer, a.rows, a.hidden, dev):.1f} us a step", flush=True)


if __name__ == "__main__":
    main()
