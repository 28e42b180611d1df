"""The operators around the block-scaled FP8 projections, as cases that can be timed.

rms_norm   residual addition, RMS norm and an 8-bit output with scales
silu_mul   the gated activation of a feed-forward layer, with an 8-bit output
gemm       FP8 x FP8 product, one scale per 128 activations of a row and per 128 x 128 weights
moe        a whole mixture-of-experts layer for a few tokens (routing, gate/up, activation, down)

8-bit formats: "fp8_block" (E4M3, one F32 scale per 128 of a row, the last block shorter where 128
does not divide the row), "fp8_row" (E4M3, one scale per row), "int8_block" (int8, one scale per 32).
Scale = amax / 448 (127 for int8), code = the value over the scale, rounded to nearest even; a block
of zeros has scale 0 and codes 0.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the norm in front of one decoded token's projections: latency
        {"name": "norm-1x5120", "op": "rms_norm", "rows": 1, "k": 5120, "fmt": "fp8_block", "residual": True},
        # a ragged prefill chunk in front of the int8 product
        {"name": "norm-2047x5120-int8", "op": "rms_norm", "rows": 2047, "k": 5120, "fmt": "int8_block", "residual": True},
        # a whole prefill in front of the row-wise FP8 product
        {"name": "norm-8192x5120-row", "op": "rms_norm", "rows": 8192, "k": 5120, "fmt": "fp8_row", "residual": True},
        # the activation of a verify batch of draft tokens
        {"name": "silu-16x17408", "op": "silu_mul", "rows": 16, "i": 17408, "fmt": "fp8_block"},
        # the activation of a prefill
        {"name": "silu-4096x17408", "op": "silu_mul", "rows": 4096, "i": 17408, "fmt": "fp8_block"},
        # decode of four requests: the weight's bytes count
        {"name": "gemm-4x17408x5120", "op": "gemm", "m": 4, "n": 17408, "k": 5120},
        # a verify batch through a down projection: few rows, long sums
        {"name": "gemm-37x5120x17408", "op": "gemm", "m": 37, "n": 5120, "k": 17408},
        # a ragged prefill chunk of a sharded layer whose last block of 128 is a half
        {"name": "gemm-600x4104x2368", "op": "gemm", "m": 600, "n": 4104, "k": 2368},
        # a whole prefill
        {"name": "gemm-8192x12288x5120", "op": "gemm", "m": 8192, "n": 12288, "k": 5120},
        # one decoded token, many small experts
        {"name": "moe-1-128x8-2048x768", "op": "moe", "t": 1, "e": 128, "topk": 8, "h": 2048, "i": 768, "renorm": True},
        # five requests, few large experts, some of them shut off by the router's mask
        {"name": "moe-5-8x2-4096x8192", "op": "moe", "t": 5, "e": 8, "topk": 2, "h": 4096, "i": 8192, "renorm": True},
        # the largest decode batch
        {"name": "moe-16-64x6-5120x1408", "op": "moe", "t": 16, "e": 64, "topk": 6, "h": 5120, "i": 1408, "renorm": False},
    ]


def _spread(rng, lo, hi, step):
    """A multiple of `step` in lo..hi, even over the logarithm (and not one that doubles to, or is, 24 blocks)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, lo, step), hi)
    return v + step if v in (12 * 128, 24 * 128) else v


def draw(rng):
    op = rng.choice(["rms_norm", "silu_mul", "gemm", "gemm", "moe", "moe"])
    if op == "rms_norm":
        fmt = rng.choice(["fp8_block", "fp8_row", "int8_block"])
        k = _spread(rng, 256, 16384, 32 if fmt == "int8_block" else 16)
        rows = _spread(rng, 1, min(8192, 8192 * 5120 // k), 1)
        return {"op": op, "rows": rows, "k": k, "fmt": fmt, "residual": rng.random() < 0.8}
    if op == "silu_mul":
        fmt = rng.choice(["fp8_block", "fp8_row", "int8_block"])
        i = _spread(rng, 256, 17408, 32 if fmt == "int8_block" else 16)
        rows = _spread(rng, 1, min(8192, 4096 * 17408 // i), 1)
        return {"op": op, "rows": rows, "i": i, "fmt": fmt}
    if op == "gemm":
        n = _spread(rng, 128, 17408, rng.choice([1, 8, 128]))
        k = _spread(rng, 128, 17408, rng.choice([16, 128, 128]))
        m = _spread(rng, 1, min(8192, 8192 * 12288 * 5120 // (n * k)), 1)
        return {"op": op, "m": m, "n": n, "k": k}
    h = _spread(rng, 512, 7168, 128)
    i = _spread(rng, 256, 4096, 128)
    e = _spread(rng, 8, max(8, min(256, 64 * 5120 * 1408 // (h * i))), 1)
    topk = rng.randint(1, min(8, e))
    t = rng.randint(1, 16)
    while t > 1 and t * topk * h * i > 96 * 5120 * 1408:
        t -= 1
    while topk > 1 and t * topk * h * i > 96 * 5120 * 1408:
        topk -= 1
    return {"op": op, "t": t, "e": e, "topk": topk, "h": h, "i": i, "renorm": rng.random() < 0.5}


def _blocks(k, b):
    return (k + b - 1) // b


def _scales_per_row(fmt, k):
    return {"fp8_block": _blocks(k, 128), "fp8_row": 1, "int8_block": k // 32}[fmt]


def work(case):
    c = case
    if c["op"] == "rms_norm":
        n = c["rows"] * c["k"]
        b = n * (7 if c["residual"] else 3) + 2 * c["k"] + 4 * c["rows"] * _scales_per_row(c["fmt"], c["k"])
        return {"bytes": b, "flops": 8 * n}
    if c["op"] == "silu_mul":
        n = c["rows"] * c["i"]
        return {"bytes": 5 * n + 4 * c["rows"] * _scales_per_row(c["fmt"], c["i"]), "flops": 8 * n}
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        kb = _blocks(k, 128)
        return {"bytes": m * k + n * k + 2 * m * n + 4 * kb * (m + _blocks(n, 128)), "flops": 2 * m * n * k}
    t, e, topk, h, i = c["t"], c["e"], c["topk"], c["h"], c["i"]
    hit = e * (1.0 - (1.0 - topk / e) ** t)          # distinct experts that t tokens choose on average
    per = 3 * h * i * (1.0 + 4.0 / (128 * 128))
    return {"bytes": hit * per + 4 * t * h + 4 * t * e, "flops": 6 * t * topk * h * i}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _acts(g, shape):
    """Activations: normal, one entry in a hundred twenty times as large."""
    x = _normal(g, shape)
    far = torch.rand(shape, generator=g, device=DEV) < 0.01
    return torch.where(far, 20.0 * x, x)


def _weight_codes(g, out):
    """E4M3 codes as a per-block quantizer leaves them for normal weights (amax at about 4 sigma)."""
    flat = out.view(-1)
    step = 1 << 26
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        part.copy_((112.0 * _normal(g, part.shape)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn))
    return out


def _weight_grid(g, shape):
    return 1.8e-4 * (0.5 + torch.rand(shape, generator=g, device=DEV))


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _code_type(fmt):
    return torch.int8 if fmt == "int8_block" else torch.float8_e4m3fn


def prepare(case, seed):
    g, c = _gen(seed), case
    s = dict(case)
    if c["op"] == "rms_norm":
        rows, k = c["rows"], c["k"]
        s["x"] = _acts(g, (rows, k)).to(torch.bfloat16)
        s["res"] = (4.0 * _normal(g, (rows, k))).to(torch.bfloat16) if c["residual"] else None
        s["w"] = (1.0 + 0.2 * _normal(g, (k,))).to(torch.bfloat16)
        s["res_out"] = _empty((rows, k), torch.bfloat16) if c["residual"] else None
        s["q"] = _empty((rows, k), _code_type(c["fmt"]))
        s["scale"] = _empty((rows, _scales_per_row(c["fmt"], k)), torch.float32)
    elif c["op"] == "silu_mul":
        rows, i = c["rows"], c["i"]
        s["gate_up"] = _acts(g, (rows, 2 * i)).to(torch.bfloat16)
        s["q"] = _empty((rows, i), _code_type(c["fmt"]))
        s["scale"] = _empty((rows, _scales_per_row(c["fmt"], i)), torch.float32)
    elif c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        s["a"], s["a_scale"] = _quantize(_acts(g, (m, k)), "fp8_block")
        s["w"] = _weight_codes(g, _empty((n, k), torch.float8_e4m3fn))
        s["w_scale"] = _weight_grid(g, (_blocks(n, 128), _blocks(k, 128)))
        s["out"] = _empty((m, n), torch.bfloat16)
    else:
        t, e, h, i = c["t"], c["e"], c["h"], c["i"]
        s["x"] = _acts(g, (t, h)).to(torch.bfloat16)
        s["logits"] = 1.5 * _normal(g, (t, e))
        # the router's mask: now and then an expert is shut off
        s["logits"][torch.rand((t, e), generator=g, device=DEV) < 0.03] = -math.inf
        s["w13"] = _weight_codes(g, _empty((e, 2 * i, h), torch.float8_e4m3fn))
        s["s13"] = _weight_grid(g, (e, 2 * i // 128, h // 128))
        s["w2"] = _weight_codes(g, _empty((e, h, i), torch.float8_e4m3fn))
        s["s2"] = _weight_grid(g, (e, h // 128, i // 128))
        s["out"] = _empty((t, h), torch.bfloat16)
        # the layer's activations in F32 and 64 KiB for the routing
        s["work"] = _empty((4 * t * c["topk"] * i + 65536,), torch.uint8)
    return s


# -------------------------------------------------------------------------------- plain forms
def _block_of(fmt, k):
    return {"fp8_block": 128, "fp8_row": k, "int8_block": 32}[fmt]


def _quantize(y, fmt):
    rows, k = y.shape
    b = _block_of(fmt, k)
    nb = _blocks(k, b)
    top = 127.0 if fmt == "int8_block" else 448.0
    z = torch.zeros((rows, nb * b), dtype=y.dtype, device=y.device)
    z[:, :k] = y
    z = z.view(rows, nb, b)
    scale = z.abs().amax(dim=2) / top
    over = torch.where(scale > 0, scale, torch.ones_like(scale))
    v = (z / over[:, :, None]).reshape(rows, nb * b)[:, :k].clamp(-top, top)
    q = v.round().to(torch.int8) if fmt == "int8_block" else v.to(torch.float8_e4m3fn)
    return q.contiguous(), scale


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = (h + s["res"].float()).to(torch.bfloat16)
    res_out = h if s["res"] is not None else None
    h = h.float()
    rstd = torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS)
    q, scale = _quantize(h * rstd * s["w"].float(), s["fmt"])
    return res_out, q, scale


def _plain_silu(s):
    i = s["i"]
    g, u = s["gate_up"][:, :i].float(), s["gate_up"][:, i:].float()
    return _quantize(g / (1.0 + torch.exp(-g)) * u, s["fmt"])


def _spread_rows(scale, k):
    """[m, blocks] -> [m, k]: each scale over its 128 elements."""
    return scale.repeat_interleave(128, dim=-1)[..., :k]


def _plain_gemm(s):
    n, k = s["n"], s["k"]
    a = s["a"].float() * _spread_rows(s["a_scale"], k)
    w = s["w"].float() * _spread_rows(s["w_scale"].repeat_interleave(128, dim=0)[:n], k)
    return (a @ w.t()).to(torch.bfloat16)


def _route(logits, topk, renorm):
    """The topk largest logits of a row (ties to the lowest expert) and their weights; a row with nothing to choose gives none."""
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :topk]
    top = logits.amax(dim=1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    chosen = p.gather(1, ids)
    total = (chosen if renorm else p).sum(dim=1, keepdim=True)
    return ids, chosen / torch.where(total > 0, total, torch.ones_like(total))


def _grid_over(w, grid, dtype):
    """[b, r, c] weights times their [b, r/128, c/128] scales."""
    b, r, c = w.shape
    v = w.to(dtype).view(b, r // 128, 128, c // 128, 128) * grid.to(dtype)[:, :, None, :, None]
    return v.view(b, r, c)


def _experts(s, ids, p, dtype):
    t, topk, i, h = s["t"], s["topk"], s["i"], s["h"]
    flat = ids.reshape(-1)
    x = s["x"].to(dtype).repeat_interleave(topk, dim=0).unsqueeze(2)
    u8 = torch.uint8
    pick = lambda w: w.view(u8)[flat].view(torch.float8_e4m3fn)  # noqa: E731
    gu = torch.matmul(_grid_over(pick(s["w13"]), s["s13"][flat], dtype), x).squeeze(2)
    gate, up = gu[:, :i], gu[:, i:]
    act = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.matmul(_grid_over(pick(s["w2"]), s["s2"][flat], dtype), act.unsqueeze(2)).view(t, topk, h)
    return (y * p.to(dtype)[:, :, None]).sum(dim=1)


# ---------------------------------------------------------------------------------------- run
def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "rms_norm":
        res_out, q, scale = _plain_norm(s)
        return {"codes": _codes(q), "scale": scale, **({"residual": res_out} if res_out is not None else {})}
    if s["op"] == "silu_mul":
        q, scale = _plain_silu(s)
        return {"codes": _codes(q), "scale": scale}
    if s["op"] == "gemm":
        return _plain_gemm(s)
    ids, p = _route(s["logits"], s["topk"], s["renorm"])
    return _experts(s, ids, p, torch.float32).to(torch.bfloat16)


def _codes(q):
    """Codes as the values they stand for (int8 ones are whole in BF16)."""
    return q.to(torch.bfloat16) if q.dtype == torch.int8 else q


def _run_own(s):
    import gemv_nvfp4_int8_amd as qp
    fmt = {"fp8_row": qp.QP_ACT_FP8_ROW, "fp8_block": qp.QP_ACT_FP8_BLOCK128, "int8_block": qp.QP_ACT_INT8_BLOCK32}
    if s["op"] == "rms_norm":
        qp.rmsnorm_residual_quant(s["x"], s["res"], s["w"], EPS, fmt[s["fmt"]], s["q"], s["scale"], s["res_out"])
        return {"codes": _codes(s["q"]), "scale": s["scale"],
                **({"residual": s["res_out"]} if s["res_out"] is not None else {})}
    if s["op"] == "silu_mul":
        qp.silu_mul_quant(s["gate_up"], fmt[s["fmt"]], s["q"], s["scale"])
        return {"codes": _codes(s["q"]), "scale": s["scale"]}
    if s["op"] == "gemm":
        qp.fp8_gemm_blockscale(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"])
        return s["out"]
    qp.moe_fp8_blockscale(s["x"], s["logits"], s["w13"], s["s13"], s["w2"], s["s2"], s["topk"], s["renorm"],
                          s["work"], s["out"])
    return s["out"]


# -------------------------------------------------------------------------------------- exact
def _exact_quant(y, fmt):
    """Scales and codes in 64 bits. The codes are given before their rounding to eight bits, so that a value beside
    a tie counts as half a step off and not as a whole one."""
    rows, k = y.shape
    b = _block_of(fmt, k)
    top = 127.0 if fmt == "int8_block" else 448.0
    col = torch.arange(k, device=y.device) // b
    scale = torch.zeros((rows, _blocks(k, b)), dtype=torch.float64, device=y.device)
    scale.scatter_reduce_(1, col.expand(rows, k), y.abs(), "amax")
    scale /= top
    each = scale[:, col]
    return torch.where(each > 0, y / torch.where(each > 0, each, 1.0), 0.0), scale


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "rms_norm":
        h = s["x"].to(f64)
        out = {}
        if s["res"] is not None:
            out["residual"] = h + s["res"].to(f64)
            # the norm is that of the residual as it is kept: the two BF16 values' sum, rounded once to BF16
            h = out["residual"].float().to(torch.bfloat16).to(f64)
        y = h / torch.sqrt((h * h).sum(dim=1, keepdim=True) / s["k"] + EPS) * s["w"].to(f64)
        out["codes"], out["scale"] = _exact_quant(y, s["fmt"])
        return out
    if s["op"] == "silu_mul":
        g, u = s["gate_up"].to(f64).split(s["i"], dim=1)
        codes, scale = _exact_quant(g * torch.sigmoid(g) * u, s["fmt"])
        return {"codes": codes, "scale": scale}
    if s["op"] == "gemm":
        m, n, k = s["m"], s["n"], s["k"]
        c = torch.zeros((m, n), dtype=f64, device=DEV)
        col = torch.arange(n, device=DEV) // 128
        for b in range(_blocks(k, 128)):
            at = slice(128 * b, min(k, 128 * b + 128))
            part = s["a"][:, at].to(f64) @ s["w"][:, at].to(f64).t()
            c += part * s["a_scale"][:, b, None].to(f64) * s["w_scale"][col, b][None, :].to(f64)
        return c
    i, h = s["i"], s["h"]
    out = torch.zeros((s["t"], h), dtype=f64, device=DEV)
    rows = s["logits"].to(f64).cpu().tolist()
    for t, row in enumerate(rows):
        # a masked expert weighs nothing; ties go to the lowest expert
        open_ = sorted((j for j in range(s["e"]) if row[j] > -math.inf), key=lambda j: (-row[j], j))
        chosen = open_[:s["topk"]]
        if not chosen:
            continue
        total = sum(math.exp(row[j] - row[chosen[0]]) for j in (chosen if s["renorm"] else open_))
        x = s["x"][t].to(f64)
        for j in chosen:
            w13 = s["w13"][j].to(f64) * s["s13"][j].to(f64).repeat_interleave(128, 0).repeat_interleave(128, 1)
            w2 = s["w2"][j].to(f64) * s["s2"][j].to(f64).repeat_interleave(128, 0).repeat_interleave(128, 1)
            gate, up = w13[:i] @ x, w13[i:] @ x
            out[t] += math.exp(row[j] - row[chosen[0]]) / total * (w2 @ (gate * torch.sigmoid(gate) * up))
    return out
