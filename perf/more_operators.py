"""The operators that complete a decoder's step, as cases that can be timed.

qk_rope     norms of queries and keys for each head, rotary positions, and the new keys and values
            put into a paged cache, in one pass over the output of the q/k/v product
attention   attention of the new tokens of several sequences over that cache
logprobs    log probabilities of given tokens, entropy and the most probable alternatives

The cache: K and V as [pages, kv_heads, page_size, d], BF16, or E4M3 with one F32 scale for each
position and head (amax / 448, values over the scale rounded to nearest even, a row of zeros has
scale 0 and codes 0).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BASE = 1e6           # of the rotary frequencies


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token behind the q/k/v product (32 + 2 x 8 heads of 128 are 6144 columns): latency
        {"name": "rope-1-32+8x128", "op": "qk_rope", "t": 1, "heads": 32, "kv": 8, "d": 128, "rot": 128,
         "layout": "half", "norm": True, "fmt": "bf16", "page": 16, "far": 40000},
        # a ragged prefill chunk of a model that turns half of each head, no norms, the cache in eight bits
        {"name": "rope-2047-40+4x128-fp8", "op": "qk_rope", "t": 2047, "heads": 40, "kv": 4, "d": 128, "rot": 64,
         "layout": "interleaved", "norm": False, "fmt": "fp8", "page": 64, "far": 131072},
        # a whole prefill
        {"name": "rope-8192-32+8x128", "op": "qk_rope", "t": 8192, "heads": 32, "kv": 8, "d": 128, "rot": 128,
         "layout": "half", "norm": True, "fmt": "bf16", "page": 16, "far": 8192},
        # one request's next token over a short context: latency
        {"name": "attn-1x1-over-700", "op": "attention", "seqs": 1, "new": 1, "kvlen": 700, "ragged": 0.0, "heads": 32,
         "kv": 8, "d": 128, "fmt": "bf16", "page": 16, "window": 0},
        # decode of many requests of different lengths: the cache's bytes count
        {"name": "attn-48x1-over-12000", "op": "attention", "seqs": 48, "new": 1, "kvlen": 12000, "ragged": 0.9,
         "heads": 32, "kv": 8, "d": 128, "fmt": "bf16", "page": 16, "window": 0},
        # a verify batch of five draft tokens each, cache in eight bits, odd group of ten heads
        {"name": "attn-16x5-over-9001-fp8", "op": "attention", "seqs": 16, "new": 5, "kvlen": 9001, "ragged": 0.5,
         "heads": 40, "kv": 4, "d": 128, "fmt": "fp8", "page": 64, "window": 0},
        # a chunk of one long prompt behind what is cached of it
        {"name": "attn-1x2000-over-32000", "op": "attention", "seqs": 1, "new": 2000, "kvlen": 32000, "ragged": 0.0,
         "heads": 32, "kv": 8, "d": 128, "fmt": "bf16", "page": 16, "window": 0},
        # prompts of different lengths, of a model with a window and small heads
        {"name": "attn-7x2500-window-1024", "op": "attention", "seqs": 7, "new": 2500, "kvlen": 2500, "ragged": 0.8,
         "heads": 64, "kv": 8, "d": 64, "fmt": "bf16", "page": 32, "window": 1024},
        # a whole prefill
        {"name": "attn-1x8192-prefill", "op": "attention", "seqs": 1, "new": 8192, "kvlen": 8192, "ragged": 0.0,
         "heads": 32, "kv": 8, "d": 128, "fmt": "bf16", "page": 16, "window": 0},
        # one sampled token of a request that asks for alternatives: latency
        {"name": "logp-1x152064", "op": "logprobs", "rows": 1, "vocab": 152064, "top": 20, "type": "bf16", "masked": 0.0},
        # a verify batch under a grammar that forbids most tokens; a vocabulary of odd size
        {"name": "logp-16x129281-f32", "op": "logprobs", "rows": 16, "vocab": 129281, "top": 5, "type": "f32",
         "masked": 0.9},
        # scoring of a prompt
        {"name": "logp-2048x152064", "op": "logprobs", "rows": 2048, "vocab": 152064, "top": 8, "type": "bf16",
         "masked": 0.0},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in lo..hi, even over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo, step), hi)


def draw(rng):
    op = rng.choice(["qk_rope", "attention", "attention", "attention", "logprobs"])
    if op == "logprobs":
        vocab = _spread(rng, 500, 262144)
        rows = _spread(rng, 1, max(1, min(8192, 2048 * 152064 // (2 * vocab))))
        return {"op": op, "rows": rows, "vocab": vocab, "top": rng.randint(0, 32), "type": rng.choice(["bf16", "f32"]),
                "masked": rng.choice([0.0, 0.0, 0.5, 0.99])}
    d = rng.choice([32, 64, 80, 96, 128, 128, 128, 192, 256])
    kv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    heads = kv * rng.choice([1, 2, 4, 5, 7, 8, 8, 10, 16])
    fmt = rng.choice(["bf16", "bf16", "fp8"])
    page = rng.choice([16, 16, 32, 64, 128, 256])
    if op == "qk_rope":
        t = _spread(rng, 1, min(8192, 8192 * 48 * 128 // ((heads + 2 * kv) * d)))
        rot = rng.choice([d, d, d // 2 // 16 * 16])
        return {"op": op, "t": t, "heads": heads, "kv": kv, "d": d, "rot": rot,
                "layout": rng.choice(["half", "interleaved"]), "norm": rng.random() < 0.6, "fmt": fmt, "page": page,
                "far": _spread(rng, 8192, 1 << 20)}
    window = _spread(rng, 100, 5000) if rng.random() < 0.3 else 0
    c = {"op": op, "seqs": 1, "new": 1, "kvlen": 1, "ragged": rng.choice([0.0, 0.5, 0.9]), "heads": heads, "kv": kv,
         "d": d, "fmt": fmt, "page": page, "window": window}
    kind = rng.choice(["decode", "verify", "chunk", "prompt"])
    if kind == "decode" or kind == "verify":
        c["new"] = 1 if kind == "decode" else rng.randint(2, 16)
        c["seqs"] = _spread(rng, 1, 200)
        c["kvlen"] = _spread(rng, 17, max(20, min(200000, 48 * 7000 * 8 * 128 // (c["seqs"] * kv * d))))
    else:
        most = 8192 * 8192 * 32 * 128 // (heads * d)           # pairs of a query and a key, times two
        c["new"] = _spread(rng, 20, min(8192, int(math.sqrt(most))))
        c["seqs"] = _spread(rng, 1, max(1, min(16, most // (c["new"] * c["new"]))))
        room = max(1, min(64000, most // (2 * c["seqs"] * c["new"])))
        c["kvlen"] = c["new"] if kind == "prompt" else c["new"] + _spread(rng, 1, max(2, room))
    return c


def _frac(x):
    return x - math.floor(x)


def _lengths(c):
    """New tokens and cached positions (the new ones among them) of each sequence: spread evenly below the case's."""
    new, total = [], []
    for i in range(c["seqs"]):
        n = max(1, round(c["new"] * (1.0 - c["ragged"] * _frac(0.7549 * i)))) if c["new"] > 16 else c["new"]
        old = round((c["kvlen"] - c["new"]) * (1.0 - c["ragged"] * _frac(0.6180 * i)))
        new.append(n)
        total.append(n + max(0, old))
    return new, total


def _first(c, n, length):
    """The first position that any of the n new tokens of a sequence sees."""
    return max(0, length - n - c["window"] + 1) if c["window"] else 0


def work(case):
    c = case
    if c["op"] == "qk_rope":
        n, kvn = c["t"] * c["d"] * (c["heads"] + 2 * c["kv"]), c["t"] * c["d"] * 2 * c["kv"]
        kept = 2 * kvn if c["fmt"] == "bf16" else kvn + 8 * c["t"] * c["kv"]
        return {"bytes": 2 * n + 2 * (n - kvn) + kept + 8 * c["t"] + 4 * c["rot"] // 2, "flops": 8 * n}
    if c["op"] == "logprobs":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * (2 if c["type"] == "bf16" else 4) + c["rows"] * (12 + 8 * c["top"]), "flops": 5 * n}
    b, pairs = 0, 0
    per = c["kv"] * (4 * c["d"] if c["fmt"] == "bf16" else 2 * c["d"] + 8)      # bytes of a cached position
    for n, length in zip(*_lengths(c)):
        b += 4 * n * c["heads"] * c["d"] + (length - _first(c, n, length)) * per
        old = length - n
        if not c["window"]:
            pairs += n * old + n * (n + 1) // 2
        else:
            short = max(0, min(n, c["window"] - old))           # rows that see all there is
            pairs += short * old + short * (short + 1) // 2 + (n - short) * c["window"]
    return {"bytes": b, "flops": 4 * pairs * c["heads"] * c["d"]}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _acts(g, shape):
    """Activations: normal, one entry in a hundred eight times as large."""
    x = _normal(g, shape)
    far = torch.rand(shape, generator=g, device=DEV) < 0.01
    return torch.where(far, 8.0 * x, x)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cache(g, c, pages):
    """K and V (codes and scales) of normal values; what no sequence holds is another one's leavings."""
    shape = (pages, c["kv"], c["page"], c["d"])
    out = {}
    for name in ("k", "v"):
        x = torch.empty(shape, dtype=torch.bfloat16 if c["fmt"] == "bf16" else torch.float8_e4m3fn, device=DEV)
        scale = None if c["fmt"] == "bf16" else torch.empty(shape[:3], dtype=torch.float32, device=DEV)
        step = max(1, (1 << 26) // (c["kv"] * c["page"] * c["d"]))
        for at in range(0, pages, step):
            part = _normal(g, (min(step, pages - at), *shape[1:]))
            if scale is None:
                x[at:at + step] = part.to(torch.bfloat16)
            else:
                x[at:at + step], scale[at:at + step] = _quantize(part)
        out[name], out[name + "_scale"] = x, scale
    return out


def prepare(case, seed):
    g, c = _gen(seed), case
    s = dict(case)
    if c["op"] == "logprobs":
        kind = torch.bfloat16 if c["type"] == "bf16" else torch.float32
        s["logits"] = torch.empty((c["rows"], c["vocab"]), dtype=kind, device=DEV)
        s["targets"] = torch.randint(0, c["vocab"], (c["rows"],), generator=g, device=DEV, dtype=torch.int32)
        for at in range(0, c["rows"], 256):
            part = s["logits"][at:at + 256]
            x = 2.5 * _normal(g, part.shape)
            x += 6.0 * (torch.rand(part.shape, generator=g, device=DEV) < 1e-4)
            if c["masked"]:
                hide = torch.rand(part.shape, generator=g, device=DEV) < c["masked"]
                # the tokens that were taken were allowed
                hide.scatter_(1, s["targets"][at:at + 256].long()[:, None], False)
                x[hide] = -math.inf
            part.copy_(x)
        new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
        s["logprob"], s["entropy"] = new(c["rows"]), new(c["rows"])
        s["ids"], s["top_logprobs"] = new(c["rows"], c["top"], dtype=torch.int32), new(c["rows"], c["top"])
        if own:
            import gemv_nvfp4_int8_amd as qp
            s["work"] = new(qp.token_logprobs_workspace(c["rows"], c["vocab"], c["top"]), dtype=torch.uint8)
        return s
    if c["op"] == "qk_rope":
        t, heads, kv, d, page = c["t"], c["heads"], c["kv"], c["d"], c["page"]
        s["qkv"] = _acts(g, (t, (heads + 2 * kv) * d)).to(torch.bfloat16)
        s["q_norm"] = (1.0 + 0.2 * _normal(g, (d,))).to(torch.bfloat16) if c["norm"] else None
        s["k_norm"] = (1.0 + 0.2 * _normal(g, (d,))).to(torch.bfloat16) if c["norm"] else None
        # a prompt's consecutive positions, up to the farthest of the case
        start = torch.randint(max(0, c["far"] - 2 * t), max(1, c["far"] - t) + 1, (1,), generator=g, device=DEV)
        s["positions"] = (start + torch.arange(t, device=DEV)).to(torch.int32)
        half = c["rot"] // 2
        s["inv_freq"] = (BASE ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)).float()
        s["rope_scale"] = 1.0 if c["far"] <= 65536 else 0.1 * math.log(c["far"] / 32768) + 1.0
        # consecutive positions fill pages that were given out in no order, beginning inside one
        pages = t // page + 3
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(t, device=DEV) + 5
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        s.update(_cache(g, c, pages))
        s["q_out"] = torch.empty((t, heads, d), dtype=torch.bfloat16, device=DEV)
        if own:
            import gemv_nvfp4_int8_amd as qp
            s["cache"] = qp.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        return s
    new, total = _lengths(c)
    s["lengths"] = list(zip(new, total))                        # the program's own count of its sequences
    t, page = sum(new), c["page"]
    widest = max(total)
    each = [-(-n // page) for n in total]
    width = -(-widest // page)
    order = torch.randperm(sum(each), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((c["seqs"], width), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(each):
        table[i, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["q_start"] = _i32([sum(new[:i]) for i in range(c["seqs"] + 1)])
    s["kv_len"] = _i32(total)
    s["max_q"] = max(new)
    s["q"] = (1.5 * _normal(g, (t, c["heads"], c["d"]))).to(torch.bfloat16)
    s["scale"] = c["d"] ** -0.5
    s.update(_cache(g, c, sum(each)))
    s["out"] = torch.empty_like(s["q"])
    if own:
        import gemv_nvfp4_int8_amd as qp
        s["cache"] = qp.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["work"] = torch.empty(qp.paged_attention_workspace(t, c["seqs"], s["max_q"], c["heads"], c["kv"], c["d"]),
                                dtype=torch.uint8, device=DEV)
    return s


# -------------------------------------------------------------------------------- plain forms
def _quantize(y):
    """E4M3 values and F32 scales of the last dimension's rows."""
    scale = y.abs().amax(dim=-1) / 448.0
    over = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (y / over[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _normed(x, w):
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w.float()


def _turned(x, cos, sin, layout):
    """The first 2 * cos.shape[-1] entries of each head turned by their angles."""
    half = cos.shape[-1]
    y = x.clone()
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_rope(s):
    t, heads, kv, d = s["t"], s["heads"], s["kv"], s["d"]
    x = s["qkv"].view(t, heads + 2 * kv, d).float()
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    if s["norm"]:
        q, k = _normed(q, s["q_norm"]), _normed(k, s["k_norm"])
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = (torch.cos(angle) * s["rope_scale"]).float(), (torch.sin(angle) * s["rope_scale"]).float()
    q, k = _turned(q, cos, sin, s["layout"]), _turned(k, cos, sin, s["layout"])
    page, where = s["slots"].long() // s["page"], s["slots"].long() % s["page"]
    for name, x in (("k", k), ("v", v)):
        if s["fmt"] == "bf16":
            s[name][page, :, where] = x.to(torch.bfloat16)
        else:
            codes, scale = _quantize(x)
            s[name].view(torch.uint8)[page, :, where] = codes.view(torch.uint8)
            s[name + "_scale"][page, :, where] = scale
    s["q_out"] = q.to(torch.bfloat16)


def _gathered(s, name, i, lo, hi):
    """Positions lo..hi-1 of sequence i as [kv, hi - lo, d] in 32 bits."""
    page = s["page"]
    ids = s["table"][i, lo // page:-(-hi // page)].long()
    x = s[name]
    x = x[ids].float() if x.dtype == torch.bfloat16 else x.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][ids][..., None]
    x = x.transpose(0, 1).reshape(s["kv"], -1, s["d"])
    return x[:, lo % page:lo % page + hi - lo]


def _plain_attention(s):
    heads, kv, d = s["heads"], s["kv"], s["d"]
    group = heads // kv
    out = torch.empty_like(s["q"])
    at = 0
    for i, (n, length) in enumerate(s["lengths"]):
        lo = _first(s, n, length)
        k, v = _gathered(s, "k", i, lo, length), _gathered(s, "v", i, lo, length)
        step = max(1, (1 << 28) // (heads * (length - lo)))
        for r in range(0, n, step):
            m = min(step, n - r)
            # rows of a key's head: the group's query heads of each token
            q = s["q"][at + r:at + r + m].float().view(m, kv, group, d).permute(1, 0, 2, 3).reshape(kv, m * group, d)
            score = torch.matmul(q, k.transpose(1, 2).contiguous()) * s["scale"]
            where = length - n + torch.arange(r, r + m, device=DEV).repeat_interleave(group)[:, None]
            key = torch.arange(lo, length, device=DEV)[None]
            seen = key <= where
            if s["window"]:
                seen &= key > where - s["window"]
            score = torch.where(seen, score, -math.inf)
            p = torch.exp(score - score.amax(dim=-1, keepdim=True))
            o = torch.matmul(p, v.contiguous()) / p.sum(dim=-1, keepdim=True)
            out[at + r:at + r + m] = o.view(kv, m, group, d).permute(1, 0, 2, 3).reshape(m, heads, d).to(torch.bfloat16)
        at += n
    s["out"] = out


def _plain_logprobs(s):
    rows, top = s["rows"], s["top"]
    parts = []
    for at in range(0, rows, 128):
        raw = s["logits"][at:at + 128]
        x = raw.float()
        y = x - x.amax(dim=1, keepdim=True)
        e = torch.exp(y)
        total = e.sum(dim=1, keepdim=True)
        norm = torch.log(total)
        target = s["targets"][at:at + 128].long()[:, None]
        entropy = norm - torch.where(e > 0, e * y, 0.0).sum(dim=1, keepdim=True) / total
        # equal logits: the lowest token first
        ids = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :top]
        parts.append((y.gather(1, target) - norm, entropy, ids, y.gather(1, ids) - norm))
    logprob, entropy, ids, best = (torch.cat(p) for p in zip(*parts))
    return {"logprob": logprob[:, 0], "entropy": entropy[:, 0], "ids": ids.to(torch.int32), "top": best}


# ---------------------------------------------------------------------------------------- run
def run(state):
    s = state
    if s["op"] == "logprobs":
        if not own:
            return _plain_logprobs(s)
        import gemv_nvfp4_int8_amd as qp
        qp.token_logprobs(s["logits"], s["targets"], s["logprob"], s["entropy"], s["ids"], s["top_logprobs"], s["work"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "ids": s["ids"], "top": s["top_logprobs"]}
    if s["op"] == "attention":
        if not own:
            _plain_attention(s)
            return s["out"]
        import gemv_nvfp4_int8_amd as qp
        qp.paged_attention(s["q"], s["cache"], s["table"], s["q_start"], s["kv_len"], s["max_q"], s["scale"],
                           s["window"], s["work"], s["out"])
        return s["out"]
    if not own:
        _plain_rope(s)
    else:
        import gemv_nvfp4_int8_amd as qp
        layout = qp.QP_ROPE_HALF if s["layout"] == "half" else qp.QP_ROPE_INTERLEAVED
        qp.qk_norm_rope_cache(s["qkv"], s["q_norm"], s["k_norm"], EPS, s["positions"], s["inv_freq"], s["rope_scale"],
                              layout, s["slots"], s["cache"], s["q_out"])
    out = {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if s["fmt"] != "bf16":
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


# -------------------------------------------------------------------------------------- exact
def exact(case, seed):
    s, f64 = prepare(case, seed), torch.float64
    if s["op"] == "logprobs":
        out = {n: [] for n in ("logprob", "entropy", "ids", "top")}
        for r in range(s["rows"]):
            x = s["logits"][r].to(f64)
            lse = torch.logsumexp(x, dim=0)
            p = torch.exp(x - lse)
            out["logprob"].append(x[s["targets"][r].long()] - lse)
            out["entropy"].append(-(p * torch.where(p > 0, x - lse, 0.0)).sum())
            out["top"].append(torch.topk(x, s["top"]).values - lse)
        return {n: torch.stack(v) if v else None for n, v in out.items()}
    if s["op"] == "qk_rope":
        t, heads, kv, d, half = s["t"], s["heads"], s["kv"], s["d"], s["rot"] // 2
        x = s["qkv"].to(f64).view(t, -1, d)
        parts = {"q": x[:, :heads], "k": x[:, heads:heads + kv]}
        turn = torch.polar(torch.full((), s["rope_scale"], dtype=f64, device=DEV).float().to(f64).expand(t, 1, half),
                           s["positions"].to(f64)[:, None, None] * s["inv_freq"].to(f64))
        out = {}
        for name, y in parts.items():
            if s["norm"]:
                y = y / torch.sqrt((y * y).sum(dim=2, keepdim=True) / d + EPS) * s[name + "_norm"].to(f64)
            a, rest = y[:, :, :2 * half], y[:, :, 2 * half:]
            if s["layout"] == "half":
                z = torch.complex(a[:, :, :half].contiguous(), a[:, :, half:].contiguous()) * turn
                a = torch.cat([z.real, z.imag], dim=2)
            else:
                z = torch.view_as_complex(a.reshape(t, -1, half, 2).contiguous()) * turn
                a = torch.view_as_real(z).reshape(t, -1, 2 * half)
            out[name] = torch.cat([a, rest], dim=2)
        out["v"] = x[:, heads + kv:]
        q = out.pop("q")
        slots = s["slots"].long()
        for name, y in list(out.items()):
            whole = s[name].to(f64) if s["fmt"] == "bf16" else s[name].float().to(f64)
            whole = whole.transpose(1, 2).reshape(-1, kv, d).clone()
            if s["fmt"] != "bf16":
                # codes before their rounding to eight bits
                scale = y.abs().amax(dim=2) / 448.0
                y = torch.where(scale[..., None] > 0, y / torch.where(scale > 0, scale, 1.0)[..., None], 0.0)
                kept = s[name + "_scale"].to(f64).transpose(1, 2).reshape(-1, kv).clone()
                kept[slots] = scale
                out[name + "_scale"] = kept.view(-1, s["page"], kv).transpose(1, 2)
            whole[slots] = y
            out[name] = whole.view(-1, s["page"], kv, d).transpose(1, 2)
        return {"q": q, **out}
    if work(case)["flops"] > 4e12:
        return None
    heads, kv, d, page, table = s["heads"], s["kv"], s["d"], s["page"], s["table"].long()
    out = torch.empty(s["q"].shape, dtype=f64, device=DEV)
    at = 0
    for i, (n, length) in enumerate(s["lengths"]):
        where = torch.arange(length, device=DEV)
        ids, inside = table[i][where // page], where % page
        for h in range(kv):
            kk, vv = (s[x][ids, h, inside].float().to(f64) if s["fmt"] == "bf16" else
                      s[x].view(torch.uint8)[ids, h, inside].view(torch.float8_e4m3fn).float().to(f64)
                      * s[x + "_scale"][ids, h, inside].to(f64)[:, None] for x in ("k", "v"))
            for head in range(h * (heads // kv), (h + 1) * (heads // kv)):
                for r in range(0, n, 1024):
                    m = min(1024, n - r)
                    pos = length - n + r + torch.arange(m, device=DEV)[:, None]
                    hide = where[None] > pos
                    if s["window"]:
                        hide |= where[None] <= pos - s["window"]
                    score = s["q"][at + r:at + r + m, head].to(f64) @ kk.t() * s["scale"]
                    out[at + r:at + r + m, head] = torch.softmax(score.masked_fill(hide, -math.inf), dim=1) @ vv
        at += n
    return out
