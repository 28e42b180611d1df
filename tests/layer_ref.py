"""Plain references in 64 bits for the operators of include/qproj_layer.h (test
infrastructure; no code shared with the library)."""
import math

import torch

F64 = torch.float64
FMT_ROW, FMT_BLOCK128, FMT_INT8 = 0, 1, 2


def block_of(fmt, k):
    return {FMT_ROW: k, FMT_BLOCK128: 128, FMT_INT8: 32}[fmt]


def top_of(fmt):
    return 127.0 if fmt == FMT_INT8 else 448.0


def rms_norm(x, residual, weight, eps):
    """(h in BF16, y in 64 bits)."""
    h = x.double()
    if residual is not None:
        # a sum of two BF16 values, rounded to F32 and then to BF16, as any
        # 32-bit program forms it
        h = h + residual.double()
    h16 = h.float().to(torch.bfloat16)
    h = h16.double()
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32)))
    return h16, h * rstd * weight.double()


def silu_mul(gate_up):
    k = gate_up.shape[1] // 2
    g, u = gate_up[:, :k].double(), gate_up[:, k:].double()
    return g / (1.0 + torch.exp(-g)) * u


def scales(y, fmt):
    rows, k = y.shape
    b = block_of(fmt, k)
    nb = -(-k // b)
    z = torch.zeros((rows, nb * b), dtype=F64, device=y.device)
    z[:, :k] = y.abs()
    return z.view(rows, nb, b).amax(dim=2) / top_of(fmt)


def per_element(scale, fmt, k):
    return scale.repeat_interleave(block_of(fmt, k), dim=1)[:, :k]


def decoded(q):
    return q.double() if q.dtype == torch.int8 else q.view(torch.float8_e4m3fn).float().double()


def encoded_value(v, fmt):
    """The code grid's nearest value of v (ties to even), in 64 bits."""
    top = top_of(fmt)
    if fmt == FMT_INT8:
        return v.round().clamp(-top, top)
    return v.float().clamp(-top, top).to(torch.float8_e4m3fn).float().double()


def assert_quantized(q, scale, y, fmt, rel):
    """q, scale against the exact values y: every scale within `rel` of its
    own, every code between the codes of the exact quotient moved by `rel`
    either way.  Scales below 1e-37 (next to the F32 subnormals, which hold
    fewer bits) are checked for size only."""
    rows, k = y.shape
    ref = scales(y, fmt)
    got = scale.reshape(ref.shape).double()
    assert torch.all((got - ref).abs() <= rel * ref + 1e-38), (got - ref).abs().max()
    each, mine = per_element(ref, fmt, k), per_element(got, fmt, k)
    ok = each > 1e-37
    v = torch.where(ok, y / torch.where(ok, each, 1.0), 0.0)
    near, far = v * (1.0 - rel), v * (1.0 + rel)
    lo = encoded_value(torch.minimum(near, far), fmt)
    hi = encoded_value(torch.maximum(near, far), fmt)
    c = decoded(q)
    bad = ok & ((c < lo) | (c > hi))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())
    # a zero scale has +0 codes only
    zero = mine == 0
    assert not (zero & (q.view(torch.uint8).reshape(rows, k) != 0)).any()


# ------------------------------------------------------------------ the product
def e4m3(q):
    return q.view(torch.float8_e4m3fn).float().double()


def gemm_blockscale(a, a_scale, w, grid):
    """(C, S, G) in 64 bits: the product, the sum of its terms' magnitudes, and
    the sum over groups of 8 neighbouring terms of a bound on the group's
    largest (the product of the operands' largest)."""
    n, k = w.shape
    av = e4m3(a) * a_scale.double().repeat_interleave(128, dim=1)[:, :k]
    wv = e4m3(w) * grid.double().repeat_interleave(128, dim=0)[:n].repeat_interleave(128, dim=1)[:, :k]
    top = lambda v: v.abs().view(v.shape[0], -1, 8).amax(dim=2)  # noqa: E731
    return av @ wv.t(), av.abs() @ wv.abs().t(), top(av) @ top(wv).t()


def assert_rounded(out, c, tol):
    """out is BF16 of something within tol of c: it lies between the BF16
    neighbours that c - tol and c + tol round to (rounding is monotone; the
    step through F32 is covered by 2^-23 of c)."""
    t = tol + 2.0 ** -23 * c.abs() + 1e-38
    lo, hi = ((c + d).float().to(torch.bfloat16).double() for d in (-t, t))
    bad = ~((out.double() >= lo) & (out.double() <= hi))
    assert not bad.any(), (int(bad.sum()), ((out.double() - c).abs() / t)[bad].max())


def assert_gemm(out, csg, k):
    """The matrix core adds 8 products at a time, aligned to the largest of
    them with 13 bits kept below it (measured): 7 * 2^-13 of it per group at
    most.  The groups and then ceil(k/128) scaled blocks are summed in F32 (one
    ulp, 2^-23, for each of at most 128 + ceil(k/128) additions and for the few
    products of scales).  That bound holds for every output; the second one,
    BF16's half ulp in the 2-norm, is where the errors' signs cancel."""
    c, s, g = csg
    assert_rounded(out, c, (140 + -(-k // 128)) * 2.0 ** -23 * s + 7 * 2.0 ** -13 * g)
    assert (out.double() - c).norm() <= 2.0 ** -8 * c.norm()


# ------------------------------------------------------------ mixture of experts
def route(row, topk, renorm):
    """[(expert, weight)] of one token's logits (a list of Python floats)."""
    open_ = sorted((j for j in range(len(row)) if row[j] > -math.inf), key=lambda j: (-row[j], j))
    chosen = open_[:topk]
    if not chosen:
        return []
    top = row[chosen[0]]
    total = sum(math.exp(row[j] - top) for j in (chosen if renorm else open_))
    return [(j, math.exp(row[j] - top) / total) for j in chosen]


def moe(x, logits, w13, s13, w2, s2, topk, renorm):
    """(out, bound): the layer in 64 bits and a bound of the F32 form's error.

    A product over K elements is a sum of K/256 + 32 additions' roundings at
    most (windows, the 4-element steps within one, the 16 slices), each 2^-23
    of the magnitudes' sum; h = silu(g) u p carries those of g (the slope of
    silu is at most 1.1) and u, 2^-17 of its two planes and 2^-20 for its own
    arithmetic; the weighted sum carries h's and its own (BF16's rounding is
    assert_rounded's)."""
    t, h = x.shape
    i = w2.shape[2]
    out = torch.zeros((t, h), dtype=F64, device=x.device)
    tol = torch.zeros_like(out)
    rows = logits.double().cpu().tolist()
    grid = lambda w, s: e4m3(w) * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)  # noqa: E731
    by_expert = {}
    for n, row in enumerate(rows):
        for j, p in route(row, topk, renorm):
            by_expert.setdefault(j, []).append((n, p))
    c1, c2 = (h / 256 + 32) * 2.0 ** -23, (i / 256 + 48) * 2.0 ** -23
    for j, users in by_expert.items():
        a, b = grid(w13[j], s13[j]), grid(w2[j], s2[j])
        at = torch.tensor([n for n, _ in users], device=x.device)
        p = torch.tensor([q for _, q in users], dtype=F64, device=x.device)[:, None]
        xv = x[at].double()
        gu, mag = xv @ a.t(), xv.abs() @ a.abs().t()
        g, u = gu[:, :i], gu[:, i:]
        sil = g / (1.0 + torch.exp(-g))
        hv = sil * u * p
        dh = p * (1.1 * u.abs() * c1 * mag[:, :i] + sil.abs() * c1 * mag[:, i:]) + hv.abs() * 2.0 ** -16
        out.index_add_(0, at, hv @ b.t())
        tol.index_add_(0, at, dh @ b.abs().t() + c2 * (hv.abs() @ b.abs().t()))
    return out, tol
