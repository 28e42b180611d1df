"""Plain references in 64 bits for the operators of include/qproj_decoder.h, and
the bounds of the F32 forms' errors (test infrastructure; no code shared with
the library)."""
import math

import torch

from tests.layer_ref import F64, assert_rounded  # noqa: F401

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
DEV = "cuda:0"
NAN_CODE = 0x7F


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


# ------------------------------------------------------------------ the cache
class Cache:
    """K and V with NaN everywhere: what a test writes is what may be read."""

    def __init__(self, pages, kv, page, d, fp8):
        self.fp8, self.page, self.pages = fp8, page, pages
        new = lambda *s, dtype: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
        self.k, self.v = (new(pages, kv, page, d, dtype=U8 if fp8 else BF16) for _ in range(2))
        self.ks, self.vs = (new(pages, kv, page, dtype=F32) if fp8 else None for _ in range(2))
        for x in (self.k, self.v):
            x.fill_(NAN_CODE if fp8 else math.nan)
        for x in (self.ks, self.vs):
            if x is not None:
                x.fill_(math.nan)

    def tensors(self):
        return [x for x in (self.k, self.v, self.ks, self.vs) if x is not None]

    def put(self, which, slots, x):
        """x [n, kv, d] F32 to `slots`, as the cache's form holds it."""
        t, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        at, off = slots.long() // self.page, slots.long() % self.page
        if not self.fp8:
            t[at, :, off] = x.to(BF16)
            return
        s = x.abs().amax(dim=2) / 448.0
        codes = (x / torch.where(s > 0, s, 1.0)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        t[at, :, off] = codes.view(U8)
        scale[at, :, off] = s

    def get(self, which, slots):
        """What the cache holds at `slots`, in 64 bits: [n, kv, d]."""
        t, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        at, off = slots.long() // self.page, slots.long() % self.page
        x = t[at, :, off]
        if not self.fp8:
            return x.double()
        return x.view(torch.float8_e4m3fn).float().double() * scale[at, :, off].double()[..., None]


# ------------------------------------------------------------------ rotary positions
def rope(x, weight, eps, positions, inv_freq, rope_scale, layout_half):
    """(y, bound) of heads x [t, heads, d] (F32 values) in 64 bits.

    The bound: the sum of squares has d roundings of 2^-24 of itself, which the
    root halves; rstd, the two products and the rotation's two products and sum
    are eight more of up to 2^-23; the angle in turns is rounded to F32 once
    (2^-25 of a turn at most, 2 pi of that), and cosine and sine are off by 2^-22."""
    d = x.shape[2]
    y = x.double()
    if weight is not None:
        f32 = lambda v: float(torch.tensor(v, dtype=F32))  # noqa: E731
        y = y / torch.sqrt((y * y).mean(dim=2, keepdim=True) + f32(eps)) * weight.double()
    out, mag = y.clone(), y.abs()
    if inv_freq is not None:
        half = inv_freq.numel()
        scale = float(torch.tensor(rope_scale, dtype=F32))
        angle = positions.double()[:, None, None] * inv_freq.double()
        c, s = torch.cos(angle) * scale, torch.sin(angle) * scale
        a, b = ((slice(0, half), slice(half, 2 * half)) if layout_half
                else (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        both = (y[..., a].abs() + y[..., b].abs()) * abs(scale)
        mag = mag.clone()
        mag[..., a], mag[..., b] = both, both
    return out, (d * 2.0 ** -25 + 12 * 2.0 ** -23) * mag


def assert_row_codes(codes, scale, y, tol):
    """E4M3 rows with a scale each, of values within tol of y [..., d]: the scale
    is within the largest value's own bound, each code between those that the
    ends of its value's range round to under the scale that was written."""
    top = y.abs().amax(dim=-1)
    s = scale.double()
    assert torch.all((s - top / 448.0).abs() <= (tol.amax(dim=-1) + 2.0 ** -23 * top) / 448.0 + 1e-38)
    e4m3 = lambda v: v.float().clamp(-448, 448).to(torch.float8_e4m3fn).float().double()  # noqa: E731
    safe = torch.where(s > 0, s, 1.0)[..., None]
    room = tol / safe + 2.0 ** -22 * (y / safe).abs()
    got = codes.view(torch.float8_e4m3fn).float().double()
    bad = (s[..., None] > 0) & ((got < e4m3(y / safe - room)) | (got > e4m3(y / safe + room)))
    assert not bad.any(), int(bad.sum())


# ------------------------------------------------------------------ attention
def attention(q, k, v, seen, scale):
    """(out, bound) of q [n, heads, d] over k, v [len, kv, d] in 64 bits, where
    row i may see position j if seen[i, j].

    The bound, relative to sum p |v|: 2^-8 for the probabilities' rounding to
    BF16; a score is a sum of d products in F32 (d + 8 roundings of 2^-24 of the
    sum of magnitudes, the scales' among them) and a probability's error is its
    score's, once over the line and once in the sum under it; the exponential
    itself 2^-21; and the running sums, 2^-24 a key for the numbers above and
    below the line."""
    n, heads, d = q.shape
    group = heads // k.shape[1]
    scale = float(torch.tensor(scale, dtype=F32))
    out, tol = torch.zeros((n, heads, d), dtype=F64, device=q.device), torch.zeros((n, heads, d), dtype=F64, device=q.device)
    if not len(k):
        return out, tol
    used = seen.any(dim=0)
    k = torch.where(used[:, None, None], k, 0.0)        # what no row sees may be NaN
    v = torch.where(used[:, None, None], v, 0.0)
    for h in range(heads):
        qh, kh, vh = q[:, h].double(), k[:, h // group], v[:, h // group]
        score = (qh @ kh.t()) * scale
        spread = (qh.abs() @ kh.abs().t()) * scale
        score = torch.where(seen, score, -math.inf)
        top = score.amax(dim=1, keepdim=True)
        p = torch.where(seen, torch.exp(score - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
        total = p.sum(dim=1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
        each = 2.0 * (d + 8) * 2.0 ** -24 * torch.where(seen, spread, 0.0).amax(dim=1, keepdim=True)
        c = 2.0 ** -8 + each + 2.0 ** -20 + 2.0 * seen.sum(dim=1, keepdim=True) * 2.0 ** -24
        out[:, h] = p @ vh
        tol[:, h] = c * (p @ vh.abs())
    return out, tol


def visible(n, length, window, holes=None, device=DEV):
    """[n, length]: which positions each of the last n rows sees."""
    pos = length - n + torch.arange(n, device=device)[:, None]
    key = torch.arange(length, device=device)[None]
    seen = key <= pos
    if window:
        seen &= key > pos - window
    if holes is not None:
        seen &= ~holes[None]
    return seen


# ------------------------------------------------------------------ log probabilities
def logprobs(logits, targets, top):
    """(logprob, entropy, ids, best, bounds) of F64 rows.  The sums' bound: 2^-23
    for each of vocab / 256 + 64 additions in a row at most (a thread's own, then
    the joins), and an exponential's error, 2^-21 and 2^-23 for each unit of its
    argument, weighted by the probabilities."""
    x = logits.double()
    m = x.amax(dim=1, keepdim=True)
    y = x - torch.where(torch.isfinite(m), m, 0.0)
    e = torch.exp(y)
    s = e.sum(dim=1, keepdim=True)
    alive = s[:, 0] > 0
    norm = torch.log(torch.where(s > 0, s, 1.0))
    p = e / torch.where(s > 0, s, 1.0)
    py = torch.where(p > 0, p * y, 0.0).sum(dim=1)
    entropy = torch.where(alive, norm[:, 0] - py, 0.0)
    ids = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :top]
    ok = (targets >= 0) & (targets < x.shape[1])
    at = torch.where(ok, targets, 0).long()[:, None]
    logprob = torch.where(ok, (y.gather(1, at) - norm)[:, 0], 0.0)
    rel = (x.shape[1] / 256 + 64) * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -23 * py.abs()
    return logprob, entropy, ids, y.gather(1, ids) - norm, rel


def assert_logprobs(got, want, rel):
    """Of log probabilities [rows, n]: equal where infinite, else within rel and
    the roundings of the difference."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine])
    room = rel[:, None] + 2.0 ** -22 * torch.where(fine, want, 0.0).abs() + 2.0 ** -22
    bad = fine & ~((got - want).abs() <= room)
    assert not bad.any(), (got[bad][:4], want[bad][:4])
