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
