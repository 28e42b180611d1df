"""Argument checks of the entry points of include/qproj_decoder.h, and the rotary
frequencies, which are computed on the host (no GPU)."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import gemv_nvfp4_int8_amd as qp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = qp.lib()
A, B = 0x10000, 0x20000          # aligned, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def nothing_is_launched():
    before = qp.launch_count()
    yield
    assert qp.launch_count() == before


def test_header_and_library_agree():
    text = open(os.path.join(ROOT, "include", "qproj_decoder.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^(?:int|uint64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M))
    assert names == {"rope_inv_freq", "qk_norm_rope_cache", "paged_attention", "paged_attention_workspace",
                     "token_logprobs", "token_logprobs_workspace"}
    out = subprocess.run(["nm", "-D", "--defined-only", qp.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def test_the_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "qproj_decoder.h"\nint main(void) { return QP_LOGPROBS_MAX_TOP - 32 + QP_KV_BF16; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "use.o")], check=True)


ROPE = dict(qkv=A, q_norm=B, k_norm=B, eps=1e-6, positions=A, inv_freq=B, rope_scale=1.0, layout=0, rot=64, slots=A, fmt=1,
            k=A, v=B, ks=A, vs=B, q_out=B, t=4, q_heads=8, kv_heads=2, d=64, pages=10, page_size=16)
ATTN = dict(q=A, fmt=1, k=A, v=B, ks=A, vs=B, table=A, q_start=B, kv_len=A, scale=0.1, window=0, work=A, bytes=1 << 40,
            out=B, t=4, seqs=2, max_q=4, q_heads=8, kv_heads=2, d=64, pages=10, page_size=16, width=5)
LOGP = dict(logits=A, fmt=0, targets=B, logprob=A, entropy=B, ids=A, best=B, work=A, bytes=1 << 40, rows=4, vocab=100, top=3)


def _call(fn, defaults, **changes):
    args = {**defaults, **changes}
    assert set(args) == set(defaults)
    return getattr(L, fn)(*args.values(), None)


def rope(**c):
    return _call("qk_norm_rope_cache", ROPE, **c)


def attn(**c):
    return _call("paged_attention", ATTN, **c)


def logp(**c):
    return _call("token_logprobs", LOGP, **c)


POINTERS = [(rope, n) for n in ("qkv", "positions", "slots", "k", "v", "ks", "vs", "q_out", "q_norm", "k_norm", "inv_freq")] + \
           [(attn, n) for n in ("q", "k", "v", "ks", "vs", "table", "q_start", "kv_len", "work", "out")] + \
           [(logp, n) for n in ("logits", "targets", "logprob", "ids", "best", "work")]


@pytest.mark.parametrize("call,name", POINTERS, ids=[f"{c.__name__}-{n}" for c, n in POINTERS])
def test_every_pointer_is_checked(call, name):
    assert call(**{name: 0}) == qp.QP_ERR_NULL
    assert call(**{name: A + 8}) == qp.QP_ERR_ALIGN


def test_a_logits_call_asks_for_something():
    assert logp(targets=0, logprob=0, entropy=0, top=0, ids=0, best=0) == qp.QP_ERR_NULL
    assert logp(entropy=A + 4) == qp.QP_ERR_ALIGN


@pytest.mark.parametrize("name", ["t", "q_heads", "kv_heads", "d", "pages", "page_size"])
def test_empty_extents(name):
    assert rope(**{name: 0}) == qp.QP_ERR_SHAPE
    assert attn(**{name: 0}) == qp.QP_ERR_SHAPE


@pytest.mark.parametrize("bad", [dict(d=24), dict(d=8), dict(d=272), dict(page_size=8), dict(page_size=48),
                                 dict(page_size=8192), dict(pages=1 << 27), dict(kv_heads=65536, q_heads=65536)])
def test_cache_shapes(bad):
    assert rope(**bad) == qp.QP_ERR_SHAPE
    assert attn(**bad) == qp.QP_ERR_SHAPE


def test_formats():
    for fmt in (-1, 2, 16):
        assert rope(fmt=fmt) == qp.QP_ERR_FORMAT
        assert attn(fmt=fmt) == qp.QP_ERR_FORMAT
        assert logp(fmt=fmt) == qp.QP_ERR_FORMAT
    assert rope(layout=2) == qp.QP_ERR_FORMAT and rope(layout=-1) == qp.QP_ERR_FORMAT


def test_rope_refusals():
    for rot in (1, 63, 66, 128):
        assert rope(rot=rot) == qp.QP_ERR_SHAPE
    assert rope(t=1 << 22) == qp.QP_ERR_SHAPE                     # 2^22 * 12 * 64 values
    assert rope(t=1, q_heads=1 << 26) == qp.QP_ERR_SHAPE
    assert rope(t=1, q_heads=0xFFFFFFFF) == qp.QP_ERR_SHAPE
    for eps in (0.0, -1.0, NAN, INF):
        assert rope(eps=eps) == qp.QP_ERR_RANGE
    for s in (NAN, INF, -INF):
        assert rope(rope_scale=s) == qp.QP_ERR_RANGE


def test_attention_refusals():
    assert attn(q_heads=9) == qp.QP_ERR_SHAPE
    for bad in (dict(seqs=0), dict(width=0), dict(t=1 << 22), dict(seqs=1 << 29), dict(width=1 << 27),
                dict(seqs=0xFFFFFFFF, width=1), dict(width=1 << 23), dict(seqs=1 << 13, width=1 << 21)):
        assert attn(**bad) == qp.QP_ERR_SHAPE, bad
    for bad in (dict(max_q=0), dict(max_q=5), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF)):
        assert attn(**bad) == qp.QP_ERR_RANGE, bad
    need = qp.paged_attention_workspace(4, 2, 4, 8, 2, 64)
    assert need > 0 and attn(bytes=need - 1) == qp.QP_ERR_SCRATCH and attn(bytes=0) == qp.QP_ERR_SCRATCH
    assert qp.paged_attention_workspace(4, 2, 5, 8, 2, 64) == 0 and qp.paged_attention_workspace(4, 2, 4, 9, 2, 64) == 0


def test_logits_refusals():
    for bad in (dict(rows=0), dict(vocab=0), dict(rows=1 << 16, vocab=1 << 15), dict(rows=1 << 24, vocab=4)):
        assert logp(**bad) == qp.QP_ERR_SHAPE, bad
    for bad in (dict(top=33), dict(top=101), dict(vocab=2)):
        assert logp(**bad) == qp.QP_ERR_RANGE, bad
    need = qp.token_logprobs_workspace(4, 100, 3)
    assert need > 0 and logp(bytes=need - 1) == qp.QP_ERR_SCRATCH
    assert qp.token_logprobs_workspace(4, 100, 33) == 0


def test_workspaces_stay_modest():
    """Scratch for partial results, whatever the lengths: not more than 1 GiB."""
    for args in ((8192, 1, 8192, 32, 8, 128), (200, 200, 1, 128, 16, 256), (1, 1, 1, 1, 1, 16), (4096, 512, 4096, 64, 8, 256)):
        assert 0 < qp.paged_attention_workspace(*args) <= 1 << 30, args
    for args in ((1, 262144, 32), (2048, 152064, 8), (1, 1, 0)):
        assert 0 < qp.token_logprobs_workspace(*args) <= 1 << 26, args


def test_a_workspace_serves_smaller_calls():
    """What is enough for the most rows of a sequence is enough for fewer."""
    for d in (16, 64, 80, 128, 192, 256):
        for heads, kv in ((8, 8), (8, 2), (40, 4), (64, 1)):
            need = [qp.paged_attention_workspace(8192, 4, n, heads, kv, d) for n in
                    (1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 100, 255, 256, 257, 1000, 8192)]
            assert all(a <= b for a, b in zip(need, need[1:])), (d, heads, kv)


def test_binding_refuses_tensors_that_do_not_fit():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        qp.KVCache(k, k)
    with pytest.raises(TypeError, match="dtype"):
        qp.KVCache(k.float(), k)
    x = torch.zeros((2, 100))
    with pytest.raises(ValueError, match="device"):
        qp.token_logprobs(x, None, None, x[:, 0].contiguous(), None, None, x)
    with pytest.raises(TypeError, match="dtype"):
        qp.token_logprobs(x.double(), None, None, x[:, 0].contiguous(), None, None, x)


# ------------------------------------------------------------------ frequencies
def test_plain_linear_and_base_frequencies():
    rot, base = 128, 5e5
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    f32 = lambda v: torch.tensor(v, dtype=torch.float64).float()  # noqa: E731
    near = lambda a, b: torch.all((a - b).abs() <= 2.0 ** -23 * b.abs())  # noqa: E731
    assert near(qp.rope_inv_freq(rot, base), f32(f))
    assert near(qp.rope_inv_freq(rot, base, qp.QP_ROPE_LINEAR, 4.0), f32([v / 4.0 for v in f]))
    b = base * 8.0 ** (rot / (rot - 2))
    assert near(qp.rope_inv_freq(rot, base, qp.QP_ROPE_BASE, 8.0), f32([b ** (-2 * i / rot) for i in range(rot // 2)]))
    # base: the first pair stays, the last turns `factor` times slower
    got = qp.rope_inv_freq(rot, base, qp.QP_ROPE_BASE, 8.0)
    assert got[0] == 1.0 and abs(f[-1] / float(got[-1]) - 8.0) < 1e-4


def test_wavelength_blend():
    rot, base, factor, low, high, original = 128, 5e5, 8.0, 1.0, 4.0, 8192
    got = qp.rope_inv_freq(rot, base, qp.QP_ROPE_WAVELENGTH, factor, low, high, original)
    kept = divided = mixed = 0
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        wave = 2 * math.pi / f
        if wave < original / high:
            want, kept = f, kept + 1
        elif wave > original / low:
            want, divided = f / factor, divided + 1
        else:
            s = (original / wave - low) / (high - low)
            want, mixed = (1 - s) * f / factor + s * f, mixed + 1
        assert abs(float(got[i]) - want) <= 2.0 ** -23 * want
    assert kept > 10 and divided > 10 and mixed > 2


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
def test_ramp_blend(rot):
    base, factor, low, high, original = 1e4, 16.0, 1.0, 32.0, 4096
    got = qp.rope_inv_freq(rot, base, qp.QP_ROPE_RAMP, factor, low, high, original)
    pair = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot // 2 - 1)
    if a >= b:
        b = a + 1e-3
    for i in range(rot // 2):
        f, r = base ** (-2 * i / rot), min(max((i - a) / (b - a), 0.0), 1.0)
        want = f / factor * r + f * (1 - r)
        assert abs(float(got[i]) - want) <= 2.0 ** -22 * want


def test_frequency_refusals():
    f = (ctypes.c_float * 128)()
    call = lambda rot=64, base=1e4, kind=0, factor=2.0, low=1.0, high=4.0, orig=4096, out=f: L.rope_inv_freq(  # noqa: E731
        out, rot, base, kind, factor, low, high, orig)
    assert call() == qp.QP_OK
    assert call(out=None) == qp.QP_ERR_NULL
    for rot in (0, 1, 63, 258, 1 << 20):
        assert call(rot=rot) == qp.QP_ERR_SHAPE
    assert call(rot=2, kind=qp.QP_ROPE_BASE) == qp.QP_ERR_SHAPE
    for kind in (-1, 5):
        assert call(kind=kind) == qp.QP_ERR_FORMAT
    for bad in (dict(base=1.0), dict(base=NAN), dict(base=INF), dict(factor=0.5), dict(factor=NAN), dict(factor=INF)):
        assert call(**bad) == qp.QP_ERR_RANGE
    for kind in (qp.QP_ROPE_WAVELENGTH, qp.QP_ROPE_RAMP):
        for bad in (dict(low=0.0), dict(low=4.0), dict(high=INF), dict(low=NAN), dict(orig=0)):
            assert call(kind=kind, **bad) == qp.QP_ERR_RANGE
