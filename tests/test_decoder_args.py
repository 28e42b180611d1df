"""Arguments of the entry points of include/qproj_decoder.h at the ends of their
ranges (no GPU)."""
import math

import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from tests.test_decoder_abi import attn, rope


def ramp(rot, base, factor, low, high, original):
    """The frequencies as the header states them, in 64 bits."""
    pair = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        share = min(max((i - a) / (b - a), 0.0), 1.0) if b > a else float(i > a)
        out.append(f / factor * share + f * (1 - share))
    return a, b, out


@pytest.mark.parametrize("rot,base,factor,low,high,original", [
    (128, 1e4, 4.0, 1.0, 32.0, 131072), (64, 1e4, 8.0, 1.0, 32.0, 262144), (128, 1e4, 40.0, 1.0, 32.0, 4096),
    (128, 5e5, 4.0, 1.0, 32.0, 8192), (64, 1e3, 2.0, 0.5, 16.0, 1 << 20), (16, 1e4, 4.0, 1.0, 4.0, 131072),
    (128, 10.0, 4.0, 1.0, 32.0, 1 << 20)])
def test_a_ramp_that_ends_behind_the_last_pair(rot, base, factor, low, high, original):
    a, b, want = ramp(rot, base, factor, low, high, original)
    got = qp.rope_inv_freq(rot, base, qp.QP_ROPE_RAMP, factor, low, high, original)
    for i, w in enumerate(want):
        assert abs(float(got[i]) - w) <= 2.0 ** -22 * w, (i, a, b)


def test_a_ramp_by_hand():
    """The pairs that make 32 turns and one over 131072 positions at base 1e4 are 45.0
    and 69.1: from 45 to 70, so that pair 63 is 18/25 of the way to a quarter."""
    got = qp.rope_inv_freq(128, 1e4, qp.QP_ROPE_RAMP, 4.0, 1.0, 32.0, 131072)
    assert abs(float(got[63]) / 1e4 ** (-126 / 128) - (0.28 + 0.72 / 4.0)) < 1e-6
    assert abs(float(got[45]) / 1e4 ** (-90 / 128) - 1.0) < 1e-6


# ------------------------------------------------------------------ the binding's whole numbers
LARGE = r"outside 0\.\.2\^32-1"


def wide(dtype, *shape):
    """A tensor of any shape that holds one element (no memory)."""
    return torch.zeros(1, dtype=dtype).expand(shape)


@pytest.mark.parametrize("change", [dict(max_q=-1), dict(max_q=(1 << 32) + 1), dict(window=-1), dict(window=(1 << 32) + 5),
                                    dict(t=(1 << 32) + 2), dict(heads=(1 << 32) + 4), dict(seqs=(1 << 32) + 1), dict(width=(1 << 32) + 3)])
def test_attention_takes_no_number_modulo_2_to_the_32(change):
    c = dict(t=2, heads=4, seqs=1, width=3, max_q=2, window=0)
    c.update(change)

    class Handle:
        d, kv_heads, device = 64, 2, 0
    i32 = torch.int32
    q = wide(torch.bfloat16, c["t"], c["heads"], 64)
    with pytest.raises(ValueError, match=LARGE):
        qp.paged_attention(q, Handle, wide(i32, c["seqs"], c["width"]), wide(i32, c["seqs"] + 1), wide(i32, c["seqs"]),
                           c["max_q"], 0.125, c["window"], wide(torch.uint8, 64), q)


@pytest.mark.parametrize("change", [dict(t=(1 << 32) + 2), dict(heads=(1 << 32) + 4), dict(layout=1 << 32), dict(half=1 << 31)])
def test_rope_takes_no_number_modulo_2_to_the_32(change):
    c = dict(t=2, heads=4, layout=qp.QP_ROPE_HALF, half=32)
    c.update(change)

    class Handle:
        d, kv_heads, device = 64, 2, 0
    with pytest.raises(ValueError, match=LARGE):
        qp.qk_norm_rope_cache(wide(torch.bfloat16, c["t"], (c["heads"] + 4) * 64), None, None, 1e-6, wide(torch.int32, c["t"]),
                              wide(torch.float32, c["half"]), 1.0, c["layout"], wide(torch.int32, c["t"]), Handle,
                              wide(torch.bfloat16, c["t"], c["heads"], 64))


@pytest.mark.parametrize("rows,vocab,top", [((1 << 32) + 1, 1, 1), (1, (1 << 32) + 1, 1), (1, 100, (1 << 32) + 1)])
def test_logprobs_takes_no_number_modulo_2_to_the_32(rows, vocab, top):
    f32 = torch.float32
    with pytest.raises(ValueError, match=LARGE):
        qp.token_logprobs(wide(f32, rows, vocab), wide(torch.int32, rows), wide(f32, rows), wide(f32, rows),
                          wide(torch.int32, rows, top), wide(f32, rows, top), wide(torch.uint8, 64))


def test_a_cache_takes_no_number_modulo_2_to_the_32():
    with pytest.raises(ValueError, match=LARGE):
        qp.KVCache(*[wide(torch.bfloat16, (1 << 32) + 1, 2, 16, 64)] * 2)


def test_frequencies_and_workspaces_take_no_number_modulo_2_to_the_32():
    for bad in (dict(rot=(1 << 32) + 4), dict(rot=-(1 << 32) + 64), dict(scaling=1 << 32), dict(original=(1 << 32) + 1),
                dict(original=-1)):
        with pytest.raises(ValueError, match=LARGE):
            qp.rope_inv_freq(**{**dict(rot=64, base=1e4, scaling=qp.QP_ROPE_RAMP, factor=2.0, low=1.0, high=4.0, original=4096), **bad})
    good = (4, 2, 4, 8, 2, 64)
    assert qp.paged_attention_workspace(*good) > 0 and qp.token_logprobs_workspace(4, 100, 3) > 0
    for i in range(6):
        for off in (1 << 32, -(1 << 32)):
            assert qp.paged_attention_workspace(*[v + off * (j == i) for j, v in enumerate(good)]) == 0
    for i in range(3):
        for off in (1 << 32, -(1 << 32)):
            assert qp.token_logprobs_workspace(*[v + off * (j == i) for j, v in enumerate((4, 100, 3))]) == 0


def test_eps_below_the_normal_numbers():
    """The reciprocal root takes a subnormal number for 0, and a head of zeros would be
    0 times infinity."""
    for eps in (1.1754942e-38, 1e-39, 1e-45):
        assert rope(eps=eps) == qp.QP_ERR_RANGE
    # (no norms: eps is not used, and rot is what is refused)
    assert rope(eps=0.0, q_norm=0, k_norm=0, rot=63) == qp.QP_ERR_SHAPE


def test_scales_that_base_2_does_not_hold():
    """Scores are kept in base 2: scale times log2(e) has to be finite."""
    for scale in (2.36e38, 3e38, 3.4028234e38):
        assert attn(scale=scale) == qp.QP_ERR_RANGE
    assert attn(scale=2.35e38, bytes=0) == qp.QP_ERR_SCRATCH
