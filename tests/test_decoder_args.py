"""Arguments of the entry points of include/qproj_decoder.h at the ends of their
ranges (no GPU)."""
import math

import pytest
import torch

import gemv_nvfp4_int8_amd as qp


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
