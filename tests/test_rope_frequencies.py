"""rope_inv_freq's scaled frequencies against their formulas, each pair computed for itself in Python floats.

Tolerance: a dozen roundings in 64 bits, one of them in an exponent of at most 15: 1e-13 relative.
"""
import math
import os
import re

import pytest

import gqa_flash_attention_gb300 as sdp


def yarn(dim, base, factor, length, fast, slow):
    """The interpolated frequencies: pairs below `low` are kept, those from `high` on divided, linear between.
    The ends are the (real-valued) pairs that turn `fast` and `slow` times in `length`, rounded outwards and held
    to [0, dim - 1]: the upper one may lie past the last pair, dim / 2 - 1."""
    def pair(turns):
        return dim / 2 * math.log(length / (turns * 2 * math.pi)) / math.log(base)

    low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), dim - 1)
    out = []
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        g = min(max((i - low) / (high - low), 0.0), 1.0)
        out.append((1 - g) * f + g * f / factor)
    return out


@pytest.mark.parametrize("dim,base,factor,length", [
    (128, 1e4, 4.0, 4096), (128, 1e4, 16.0, 32768), (64, 5e5, 8.0, 8192), (256, 1e6, 2.0, 262144), (96, 1e4, 40.0, 4096),
    # the ramp ends past the last pair
    (64, 1e4, 4.0, 65536), (128, 1e4, 4.0, 131072), (256, 1e4, 32.0, 1 << 20), (16, 100.0, 4.0, 4096),
])
def test_yarn(dim, base, factor, length):
    got = sdp.rope_inv_freq(dim, base, scaling="yarn", factor=factor, original_length=length)
    want = yarn(dim, base, factor, length, 32.0, 1.0)
    for i, (x, y) in enumerate(zip(got.tolist(), want)):
        assert abs(x - y) <= 1e-13 * y, (i, x / y)


def test_yarn_divides_no_pair_fully_that_turns_often_enough():
    plain = sdp.rope_inv_freq(64, 1e4)
    f = sdp.rope_inv_freq(64, 1e4, scaling="yarn", factor=4.0, original_length=65536)
    turns = 65536 * plain / (2 * math.pi)
    assert turns[31] > 1.3  # more than beta_slow, so between kept and divided
    assert (f[turns > 1] > 1.01 * plain[turns > 1] / 4).all()
    assert abs(plain[31].item() / f[31].item() - 13 / (2 + 11 / 4)) < 1e-12  # pairs 20 to 33: 11 of 13 steps


def test_yarn_keeps_every_pair_of_a_length_in_which_all_turn_often():
    """Both ends lie past the last pair."""
    f = sdp.rope_inv_freq(64, 100.0, scaling="yarn", factor=8.0, original_length=1 << 24)
    assert (f == sdp.rope_inv_freq(64, 100.0)).all()


def test_the_documented_yarn_table_carries_its_attention_factor():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as readme:
        lines = re.findall(r"^(?:f|table) = .*$", readme.read(), re.M)
    scope = {"sdp": sdp, "math": math}
    exec("\n".join(lines).replace('device="cuda"', 'device="cpu"'), scope)
    assert "yarn" in lines[0] and scope["table"].turns.shape == (64,)
    assert abs(scope["table"].mscale - (0.1 * math.log(4) + 1)) < 1e-12
