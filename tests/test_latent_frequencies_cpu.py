"""Scaled frequencies against their definition, pair by pair, for short and long trained lengths."""
import math

import pytest

import block_scaled_fp8_04_amd as bfp8


@pytest.mark.parametrize("dim,base", [(64, 1e4), (128, 1e4), (64, 5e5), (128, 1e6), (2, 1e4), (6, 100.0)])
@pytest.mark.parametrize("trained", [4, 100, 2048, 4096, 32768, 131072, 1 << 20, 10 ** 9])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (8.0, 8.0), (300.0, 2.5)])
def test_every_pair_follows_its_turns(dim, base, trained, fast, slow):
    factor = 4.0
    plain = bfp8.rope_frequencies(dim, base, device="cpu")[0].double()
    scaled, amplitude = bfp8.rope_frequencies(dim, base, factor, trained, fast, slow, device="cpu")
    assert amplitude == 0.1 * math.log(factor) + 1
    kept = []
    for i in range(dim // 2):
        turns = trained * base ** (-2.0 * i / dim) / (2 * math.pi)
        ratio = float(scaled[i].double() / plain[i])
        near = 2.0 ** -22                                  # two values rounded to fp32
        if turns > fast * (1 + 1e-9):
            assert abs(ratio - 1) <= near, (i, turns, ratio)
        elif turns < slow * (1 - 1e-9):
            assert abs(ratio - 1 / factor) <= near, (i, turns, ratio)
        else:
            assert 1 / factor - near <= ratio <= 1 + near
            assert ratio > 1 / factor + near or turns < slow * (1 + 1e-9), (i, turns, ratio)
        # the part that is kept falls linearly over the pairs in between
        kept.append((ratio - 1 / factor) / (1 - 1 / factor))
    between = [k for k in kept if 1e-6 < k < 1 - 1e-6]
    steps = [a - b for a, b in zip(between, between[1:])]
    assert all(abs(s - steps[0]) < 1e-5 for s in steps)
    assert all(a >= b - 1e-6 for a, b in zip(kept, kept[1:]))


def test_a_last_pair_of_several_turns_is_mixed():
    """2.78 turns in 131072 tokens, between 1 and 32: neither kept nor fully divided.  The ramp goes over
    the pairs that make 32 turns and 1 turn as real numbers, 22.498 and 34.539, so from 22 to 35."""
    plain, _ = bfp8.rope_frequencies(64, device="cpu")
    scaled, _ = bfp8.rope_frequencies(64, factor=4.0, trained_len=131072, device="cpu")
    part = (31 - 22) / (35 - 22)
    assert abs(float(scaled[31].double() / plain[31].double()) - (part / 4 + 1 - part)) < 1e-6
