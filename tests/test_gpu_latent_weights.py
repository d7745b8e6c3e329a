"""Weights of bfp8_attn_latent that lie far below the largest: what they lose is bounded, however many tokens
there are, and wherever in a tile they stand."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
from gpu_helpers import announce, dev
from kv_helpers import i32
from kv_reference import VALUES

pytestmark = pytest.mark.gpu

ONE, MOST = 0x38, 0x7E                                     # codes of 1 and of 448


def attend(x, codes, scales, H, workspace, what):
    """One query row for H heads whose logits are x (sums of three bf16 at most), over tokens whose 512 codes
    are all codes[t]; returns the output as one number, and lse, of heads that are all alike."""
    n, B = len(x), 128
    pages = -(-n // B)
    cache = bfp8.latent_cache_buffers(pages, B, dev())
    cache[0].fill_(0x7F)
    cache[1].fill_(float("nan"))
    cache[2].fill_(float("nan"))
    cache[0].flatten(0, 1)[:n] = torch.from_numpy(np.asarray(codes, np.uint8)).to(dev())[:, None]
    cache[1].flatten()[:n] = torch.from_numpy(np.asarray(scales, np.float32)).to(dev())
    cache[2].flatten(0, 1)[:n] = 0
    left = torch.from_numpy(np.asarray(x, np.float64))
    for d in range(3):
        part = left.bfloat16()
        cache[2].flatten(0, 1)[:n, d] = part.to(dev())
        left = left - part.double()
    assert (left == 0).all()
    ql = torch.zeros(1, H, 512, dtype=torch.bfloat16, device=dev())
    qr = torch.zeros(1, H, 64, dtype=torch.bfloat16, device=dev())
    qr[..., :3] = 1
    out, lse = torch.empty_like(ql), torch.empty(1, H, device=dev())
    ws = bfp8.attn_latent_workspace(1, 1, H, dev()) if workspace else None
    announce(f"latent weights {what} n={n} H={H} ws={workspace}")
    bfp8.bfp8_attn_latent(ql, qr, *cache, i32([range(pages)]), i32([0, 1]), i32([n]), 1, 1.0, out, lse, ws)
    torch.cuda.synchronize()
    assert (out == out[0, 0, 0]).all() and (lse == lse[0, 0]).all()
    return float(out[0, 0, 0]), float(lse[0, 0])


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("top", [16.0, 16.75, 17.25])
def test_lse_of_one_token_above_a_long_tail(H, workspace, top):
    """131071 tokens at 2^-23 to 2^-24.9 of the largest.  The fp32 exponent and its power are off by 2^-22 of
    their size, top log2 e and one, together, the logarithm by 2^-23 of the result; 2048 tiles' sums are added
    one after another, each rounded by 2^-25 at most of a sum that is between 1/2 and 1: 2^-13 of it."""
    n = 131072
    x = np.zeros(n)
    x[70] = top
    _, lse = attend(x, [ONE] * n, [1.0] * n, H, workspace, f"norm, top {top}")
    want = top + np.log1p((n - 1) * np.exp(-top))
    bound = 2.0 ** -22 * (top * 1.5 + 1) + 2.0 ** -23 * want + 2.0 ** -13
    announce(f"lse {lse:.8g} want {want:.8g} bound {bound:.3g}")
    assert abs(lse - want) <= bound


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("exponent", [23, 24, 25, 26, 27, 28, 30, 40, 100])
def test_far_logits_that_grow(H, exponent):
    """Logits whose steps are 1 and more: neighbours are 2^16 and more apart, whatever the reference is rounded
    to.  All values are 1, so the output is 1 but for its own rounding, and lse off by the rounding of the
    logits' product and power, 2^-22 of their size."""
    rng = np.random.default_rng(exponent)
    step = 2.0 ** (exponent - 23)                           # fp32's there
    for sign in (1, -1):
        for _ in range(4):
            # a few steps up from tile to tile, and within one
            x = sign * 2.0 ** exponent + step * (np.repeat(np.cumsum(rng.integers(0, 4, 10)), 64) + rng.integers(0, 3, 640))
            x = x[:rng.integers(1, 640)]
            out, lse = attend(x, [ONE] * len(x), [1.0] * len(x), H, False, f"far {sign} 2^{exponent}")
            assert out == 1.0
            assert abs(lse - x.max()) <= 2.0 ** -22 * 1.5 * np.abs(x).max() + np.log(len(x))


def check(x, codes, scales, H, workspace, what):
    """Against 64 bits.  Counted: the output's rounding, 2^-8 of it; a weight's rounding to fp16, 2^-11 of
    it; a logit's x log2 e + e_t and its power in fp32, 2^-22 of their size and 2^-22; and three halves of
    fp16's last step, 2^-24, below its normal range (a weight's rounding, and twice when two halves of a
    tile are brought to one reference), where the largest weight is 2^6 or more: 2^-29 of the largest
    contribution for a token's code."""
    x, v, s = np.asarray(x, np.float64), VALUES[np.asarray(codes)], np.asarray(scales, np.float64)
    p = np.exp(x - x.max())
    norm = p.sum()
    want, want_lse = (p * v * s).sum() / norm, x.max() + np.log(norm)
    slack = 2.0 ** -22 * (1.5 * np.abs(x).max() + 33)
    bound = 2.0 ** -8 * abs(want) + (2.0 ** -11 + 2 * slack) * (p * np.abs(v) * s).sum() / norm + \
        2.0 ** -29 * (p * s).max() * np.abs(v).sum() / norm
    out, lse = attend(x, codes, scales, H, workspace, what)
    announce(f"got {out:.6g} want {want:.6g} bound {bound:.3g}, lse {lse:.7g} want {want_lse:.7g}")
    assert abs(out - want) <= bound, (out, want, bound)
    # a sum of n fp32 in chains of n / 32 and less, and the logarithm
    assert abs(lse - want_lse) <= slack + 2.0 ** -21 * (1 + abs(want_lse)) + 2.0 ** -24 * np.sqrt(len(x))


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("workspace", [False, True])
def test_one_token_above_a_long_tail(H, workspace):
    """131071 tokens at 2^-24.2 of the largest hold 0.7 % of the sum."""
    n = 131072
    x = np.zeros(n)
    x[70] = 16.75
    check(x, [ONE] * n, [1.0] * n, H, workspace, "tail")


@pytest.mark.parametrize("H", [16, 64])
def test_a_tail_of_many_sizes(H):
    """Weights from 2^-20 to 2^-27 of the largest, values of one sign."""
    rng = np.random.default_rng(71)
    n = 100003
    x = rng.integers(-150, -110, n) / 8.0
    x[n // 2] = 0
    check(x, rng.integers(ONE, MOST, n), 2.0 ** rng.integers(-1, 2, n), H, False, "sizes")


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("leap", [5.5, 15.5, 16.5, 18.5, 22.0, 26.0, 31.0])
@pytest.mark.parametrize("tall", [0, 1])
def test_one_half_of_a_tile_leaps(H, leap, tall):
    """A tile's half leaps up; the other half's tokens, 2^7.94 above the reference so far, keep their
    share of a sum in which their values are 448 times the tallest token's."""
    x = np.zeros(192)
    half = np.arange(64, 128) if tall else np.arange(64, 128)[::-1]
    x[half[:32]] = 5.5
    x[half[63]] = leap
    codes = np.full(192, MOST)
    codes[half[63]] = ONE
    check(x, codes, np.ones(192), H, False, f"leap {leap}")


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("n", [1, 2, 63, 200, 9000])
def test_a_cache_of_zeros(H, workspace, n):
    """Scales of zero: values of nothing, and every token counts."""
    out, lse = attend(np.zeros(n), [0] * n, [0.0] * n, H, workspace, "zeros")
    assert out == 0 and abs(lse - np.log(n)) <= 2.0 ** -20 * (1 + np.log(n))


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("exponent", [-22, 0, 8, 30])
def test_zeros_beside_others(H, exponent):
    """Tokens of scale zero next to one of another scale: they halve, or thin, its share."""
    for n in (2, 64, 300):
        scales = np.zeros(n)
        scales[n - 1] = 2.0 ** exponent
        codes = np.full(n, 0)
        codes[n - 1] = ONE
        check(np.zeros(n), codes, scales, H, False, f"2^{exponent} beside zeros")
