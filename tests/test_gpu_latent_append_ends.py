"""bfp8_latent_append where squares leave the range of fp32, and for tokens without a position."""
import numpy as np
import pytest
import torch

from kv_helpers import bf16
from test_gpu_latent_cache import check_append, freq, pool, run_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-6, 1e-30, 0.0])
def test_norms_of_the_largest_and_smallest_rows(eps):
    """Rows whose squares, or their sum, pass fp32 at either end are normed as the formula says; the error
    of the root's argument in them is that of an ordinary row, so check_append's bounds hold."""
    rng = np.random.default_rng(61)
    kv = rng.standard_normal((14, 576))
    for t, size in enumerate([2.0 ** 124, 2.0 ** 100, 2.0 ** 63, 2.0 ** 59, 2.0 ** -60, 2.0 ** -64, 2.0 ** -75, 2.0 ** -110]):
        kv[t, :512] *= size
    kv[8, 3] = 3.0e38
    kv[9, 500] = -1e30
    kv[10, :512], kv[10, 9] = 0, 2.0 ** 120
    kv[11, :512], kv[11, 9] = 0, 2.0 ** -70
    kv[12, :512] = 2.0 ** 61                                # no square passes fp32, their sum does
    kv = bf16(kv)
    weight = bf16(1 + 0.2 * rng.standard_normal(512))
    cache = pool(1, 32, rng)
    before = [x.clone() for x in cache]
    slots, pos = rng.permutation(32)[:14], rng.integers(0, 9999, 14)
    run_append(kv, slots, pos, freq(64), cache, norm_weight=weight, eps=eps)
    assert torch.isfinite(cache[1][0, slots]).all()
    check_append(kv, slots, pos, freq(64), before, cache, True, 1.0, weight, eps)


def test_rows_that_are_not_finite_stay_poisoned():
    rng = np.random.default_rng(62)
    for at, value in ((0, np.inf), (511, -np.inf), (7, np.nan)):
        kv = rng.standard_normal((3, 576))
        kv[1, at] = value
        kv[2, :512] *= 2.0 ** 100
        kv, weight = bf16(kv), bf16(np.ones(512))
        for eps in (1e-6, 0.0):
            cache = pool(1, 32, rng)
            before = [x.clone() for x in cache]
            run_append(kv, [4, 5, 6], [1, 2, 3], freq(64), cache, norm_weight=weight, eps=eps)
            assert torch.isnan(cache[1][0, 4:7]).tolist() == [False, True, False]
            check_append(kv, np.array([4, 5, 6]), np.array([1, 2, 3]), freq(64), before, cache, True, 1.0, weight, eps)
    # nothing but zeros, and no eps: 0 / 0
    cache = pool(1, 32, rng)
    kv = torch.zeros_like(kv)
    run_append(kv, [1, 2, 3], [0, 0, 0], freq(64), cache, norm_weight=weight, eps=0.0)
    assert torch.isnan(cache[1][0, 1:4]).all() and (cache[0][0, 1:4] == 0).all()


@pytest.mark.parametrize("T", [1, 2, 9])
@pytest.mark.parametrize("interleaved", [True, False])
def test_tokens_without_a_position_are_skipped(T, interleaved):
    """As by bfp8_rope; their slots keep what they hold, and their neighbours are stored."""
    rng = np.random.default_rng(63 + T)
    for gone in range(min(T, 3)):
        kv = bf16(rng.standard_normal((T, 576)))
        slots, pos = rng.permutation(32)[:T], rng.integers(0, 9999, T)
        pos[gone] = (-1, -2 ** 31, -77)[gone]
        cache = pool(1, 32, rng)
        before = [x.clone() for x in cache]
        run_append(kv, slots, pos, freq(64), cache, interleaved=interleaved)
        kept = np.where(pos < 0, -1, slots)
        check_append(kv, kept, pos, freq(64), before, cache, interleaved, 1.0, None, 1e-6)
