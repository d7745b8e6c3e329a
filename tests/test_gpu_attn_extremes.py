"""Keys and values near the largest bf16 numbers: 248 * 2^120 and above round to the code of 256 at a
scale of 2^120.  Rows that do not see such a token are what they are without it, the others follow the
definition."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
import kv_terms
from gpu_helpers import announce, dev
from kv_helpers import attend, bf16, f64

pytestmark = pytest.mark.gpu

LARGEST = 255 * 2.0 ** 120                                  # of bf16


def cached(k, v, B):
    """The keys and values [n, 1, D] appended to a cache whose pages lie backwards in the pool."""
    n, dk, dv = len(k), k.shape[2], v.shape[2]
    P = -(-n // B)
    table = np.arange(P)[::-1].reshape(1, P).astype(np.int32)
    cache = bfp8.kv_cache_buffers(P, 1, B, dk, dv, dev())
    slots = [int(table[0, i // B]) * B + i % B for i in range(n)]
    bfp8.bfp8_kv_append(bf16(k), bf16(v), torch.tensor(slots, dtype=torch.int32, device=dev()), *cache)
    return cache, table


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("size", [1.0, 248 / 255, 247 / 255])
@pytest.mark.parametrize("new,at", [(4, 39), (4, 38), (40, 39), (40, 7)])
def test_the_largest_values(dk, dv, size, new, at):
    rng = np.random.default_rng(dk + at)
    n, G, B = 40, 4, 32
    k, v = rng.standard_normal((n, 1, dk)), rng.standard_normal((n, 1, dv))
    v[at, 0, 5], v[at, 0, 20] = size * LARGEST, -size * LARGEST
    q = bf16(rng.standard_normal((new, G, dk)))
    off = np.array([0, new])
    cache, table = cached(k, v, B)
    # the page's scale is the large elements': without them the same codes at the same scale
    calm = [x.clone() for x in cache]
    calm[2][int(table[0, at // B]), 0, :, at % B] = 0
    blind = max(at - (n - new), 0)                           # rows that do not see the token
    for ws in (True, False):
        announce(f"largest values {dk}/{dv} size={size:.3f} new={new} at={at} workspace={ws}")
        out, lse = attend(q, cache, table, off, [n], new, dk ** -0.5, ws)
        want, _ = attend(q, calm, table, off, [n], new, dk ** -0.5, ws)
        assert torch.isfinite(out[:blind].float()).all(), "a row that does not see the token"
        assert torch.equal(out[:blind], want[:blind])
        # no weight of this row passes 0.9, so its exact result is a bf16 number
        kv_terms.check(f64(out), f64(lse), f64(q), [x.cpu().numpy() for x in cache], table, off, [n], dk ** -0.5,
                       "rows that see the token")


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("new", [4, 40])
def test_the_largest_keys(dk, dv, new):
    """One token's key has the largest element: queries with 0 there ignore it, a positive one picks the
    token, a negative one passes it over."""
    rng = np.random.default_rng(dk + new)
    n, G, B, at = 80, 4, 32, 33
    k, v = rng.standard_normal((n, 1, dk)), rng.standard_normal((n, 1, dv))
    k[at, 0] = 0.0
    k[at, 0, 5] = LARGEST
    q = rng.standard_normal((new, G, dk))
    q[:, 0, 5], q[:, 1, 5], q[:, 2, 5], q[:, 3, 5] = 0.0, 2.0 ** -10, -2.0 ** -10, 2.0 ** -100
    q = bf16(q)
    off = np.array([0, new])
    cache, table = cached(k, v, B)
    arrays = [x.cpu().numpy() for x in cache]
    # the largest element sets its page's scale: all other keys of the page are zeros
    assert np.count_nonzero(arrays[0][table[0, 1]] & 0x7F) == 1
    for ws in (True, False):
        announce(f"largest keys {dk}/{dv} new={new} workspace={ws}")
        out, lse = attend(q, cache, table, off, [n], new, dk ** -0.5, ws)
        got = f64(out)
        want, want_lse, weight, slack = kv_terms.attention(f64(q), *arrays, table, off, [n], dk ** -0.5)
        picked = want_lse > 1000.0
        assert picked[:, 1].all() and not picked[:, [0, 2]].any()
        assert np.isfinite(got).all()
        assert np.array_equal(got[picked], want[picked])     # the token's value, a bf16 number
        # the logits that count are those of the other tokens, a few units: what the large one's adds
        # to the bound of the sums does not apply
        few = np.full_like(slack, 2.0 ** -20 * 64)
        rest = ~picked
        err = np.abs(got - want)[rest] / kv_terms.bound(want, weight, few)[rest]
        assert err.max() <= 1.0, f"worst err/bound {err.max():.3f}"
