"""A long chunk of new tokens beside requests that decode one token each, long and short: the launch without
parts, whose row tiles are 64 rows for all of them."""
import numpy as np
import pytest

import block_scaled_fp8_04_amd as bfp8
from kv_helpers import offsets
from latent_helpers import LatentCache, attend, check, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("where", [0, 3, 7])
def test_a_chunk_beside_long_requests(where):
    rng = np.random.default_rng(81 + where)
    H, new, kv = 16, [1] * 8, [9000, 1, 64, 700, 65, 4097, 2, 129]
    new[where], kv[where] = 520, 600
    assert bfp8.bfp8_attn_latent_workspace_size(8, 520, H) == 0
    cache = LatentCache(rng, kv, 64)
    ql, qr = queries(rng, sum(new), H)
    q_off = offsets(new)
    out, lse = attend(ql, qr, cache.gpu(), cache.table, q_off, kv, 520, 192 ** -0.5)
    check(out, lse, ql, qr, cache.arrays, cache.table, q_off, kv, 192 ** -0.5, f"chunk at {where}")
