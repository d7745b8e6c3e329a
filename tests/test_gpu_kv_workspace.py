"""Attention of sizes whose workspace is empty takes any workspace, and none, alike."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
from gpu_helpers import announce, dev
from kv_helpers import Cache, bf16, check_attention, f64, i32, offsets

pytestmark = pytest.mark.gpu


def test_an_empty_workspace():
    rng = np.random.default_rng(1)
    H, new, kv = 32, [70, 1, 0, 66, 3, 1, 1, 9], [90, 300, 0, 66, 40, 1, 129, 200]
    cache = Cache(rng, kv, H, 64, 128, 128)
    q_off = offsets(new)
    T = int(q_off[-1])
    q = bf16(rng.standard_normal((T, H, 128)))
    assert bfp8.bfp8_attn_paged_workspace_size(len(kv), max(new), H, H, 128, 128) == 0
    args = (q, *cache.gpu(), i32(cache.table), i32(q_off), i32(kv), i32(offsets([-(-n // 128) for n in kv])),
            max(new), 0.1)
    announce("attention with an empty workspace")
    outs = []
    for ws in (None, torch.zeros(0, dtype=torch.uint8, device=dev()), torch.zeros(16, dtype=torch.uint8, device=dev())):
        out = torch.empty(T, H, 128, dtype=torch.bfloat16, device=dev())
        lse = torch.empty(T, H, device=dev())
        bfp8.bfp8_attn_paged(*args, out, lse, ws)
        torch.cuda.synchronize()
        outs.append((out, lse))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    check_attention(*outs[0], f64(q), cache.arrays, cache.table, q_off, kv, 0.1, "empty workspace")
