"""Exact sizes of attention's workspace: partial results of 16 columns, two a workgroup, where columns
are few; parts of 128 columns where they are many; nothing where no launch of these sizes is split."""
import pytest

import block_scaled_fp8_04_amd as bfp8

size = bfp8.bfp8_attn_paged_workspace_size


@pytest.mark.parametrize("R,max_new,hq,hkv,dk,groups", [
    (1, 1, 16, 4, 128, 512), (64, 1, 64, 8, 128, 512), (4096, 64, 32, 32, 192, 512),      # 64 columns at most
    (3, 4, 12, 4, 64, 1024), (64, 8, 64, 8, 64, 1024)])
def test_few_columns(R, max_new, hq, hkv, dk, groups):
    dv = min(dk, 128)
    assert size(R, max_new, hq, hkv, dk, dv) == groups * 2 * 16 * (dv + 2) * 4


@pytest.mark.parametrize("R,max_new,hq,hkv,parts", [
    (1, 100, 4, 1, 4 * 16),             # 400 columns: four blocks of 128, sixteen parts each
    (1, 2048, 32, 8, 512),              # 65 blocks of eight KV heads: as many parts as run at once
    (255, 100, 1, 1, 512)])             # one token a request: 255 blocks, two parts each
def test_many_columns(R, max_new, hq, hkv, parts):
    assert size(R, max_new, hq, hkv, 128, 128) == parts * 128 * 130 * 4


@pytest.mark.parametrize("R,max_new,hq,hkv", [
    (256, 100, 1, 1), (8, 500, 32, 32), (32, 65, 8, 8), (64, 512, 64, 8), (4096, 2048, 128, 128),
    (1, 1, 32768, 256)])
def test_never_split(R, max_new, hq, hkv):
    """A block for every request and KV head already takes every CU."""
    assert size(R, max_new, hq, hkv, 128, 128) == 0
    assert size(R, max_new, hq, hkv, 64, 64) == 0
