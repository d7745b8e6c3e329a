"""bfp8_latent_gather behind rows that belong to no request: the first request's rows do not begin at 0."""
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
from gpu_helpers import dev
from kv_helpers import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [1, 5, 8, 70, 40001])
@pytest.mark.parametrize("start", [0, 3, 100])
def test_rows_before_the_first_request_are_left_alone(first, start):
    """40001 rows: the kernel for many rows as well."""
    torch.manual_seed(first + start)
    B, counts, starts = 64, [3, 0, 40], [start, 7, 2 * start]
    codes = torch.randint(0, 127, (12, B, 512), dtype=torch.uint8, device=dev())
    scales = torch.randint(-9, 9, (12, B), device=dev()).float().exp2()
    keys = torch.randn(12, B, 64, device=dev()).bfloat16()
    table = torch.randperm(12, device=dev()).to(torch.int32).view(3, 4)
    ends = [first, first + 3, first + 3, first + 43]
    latent = torch.full((first + 50, 512), -7.0, dtype=torch.bfloat16, device=dev())
    rope = torch.full((first + 50, 64), -7.0, dtype=torch.bfloat16, device=dev())
    bfp8.bfp8_latent_gather(codes, scales, keys, table, i32(ends), latent, rope, i32(starts))
    for r, n in enumerate(counts):
        pages = table[r].long()
        values = (codes[pages].view(torch.float8_e4m3fn).float() * scales[pages][..., None]).flatten(0, 1)
        at = slice(starts[r], starts[r] + n)
        assert torch.equal(latent[ends[r]:ends[r + 1]].float(), values[at])
        assert torch.equal(rope[ends[r]:ends[r + 1]], keys[pages].flatten(0, 1)[at])
    for rows in (latent, rope):
        assert (rows[:first] == -7).all(), "rows in front of the first request"
        assert (rows[first + 43:] == -7).all(), "rows behind the last request"
    got = bfp8.latent_gather((codes, scales, keys), table, i32(ends), first + 50, i32(starts))
    assert (got[0][:first] == 0).all() and (got[1][:first] == 0).all()
    assert torch.equal(got[0][first:first + 43], latent[first:first + 43])
