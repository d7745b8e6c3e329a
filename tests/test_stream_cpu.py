"""The allocating calls on a stream that is named: every array they make or fill belongs to it.

A fill that is queued on another stream than the kernels may land behind them, and memory that is
handed back to another stream's pool may be written again while they read it."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
from block_scaled_fp8_04_amd import _lib

# a device that only names itself: the library's calls are recorded, not made
GPU = SimpleNamespace(type="cuda", index=0)


class Like:
    """A GPU tensor's shape and device."""

    def __init__(self, *shape):
        self.shape, self.device = tuple(shape), GPU

    def __getitem__(self, _):
        return self


def calls():
    x, s = Like(256, 256), Like(256, 2)
    w, ws = Like(256, 256), Like(2, 2)
    moe, plan = Like(4, 2), SimpleNamespace(q_offsets=0, kv_lens=0, tile_offsets=0)
    cache = (Like(8, 2, 64, 128), Like(8, 2), Like(8, 2, 128, 64), Like(8, 2))
    return {
        "act_quant": (x,), "act_quant_ue8m0": (x,), "weight_dequant": (w, ws), "gemm": (x, s, w, ws),
        "gemm_ue8m0": (x, s, w, ws), "gemm_grouped": (x, s, Like(2, 256, 256), Like(2, 2, 2), Like(3)),
        "gemm_bf16": (x, w), "linear_bf16": (x, w, ws), "linear_fp8": (x, w, ws),
        "gemm_act_quant": (x, s, w, ws), "gemm_swiglu_act_quant": (x, s, w, ws),
        "moe_dispatch": (moe, 0, 4), "moe_combine": (x, moe, moe),
        "moe_experts_fp8": (Like(4, 256), moe, moe, Like(4, 256, 256), Like(4, 2, 2), 0),
        "kv_plan": (Like(4), Like(4), Like(9), Like(4, 3), 64, 16),
        "attn_paged": (Like(4, 4, 128), cache, Like(4, 3), plan, 1),
    }


@pytest.mark.parametrize("handle", [None, 0, 0x1234])
@pytest.mark.parametrize("name", sorted(calls()))
def test_arrays_belong_to_the_stream(name, handle, monkeypatch):
    current, made, launched = ["current"], [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def array(*shape, **kw):
        made.append(current[-1])
        return Like(*(shape[0] if isinstance(shape[0], (tuple, torch.Size)) else shape))

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: h)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    monkeypatch.setattr(torch, "empty", array)
    monkeypatch.setattr(torch, "zeros", array)
    for entry in dir(_lib):
        if entry.startswith("bfp8_") and not entry.endswith("_size"):
            monkeypatch.setattr(_lib, entry, lambda *a, **kw: launched.append(kw.get("stream", a[-1])))
    getattr(bfp8, name)(*calls()[name], stream=handle)
    assert current == ["current"]
    assert launched and all(s == handle for s in launched)
    assert made and set(made) == {"current" if handle is None else handle}
