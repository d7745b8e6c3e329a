"""The C ABI of rotary positions and of the latent cache without a GPU (refusals, before any HIP call), the
frequencies, and the plain implementations the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
import latent_reference as ref
from block_scaled_fp8_04_amd import _lib
from kv_reference import VALUES, encode, scale_of

FAKE = ctypes.c_void_p(0x10000)            # aligned, never dereferenced: every call is rejected
ODD = ctypes.c_void_p(0x10002)
ODDER = ctypes.c_void_p(0x10001)
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return _lib.library()


def rope(lib, **kw):
    a = dict(x=FAKE, xt=1024, xh=64, pos=FAKE, freq=FAKE, out=FAKE, ot=1024, oh=64, T=4, H=16, D=64, il=1, amp=1.0)
    a.update(kw)
    return lib.bfp8_rope(a["x"], a["xt"], a["xh"], a["pos"], a["freq"], a["out"], a["ot"], a["oh"], a["T"], a["H"],
                         a["D"], a["il"], a["amp"], None)


def test_rope_refusals(lib):
    for amp in (math.nan, math.inf):
        assert rope(lib, amp=amp) == _lib.BFP8_ERR_ARG
    for kw in (dict(T=-1), dict(T=1 << 24), dict(H=0), dict(H=65536), dict(D=0), dict(D=7), dict(D=-2), dict(D=1026),
               dict(xt=-1), dict(xh=-1), dict(ot=-1), dict(oh=-1)):
        assert rope(lib, **kw) == _lib.BFP8_ERR_SHAPE, kw
    for name in ("x", "pos", "freq", "out"):
        assert rope(lib, **{name: None}) == _lib.BFP8_ERR_NULL, name
    for name in ("pos", "freq"):
        assert rope(lib, **{name: ODD}) == _lib.BFP8_ERR_ALIGN, name
    for name in ("x", "out"):
        assert rope(lib, **{name: ODDER}) == _lib.BFP8_ERR_ALIGN, name
    assert rope(lib, T=0, x=None) == _lib.BFP8_OK


def append(lib, **kw):
    a = dict(kv=FAKE, kt=576, w=FAKE, eps=1e-6, slots=FAKE, pos=FAKE, freq=FAKE, il=1, amp=1.0, T=4, codes=FAKE,
             scales=FAKE, rope=FAKE, P=8, B=64)
    a.update(kw)
    return lib.bfp8_latent_append(a["kv"], a["kt"], a["w"], a["eps"], a["slots"], a["pos"], a["freq"], a["il"],
                                  a["amp"], a["T"], a["codes"], a["scales"], a["rope"], a["P"], a["B"], None)


def test_append_refusals(lib):
    for kw in (dict(B=16), dict(B=48), dict(B=0), dict(B=256), dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf),
               dict(amp=math.inf)):
        assert append(lib, **kw) == _lib.BFP8_ERR_ARG, kw
    for kw in (dict(T=-1), dict(T=1 << 26), dict(kt=-1), dict(P=-1), dict(P=BIG // 64)):
        assert append(lib, **kw) == _lib.BFP8_ERR_SHAPE, kw
    for name in ("kv", "slots", "pos", "freq", "codes", "scales", "rope"):
        assert append(lib, **{name: None}) == _lib.BFP8_ERR_NULL, name
    for name in ("slots", "pos", "freq", "codes", "scales", "rope"):
        assert append(lib, **{name: ODD}) == _lib.BFP8_ERR_ALIGN, name
    for name in ("kv", "w"):
        assert append(lib, **{name: ODDER}) == _lib.BFP8_ERR_ALIGN, name
    assert append(lib, T=0, kv=None) == _lib.BFP8_OK and append(lib, P=0, codes=None) == _lib.BFP8_OK


def gather(lib, **kw):
    a = dict(codes=FAKE, scales=FAKE, rope=FAKE, P=8, B=64, table=FAKE, W=4, off=FAKE, starts=None, R=2, N=10, lat=FAKE,
             lt=512, out=FAKE, ot=64)
    a.update(kw)
    return lib.bfp8_latent_gather(a["codes"], a["scales"], a["rope"], a["P"], a["B"], a["table"], a["W"], a["off"],
                                  a["starts"], a["R"], a["N"], a["lat"], a["lt"], a["out"], a["ot"], None)


def test_gather_refusals(lib):
    assert gather(lib, B=16) == _lib.BFP8_ERR_ARG
    for kw in (dict(R=-1), dict(N=-1), dict(N=1 << 30), dict(P=-1), dict(P=BIG // 64), dict(W=-1), dict(W=BIG // 64),
               dict(lt=-8), dict(ot=-8)):
        assert gather(lib, **kw) == _lib.BFP8_ERR_SHAPE, kw
    assert gather(lib, R=bfp8.KV_MAX_REQUESTS + 1) == _lib.BFP8_ERR_GROUPS
    for name in ("codes", "scales", "rope", "table", "off", "lat", "out"):
        assert gather(lib, **{name: None}) == _lib.BFP8_ERR_NULL, name
    for name in ("codes", "scales", "rope", "table", "off", "starts", "lat", "out"):
        assert gather(lib, **{name: ODD}) == _lib.BFP8_ERR_ALIGN, name
    assert gather(lib, lt=513) == gather(lib, ot=68) == _lib.BFP8_ERR_ALIGN
    for kw in (dict(R=0), dict(N=0), dict(P=0), dict(W=0)):
        assert gather(lib, codes=None, **kw) == _lib.BFP8_OK


def attn(lib, **kw):
    a = dict(ql=FAKE, qlt=8192, qlh=512, qr=FAKE, qrt=1024, qrh=64, codes=FAKE, scales=FAKE, rope=FAKE, P=8, B=64,
             table=FAKE, W=4, off=FAKE, kv=FAKE, R=2, T=2, max_new=1, H=16, scale=0.1, out=FAKE, ot=8192, oh=512,
             lse=None, ws=None, wsb=0)
    a.update(kw)
    return lib.bfp8_attn_latent(a["ql"], a["qlt"], a["qlh"], a["qr"], a["qrt"], a["qrh"], a["codes"], a["scales"],
                                a["rope"], a["P"], a["B"], a["table"], a["W"], a["off"], a["kv"], a["R"], a["T"],
                                a["max_new"], a["H"], a["scale"], a["out"], a["ot"], a["oh"], a["lse"], a["ws"],
                                a["wsb"], None)


def test_attention_refusals(lib):
    assert attn(lib, B=48) == _lib.BFP8_ERR_ARG
    for s in (math.nan, math.inf, -math.inf):
        assert attn(lib, scale=s) == _lib.BFP8_ERR_ARG
    for kw in (dict(R=-1), dict(T=-1), dict(T=(1 << 29) // 16), dict(max_new=-1), dict(max_new=0),
               dict(max_new=BIG // 16), dict(H=0), dict(H=65536), dict(qlt=-1), dict(qlh=-1), dict(qrt=-1),
               dict(qrh=-1), dict(ot=-8), dict(oh=-8), dict(P=-1), dict(P=BIG // 64), dict(W=-1), dict(W=BIG // 64)):
        assert attn(lib, **kw) == _lib.BFP8_ERR_SHAPE, kw
    assert attn(lib, R=bfp8.KV_MAX_REQUESTS + 1) == _lib.BFP8_ERR_GROUPS
    for name in ("ql", "qr", "codes", "scales", "rope", "table", "off", "kv", "out"):
        assert attn(lib, **{name: None}) == _lib.BFP8_ERR_NULL, name
    for name in ("codes", "scales", "rope", "table", "off", "kv", "out", "lse", "ws"):
        assert attn(lib, **{name: ODD}) == _lib.BFP8_ERR_ALIGN, name
    assert attn(lib, ql=ODDER) == attn(lib, qr=ODDER) == _lib.BFP8_ERR_ALIGN
    assert attn(lib, ot=8190) == attn(lib, oh=516) == _lib.BFP8_ERR_ALIGN
    assert attn(lib, R=0, ql=None) == attn(lib, T=0, ql=None) == _lib.BFP8_OK


def test_attention_workspace(lib):
    size = bfp8.bfp8_attn_latent_workspace_size
    for R, mn, H in ((1, 1, 16), (64, 1, 128), (3, 4, 20), (5, 60, 64)):
        n = size(R, mn, H)
        assert n > 0 and n % 16 == 0
        assert attn(lib, R=R, T=R * mn, max_new=mn, H=H, ws=FAKE, wsb=n - 16) == _lib.BFP8_ERR_WORKSPACE
    # as many items as fill the chip are not split
    assert size(4096, 1, 16) == size(8, 2048, 128) == 0
    assert size(0, 1, 16) == size(1, 0, 16) == size(1, 1, 0) == size(5000, 1, 16) == size(-1, 1, 16) == 0
    assert size(1, BIG, 16) == size(1, 1, 70000) == 0


def test_binding_refusals():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    f = torch.ones(32)
    cache = bfp8.latent_cache_buffers(3, 64, "cpu")
    for call in (lambda: bfp8.bfp8_rope(x, i, f, x),
                 lambda: bfp8.bfp8_latent_append(torch.zeros(4, 576, dtype=torch.bfloat16), i, i, f, *cache),
                 lambda: bfp8.bfp8_latent_gather(*cache, torch.zeros(3, 2, dtype=torch.int32), i, x[:, 0], x[:, 0]),
                 lambda: bfp8.bfp8_attn_latent(torch.zeros(4, 2, 512, dtype=torch.bfloat16), x, *cache,
                                               torch.zeros(3, 2, dtype=torch.int32), i, i[:3], 1, 1.0, x)):
        with pytest.raises(ValueError):
            call()
    for bad in ((cache[0].float(), cache[1], cache[2]), (cache[0], cache[1].double(), cache[2]),
                (cache[0][..., :500], cache[1], cache[2]), (cache[0], cache[1], cache[2].float())):
        with pytest.raises((ValueError, TypeError)):
            _lib._latent_shape(torch.device("cpu"), *bad)
    for kw in (dict(dim=7), dict(dim=0), dict(dim=64, factor=0.5), dict(dim=64, base=1.0), dict(dim=64, slow=40.0)):
        with pytest.raises(ValueError):
            bfp8.rope_frequencies(device="cpu", **kw)


def test_frequencies():
    f, a = bfp8.rope_frequencies(64, device="cpu")
    assert a == 1.0 and np.allclose(f.numpy(), 1e4 ** (-np.arange(32) / 32), rtol=2.0 ** -23)
    g, a = bfp8.rope_frequencies(64, factor=40.0, device="cpu")
    assert a == 0.1 * math.log(40) + 1
    turns = f.double().numpy() * 4096 / (2 * math.pi)          # within the trained length
    ratio = (g.double() / f.double()).numpy()
    assert (ratio[turns > 40] == 1).all() and np.allclose(ratio[turns < 0.8], 1 / 40, rtol=1e-6)
    assert (np.diff(ratio) <= 1e-6).all()


def test_stream_of_the_allocating_calls(monkeypatch):
    """New arrays are made on the stream that the kernels take."""
    import contextlib
    from types import SimpleNamespace
    gpu = SimpleNamespace(type="cuda", index=0)

    class Like:
        def __init__(self, *shape):
            self.shape, self.device = shape, gpu
    current, made, launched = ["current"], [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: h)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, lambda *a, **kw: made.append(current[-1]) or Like(1))
    for entry in ("bfp8_rope", "bfp8_latent_gather", "bfp8_attn_latent"):
        monkeypatch.setattr(_lib, entry, lambda *a, **kw: launched.append(a[-1]))
    monkeypatch.setattr(_lib, "bfp8_attn_latent_workspace_size", lambda *a: 64)
    plan = SimpleNamespace(q_offsets=0, kv_lens=0)
    cache = (Like(8, 64, 512), Like(8, 64), Like(8, 64, 64))
    bfp8.rope(Like(4, 2, 64), 0, 0, stream=0x1234)
    bfp8.latent_gather(cache, Like(4, 3), 0, 9, stream=0x1234)
    bfp8.attn_latent(Like(4, 16, 512), 0, cache, Like(4, 3), plan, 1, 1.0, stream=0x1234)
    assert len(made) == 5 and set(made) == {0x1234} and launched == [0x1234] * 3 and current == ["current"]


def test_reference_attention_is_softmax():
    """Against torch's softmax in 64 bits on one dense request."""
    rng = np.random.default_rng(1)
    B, n, H = 32, 70, 2
    c = rng.standard_normal((n, 512))
    codes, scales = np.zeros((4, B, 512), np.uint8), np.ones((4, B), np.float32)
    rope = rng.standard_normal((4, B, 64))
    table = np.array([[2, 0, 3]])
    dense, k = np.zeros((n, 512)), np.zeros((n, 64))
    for t in range(n):
        at = table[0, t // B], t % B
        scales[at] = scale_of(np.abs(c[t]).max())
        codes[at] = encode(c[t] / scales[at])
        dense[t], k[t] = VALUES[codes[at]] * scales[at], rope[at]
    assert np.abs(dense - c).max() < 2.0 ** -3
    ql, qr = rng.standard_normal((5, H, 512)), rng.standard_normal((5, H, 64))
    out, lse, bound, _ = ref.attention(ql, qr, (codes, scales, rope), table, [0, 5], [n], 0.1)
    z = torch.from_numpy(np.einsum("thd,nd->thn", ql, dense) + np.einsum("thd,nd->thn", qr, k)) * 0.1
    z.masked_fill_(torch.arange(n)[None, None, :] > (n - 5 + torch.arange(5))[:, None, None], -math.inf)
    want = torch.einsum("thn,nd->thd", z.softmax(2), torch.from_numpy(dense))
    assert np.allclose(out, want.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(z, 2).numpy(), rtol=1e-12)
    assert (bound > 0).all() and bound.max() < 0.05


def test_reference_rotation():
    """As multiplication by e^(i angle); turning back undoes it."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 3, 16))
    f = rng.random(8)
    pos = rng.integers(0, 50, 6)
    il = ref.rotate(x, pos, f, True, 1.0)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * pos[:, None, None] * f)
    assert np.allclose(il[..., 0::2], z.real) and np.allclose(il[..., 1::2], z.imag)
    half = ref.rotate(np.concatenate([x[..., 0::2], x[..., 1::2]], -1), pos, f, False, 1.0)
    assert np.allclose(half, np.concatenate([il[..., 0::2], il[..., 1::2]], -1))
    assert np.allclose(ref.rotate(il, pos, -f, True, 1.0), x)
