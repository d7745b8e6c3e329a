"""Operators of attention over a shared latent: plain forms, the library's calls, and the cases to measure.

Keys and values of all heads come from one latent vector of 512 a token, next to 64 rotated dims that
all heads share.  The cache holds the latent in e4m3 with one power-of-two scale per token, and the
rotated key in bf16.

  rope           rotary positions of query heads: interleaved or half layout, a part of the head, any
                 table of frequencies (scaled ones for long contexts) and an amplitude
  latent_append  a projection's rows [T, 512 + 64] -> RMS norm of the latent, rotation of the key,
                 quantized into the slots of a paged cache
  latent_gather  cached tokens of each request back to bf16 rows (the expanded form's input)
  attn_latent    the absorbed form: softmax(scale (q_latent c^T + q_rope r^T)) c of each request's new
                 tokens over its pages, causal at the end of the request

`run` computes them in elementary torch operations in 32 bits (angles in 64), or (own) by the library's
calls.
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE = 512, 64
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-4
EPS = 1e-6


# ------------------------------------------------------------------------------- cases

def listed():
    def rope(name, T, heads, dim, first, rot, interleaved, far, scaled):
        return {"name": name, "op": "rope", "tokens": T, "heads": heads, "dim": dim, "first": first,
                "rot": rot, "interleaved": interleaved, "far": far, "scaled": scaled}

    def serve(name, op, R, ctx, new, page, heads=1, idle=0, lse=False, norm=False, interleaved=True):
        return {"name": name, "op": op, "requests": R, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
                "new_lo": new[0], "new_hi": new[1], "page": page, "heads": heads, "idle": idle,
                "lse": lse, "norm": norm, "interleaved": interleaved}
    return [
        # the rotated part of a decode step's queries, out of heads of 128 + 64
        rope("rope-decode", 64, 128, 192, 128, 64, True, 8192, False),
        # prompts of a model that rotates whole heads in halves, positions past the trained length
        rope("rope-prompts", 8192, 32, 128, 0, 128, False, 131072, True),
        # one token of each of 64 requests enters the cache: latency
        serve("append-decode", "append", 64, (1, 8192), (1, 1), 64, norm=True),
        # prompts of ragged lengths, keys rotated in halves
        serve("append-prompts", "append", 8, (0, 200), (1024, 4096), 64, norm=True, interleaved=False),
        # a few cached prefixes read back before their prompts' chunks
        serve("gather-prefix", "gather", 5, (30, 700), (0, 0), 32),
        # a long context read back to be expanded to full heads
        serve("gather-long", "gather", 3, (20000, 131072), (0, 0), 128),
        # a single user's next token on one of eight GPUs (16 heads): latency
        serve("attn-one", "attn", 1, (1030, 1030), (1, 1), 64, heads=16),
        # the ordinary decode step with all 128 heads on one GPU
        serve("attn-decode", "attn", 64, (512, 8192), (1, 1), 64, heads=128),
        # the same with the heads shared by eight GPUs: the cache's bytes count
        serve("attn-decode-16", "attn", 64, (512, 8192), (1, 1), 64, heads=16),
        # few requests, very long caches: work is split over tokens
        serve("attn-long", "attn", 2, (50000, 131072), (1, 1), 128, heads=128),
        # three drafted tokens per request to verify, an odd number of heads, short pages, idle slots
        serve("attn-draft", "attn", 24, (100, 6000), (3, 3), 32, heads=20, idle=8, lse=True),
        # a short chunk of new tokens for some requests next to single ones
        serve("attn-mixed", "attn", 12, (0, 3000), (1, 60), 64, heads=64, idle=6),
    ]


def _log_int(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 200)


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(["rope", "append", "gather", "attn", "attn", "attn"])
        if op == "rope":
            rot = 2 * rng.choice([16, 32, 32, 48, 64])
            part = rng.random() < 0.5
            first = 8 * rng.randint(0, 16) if part else 0
            c = {"op": op, "tokens": _log_int(rng, 1, 16384), "heads": _log_int(rng, 1, 128),
                 "dim": first + rot + (8 * rng.randint(0, 4) if part else 0), "first": first, "rot": rot,
                 "interleaved": rng.random() < 0.5, "far": _log_int(rng, 64, 500000),
                 "scaled": rng.random() < 0.5}
            if _cost(c) > 0.9 * top[op]:
                continue
            return c
        c = {"op": op, "requests": _log_int(rng, 1, 200), "page": rng.choice([32, 64, 128]), "heads": 1,
             "idle": rng.choice([0, 0, 5, 16]), "lse": False, "norm": False, "interleaved": True}
        c["ctx_hi"] = _log_int(rng, 1, 100000)
        c["ctx_lo"] = _log_int(rng, 1, c["ctx_hi"]) - 1
        c["new_lo"] = c["new_hi"] = 0 if op == "gather" else 1
        if op == "append":
            c["ctx_hi"] = min(c["ctx_hi"], 8192)
            c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])
            c["norm"], c["interleaved"] = rng.random() < 0.7, rng.random() < 0.5
            if rng.random() < 0.6:
                c["new_hi"] = _log_int(rng, 2, 8192)
                c["new_lo"] = _log_int(rng, 1, c["new_hi"])
        if op == "attn":
            c["heads"] = rng.choice([1, 5, 8, 16, 16, 20, 32, 40, 64, 128, 128])
            c["lse"] = rng.random() < 0.3
            kind = rng.choice(["one", "one", "draft", "mixed"])
            if kind == "draft":
                c["new_lo"] = c["new_hi"] = rng.randint(2, 6)
            elif kind == "mixed":
                c["new_hi"] = _log_int(rng, 2, 100)
        ctx, new = _lens(c)
        total = ctx + new
        if total.sum() < 1 or (op != "gather" and new.sum() < 1) or _cost(c) > 0.9 * top[op]:
            continue
        R, L, Q = len(ctx), int(total.max()), max(1, int(new.max()))
        # the plain form pads every request to the longest one
        if int(total.sum()) + R * c["page"] > 800000:
            continue
        if op == "attn" and (R * (L + c["page"]) > 3e6 or R * c["heads"] * Q * (L + c["page"]) > 2e9):
            continue
        return c


def _spread(lo, hi, u):
    """Whole numbers of [lo, hi], even over their logarithm."""
    if lo == hi:
        return np.full(u.shape, lo, np.int64)
    v = np.exp(math.log(lo + 1) + (math.log(hi + 2) - math.log(lo + 1)) * u) - 1
    return np.clip(np.floor(v).astype(np.int64), lo, hi)


def _lens(case):
    """The requests' cached and new token counts, in an order that the seed shuffles."""
    r = np.arange(1, case["requests"] + 1)
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], (r * 0.6180339887498949) % 1.0)
    new = _spread(case["new_lo"], case["new_hi"], (r * 0.4142135623730951) % 1.0)
    if case["idle"]:
        gone = r % case["idle"] == 0
        ctx, new = np.where(gone, 0, ctx), np.where(gone, 0, new)
    return ctx, new


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["rot"]
        return {"bytes": float(4 * n + 4 * case["tokens"] + 2 * case["rot"]), "flops": float(3 * n)}
    ctx, new = _lens(case)
    T, total = int(new.sum()), ctx + new
    row = LATENT + 4 + 2 * ROPE                         # a cached token
    if case["op"] == "append":
        return {"bytes": float(T * (2 * (LATENT + ROPE) + row + 8) + (2 * LATENT if case["norm"] else 0)),
                "flops": float(T * (6 * LATENT + 3 * ROPE))}
    if case["op"] == "gather":
        return {"bytes": float(int(total.sum()) * (row + 2 * (LATENT + ROPE))),
                "flops": float(int(total.sum()) * LATENT)}
    live = np.where(new > 0, total, 0)
    H = case["heads"]
    pairs = int((new * ctx + new * (new + 1) // 2).sum())
    return {"bytes": float(int(live.sum()) * row + 2 * T * H * (2 * LATENT + ROPE) +
                           (4 * T * H if case["lse"] else 0)),
            "flops": float(2 * pairs * H * (2 * LATENT + ROPE))}


# ------------------------------------------------------------------------------ states

def _frequencies(rot, scaled):
    """1e4 ** (-2 i / rot); scaled: by a factor of 40 where a trained length of 4096 holds less than
    one turn, by none where it holds over 32, in between linearly."""
    i = np.arange(rot // 2)
    f = 1e4 ** (-2.0 * i / rot)
    if scaled:
        turns_at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(1e4))   # noqa: E731
        lo, hi = max(math.floor(turns_at(32)), 0), min(math.ceil(turns_at(1)), rot // 2 - 1)
        keep = 1 - np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        f = f / 40 * (1 - keep) + f * keep
    return f.astype(np.float32), (0.1 * math.log(40) + 1.0) if scaled else 1.0


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _pow2_scale(amax):
    """max(amax, floor) / 448, rounded up to a power of two."""
    m, e = torch.frexp(amax.clamp_min(AMAX_FLOOR) / E4M3_MAX)
    return torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "rope":
        T, H, D, rot = case["tokens"], case["heads"], case["dim"], case["rot"]
        f, amplitude = _frequencies(rot, case["scaled"])
        x = torch.randn(T, H, D, generator=g, device=dev).to(torch.bfloat16)
        return {"case": case, "x": x[:, :, case["first"]:case["first"] + rot],
                "positions": torch.randint(0, case["far"], (T,), generator=g, device=dev).to(torch.int32),
                "inv_freq": torch.from_numpy(f).to(dev), "amplitude": amplitude}

    ctx, new = _lens(case)
    order = np.random.RandomState(seed % (1 << 32)).permutation(len(ctx))
    ctx, new = ctx[order], new[order]
    total, B, R = ctx + new, case["page"], len(ctx)
    need = -(-total // B)
    width = int(need.max()) + 1
    P = int(need.sum()) + int(need.sum()) // 16 + 2
    perm = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    # each request's pages lie anywhere in the pool; entries past them are stale
    first = torch.from_numpy(np.cumsum(need) - need).to(dev)
    j = torch.arange(width, device=dev)
    table = perm[(first[:, None] + j[None, :]).clamp_max(P - 1)].contiguous()
    T = int(new.sum())

    def sums(n):
        return torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(dev, torch.int32)
    # normal latents whose size differs from token to token, quantized
    x = torch.empty(P, B, LATENT, device=dev).normal_(generator=g)
    x *= torch.empty(P, B, 1, device=dev).log_normal_(0.0, 0.3, generator=g)
    s = _pow2_scale(x.abs().amax(dim=2))
    st = {"case": case, "T": T, "R": R, "max_new": int(new.max()), "block_table": table,
          "latent_cache": _e4m3(x.div_(s[:, :, None])).view(torch.uint8), "latent_scales": s,
          "rope_cache": torch.randn(P, B, ROPE, generator=g, device=dev).to(torch.bfloat16)}
    del x
    if case["op"] == "gather":
        st["row_offsets"] = sums(total)
        st["rows"] = int(total.sum())
        return st
    live = np.where(new > 0, total, 0)
    st["q_offsets"], st["kv_lens"] = sums(new), torch.from_numpy(live).to(dev, torch.int32)
    if case["op"] == "append":
        t = torch.arange(T, device=dev)
        r = torch.searchsorted(st["q_offsets"].long(), t, right=True) - 1
        pos = torch.from_numpy(ctx).to(dev)[r] + t - st["q_offsets"].long()[r]
        st["positions"] = pos.to(torch.int32)
        st["slot_map"] = (table.long()[r, pos // B] * B + pos % B).to(torch.int32)
        # the last columns of a wider projection: strided rows
        wide = torch.randn(T, 1536 + LATENT + ROPE, generator=g, device=dev).to(torch.bfloat16)
        st["kv"] = wide[:, 1536:]
        f, st["amplitude"] = _frequencies(ROPE, True)
        st["inv_freq"] = torch.from_numpy(f).to(dev)
        st["norm_weight"] = (1 + 0.2 * torch.randn(LATENT, generator=g, device=dev)).to(torch.bfloat16) \
            if case["norm"] else None
        return st
    # logits of a few units: some tokens matter much more than others
    H = case["heads"]
    st["q_latent"] = (1.2 * torch.randn(T, H, LATENT, generator=g, device=dev)).to(torch.bfloat16)
    st["q_rope"] = (1.2 * torch.randn(T, H, ROPE, generator=g, device=dev)).to(torch.bfloat16)
    st["scale"] = (128 + 64) ** -0.5
    return st


# --------------------------------------------------------------------------- plain forms

def _rotate(x, positions, inv_freq, amplitude, interleaved):
    """x [T, H, rot] in 32 bits, rotated by its tokens' angles (formed in 64)."""
    angle = positions.double()[:, None] * inv_freq.double()[None, :]
    cos, sin = ((amplitude * f(angle)).float()[:, None, :] for f in (torch.cos, torch.sin))
    half = x.shape[2] // 2
    a, b = (x[:, :, 0::2], x[:, :, 1::2]) if interleaved else (x[:, :, :half], x[:, :, half:])
    lo, hi = a * cos - b * sin, a * sin + b * cos
    return torch.stack([lo, hi], 3).flatten(2) if interleaved else torch.cat([lo, hi], 2)


def _append_plain(st):
    c, B = st["case"], st["case"]["page"]
    x = st["kv"].float()
    y, k = x[:, :LATENT], x[:, LATENT:]
    if c["norm"]:
        y = y * torch.rsqrt((y * y).mean(dim=1, keepdim=True) + EPS) * st["norm_weight"].float()
    s = _pow2_scale(y.abs().amax(dim=1))
    slot = st["slot_map"].long()
    page, off = slot // B, slot % B
    st["latent_cache"][page, off] = _e4m3(y / s[:, None]).view(torch.uint8)
    st["latent_scales"][page, off] = s
    k = _rotate(k[:, None], st["positions"], st["inv_freq"], st["amplitude"], c["interleaved"])[:, 0]
    st["rope_cache"][page, off] = k.to(torch.bfloat16)
    return _append_outputs(st)


def _append_outputs(st):
    return {"latent": st["latent_cache"].view(torch.float8_e4m3fn), "scales": st["latent_scales"],
            "rope": st["rope_cache"]}


def _gather_plain(st):
    B, off = st["case"]["page"], st["row_offsets"].long()
    t = torch.arange(st["rows"], device=off.device)
    r = torch.searchsorted(off, t, right=True) - 1
    pos = t - off[r]
    page = st["block_table"].long()[r, pos // B]
    codes = st["latent_cache"].view(torch.float8_e4m3fn)[page, pos % B].float()
    return [(codes * st["latent_scales"][page, pos % B][:, None]).to(torch.bfloat16),
            st["rope_cache"][page, pos % B]]


def _attend_plain(st):
    """Every request padded to the longest one."""
    c, dev = st["case"], st["q_latent"].device
    H, B, R, T, Q = c["heads"], c["page"], st["R"], st["T"], st["max_new"]
    kv_len, q_off = st["kv_lens"].long(), st["q_offsets"].long()
    n_new = q_off[1:] - q_off[:-1]
    table = st["block_table"].long()
    L = table.shape[1] * B
    v = st["latent_cache"].view(torch.float8_e4m3fn)[table].float() * st["latent_scales"][table][..., None]
    v = v.reshape(R, L, LATENT)
    k = torch.cat([v, st["rope_cache"][table].float().reshape(R, L, ROPE)], 2)
    i = torch.arange(Q, device=dev)
    q = torch.cat([st["q_latent"], st["q_rope"]], 2).float()
    q = q[(q_off[:-1, None] + i[None, :]).clamp_max(T - 1)].reshape(R, Q * H, LATENT + ROPE)
    s = (torch.matmul(q, k.transpose(1, 2)) * st["scale"]).reshape(R, Q, H, L)
    pos = torch.where(i[None, :] < n_new[:, None], kv_len[:, None] - n_new[:, None] + i[None, :], -1)
    seen = torch.arange(L, device=dev)[None, None, :] <= pos[:, :, None]
    s = s.masked_fill(~seen[:, :, None], -math.inf)
    m = s.amax(dim=3, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(s - m)
    del s
    norm = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p.reshape(R, Q * H, L), v).reshape(R, Q, H, LATENT)
    o = torch.where(norm > 0, o / norm, 0)
    lse = torch.where(norm > 0, m + torch.log(norm), -math.inf)[..., 0]
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(q_off, t, right=True) - 1
    at = t - q_off[r]
    return o[r, at].to(torch.bfloat16), lse[r, at]


def run(st):
    c = st["case"]
    if own:
        return _run_own(st)
    if c["op"] == "rope":
        return _rotate(st["x"].float(), st["positions"], st["inv_freq"], st["amplitude"],
                       c["interleaved"]).to(torch.bfloat16)
    if c["op"] == "append":
        return _append_plain(st)
    if c["op"] == "gather":
        return _gather_plain(st)
    o, lse = _attend_plain(st)
    return [o, lse] if c["lse"] else [o]


# ------------------------------------------------------------------------ the library's calls

def _run_own(st):
    import block_scaled_fp8_04_amd as bfp8

    c = st["case"]
    if c["op"] == "rope":
        if "out" not in st:
            st["out"] = torch.empty(st["x"].shape, dtype=torch.bfloat16, device=st["x"].device)
        bfp8.bfp8_rope(st["x"], st["positions"], st["inv_freq"], st["out"],
                       interleaved=c["interleaved"], amplitude=st["amplitude"])
        return st["out"]
    cache = st["latent_cache"], st["latent_scales"], st["rope_cache"]
    if c["op"] == "append":
        bfp8.bfp8_latent_append(st["kv"], st["slot_map"], st["positions"], st["inv_freq"], *cache,
                                norm_weight=st["norm_weight"], eps=EPS, interleaved=c["interleaved"],
                                amplitude=st["amplitude"])
        return _append_outputs(st)
    dev = st["block_table"].device
    if c["op"] == "gather":
        if "latent" not in st:
            st["latent"] = torch.empty(st["rows"], LATENT, dtype=torch.bfloat16, device=dev)
            st["rope"] = torch.empty(st["rows"], ROPE, dtype=torch.bfloat16, device=dev)
        bfp8.bfp8_latent_gather(*cache, st["block_table"], st["row_offsets"], st["latent"], st["rope"])
        return [st["latent"], st["rope"]]
    if "out" not in st:
        T, H = st["T"], c["heads"]
        st["out"] = torch.empty(T, H, LATENT, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty(T, H, dtype=torch.float32, device=dev) if c["lse"] else None
        st["workspace"] = bfp8.attn_latent_workspace(st["R"], st["max_new"], H, dev)
    bfp8.bfp8_attn_latent(st["q_latent"], st["q_rope"], *cache, st["block_table"], st["q_offsets"],
                          st["kv_lens"], st["max_new"], st["scale"], st["out"], st["lse"],
                          st["workspace"])
    return [st["out"], st["lse"]] if c["lse"] else [st["out"]]


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definitions in 64 bits; a cached code's exact value is the unrounded quotient."""
    if work(case)["flops"] > 3e12:
        return None
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "gather": _exact_gather,
            "attn": _exact_attention}[case["op"]](st)


def _turned(x, positions, inv_freq, amplitude, interleaved):
    """Pairs as complex numbers, times amplitude e^(i angle)."""
    x = x.double()
    half = x.shape[-1] // 2
    pairs = x.unflatten(-1, (half, 2)) if interleaved else x.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous())
    angle = positions.double()[:, None] * inv_freq.double()
    z = z * torch.polar(torch.full_like(angle, amplitude), angle).reshape(
        (x.shape[0],) + (1,) * (x.dim() - 2) + (half,))
    pairs = torch.view_as_real(z)
    return (pairs if interleaved else pairs.transpose(-1, -2)).flatten(-2)


def _exact_rope(st):
    return _turned(st["x"], st["positions"], st["inv_freq"], st["amplitude"], st["case"]["interleaved"])


def _exact_append(st):
    kv = st["kv"].double()
    y = kv[:, :LATENT]
    if st["norm_weight"] is not None:
        y = y / torch.sqrt(y.square().sum(1, keepdim=True) / LATENT + EPS) * st["norm_weight"].double()
    s = torch.exp2(torch.ceil(torch.log2(y.abs().amax(1).clamp_min(AMAX_FLOOR) / E4M3_MAX)))
    codes = st["latent_cache"].view(torch.float8_e4m3fn).double().flatten(0, 1)
    scales, rope = st["latent_scales"].double().flatten(), st["rope_cache"].double().flatten(0, 1)
    slot = st["slot_map"].long()
    codes[slot] = y / s[:, None]
    scales[slot] = s
    rope[slot] = _turned(kv[:, LATENT:], st["positions"], st["inv_freq"], st["amplitude"],
                         st["case"]["interleaved"])
    B = st["case"]["page"]
    return {"latent": codes.unflatten(0, (-1, B)), "scales": scales.unflatten(0, (-1, B)),
            "rope": rope.unflatten(0, (-1, B))}


def _request(st, r, n):
    """Request r's first n tokens: latents and rotated keys."""
    pages = st["block_table"][r, :-(-n // st["case"]["page"])].long()
    c = st["latent_cache"][pages].view(torch.float8_e4m3fn).double() * st["latent_scales"][pages].double()[..., None]
    return c.flatten(0, 1)[:n], st["rope_cache"][pages].double().flatten(0, 1)[:n]


def _exact_gather(st):
    n = torch.diff(st["row_offsets"]).tolist()
    rows = [_request(st, r, k) for r, k in enumerate(n)]
    return [torch.cat([x[i] for x in rows]) for i in (0, 1)]


def _exact_attention(st):
    """Request by request: gather the tokens, mask, softmax, average."""
    H, T, dev = st["case"]["heads"], st["T"], st["q_latent"].device
    out = torch.zeros(T, H, LATENT, dtype=torch.float64, device=dev)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    offs, lens = st["q_offsets"].tolist(), st["kv_lens"].tolist()

    def token(t, c, k, seen):
        z = st["q_latent"][t].double() @ c[:seen].T.contiguous() + st["q_rope"][t].double() @ k[:seen].T.contiguous()
        z = z * st["scale"]
        top = torch.logsumexp(z, dim=1)
        out[t] = torch.exp(z - top[:, None]) @ c[:seen]
        lse[t] = top

    def request(r):
        a, b, n = offs[r], offs[r + 1], lens[r]
        c, k = _request(st, r, n)
        list(map(lambda t: token(t, c, k, n - (b - 1 - t)), range(a, b)))
    list(map(request, [r for r, n in enumerate(lens) if n > 0]))
    return [out, lse] if st["case"]["lse"] else [out]
