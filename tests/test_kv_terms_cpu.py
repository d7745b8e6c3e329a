"""The bound of the attention tests: it holds for the roundings that the library states, and a weight
without its remainder, of any token, breaks it."""
import numpy as np
import pytest

import kv_reference as ref
import kv_terms


def bf16(x):
    """float32 rounded to bf16, to nearest even, as float32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + (b >> 16 & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def emulate(q, case, scale, keep=None):
    """Attention with the stated roundings (one accumulator, all of a case's queries see all
    tokens): p's remainder enters where keep [n] is 1."""
    pages, n = case.table[0], case.n
    k = ref.VALUES[case.k[pages, 0]].reshape(-1, q.shape[-1])[:n]
    v = ref.VALUES[case.v[pages, 0]].transpose(0, 2, 1).reshape(-1, case.v.shape[2])[:n]
    c = np.float32(scale * np.log2(np.e))
    s = (q @ k.T).astype(np.float32)
    m = np.ceil((s * c).max(axis=-1, keepdims=True))
    p = np.exp2((s.astype(np.float64) * c - m).astype(np.float32)).astype(np.float32)
    hi = bf16(p)
    lo = bf16(p - hi)
    w = hi.astype(np.float64) + lo * (1.0 if keep is None else keep)
    return bf16(((w @ v) / p.astype(np.float64).sum(axis=-1, keepdims=True)).astype(np.float32))


def case(dk, at=64, n=160):
    c = kv_terms.Cancelling(dk, at, n, 32, dk, min(dk, 128), draws=8)
    return c, c.q.reshape(-1, 1, dk)


def worst(c, q, got):
    # every query is the last one: a request of its own over the same pages
    T = q.shape[0]
    want, _, weight, slack = kv_terms.attention(q, *c.arrays, np.repeat(c.table, T, 0), np.arange(T + 1),
                                                [c.n] * T, 1.0)
    err = np.abs(got[:, None] - want) / kv_terms.bound(want, weight, slack)
    return err[:, 0].max(axis=1)


@pytest.mark.parametrize("dk", [64, 128])
def test_the_stated_roundings_stay_within(dk):
    c, q = case(dk)
    assert worst(c, q, emulate(q[:, 0], c, 1.0)).max() <= 1.0


@pytest.mark.parametrize("dk", [64, 128])
def test_a_lost_remainder_does_not(dk):
    c, q = case(dk)
    assert worst(c, q, emulate(q[:, 0], c, 1.0, np.zeros(c.n))).max() > 2.0
    for token in range(c.at, c.at + c.HOT):
        keep = np.ones(c.n)
        keep[token] = 0
        assert worst(c, q, emulate(q[:, 0], c, 1.0, keep)).max() > 1.25, f"token {token} of {c.HOT}"


def test_remainders_that_change_places_do_not():
    """p's remainders taken from the token next to it, or from eight tokens on."""
    c, q = case(64)
    pages = c.table[0]
    k = ref.VALUES[c.k[pages, 0]].reshape(-1, 64)[:c.n]
    v = ref.VALUES[c.v[pages, 0]].transpose(0, 2, 1).reshape(-1, 64)[:c.n]
    s = (q[:, 0] @ k.T).astype(np.float32)
    log2e = np.float32(np.log2(np.e))
    p = np.exp2(s * log2e - np.ceil((s * log2e).max(axis=1, keepdims=True))).astype(np.float32)
    lo = p - bf16(p)
    for by in (1, 8, 16):
        w = bf16(p).astype(np.float64) + np.roll(lo, by, axis=1)
        got = bf16(((w @ v) / p.astype(np.float64).sum(axis=1, keepdims=True)).astype(np.float32))
        assert worst(c, q, got).max() > 2.0, f"moved by {by}"


def test_both_references_agree():
    rng = np.random.default_rng(5)
    B, kv, new = 32, [70, 0, 3, 9, 40], [5, 0, 1, 12, 2]
    P = 12
    arrays = (rng.integers(0, 127, (P, 2, B, 64), dtype=np.uint8), np.full((P, 2), 2.0 ** -6, np.float32),
              rng.integers(0, 127, (P, 2, 64, B), dtype=np.uint8), np.full((P, 2), 2.0 ** -3, np.float32))
    table = rng.permutation(P)[:10].reshape(5, 2)
    table = np.concatenate([table, table[:, :1]], axis=1)
    q_off = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((q_off[-1] + 1, 6, 64))
    a = ref.attention(q, *arrays, table, q_off, kv, 0.2)
    b = kv_terms.attention(q, *arrays, table, q_off, kv, 0.2)
    for x, y in zip(a[:2], b[:2]):
        assert np.allclose(x, y, rtol=1e-11, atol=1e-12, equal_nan=True)
    live = ~np.isnan(a[1])
    assert np.allclose(a[2][live], b[2][live], rtol=1e-11) and np.allclose(a[3][live], b[3][live], rtol=1e-11)
