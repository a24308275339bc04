"""qk_kv_append over numbers of heads at the borders of its turns: a CTA takes 256 / (D / 4) heads side by side and loads the
queries of four such turns together. Many tokens of one call against the definition."""
import numpy as np
import pytest

from oracle import kv as OK
from tests.kv_helpers import random_pages
from tests.test_gpu_kv_cache import append, rows

pytestmark = pytest.mark.gpu


def check(geo, T, Hq, kind, seed):
    n_pages, P, Hkv, D = geo
    rng = np.random.default_rng(seed)
    x = rows(rng, T, Hq + 2 * Hkv, D, "f32")
    slots = rng.permutation(n_pages * P)[:T]
    pages = random_pages(rng, geo)
    dims = D - 8
    pos = rng.integers(0, 5000, (2, T))
    freqs = rng.uniform(0.0, 1.0, (2, dims // 2)).astype(np.float32)
    rope = None if kind is None else (kind, dims, pos, freqs)
    q, got = append(geo, pages, x, "f32", Hq, slots, rope, "f32")
    want = pages.copy()
    ref = x[:, :Hq + Hkv].astype(np.float64) if kind is None else OK.rotate(x[:, :Hq + Hkv], kind, dims, pos, freqs)
    for t in range(T):
        codes, d = OK.q4_block(np.concatenate([ref[t, Hq:], x[t, Hq + Hkv:]]).astype(np.float32).reshape(2, Hkv, D // 32, 32))
        OK.put(want, geo, int(slots[t]), codes.reshape(2, Hkv, D), d)
    if kind is None:
        assert np.array_equal(got, want)
        assert Hq == 0 or np.array_equal(q, x[:, :Hq])
        return
    # rotated: c and s within 2^-22, three roundings of 2^-24, of a pair's |x| + |y| <= 2 max
    size = np.abs(x).max() * 2
    if Hq:
        assert np.abs(q - ref[:, :Hq]).max() <= size * (2.0 ** -22 + 3 * 2.0 ** -24)
    # a key's code is off by one where its quotient is next to a border, and a scale by binary16's rounding
    k0, v0 = OK.values(want, geo)
    k1, v1 = OK.values(got, geo)
    assert np.array_equal(v0, v1)
    other = np.setdiff1d(np.arange(n_pages * P), slots)
    assert np.array_equal(k0[other], k1[other])
    d = np.abs(ref[:, Hq:].reshape(T, Hkv, D // 32, 32)).max(-1, keepdims=True) / 8
    off = np.abs(k1[slots].reshape(T, Hkv, D // 32, 32) - k0[slots].reshape(T, Hkv, D // 32, 32))
    assert (off <= d * 1.01 + 1e-6).all() and (off > d * 0.01).mean() <= 1e-3


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", ["one", "a turn", "four turns less one", "four turns", "four turns and one", "nine turns and two"])
@pytest.mark.parametrize("kind", [None, "halves", "adjacent"])
def test_numbers_of_query_heads(D, heads, kind):
    turn = 256 // (D // 4)
    Hq = {"one": 1, "a turn": turn, "four turns less one": 4 * turn - 1, "four turns": 4 * turn, "four turns and one": 4 * turn + 1,
          "nine turns and two": 9 * turn + 2}[heads]
    check((3, 16, 2, D), 5, Hq, kind, Hq)


@pytest.mark.parametrize("D,Hkv", [(64, 1), (64, 7), (64, 8), (64, 9), (128, 3), (128, 4), (128, 5), (256, 1), (256, 2), (256, 3), (64, 256)])
@pytest.mark.parametrize("kind", [None, "halves"])
def test_numbers_of_cache_heads(D, Hkv, kind):
    check((2, 16, Hkv, D), 6, 0 if Hkv % 2 else 3, kind, Hkv)


@pytest.mark.parametrize("kind", [None, "halves", "adjacent"])
def test_many_tokens_of_one_call(kind):
    check((20, 64, 2, 64), 1200, 5, kind, 7)
