"""Pins of the CPU definitions of the 4-bit cache: the layout is a bijection, blocks worked by hand, rotation and
attention against facts outside themselves."""
import numpy as np
import pytest

from oracle import kv as OK
from quantized_activation_q4_gb300 import binding as qk


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_uses_every_nibble_once(D):
    kb, ksh, vb, vsh = OK.code_places(D)
    nibbles = np.concatenate([(2 * b + s // 4).ravel() for b, s in ((kb, ksh), (vb, vsh))])
    sk, sv = OK.scale_places(D)
    for s in (sk, sv):
        nibbles = np.concatenate([nibbles] + [(2 * s.ravel() + k) for k in range(4)])
    assert np.array_equal(np.sort(nibbles), np.arange(2 * 18 * D))
    # a byte belongs to one token
    for byte in (kb, vb):
        owner = {}
        for i in range(16):
            for x in byte[i]:
                assert owner.setdefault(int(x), i) == i
    assert qk.qk_kv_page_bytes(64, 3, D) == 3 * 4 * 18 * D
    assert qk.qk_kv_page_bytes(24, 3, D) == 0 and qk.qk_kv_page_bytes(16, 0, D) == 0 and qk.qk_kv_page_bytes(16, 1, 96) == 0


def test_blocks_by_hand():
    x = np.zeros(32, dtype=np.float32)
    c, d = OK.q4_block(x)
    assert (c == 8).all() and d == 0
    x[3], x[5] = 4.0, -4.0                       # equal magnitudes: the first gives the scale
    c, d = OK.q4_block(x)
    assert d == np.float16(-0.5) and c[3] == 0 and c[5] == 15 and c[0] == 8
    x[3], x[5] = -4.0, 4.0
    c, d = OK.q4_block(x)
    assert d == np.float16(0.5) and c[3] == 0 and c[5] == 15
    x[7], x[8], x[9] = 0.25, 0.75, -0.25         # ties to even
    c, d = OK.q4_block(x)
    assert (c[7], c[8], c[9]) == (8, 10, 8)
    x[4] = np.nan
    assert OK.q4_block(x)[0][4] == 8
    x[6] = np.inf
    c, d = OK.q4_block(x)
    assert d == np.float16(-65504) and c[6] == 0 and c[3] == 8


def test_values_return_what_put_stored():
    rng = np.random.default_rng(5)
    geo = (3, 32, 2, 64)
    pages = rng.integers(0, 256, (3, 2, 2, 18 * 64), dtype=np.uint8)
    x = rng.normal(size=(2, 2, 2, 32)).astype(np.float32)
    codes, d = OK.q4_block(x)
    before = pages.copy()
    OK.put(pages, geo, 41, codes.reshape(2, 2, 64), d)
    k, v = OK.values(pages, geo)
    want = (codes - 8) * d[..., None].astype(np.float64)
    assert np.array_equal(k[41], want[0].reshape(2, 64)) and np.array_equal(v[41], want[1].reshape(2, 64))
    assert np.abs(want - x).max() <= np.abs(d).max() * 1.01
    k0, v0 = OK.values(before, geo)
    keep = np.arange(96) != 41
    assert np.array_equal(k[keep], k0[keep], equal_nan=True) and np.array_equal(v[keep], v0[keep], equal_nan=True)


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(6)
    x, y = rng.normal(size=(2, 1, 1, 64))
    f = (10000.0 ** (-np.arange(32) / 32))[None].astype(np.float32)
    for kind in ("halves", "adjacent"):
        dots = []
        for base in (0, 1000, 100000):
            a = OK.rotate(x, kind, 64, np.array([[base + 7]]), f)
            b = OK.rotate(y, kind, 64, np.array([[base]]), f)
            assert np.isclose(np.linalg.norm(a), np.linalg.norm(x), rtol=1e-14)
            dots.append(float((a * b).sum()))
        assert np.allclose(dots, dots[0], rtol=0, atol=1e-9)


def test_attention_of_equal_keys_is_the_mean_and_a_sink_takes_its_share():
    rng = np.random.default_rng(7)
    v = rng.normal(size=(5, 1, 64))
    k = np.ones((5, 1, 64))
    q = rng.normal(size=(2, 2, 64))
    out, _ = OK.attention(q, k, v, np.ones(5, bool), 2, 0.1)
    assert np.allclose(out[1], v[:, 0].mean(0)) and np.allclose(out[0], v[:4, 0].mean(0))
    out, _ = OK.attention(q, k, v, np.ones(5, bool), 2, 0.1, window=2)
    assert np.allclose(out[1], v[3:, 0].mean(0)) and np.allclose(out[0], v[2:4, 0].mean(0))
    s = 0.1 * q[1, 0].sum()
    out, _ = OK.attention(q, k, v, np.ones(5, bool), 2, 0.1, sinks=np.array([s + np.log(5), 0.0]))
    assert np.allclose(out[1, 0], v[:, 0].mean(0) / 2)
    out, parts = OK.attention(q, k[:0], v[:0], np.ones(0, bool), 2, 0.1)
    assert (out == 0).all()
