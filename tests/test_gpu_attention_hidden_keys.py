"""A key that a row does not see leaves nothing in it, whatever its values are."""
import numpy as np
import pytest

from oracle import kv as OK
from tests.kv_helpers import bound_of, decode_error, expected, poison, run_attention
from tests.test_gpu_attention import case, check, queries

pytestmark = pytest.mark.gpu

HALF_MAX = 65504.0


def set_scales(pages, geo, slot, k=None, v=None):
    """The scales of one token's key or value blocks."""
    _, P, _, D = geo
    g = pages[slot // P, :, slot % P // 16]
    for places, d in zip(OK.scale_places(D), (k, v)):
        if d is not None:
            raw = int(np.float16(d).view(np.uint16))
            s = places[slot % 16]
            g[:, s], g[:, s + 1] = raw & 255, raw >> 8


@pytest.mark.parametrize("D,Hkv,G,window", [(64, 1, 2, 0), (128, 2, 3, 0), (256, 1, 1, 0), (128, 1, 4, 60)])
@pytest.mark.parametrize("call,n", [("prefill", 200), ("prefill", 3), ("decode", 8)])
def test_large_values_at_tokens_that_are_not_seen(call, n, D, Hkv, G, window):
    """Values up to 8 * 60000 at some tokens. The prefill takes them as 65504; rows that do not see them are as always."""
    rng = np.random.default_rng(D + n)
    lens = [200]
    geo, pages, table = case(rng, D, Hkv, 16, lens)
    for j in (60, 150, 199):
        set_scales(pages, geo, int(table[0, j // 16]) * 16 + j % 16, v=60000.0)
    q = queries(rng, n, Hkv * G, D, "f32")
    out, _ = run_attention(geo, pages, table, lens, q, [n], "f32", 0.05, window, None, "f32", False, call)
    k, v = OK.values(pages, geo)
    slots = table[0, np.arange(200) // 16] * 16 + np.arange(200) % 16
    kk, vv = k[slots], v[slots]
    if call == "prefill":
        vv = np.clip(vv, -HALF_MAX, HALF_MAX)
    want, parts = OK.attention(q.astype(np.float64), kk, vv, np.ones(200, bool), n, 0.05, window)
    check(out, want, decode_error(vv, want, parts, G, call == "prefill"), "f32")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_keys(D):
    """Keys beyond binary16's range: the prefill takes them as 65504 too, visible or not."""
    rng = np.random.default_rng(D)
    n, G, lens = 100, 2, [100]
    geo, pages, table = case(rng, D, 1, 16, lens)
    for j in (20, 77):
        set_scales(pages, geo, int(table[0, j // 16]) * 16 + j % 16, k=60000.0)
    q = queries(rng, n, G, D, "f32")
    out, _ = run_attention(geo, pages, table, lens, q, [n], "f32", 1e-6, 0, None, "f32", False, "prefill")
    k, v = OK.values(pages, geo)
    slots = table[0, np.arange(100) // 16] * 16 + np.arange(100) % 16
    kk = np.clip(k[slots], -HALF_MAX, HALF_MAX)
    want, parts = OK.attention(q.astype(np.float64), kk, v[slots], np.ones(100, bool), n, 1e-6)
    check(out, want, decode_error(v[slots], want, parts, G, True), "f32")


@pytest.mark.parametrize("call,D,Hkv,G,n", [
    ("prefill", 128, 2, 4, 10), ("prefill", 64, 1, 3, 130), ("prefill", 256, 1, 2, 70),
    ("decode", 128, 2, 4, 1), ("decode", 64, 1, 16, 1), ("decode", 256, 1, 4, 2), ("decode", 128, 1, 8, 8),
])
@pytest.mark.parametrize("window", [1, 40, 77])
def test_nothing_in_front_of_the_first_visible_key_is_used(call, D, Hkv, G, n, window):
    """Scales of NaN and infinity at every token below the first that any row sees, in its group of 16 too."""
    rng = np.random.default_rng(D + window + n)
    lens = [300, 1000, 170, n]
    geo, pages, table = case(rng, D, Hkv, 16, lens)
    seen = []
    for b, length in enumerate(lens):
        j = np.arange(max(0, length - n + 1 - window), length)
        seen.append(table[b, j // 16].astype(np.int64) * 16 + j % 16)
    poison(pages, geo, np.concatenate(seen))
    q = queries(rng, n * len(lens), Hkv * G, D, "f32")
    out, _ = run_attention(geo, pages, table, lens, q, [n] * len(lens), "f32", 0.1, window, None, "f32", False, call)
    want, parts = expected(geo, pages, table, lens, q, [n] * len(lens), 0.1, window, None)
    check(out, want, bound_of(parts, call == "prefill"), "f32")
