"""A NaN in a query row and head makes that row and head NaN, whatever the sinks."""
import numpy as np
import pytest

from tests.kv_helpers import run_attention
from tests.test_gpu_attention import case, queries

pytestmark = pytest.mark.gpu

SHAPES = [(64, 1, 2, [40, 300, 0], 3), (128, 2, 4, [333, 70], 5), (256, 1, 3, [90, 200], 2)]


def inputs(D, Hkv, G, lens, n, kind):
    rng = np.random.default_rng(D + n)
    geo, pages, table = case(rng, D, Hkv, 32, lens)
    q = queries(rng, n * len(lens), Hkv * G, D, "f32")
    sink = {"none": None, "finite": rng.standard_normal(Hkv * G), "large": np.full(Hkv * G, 80.0),
            "minus infinity": np.full(Hkv * G, -np.inf)}[kind]
    return geo, pages, table, q, None if sink is None else sink.astype(np.float32)


@pytest.mark.parametrize("call", ["decode", "prefill"])
@pytest.mark.parametrize("kind", ["finite", "large", "minus infinity"])
@pytest.mark.parametrize("D,Hkv,G,lens,n", SHAPES)
def test_with_sinks(call, kind, D, Hkv, G, lens, n):
    geo, pages, table, q, sink = inputs(D, Hkv, G, lens, n, kind)
    run = lambda: run_attention(geo, pages, table, lens, q, [n] * len(lens), "f32", 0.1, 0, sink, "f32", False, call)[0]
    clean = run()
    assert np.isfinite(clean).all()
    at = [(0, Hkv * G - 1), (n - 1, 0), (n, 1)]
    for i, h in at:
        q[i, h, 33] = np.nan
    got = run()
    for i, h in at:
        assert np.isnan(got[i, h]).all()
        got[i, h] = clean[i, h]
    assert np.array_equal(got, clean)
