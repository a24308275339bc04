"""Queries, logits and values of very large and very small sizes."""
import numpy as np
import pytest

from tests.kv_helpers import bound_of, expected, run_attention
from tests.test_gpu_attention import case, check, queries

pytestmark = pytest.mark.gpu


def least_steps(parts, shape):
    """What binary16's least step adds to a bound of the ordinary roundings, for scales of the values up to 1.

    The weight of the largest logit is held as 2^6 at least and a weight is off by half of 2^-24 where it is subnormal:
    2^-31 of the largest weight a key, times the key's value. A product of weight and scale is off by as much, times a
    code's 8: 2^-28 of the largest weight, which is 2^-28 of it times the largest value where that is 1 or more."""
    more, at = np.zeros(shape), 0
    for v, out, of_rows, G in parts:
        for h, i, keys, p, _ in of_rows:
            if len(p):
                more[at + i, h] = len(p) * 2.0 ** -28 * p.max() * max(1.0, np.abs(v[keys, h // G]).max())
        at += len(out)
    return more


SHAPES = [("decode", 128, 2, 4, 1), ("decode", 64, 1, 16, 1), ("decode", 256, 1, 4, 2), ("decode", 128, 1, 8, 8),
          ("prefill", 64, 1, 3, 70), ("prefill", 128, 2, 4, 10), ("prefill", 256, 1, 2, 20)]


@pytest.mark.parametrize("call,D,Hkv,G,n", SHAPES)
@pytest.mark.parametrize("size,scale", [(1e37, 1e-38 * 5), (3e37, 2e-38), (1e35, 1e-36), (1e-37, 1e36), (1e-38, 1e37), (1e-32, 1e31)])
def test_rows_of_extreme_queries(call, D, Hkv, G, n, size, scale):
    """Finite rows up to binary32's largest and down to its smallest normal numbers, with scales that bring their logits
    to ordinary sizes."""
    rng = np.random.default_rng(D + n)
    lens = [150, 33]
    geo, pages, table = case(rng, D, Hkv, 16, lens)
    scale = float(np.float32(scale))
    q = queries(rng, 2 * n, Hkv * G, D, "f32")
    q = (q.astype(np.float64) * size).astype(np.float32)
    assert np.isfinite(q).all()
    out, _ = run_attention(geo, pages, table, lens, q, [n, n], "f32", scale, 0, None, "f32", False, call)
    want, parts = expected(geo, pages, table, lens, q, [n, n], scale, 0, None)
    check(out, want, bound_of(parts, call == "prefill") + least_steps(parts, want.shape), "f32")
