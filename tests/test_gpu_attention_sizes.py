"""Queries, logits and values of very large and very small sizes."""
import numpy as np
import pytest

from oracle import kv as OK
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


@pytest.mark.parametrize("call,D,Hkv,G,n,lens", [s + ([150, 33, 700],) for s in SHAPES] + [
    ("prefill", 128, 1, 2, 3, [4000, 20, 2300])])             # (the last: keys shared out and joined)
@pytest.mark.parametrize("power", [10, 20, 26, 60])
@pytest.mark.parametrize("kind", ["both signs", "negative"])
@pytest.mark.parametrize("sink", [None, 3.0])
@pytest.mark.parametrize("value_size", [1.0, 2048.0])
def test_huge_logits(call, D, Hkv, G, n, lens, power, kind, sink, value_size):
    """Logits of 2^power times multiples of 32: all weight lies on the keys of the largest one, in equal parts.

    Queries and keys are powers of two times small whole numbers in one column, so equal logits are equal in every
    arithmetic and different ones are 2^15 apart at least. Values are off by 2^-11 (prefill), the common weight by 2^-11
    twice, sums of n terms by n 2^-23."""
    rng = np.random.default_rng(D + n + power)
    geo, pages, table = case(rng, D, Hkv, 16, lens)
    view = pages.reshape(-1, 18 * D)
    kb, ks, _, _ = OK.code_places(D)
    sk, sv = OK.scale_places(D)
    half = lambda at: view[:, at.reshape(-1)].astype(np.uint16) | view[:, at.reshape(-1) + 1].astype(np.uint16) << 8
    def put(at, x):
        raw = x.astype(np.float16).view(np.uint16)
        view[:, at.reshape(-1)], view[:, at.reshape(-1) + 1] = raw & 255, raw >> 8
    with np.errstate(invalid="ignore", over="ignore"):
        old = half(sk).view(np.float16)
        put(sk, np.where(np.isfinite(old), 32.0, old))
        put(sv, half(sv).view(np.float16).astype(np.float64) * value_size)
    if kind == "negative":     # codes 0..7 of the column: every key is below zero
        for i in range(16):
            view[:, kb[i, 0]] &= np.uint8(~(8 << ks[i, 0]) & 255)
    rows = n * len(lens)
    q = np.zeros((rows, Hkv * G, D), dtype=np.float32)
    q[:, :, 0] = 2.0 ** power
    s = None if sink is None else np.full(Hkv * G, sink, dtype=np.float32)
    out, _ = run_attention(geo, pages, table, lens, q, [n] * len(lens), "f32", 1.0, 0, s, "f32", False, call)
    want, parts = expected(geo, pages, table, lens, q, [n] * len(lens), 1.0, 0, s)
    at, tol = 0, np.zeros_like(want)
    for v, o, ps, _ in parts:
        for h, i, keys, p, _ in ps:
            if len(p):
                assert ((p == 0) | (np.abs(p - p.max()) <= 1e-9 * p.max())).all()
                tol[at + i, h] = (2.0 ** -9 + len(p) * 2.0 ** -23) * (p @ np.abs(v[keys, h // G]))
        at += n
    assert (np.abs(out - want) <= tol).all(), np.nanmax(np.abs(out - want) - tol)


@pytest.mark.parametrize("call,D,Hkv,G,n", SHAPES)
@pytest.mark.parametrize("sign", [1, -1])
def test_far_logits_before_ordinary_ones(call, D, Hkv, G, n, sign):
    """Keys of logits of about -8e6 (or of 8e6 that no row sees, in front of a window) and then ordinary ones: the far ones
    get nothing and leave nothing of their size.

    The first column's query is 64 times the others, which adds half of 2^-24 times 2^7 a query to the scores' errors."""
    rng = np.random.default_rng(D + n)
    lens, far = [400, 290], 200
    geo, pages, table = case(rng, D, Hkv, 16, lens)
    kb, ks, _, _ = OK.code_places(D)
    sk, _ = OK.scale_places(D)
    for b, length in enumerate(lens):
        for j in range(length):
            g, i = pages[table[b, j // 16], :, j % 16 // 16], j % 16
            code = (0 if sign > 0 else 15) if j < far else 8
            g[:, kb[i, 0]] = g[:, kb[i, 0]] & ~np.uint8(15 << ks[i, 0]) | np.uint8(code << ks[i, 0])
            if j < far:
                raw = int(np.float16(-8000.0 if sign < 0 and j % 3 else 8000.0).view(np.uint16))
                g[:, sk[i, 0]], g[:, sk[i, 0] + 1] = raw & 255, raw >> 8
    window = 0 if sign > 0 else 60
    q = (rng.normal(size=(2 * n, Hkv * G, D)) * 8 / D ** 0.5).astype(np.float32)
    q[:, :, 0] = 64.0
    out, _ = run_attention(geo, pages, table, lens, q, [n, n], "f32", 2.0, window, None, "f32", False, call)
    want, parts = expected(geo, pages, table, lens, q, [n, n], 2.0, window, None)
    bound = bound_of(parts, call == "prefill") + least_steps(parts, want.shape)
    at = 0
    k, _ = OK.values(pages, geo)
    for b, (v, o, ps, _) in enumerate(parts):
        slots = table[b, np.arange(lens[b]) // 16] * 16 + np.arange(lens[b]) % 16
        for h, i, keys, p, _ in ps:
            if len(p):
                kk, vv = k[slots[keys], h // G], v[keys, h // G]
                bound[at + i, h] += (p * 2.0 ** -18 * 2.0 * np.abs(kk[:, 1:]).sum(1)) @ (np.abs(vv) + np.abs(o[i, h]))
        at += n
    check(out, want, bound, "f32")
