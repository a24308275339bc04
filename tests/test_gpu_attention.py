"""qk_attn_decode and qk_attn_prefill against the definition in binary64, within the bound of tests/kv_helpers.py."""
import numpy as np
import pytest

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from tests.kv_helpers import (HB16, bf16, bound_of, expected, page_table, poison, random_pages, run_attention)

pytestmark = pytest.mark.gpu


def case(rng, D, Hkv, P, lens, n_pages=None):
    need = sum(-(-max(0, int(n)) // P) for n in lens) + 2
    geo = (n_pages or need, P, Hkv, D)
    pages = random_pages(rng, geo)
    table, slots = page_table(rng, geo, [max(0, n) for n in lens])
    poison(pages, geo, np.concatenate(slots) if slots else [])
    return geo, pages, table


def queries(rng, rows, Hq, D, elem, size=1.5):
    q = (size * rng.normal(size=(rows, Hq, D))).astype(np.float32)
    return bf16(q) if elem == "bf16" else q


def check(got, want, bound, out_elem, what=""):
    tol = bound + (HB16 * (np.abs(want) + bound) if out_elem == "bf16" else 2.0 ** -24 * np.abs(want))
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{what}: off by {np.nanmax(err - tol):.3e} over a bound of about {tol.mean():.3e}"


def image_is_of(img, out):
    """The image is the quantiser's of the F32 rows."""
    rows, Hq, D = out.shape
    blocks = Hq * D // 32
    if isinstance(img, tuple):
        q, d = O.quantize_q8_0(out.reshape(rows, -1), row_blocks=img[1].shape[1])
        assert np.array_equal(img[0].reshape(rows, -1), q.reshape(rows, -1)) and np.array_equal(img[1], d.reshape(rows, -1))
    else:
        want = O.quantize_q8_1(out.reshape(rows, -1), row_blocks=img.shape[1])
        assert np.array_equal(img.reshape(rows, -1), want.reshape(rows, -1))


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 255, 257]


@pytest.mark.parametrize("D,Hkv,G,P", [(64, 1, 1, 16), (64, 2, 4, 64), (128, 4, 7, 64), (128, 1, 16, 32), (128, 2, 8, 16),
                                       (256, 2, 2, 128), (256, 1, 9, 16), (64, 3, 5, 48)])
@pytest.mark.parametrize("T", [1, 3, 8])
def test_decode_lengths(D, Hkv, G, P, T):
    rng = np.random.default_rng(D + G + T)
    geo, pages, table = case(rng, D, Hkv, P, LENS)
    q = queries(rng, len(LENS) * T, Hkv * G, D, "f32")
    rows = [T] * len(LENS)
    out, img = run_attention(geo, pages, table, LENS, q, rows, "f32", D ** -0.5, 0, None, "f32", True, "decode",
                             spare_blocks=2)
    want, parts = expected(geo, pages, table, LENS, q, rows, D ** -0.5, 0, None)
    check(out, want, bound_of(parts, False), "f32")
    image_is_of(img, out)
    empty = [b * T + i for b, n in enumerate(LENS) for i in range(T) if n - T + i < 0]
    assert (out[empty] == 0).all()


@pytest.mark.parametrize("call,T", [("decode", 1), ("decode", 5), ("prefill", 5), ("prefill", 70)])
@pytest.mark.parametrize("window,sinks", [(1, False), (16, True), (37, False), (130, True), (0, True)])
def test_window_and_sinks(call, T, window, sinks):
    rng = np.random.default_rng(window + T)
    D, Hkv, G, P = 128, 2, 3, 32
    lens = [0, 1, 40, 90, 300, 517]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    q = queries(rng, len(lens) * T, Hkv * G, D, "bf16")
    s = rng.normal(size=Hkv * G).astype(np.float32) * 2 if sinks else None
    if sinks:
        s[0], s[1] = 60.0, -np.inf
    rows = [T] * len(lens)
    out, img = run_attention(geo, pages, table, lens, q, rows, "bf16", 0.1, window, s, "f32", True, call)
    want, parts = expected(geo, pages, table, lens, q, rows, 0.1, window, s)
    check(out, want, bound_of(parts, call == "prefill"), "f32")
    image_is_of(img, out)


@pytest.mark.parametrize("call", ["decode", "prefill"])
@pytest.mark.parametrize("elem,out_elem,image,pad", [("bf16", "bf16", False, 0), ("f32", "bf16", True, 5),
                                                     ("bf16", None, True, 3), ("f32", "f32", False, 1)])
def test_types_strides_and_live_sequences(call, elem, out_elem, image, pad):
    rng = np.random.default_rng(pad)
    D, Hkv, G, P = 64, 2, 3, 16
    lens, T, live = [70, 5, 130, 64, 9], 2, 3
    geo, pages, table = case(rng, D, Hkv, P, lens)
    q = queries(rng, len(lens) * T, Hkv * G, D, elem)
    rows = [T] * len(lens)
    out, img = run_attention(geo, pages, table, lens, q, rows, elem, 0.2, 0, None, out_elem, image, call, live, pad, 1)
    want, parts = expected(geo, pages, table, lens, q, rows, 0.2, 0, None)
    n = live * T
    if out is not None:
        check(out[:n], want[:n], bound_of(parts, call == "prefill")[:n], out_elem)
        assert np.isnan(out[n:]).all()
    if img is not None:
        full, whole = run_attention(geo, pages, table, lens, q, rows, elem, 0.2, 0, None, "f32", True, call, live, 0, 1)
        if call == "decode":
            assert np.array_equal(img[:n], whole[:n]) and (img[n:] == 0xA5).all()
            image_is_of(img[:n], full[:n])
        else:
            assert np.array_equal(img[0][:n], whole[0][:n]) and np.array_equal(img[1][:n], whole[1][:n])
            assert (img[0][n:] == 0x25).all() and (img[1][n:] == 0x2525).all()
            image_is_of((img[0][:n], img[1][:n]), full[:n])


@pytest.mark.parametrize("call,T", [("decode", 2), ("prefill", 2), ("prefill", 150)])
def test_pages_outside_the_cache_are_not_visible(call, T):
    rng = np.random.default_rng(11)
    D, Hkv, G, P = 128, 2, 4, 16
    lens = [100, 260, 30, 16]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    table[0, 2], table[1, 0], table[1, 7], table[1, 8] = -1, geo[0], 2 ** 31 - 1, -2 ** 31
    table[2, :2] = -5                                     # a sequence without any page
    q = queries(rng, len(lens) * T, Hkv * G, D, "f32")
    rows = [T] * len(lens)
    lens_given = [100, 260, 30, 2 ** 31 - 1]              # clamped to the page table; its further pages are -1
    out, _ = run_attention(geo, pages, table, lens_given, q, rows, "f32", 0.1, 0, None, "f32", True, call)
    lens_seen = [100, 260, 30, table.shape[1] * P]
    k = np.arange(16, table.shape[1] * P)
    table_seen = table.copy()
    want, parts = expected(geo, pages, table_seen, lens_seen, q, rows, 0.1, 0, None)
    check(out, want, bound_of(parts, call == "prefill"), "f32")
    assert (out[2 * T:3 * T] == 0).all()
    out, _ = run_attention(geo, pages, table, [-7, -2 ** 31, 0, 16], q, rows, "f32", 0.1, 0, None, "f32", True, call)
    assert (out[:3 * T] == 0).all()


@pytest.mark.parametrize("D,Hkv,G,P", [(64, 1, 2, 16), (128, 2, 7, 64), (256, 1, 3, 32), (128, 1, 1, 256)])
@pytest.mark.parametrize("rows,past", [([1, 2, 127, 128, 129], [0, 3, 0, 64, 1]), ([300, 1, 0, 40], [0, 500, 20, 129])])
def test_prefill_ragged(D, Hkv, G, P, rows, past):
    rng = np.random.default_rng(D + G + rows[0])
    lens = [n + p for n, p in zip(rows, past)]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    q = queries(rng, sum(rows), Hkv * G, D, "bf16")
    out, img = run_attention(geo, pages, table, lens, q, rows, "bf16", D ** -0.5, 0, None, "f32", True, "prefill",
                             spare_blocks=1)
    want, parts = expected(geo, pages, table, lens, q, rows, D ** -0.5, 0, None)
    check(out, want, bound_of(parts, True), "f32")
    image_is_of(img, out)


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_long_and_peaked(call):
    """A long sequence with a few large logits and many small ones; values and queries of very different sizes."""
    rng = np.random.default_rng(3)
    D, Hkv, G, P = 128, 1, 4, 64
    lens, T = [20000, 777], 2
    geo, pages, table = case(rng, D, Hkv, P, lens)
    view = pages.reshape(geo[0], Hkv, P // 16, 18 * D)
    first = table[0, 0]
    for s, size in ((8 * D, 4.0), (17 * D, 0.25)):        # the first page's keys four times as large, its values a quarter
        raw = view[first, :, :, s:s + D].copy().view(np.float16)
        view[first, :, :, s:s + D] = (raw.astype(np.float32) * size).astype(np.float16).view(np.uint8)
    second = table[0, 1]
    raw = view[second, :, :, 17 * D:].copy().view(np.float16)
    view[second, :, :, 17 * D:] = (raw.astype(np.float32) * 3000).astype(np.float16).view(np.uint8)
    q = queries(rng, 2 * T, G, D, "f32")
    q[0] *= 1e-4
    q[1, 1] *= 30
    q[2, 0] *= 1e6
    q[3, 2] = 0
    rows = [T, T]
    out, _ = run_attention(geo, pages, table, lens, q, rows, "f32", D ** -0.5, 0, None, "f32", False, call)
    want, parts = expected(geo, pages, table, lens, q, rows, D ** -0.5, 0, None)
    check(out, want, bound_of(parts, call == "prefill"), "f32")


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_same_call_same_bytes(call):
    rng = np.random.default_rng(4)
    D, Hkv, G, P = 128, 2, 7, 64
    lens, T = [3000, 1, 400, 1234, 64], 3
    geo, pages, table = case(rng, D, Hkv, P, lens)
    q = queries(rng, len(lens) * T, Hkv * G, D, "bf16")
    a, b = (run_attention(geo, pages, table, lens, q, [T] * 5, "bf16", 0.1, 0, None, "f32", False, call)[0]
            for _ in range(2))
    assert np.array_equal(a, b)


@pytest.mark.parametrize("D,Hkv,G,P", [(64, 2, 3, 64), (128, 1, 7, 16), (256, 1, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(0, False), (1500, True), (0, True)])
def test_prefill_behind_a_long_past(D, Hkv, G, P, window, sinks):
    """Few rows and many keys: the keys of a tile are shared out and joined again, some shares of them empty."""
    rng = np.random.default_rng(D + window)
    rows, past = [9, 70, 1, 3], [4000, 2300, 0, 100]
    lens = [n + p for n, p in zip(rows, past)]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    table[1, 3] = -1
    q = queries(rng, sum(rows), Hkv * G, D, "bf16")
    s = rng.normal(size=Hkv * G).astype(np.float32) * 3 if sinks else None
    out, img = run_attention(geo, pages, table, lens, q, rows, "bf16", D ** -0.5, window, s, "f32", True, "prefill",
                             spare_blocks=1)
    want, parts = expected(geo, pages, table, lens, q, rows, D ** -0.5, window, s)
    check(out, want, bound_of(parts, True), "f32")
    image_is_of(img, out)
    low, _ = run_attention(geo, pages, table, lens, q, rows, "bf16", D ** -0.5, window, s, "bf16", False, "prefill", live=3)
    n = sum(rows[:3])
    assert np.array_equal(low[:n], bf16(out[:n])) and np.isnan(low[n:]).all()


@pytest.mark.parametrize("D,Hkv,G,P,T", [(128, 2, 4, 64, 8), (64, 1, 16, 16, 2), (256, 2, 4, 32, 4), (256, 1, 8, 128, 2),
                                         (128, 1, 11, 48, 7)])
@pytest.mark.parametrize("window", [0, 700])
def test_decode_of_many_columns_over_long_sequences(D, Hkv, G, P, T, window):
    """More than 16 query columns (8 at head_dim 256), sequences longer than a share of the keys, sinks, a lost page."""
    rng = np.random.default_rng(D + G + T)
    lens = [5000, 3, 2600, 64, 0, 1300]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    table[0, 2] = geo[0] + 7
    q = queries(rng, len(lens) * T, Hkv * G, D, "bf16")
    s = rng.normal(size=Hkv * G).astype(np.float32) * 2
    rows = [T] * len(lens)
    out, img = run_attention(geo, pages, table, lens, q, rows, "bf16", D ** -0.5, window, s, "f32", True, "decode", live=5,
                             spare_blocks=1)
    n = 5 * T
    want, parts = expected(geo, pages, table, lens, q, rows, D ** -0.5, window, s)
    check(out[:n], want[:n], bound_of(parts, False)[:n], "f32")
    assert np.isnan(out[n:]).all() and (img[n:] == 0xA5).all()
    image_is_of(img[:n], out[:n])


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_sequences_that_share_pages(call):
    """A prefix whose pages several sequences have in their tables."""
    rng = np.random.default_rng(31)
    D, Hkv, G, P, T = 128, 2, 3, 32, 3
    lens = [300, 290, 128]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    table[1, :4] = table[0, :4]
    table[2, :4] = table[0, :4]
    q = queries(rng, 9, Hkv * G, D, "f32")
    out, _ = run_attention(geo, pages, table, lens, q, [T] * 3, "f32", 0.1, 0, None, "f32", False, call)
    want, parts = expected(geo, pages, table, lens, q, [T] * 3, 0.1, 0, None)
    check(out, want, bound_of(parts, call == "prefill"), "f32")
