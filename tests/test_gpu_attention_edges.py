"""The cache's and the attention's calls at their edges: bytes around every output stay as they were, NaN stays in its row,
windows and buckets of extreme sizes, a workspace full of NaN, queries on another stream than the cache's writer."""
import numpy as np
import pytest

from quantized_activation_q4_gb300 import binding as qk
from tests.kv_helpers import bound_of, expected, page_table, random_pages, run_attention
from tests.test_gpu_attention import case, check, queries

pytestmark = pytest.mark.gpu

BAND = 4096


class Banded:
    """A buffer of n bytes between two bands of canaries."""

    def __init__(self, n, fill=0x5A):
        import torch
        self.n = n
        self.raw = torch.full((2 * BAND + (n + 255) // 256 * 256,), 0xC3, dtype=torch.uint8, device="cuda")
        self.view = self.raw[BAND:BAND + n]
        self.view.fill_(fill)

    def intact(self):
        import torch
        torch.cuda.synchronize()
        return bool((self.raw[:BAND] == 0xC3).all()) and bool((self.raw[BAND + self.n:] == 0xC3).all())


@pytest.mark.parametrize("D,Hkv,G,P,T", [(64, 1, 3, 16, 1), (128, 2, 7, 64, 3), (256, 1, 2, 32, 8), (128, 3, 16, 48, 2)])
def test_bytes_around_outputs_and_workspaces(D, Hkv, G, P, T):
    import torch
    rng = np.random.default_rng(D + T)
    Hq, lens = Hkv * G, [0, 17, 300, 2500]
    geo = (sum(-(-n // P) for n in lens) + 1, P, Hkv, D)
    table, _ = page_table(rng, geo, lens, spare=0)
    pages = Banded(geo[0] * qk.qk_kv_page_bytes(P, Hkv, D))
    pages.view.copy_(torch.from_numpy(random_pages(rng, geo).reshape(-1)))
    before = pages.view.clone()
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    td, ld = i32(table), i32(lens)
    rows, width = len(lens) * T, Hq * D
    q = torch.randn((rows, width), device="cuda").bfloat16()
    cache = qk.make_kv_cache(pages.view, *geo)
    out, img = Banded(rows * width * 4), Banded(rows * width // 32 * 36)
    attn = qk.make_attn(q, "bf16", width, Hq, td, table.shape[1], ld, 0.1, 0, None, out.view, "f32", width)
    ws = Banded(qk.qk_attn_decode_workspace_bytes(cache, Hq, len(lens), T), 0xFF)
    qk.qk_attn_decode(cache, attn, len(lens), T, img.view, width // 32, ws.view, ws.n)
    assert out.intact() and img.intact() and ws.intact() and pages.intact()
    first = i32(np.arange(len(lens) + 1) * T)
    qs, d = Banded(rows * width), Banded(rows * width // 32 * 2)
    wp = Banded(qk.qk_attn_prefill_workspace_bytes(cache, len(lens), table.shape[1] * P), 0xFF)
    qk.qk_attn_prefill(cache, attn, len(lens), rows, first, table.shape[1] * P, qs.view, d.view, width // 32, wp.view, wp.n)
    assert out.intact() and qs.intact() and d.intact() and wp.intact() and pages.intact()
    assert torch.equal(pages.view, before)
    # append and read
    n = 2 * P + 3
    x = torch.randn((n, (Hq + 2 * Hkv) * D), device="cuda")
    qo, kv = Banded(n * width * 2), Banded(n * 2 * Hkv * D * 4)
    slots = i32(np.arange(n) % (geo[0] * P))
    w = x.shape[1]
    qk.qk_kv_append(cache, "f32", x, w, Hq, x[:, width:], w, x[:, width + Hkv * D:], w, min(n, geo[0] * P), slots, None, "bf16",
                    qo.view, width)
    qk.qk_kv_read(cache, slots, n, "f32", kv.view, 2 * Hkv * D)
    assert qo.intact() and kv.intact() and pages.intact()
    assert qk.qk_device_faults() == 0


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_nan_stays_in_its_row_and_head(call):
    rng = np.random.default_rng(21)
    D, Hkv, G, P, T = 128, 2, 4, 32, 2
    lens = [100, 333]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    q = queries(rng, 4, Hkv * G, D, "f32")
    clean, _ = run_attention(geo, pages, table, lens, q, [T, T], "f32", 0.1, 0, None, "f32", False, call)
    q[1, 5, 77] = np.nan
    got, _ = run_attention(geo, pages, table, lens, q, [T, T], "f32", 0.1, 0, None, "f32", False, call)
    assert np.isnan(got[1, 5]).all()
    got[1, 5] = clean[1, 5]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_a_window_wider_than_any_sequence_is_none(call):
    rng = np.random.default_rng(22)
    D, Hkv, G, P, T = 64, 1, 2, 16, 3
    lens = [1, 90, 700]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    q = queries(rng, 9, G, D, "f32")
    a, b, c = (run_attention(geo, pages, table, lens, q, [T] * 3, "f32", 0.1, w, None, "f32", False, call)[0]
               for w in (0, 2 ** 31 - 1, 1 << 30))
    assert np.array_equal(a, b) and np.array_equal(a, c)


def test_a_bucket_of_many_sequences():
    """More sequences than a CTA has threads, most of them empty; more rows than a grid's second dimension."""
    rng = np.random.default_rng(23)
    D, Hkv, G, P, B = 64, 1, 1, 16, 70000
    lens = np.zeros(B, dtype=np.int64)
    some = np.sort(rng.choice(B, 40, replace=False))
    lens[some] = rng.integers(1, 300, 40)
    lens[B - 1] = 33
    geo, pages, table = case(rng, D, Hkv, P, lens)
    q = queries(rng, B, G, D, "f32")
    out, _ = run_attention(geo, pages, table, lens, q, [1] * B, "f32", 0.1, 0, None, "f32", False, "decode")
    busy = np.flatnonzero(lens)
    want, parts = expected(geo, pages, table[busy], lens[busy], q[busy], [1] * len(busy), 0.1, 0, None)
    check(out[busy], want, bound_of(parts, False), "f32")
    assert (out[lens == 0] == 0).all()
    keep = busy[:30]
    rows = np.zeros(300, dtype=np.int64)
    rows[:30] = 2
    out, _ = run_attention(geo, pages, np.concatenate([table[keep], np.full((270, table.shape[1]), -1, np.int32)]),
                           np.concatenate([lens[keep], np.zeros(270, np.int64)]), q[:60], rows, "f32", 0.1, 0, None, "f32",
                           False, "prefill")
    want, parts = expected(geo, pages, table[keep], lens[keep], q[:60], [2] * 30, 0.1, 0, None)
    check(out, want, bound_of(parts, True), "f32")


def test_values_of_large_and_small_scales():
    """Values' scales from binary16's smallest to its largest, in one sequence and across pages."""
    rng = np.random.default_rng(24)
    D, Hkv, G, P, T = 128, 1, 3, 16, 2
    lens = [400, 64]
    geo, pages, table = case(rng, D, Hkv, P, lens)
    view = pages.reshape(geo[0], 1, 1, 18 * D)
    for b, page in enumerate(table[0, :25]):
        size = 2.0 ** rng.integers(-20, 12)
        raw = view[page, 0, 0, 17 * D:].copy().view(np.float16).astype(np.float64) * size
        view[page, 0, 0, 17 * D:] = raw.astype(np.float16).view(np.uint8)
    view[table[1, 1], 0, 0, 17 * D:] = np.full(D // 2, 8000, dtype=np.float16).view(np.uint8)
    q = queries(rng, 2 * T, G, D, "f32")
    for call in ("decode", "prefill"):
        out, _ = run_attention(geo, pages, table, lens, q, [T, T], "f32", 0.1, 0, None, "f32", False, call)
        want, parts = expected(geo, pages, table, lens, q, [T, T], 0.1, 0, None)
        # binary16 holds a weight times a scale to 2^-25 of 2^14 / the largest scale at least: far below the bound here
        check(out, want, bound_of(parts, call == "prefill"), "f32", call)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("call,D,Hkv,G,lens,n", [
    ("prefill", 128, 2, 4, [4000, 0, 2500], 3),        # few rows behind many keys: shares of the keys, joined
    ("prefill", 256, 1, 2, [2048, 3, 3333], 5),
    ("decode", 128, 4, 8, [700, 0, 90] + [300] * 29, 2),   # 2048 heads of rows: the join of many
    ("decode", 64, 1, 4, [9000, 1, 0], 1),             # the join of few, many partial results
    ("decode", 128, 1, 8, [2000, 5, 0], 8),            # many columns
])
def test_nan_stays_in_its_row_and_head_over_joined_keys(call, D, Hkv, G, lens, n, sinks):
    rng = np.random.default_rng(D + n)
    geo, pages, table = case(rng, D, Hkv, 32, lens)
    rows = n * len(lens)
    q = queries(rng, rows, Hkv * G, D, "f32")
    sink = rng.standard_normal(Hkv * G).astype(np.float32) if sinks else None
    clean, _ = run_attention(geo, pages, table, lens, q, [n] * len(lens), "f32", 0.1, 0, sink, "f32", False, call)
    assert np.isfinite(clean).all()
    at = [(0, Hkv * G - 1), (n - 1, 0)]                # a row and head of the longest sequence
    for i, h in at:
        q[i, h, 33] = np.nan
    got, _ = run_attention(geo, pages, table, lens, q, [n] * len(lens), "f32", 0.1, 0, sink, "f32", False, call)
    for i, h in at:
        assert np.isnan(got[i, h]).all()
        got[i, h] = clean[i, h]
    assert np.array_equal(got, clean)
