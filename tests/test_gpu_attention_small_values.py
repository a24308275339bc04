"""Decode over values whose scales are all small, all large or change: weights far below the largest keep their part."""
import numpy as np
import pytest

from oracle import kv as OK
from quantized_activation_q4_gb300 import binding as qk
from tests.kv_helpers import bound_of, expected, run_attention
from tests.test_gpu_attention import case, queries

pytestmark = pytest.mark.gpu

SHAPES = [(64, 1, 4, 1), (64, 1, 16, 1), (128, 1, 7, 1), (128, 1, 8, 2), (256, 1, 4, 1),      # one kernel
          (128, 1, 8, 8), (64, 1, 8, 4), (256, 1, 8, 2), (256, 1, 8, 4)]                     # the one of many columns


@pytest.mark.parametrize("D,Hkv,G,T", SHAPES)
@pytest.mark.parametrize("k", [8, 11, 14])
@pytest.mark.parametrize("size", [1.1 * 2.0 ** -4, 1.1 * 2.0 ** -8, 1.1 * 2.0 ** -14, 1.1 * 2.0 ** -16, 1.5 * 2.0 ** -20, 2.0 ** -24,
                                  0.3, 8.8, 600.0, 60000.0])
def test_one_peak_and_a_long_flat_tail(D, Hkv, G, T, k, size):
    """All values are equal, so the output is that value whatever the weights: keys 1.37 * 2^-k below the peak.

    Many sequences over the same pages, so that a share of the keys is a whole sequence or two. The weight is rounded to
    binary16 and so is its product with the scale: 2^-10 in all. The least step adds 2^-28 of the peak's weight times the
    largest value a key (2^-25 for scales of 64 and more, whose weights are held lower), sums add 2^-23 for each of the
    512 steps of 16 keys and of the parts joined."""
    import torch
    n, P, B = 8192, 256, 1200
    geo = (n // P, P, Hkv, D)
    g = np.zeros((n // P, Hkv, P // 16, 18 * D), dtype=np.uint8)
    kb, ks, vb, vs = OK.code_places(D)
    view = g.reshape(-1, 18 * D)
    view[:, :8 * D] = 0x88
    view[:, 8 * D:9 * D] = np.ones(D // 2, dtype=np.float16).view(np.uint8)
    view[:, 9 * D:17 * D] = 0xFF                          # (15 - 8) * d everywhere
    view[:, 17 * D:] = np.full(D // 2, size, dtype=np.float16).view(np.uint8)
    first = view.reshape(n // P, P // 16, 18 * D)[0]
    for group in range(0, 16, 4):                         # a peak for each warp: tokens 0, 64, 128, 192
        byte, shift = kb[0, 0], ks[0, 0]
        first[group, byte] = (first[group, byte] & ~(15 << shift)) | (15 << shift)
    scale = float(np.float32((k * np.log(2.0) - np.log(1.37)) / 7))
    Hq, width = Hkv * G, Hkv * G * D
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    table, lens = i32(np.tile(np.arange(n // P), (B, 1))), i32(np.full(B, n))
    q = torch.zeros((B * T, Hq, D), device="cuda")
    q[:, :, 0] = 1.0
    out = torch.full((B * T, width), float("nan"), device="cuda")
    pd = torch.from_numpy(g.reshape(-1)).cuda()
    cache = qk.make_kv_cache(pd, *geo)
    attn = qk.make_attn(q, "f32", width, Hq, table, n // P, lens, scale, 0, None, out, "f32", width)
    ws = torch.full((qk.qk_attn_decode_workspace_bytes(cache, Hq, B, T),), 0xFF, dtype=torch.uint8, device="cuda")
    qk.qk_attn_decode(cache, attn, B, T, None, 0, ws, ws.numel())
    torch.cuda.synchronize()
    value = 7.0 * float(np.float16(size))
    off = float((out.double() / value - 1).abs().max())
    assert off <= 2.0 ** -10 + n * 2.0 ** (-25 if size >= 64 else -28) + 2 * 512 * 2.0 ** -23, off
    assert qk.qk_device_faults() == 0


@pytest.mark.parametrize("D,Hkv,G,T", SHAPES)
@pytest.mark.parametrize("order", ["rising", "falling", "a large one last"])
def test_scales_that_change_along_a_sequence(D, Hkv, G, T, order):
    """Sequences whose values' scales go from 2^-20 up to 8 or down again, against the definition.

    Beside the bound of the ordinary roundings a key adds 2^-28 of the largest weight times the largest value and, where
    scales are above 1, the largest scale."""
    rng = np.random.default_rng(D + T)
    lens = [3000, 700, 90]
    geo, pages, table = case(rng, D, Hkv, 16, lens)
    view = pages.reshape(geo[0], Hkv, 18 * D)
    for b, length in enumerate(lens):
        used = -(-length // 16)
        for i in range(used):
            x = i / max(1, used - 1)
            power = {"rising": -20 + 23 * x, "falling": 3 - 23 * x, "a large one last": 3 if i == used - 1 else -14}[order]
            with np.errstate(invalid="ignore"):
                raw = view[table[b, i], :, 17 * D:].copy().view(np.float16).astype(np.float64) * 2.0 ** int(power)
            view[table[b, i], :, 17 * D:] = raw.astype(np.float16).view(np.uint8)
    q = queries(rng, T * len(lens), Hkv * G, D, "f32")
    rows = [T] * len(lens)
    out, _ = run_attention(geo, pages, table, lens, q, rows, "f32", 0.1, 0, None, "f32", False, "decode")
    want, parts = expected(geo, pages, table, lens, q, rows, 0.1, 0, None)
    more, at = np.zeros_like(want), 0
    for v, o, ps, _ in parts:
        for h, i, keys, p, _ in ps:
            if len(p):
                top = np.abs(v[keys, h // G]).max()
                more[at + i, h] = len(p) * 2.0 ** -28 * p.max() * top * max(1.0, top / 7)
        at += T
    tol = bound_of(parts, False) + 2.0 ** -24 * np.abs(want) + more
    assert (np.abs(out - want) <= tol).all(), np.nanmax(np.abs(out - want) - tol)
