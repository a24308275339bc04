"""Caches, rows and error bounds for the tests of the 4-bit cache and its attention."""
from __future__ import annotations

import numpy as np

from oracle import kv as OK
from quantized_activation_q4_gb300 import binding as qk


def bf16(x: np.ndarray) -> np.ndarray:
    """x rounded to bfloat16, as binary32."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().float().numpy()


def to_dev(x: np.ndarray, elem: str):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    return t.bfloat16() if elem == "bf16" else t


def random_pages(rng, geometry) -> np.ndarray:
    """Random codes, scales of either sign between 0.05 and 0.4."""
    n_pages, P, Hkv, D = geometry
    g = rng.integers(0, 256, (n_pages, Hkv, P // 16, 18 * D), dtype=np.uint8)
    for lo in (8 * D, 17 * D):
        d = rng.uniform(0.05, 0.4, g.shape[:3] + (D // 2,)) * rng.choice([-1, 1], g.shape[:3] + (D // 2,))
        g[..., lo:lo + D] = d.astype(np.float16).view(np.uint8)
    return g


def poison(pages: np.ndarray, geometry, used) -> None:
    """Scales of every slot outside `used` become NaN and infinities, their codes 255s."""
    n_pages, P, Hkv, D = geometry
    kb, _, vb, _ = OK.code_places(D)
    sk, sv = OK.scale_places(D)
    used = set(int(s) for s in used)
    for slot in range(n_pages * P):
        if slot in used:
            continue
        g = pages[slot // P, :, slot % P // 16]
        i = slot % 16
        g[:, kb[i]] = 255
        g[:, vb[i]] = 255
        bits = (0x7E00, 0x7C00, 0xFC00)[slot % 3]
        for s in (sk[i], sv[i]):
            g[:, s], g[:, s + 1] = bits & 255, bits >> 8


def page_table(rng, geometry, lens, spare=1):
    """Disjoint random pages for every sequence; unused entries -1. Returns table [B, stride] and each key's slot."""
    n_pages, P, _, _ = geometry
    need = [-(-int(n) // P) for n in lens]
    assert sum(need) <= n_pages
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max(1, max(need, default=1)) + spare), -1, dtype=np.int32)
    slots, at = [], 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        j = np.arange(int(lens[b]))
        slots.append(table[b, j // P].astype(np.int64) * P + j % P if len(j) else np.zeros(0, dtype=np.int64))
    return table, slots


# Half steps of the roundings, relative to the value.
H16, HB16 = 2.0 ** -11, 2.0 ** -8


def decode_error(v, out, parts, G, kv_rounded=False):
    """A bound of |computed - exact| for the attention, columnwise [n, Hq, D].

    A weight exp(s_j) is off by a relative eps_j: the operands of s_j are rounded to binary16, the queries always, the
    keys where the kernel stores them in binary16 (kv_rounded), so s_j is off by 2^-11 a_j for each, with
    a_j = scale * sum |q k_j|; the weight itself is rounded (twice where it is multiplied by a value's scale: 2^-10
    covers both). Binary32 adds: sums of N terms N * 2^-24 (doubled: the tensor cores cut instead of rounding), the
    exponent's argument |s| 2^-23 (|s| <= a_j), the exponential 2^-21. Then out = sum w v / sum w is off by
    sum_j p_j eps_j (|v_j| + |out|); binary16 values add 2^-11 |v_j|."""
    bound = np.zeros_like(out)
    for h, i, keys, p, a in parts:
        if not len(p):
            continue
        eps = a * (H16 * (2 if kv_rounded else 1) + 2.0 ** -22) + 2 * H16 + (len(p) + 64) * 2.0 ** -23 + 2.0 ** -20
        eps = np.expm1(np.minimum(eps, 40.0))
        av = np.abs(v[keys, h // G])
        far = (p * eps) @ (av + np.abs(out[i, h]))
        # whatever the weights, the output lies between the values
        bound[i, h] = np.minimum(far, (1 + 2.0 ** -8) * av.max(0) + np.abs(out[i, h])) + (H16 * (p @ av) if kv_rounded else 0)
    return bound


def run_attention(geometry, pages, table, lens, q, q_rows, elem, scale, window, sinks, out_elem, image, call, live=None,
                  pad=0, spare_blocks=0, max_kv=None):
    """One call of qk_attn_decode or qk_attn_prefill on the device. q [rows, Hq, D]; q_rows: rows of each sequence.

    Returns (out or None, image bytes [rows, blocks, 36] or None). Outputs start from NaN / 0xA5 bytes."""
    import torch
    n_pages, P, Hkv, D = geometry
    rows, Hq = q.shape[0], q.shape[1]
    width = Hq * D
    qd = torch.full((max(1, rows), width + pad), float("nan"), device="cuda")
    qd[:rows, :width] = torch.from_numpy(q.reshape(rows, width).astype(np.float32)).cuda()
    qd = qd.bfloat16() if elem == "bf16" else qd
    t32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
    td, ld, pd = t32(table), t32(lens), torch.from_numpy(pages.reshape(-1)).cuda()
    sd = None if sinks is None else torch.from_numpy(sinks.astype(np.float32)).cuda()
    out = None
    if out_elem:
        out = torch.full((max(1, rows), width + pad), float("nan"), device="cuda")
        out = out.bfloat16() if out_elem == "bf16" else out
    blocks = width // 32 + spare_blocks
    cache = qk.make_kv_cache(pd, n_pages, P, Hkv, D)
    attn = qk.make_attn(qd, elem, width + pad, Hq, td, table.shape[1], ld, scale, window, sd, out, out_elem or "f32",
                        width + pad)
    lv = None if live is None else t32([live])
    B = len(lens)
    img = None
    if call == "decode":
        T = q_rows[0]
        n = qk.qk_attn_decode_workspace_bytes(cache, Hq, B, T)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        if image:
            img = torch.full((rows, blocks, 36), 0xA5, dtype=torch.uint8, device="cuda")
        qk.qk_attn_decode(cache, attn, B, T, img, blocks, ws, n, lv)
        torch.cuda.synchronize()
        got = None if img is None else img.cpu().numpy()
    else:
        first = t32(np.concatenate([[0], np.cumsum(q_rows)]))
        max_kv = max_kv or table.shape[1] * P
        n = qk.qk_attn_prefill_workspace_bytes(cache, B, max_kv)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        qs = d = None
        if image:
            qs = torch.full((rows, blocks * 32), 0x25, dtype=torch.int8, device="cuda")
            d = torch.full((rows, blocks), 0x2525, dtype=torch.int16, device="cuda")
        qk.qk_attn_prefill(cache, attn, B, rows, first, max_kv, qs, d, blocks, ws, n, lv)
        torch.cuda.synchronize()
        got = None if qs is None else (qs.cpu().numpy(), d.cpu().numpy().view(np.uint16))
    o = None
    if out is not None:
        full = out.float().cpu().numpy()
        assert np.isnan(full[:, width:]).all()          # nothing is written between rows
        o = full[:rows, :width].reshape(rows, Hq, D)
    assert qk.qk_device_faults() == 0
    return o, got


def expected(geometry, pages, table, lens, q, q_rows, scale, window, sinks):
    """(out [rows, Hq, D], parts per sequence, values): the definition in binary64, q as given."""
    n_pages, P, Hkv, D = geometry
    k, v = OK.values(pages, geometry)
    outs, bounds_of, at = [], [], 0
    G = q.shape[1] // Hkv
    for b, n in enumerate(q_rows):
        L = min(max(int(lens[b]), 0), table.shape[1] * P)
        j = np.arange(L)
        page = table[b, j // P] if L else np.zeros(0, dtype=np.int64)
        there = (page >= 0) & (page < n_pages)
        slot = np.where(there, page, 0).astype(np.int64) * P + j % P
        kk = np.where(there[:, None, None], k[slot], 0.0) if L else np.zeros((0, Hkv, D))
        vv = np.where(there[:, None, None], v[slot], 0.0) if L else np.zeros((0, Hkv, D))
        o, parts = OK.attention(q[at:at + n].astype(np.float64), kk, vv, there, n, scale, window, sinks)
        outs.append(o)
        bounds_of.append((vv, o, parts, G))
        at += n
    return np.concatenate(outs) if outs else np.zeros((0,) + q.shape[1:]), bounds_of


def bound_of(bounds_of, kv_rounded):
    return np.concatenate([decode_error(v, o, parts, G, kv_rounded) for v, o, parts, G in bounds_of])
