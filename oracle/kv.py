"""The 4-bit key/value cache and its attention on the CPU: plain numpy, from the definitions in include/qk.h.

Shares no code with the GPU path. Binary64 except the 4-bit blocks, whose arithmetic the definition fixes to binary32.
"""
from __future__ import annotations

import numpy as np

GROUP = 16


def group_bytes(D: int) -> int:
    return 18 * D


def code_places(D: int):
    """(k byte, k shift, v byte, v shift) of token i, column x inside a group: four [16, D] arrays."""
    i, x = np.arange(GROUP)[:, None], np.arange(D)[None, :]
    b, W = x // 32, min(4, D // 32)
    kb = ((b // W * 16 + i) * 4 + x % 16 // 4) * 4 * W + b % W * 4 + x % 4
    vb = 9 * D + ((x // 64 * 8 + x % 8) * 4 + i % 8 // 2) * 16 + x // 16 % 4 * 4 + 2 * (i % 2) + i // 8
    whole = np.zeros((GROUP, D), dtype=np.int64)
    return kb + whole, 4 * (x % 32 >= 16) + whole, vb + whole, 4 * (x % 16 >= 8) + whole


def scale_places(D: int):
    """(k byte, v byte) of the scale of token i, block b: two [16, D / 32] arrays."""
    i, b, nb = np.arange(GROUP)[:, None], np.arange(D // 32)[None, :], D // 32
    return 8 * D + 2 * (i * nb + b), 17 * D + 2 * ((i % 8 // 2 * nb + b) * 4 + i % 2 + i // 8 * 2)


def q4_block(x: np.ndarray):
    """x [..., 32] binary32 -> codes 0..15 and half scales [...]."""
    x = np.asarray(x, dtype=np.float32)
    clean = np.where(np.isnan(x), np.float32(0), x)
    first = np.argmax(np.abs(clean), axis=-1)[..., None]
    e = np.take_along_axis(clean, first, -1)
    d = np.clip(e / np.float32(-8), np.float32(-65504), np.float32(65504))
    with np.errstate(all="ignore"):
        r = np.rint(np.where(d != 0, clean / np.where(d != 0, d, np.float32(1)), np.float32(0)))
    codes = np.clip(np.nan_to_num(r, nan=0.0, posinf=100, neginf=-100), -8, 7).astype(np.int64) + 8
    return codes, d[..., 0].astype(np.float16)


def put(pages: np.ndarray, geometry, slot: int, codes: np.ndarray, scales: np.ndarray) -> None:
    """Stores one token: codes [2, Hkv, D] (k, v) and half scales [2, Hkv, D/32], into pages (uint8, in place).
    geometry = (n_pages, P, Hkv, D)."""
    n_pages, P, Hkv, D = geometry
    if slot < 0 or slot >= n_pages * P:
        return
    view = pages.reshape(n_pages, Hkv, P // GROUP, group_bytes(D))
    page, at = slot // P, slot % P
    kb, ksh, vb, vsh = (z[at % GROUP] for z in code_places(D))
    sk, sv = (z[at % GROUP] for z in scale_places(D))
    for h in range(Hkv):
        g = view[page, h, at // GROUP]
        for byte, shift, c, sb, s in ((kb, ksh, codes[0, h], sk, scales[0, h]), (vb, vsh, codes[1, h], sv, scales[1, h])):
            g[byte] = 0
            np.add.at(g, byte, (c << shift).astype(np.uint8))
            raw = s.astype(np.float16).view(np.uint16)
            g[sb], g[sb + 1] = (raw & 255).astype(np.uint8), (raw >> 8).astype(np.uint8)


def values(pages: np.ndarray, geometry):
    """Every token's values: k and v [n_pages * P, Hkv, D] in binary64."""
    n_pages, P, Hkv, D = geometry
    g = pages.reshape(n_pages, Hkv, P // GROUP, group_bytes(D))
    kb, ksh, vb, vsh = code_places(D)
    out = []
    for byte, shift, sb in ((kb, ksh, scale_places(D)[0]), (vb, vsh, scale_places(D)[1])):
        code = (g[..., byte] >> shift) & 15
        d = (g[..., sb].astype(np.uint16) | g[..., sb + 1].astype(np.uint16) << 8).view(np.float16).astype(np.float64)
        with np.errstate(invalid="ignore"):
            v = (code.astype(np.float64) - 8) * np.repeat(d, 32, axis=-1)
        out.append(v.transpose(0, 2, 3, 1, 4).reshape(n_pages * P, Hkv, D))
    return out


def rotate(x: np.ndarray, kind: str, dims: int, positions: np.ndarray, freqs: np.ndarray) -> np.ndarray:
    """x [T, heads, D] by positions [A, T] and freqs [A, dims / 2]; the angle in extended precision."""
    p, f = positions.astype(np.longdouble), freqs.astype(np.longdouble)
    angle = (p[:, :, None] * f[:, None, :]).sum(0)
    c, s = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
    x = x.astype(np.float64).copy()
    i = np.arange(dims // 2)
    lo, hi = (i, i + dims // 2) if kind == "halves" else (2 * i, 2 * i + 1)
    a, b = x[..., lo].copy(), x[..., hi].copy()
    x[..., lo], x[..., hi] = a * c - b * s, b * c + a * s
    return x


def visible(length: int, n: int, i: int, window: int):
    end = length - n + i + 1
    return (max(0, end - window) if window else 0), max(0, end)


def attention(q, k, v, there, n, scale, window=0, sinks=None):
    """q [n, Hq, D], k and v [L, Hkv, D] of one sequence, there [L] whether a key's page exists.

    Returns out [n, Hq, D] and, for error bounds: p (weights after normalisation) as a list of (head, row, keys, p, a)
    where a_j = scale * sum_x |q_x k_jx|."""
    L, Hkv, D = k.shape
    Hq = q.shape[1]
    G = Hq // Hkv
    out = np.zeros((n, Hq, D))
    parts = []
    for i in range(n):
        lo, hi = visible(L, n, i, window)
        keys = np.arange(lo, hi)
        keys = keys[there[lo:hi]]
        for h in range(Hq):
            kk, vv = k[keys, h // G], v[keys, h // G]
            s = scale * (kk @ q[i, h])
            top = max([s.max()] if len(s) else [-np.inf])
            if sinks is not None:
                top = max(top, float(sinks[h]))
            if not np.isfinite(top):
                parts.append((h, i, keys, np.zeros(0), np.zeros(0)))
                continue
            w = np.exp(s - top)
            total = w.sum() + (np.exp(float(sinks[h]) - top) if sinks is not None else 0.0)
            p = w / total
            out[i, h] = p @ vv
            parts.append((h, i, keys, p, scale * (np.abs(kk) @ np.abs(q[i, h]))))
    return out, parts
