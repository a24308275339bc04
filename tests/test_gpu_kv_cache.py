"""qk_kv_append and qk_kv_read against the definitions: bytes where nothing is rotated, else the codes next to what
binary64 gives."""
import numpy as np
import pytest

from oracle import kv as OK
from quantized_activation_q4_gb300 import binding as qk
from tests.kv_helpers import HB16, bf16, random_pages, to_dev

pytestmark = pytest.mark.gpu


def append(geo, pages, x, elem, Hq, slots, rope, q_elem, pad=0, q_pad=0, live=None, fused=True):
    """Returns (q rows or None, pages) after one call. x [T, Hq + 2 Hkv, D] binary32, rounded to elem by the caller."""
    import torch
    n_pages, P, Hkv, D = geo
    T, heads = x.shape[0], x.shape[1]
    pd = torch.from_numpy(pages.reshape(-1).copy()).cuda()
    cache = qk.make_kv_cache(pd, n_pages, P, Hkv, D)
    sd = torch.from_numpy(np.asarray(slots, dtype=np.int32)).cuda()
    if fused:
        buf = to_dev(np.full((T, heads * D + pad), np.nan), elem)
        buf[:, :heads * D] = to_dev(x.reshape(T, -1), elem)
        q, k, v = buf, buf[:, Hq * D:], buf[:, (Hq + Hkv) * D:]
        st = (heads * D + pad,) * 3
    else:   # separate buffers, each with its own stride and an odd first element
        q, k, v, st = None, None, None, []
        parts = []
        for i, (lo, hi) in enumerate(((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, heads))):
            w = (hi - lo) * D
            b = to_dev(np.full((T * (w + pad + i) + 1,), np.nan), elem)
            view = b[1:].view(T, w + pad + i)
            if w:
                view[:, :w] = to_dev(x[:, lo:hi].reshape(T, -1), elem)
            parts.append(view)
            st.append(w + pad + i)
        q, k, v = parts
    r = None
    if rope is not None:
        kind, dims, pos, freqs = rope
        pos_d = torch.from_numpy(np.ascontiguousarray(pos, dtype=np.int32)).cuda()
        f_d = torch.from_numpy(np.ascontiguousarray(freqs, dtype=np.float32)).cuda()
        r = qk.make_rope(kind, dims, pos.shape[0], pos_d, f_d)
    q_out = to_dev(np.full((T, Hq * D + q_pad), np.nan), q_elem) if Hq else None
    lv = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    qk.qk_kv_append(cache, elem, q if Hq else None, st[0], Hq, k, st[1], v, st[2], T, sd, r, q_elem, q_out, Hq * D + q_pad, lv)
    torch.cuda.synchronize()
    qo = None
    if Hq:
        qo = q_out.float().cpu().numpy()
        assert np.isnan(qo[:, Hq * D:]).all()
        qo = qo[:, :Hq * D].reshape(T, Hq, D)
    return qo, pd.cpu().numpy().reshape(pages.shape)


def rows(rng, T, heads, D, elem):
    x = rng.normal(size=(T, heads, D)).astype(np.float32) * rng.uniform(0.1, 4, (T, heads, 1)).astype(np.float32)
    return bf16(x) if elem == "bf16" else x


@pytest.mark.parametrize("D,Hq,Hkv,P", [(64, 3, 1, 16), (128, 28, 4, 64), (256, 2, 2, 32), (64, 0, 5, 48)])
@pytest.mark.parametrize("elem,fused,pad", [("f32", True, 0), ("bf16", True, 4), ("f32", False, 3), ("bf16", False, 1)])
def test_unrotated_rows_are_stored_byte_for_byte(D, Hq, Hkv, P, elem, fused, pad):
    rng = np.random.default_rng(D + Hq + pad)
    geo, T = (5, P, Hkv, D), 37
    pages = random_pages(rng, geo)
    x = rows(rng, T, Hq + 2 * Hkv, D, elem)
    x[4, :, :32] = 0                                     # a block of zeros
    x[5, :, 7] = -(x[5, :, 9]) * 0 - 9.0                 # equal magnitudes of either sign
    x[5, :, 9] = 9.0
    x[6, :, 40] = np.nan
    x[7, :, 3] = np.inf
    x[8, :, 33] = 3e38
    x[9, :, 32:64] *= 1e-30
    if elem == "bf16":
        x = bf16(x)
    slots = rng.permutation(5 * P)[:T]
    slots[10], slots[11], slots[12] = -1, 5 * P, 2 ** 31 - 1       # not stored
    want = pages.copy()
    for t in range(T):
        codes, d = OK.q4_block(x[t, Hq:].reshape(2, Hkv, D // 32, 32))
        OK.put(want, geo, int(slots[t]), codes.reshape(2, Hkv, D), d)
    q, got = append(geo, pages, x, elem, Hq, slots, None, "f32", pad, 5, None, fused)
    assert np.array_equal(got, want)
    if Hq:
        assert np.array_equal(q, x[:, :Hq], equal_nan=True)


ROPES = [("halves", 64, 64, 1), ("adjacent", 64, 64, 1), ("halves", 128, 96, 3), ("adjacent", 128, 40, 2),
         ("halves", 256, 8, 1), ("adjacent", 256, 256, 4), ("halves", 128, 128, 4)]


@pytest.mark.parametrize("kind,D,dims,axes", ROPES)
@pytest.mark.parametrize("elem,q_elem", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_rotated_rows(kind, D, dims, axes, elem, q_elem):
    rng = np.random.default_rng(D + dims + axes)
    geo, T, Hq, Hkv = (4, 32, 2, D), 53, 6, 2
    pages = random_pages(rng, geo)
    x = rows(rng, T, Hq + 2 * Hkv, D, elem)
    pos = rng.integers(0, 40000, (axes, T))
    pos[:, 0], pos[:, 1] = 0, 1
    pos[0, 2], pos[0, 3], pos[0, 4], pos[-1, 5] = 2 ** 31 - 1, -2 ** 31, 10 ** 6, -777
    freqs = rng.uniform(0.0, 1.0, (axes, dims // 2)).astype(np.float32)
    freqs[0, 0] = 1.0
    if axes > 1:
        freqs[1:, ::2] = 0.0
    slots = rng.permutation(4 * 32)[:T]
    live = 50
    q, got = append(geo, pages, x, elem, Hq, slots, (kind, dims, pos, freqs), q_elem, 0, 0, live, True)
    ref = OK.rotate(x[:, :Hq + Hkv], kind, dims, pos, freqs)
    # a column is x c +- y s: c and s within 2^-22, three roundings of 2^-24 of |x| + |y| <= sqrt(2) of the pair's length
    i = np.arange(dims // 2)
    lo, hi = (i, i + dims // 2) if kind == "halves" else (2 * i, 2 * i + 1)
    size = np.zeros_like(ref)
    size[..., lo] = size[..., hi] = np.abs(x[:, :Hq + Hkv][..., lo]) + np.abs(x[:, :Hq + Hkv][..., hi])
    err = size * (2.0 ** -22 + 3 * 2.0 ** -24)
    tol = err[:live, :Hq] + (HB16 * np.abs(ref[:live, :Hq]) if q_elem == "bf16" else 0)
    assert (np.abs(q[:live] - ref[:live, :Hq]) <= tol * 1.001).all()
    assert np.isnan(q[live:]).all()
    # stored codes: those of binary64, or their neighbour where the quotient is that near a border
    want = pages.copy()
    gv, wv = got.reshape(4, 2, 2, 18 * D), None
    for t in range(live):
        kv = np.concatenate([ref[t, Hq:], x[t, Hq + Hkv:].astype(np.float64)]).reshape(2, Hkv, D // 32, 32)
        e = np.concatenate([err[t, Hq:], np.zeros((Hkv, D))]).reshape(2, Hkv, D // 32, 32)
        top = np.abs(kv).max(-1, keepdims=True)
        g = gv[slots[t] // 32, :, slots[t] % 32 // 16]
        s = slots[t] % 16
        kb, ksh, vb, vsh = (z[s] for z in OK.code_places(D))
        sk, sv = (z[s] for z in OK.scale_places(D))
        codes = np.stack([g[:, kb] >> ksh & 15, g[:, vb] >> vsh & 15]).reshape(kv.shape).astype(np.int64)
        d = np.stack([g[:, b].astype(np.uint16) | g[:, b + 1].astype(np.uint16) << 8 for b in (sk, sv)]).view(np.float16)
        d = d.astype(np.float64)[..., None]
        assert (np.abs(np.abs(d) - top / 8) <= top / 8 * 2.0 ** -11 + e.max(-1, keepdims=True) / 8 + 2.0 ** -25).all()
        sign = np.sign(d)
        exact = sign * kv / (top / 8)
        slack = (e + e.max(-1, keepdims=True)) / (top / 8) + 1e-6
        assert (np.abs(codes - 8 - np.clip(exact, -8, 7)) <= 0.5 + slack).all()
        # the value of the largest magnitude has code 0
        assert (np.take_along_axis(codes, np.abs(kv).argmax(-1)[..., None], -1) == 0).mean() >= 0.99
    # every other slot is as it was
    k0, v0 = OK.values(pages, geo)
    k1, v1 = OK.values(got, geo)
    other = np.setdiff1d(np.arange(128), slots[:live])
    assert np.array_equal(k0[other], k1[other]) and np.array_equal(v0[other], v1[other])


@pytest.mark.parametrize("D,Hkv,P", [(64, 1, 16), (128, 4, 64), (256, 3, 16), (128, 8, 256)])
@pytest.mark.parametrize("elem", ["f32", "bf16"])
def test_read(D, Hkv, P, elem):
    import torch
    rng = np.random.default_rng(D + P)
    geo, n, pad = (3, P, Hkv, D), 41, 3
    pages = random_pages(rng, geo)
    slots = rng.integers(0, 3 * P, n)                    # slots may repeat
    slots[3], slots[4], slots[5] = -1, 3 * P, 2 ** 31 - 1
    pd = torch.from_numpy(pages.reshape(-1)).cuda()
    width = 2 * Hkv * D
    out = to_dev(np.full((n, width + pad), np.nan), elem)
    live = torch.tensor([38], dtype=torch.int32, device="cuda")
    qk.qk_kv_read(qk.make_kv_cache(pd, *geo), torch.from_numpy(slots.astype(np.int32)).cuda(), n, elem, out, width + pad, live)
    torch.cuda.synchronize()
    got = out.float().cpu().numpy()
    k, v = OK.values(pages, geo)
    skipped = [3, 4, 5, 38, 39, 40]
    assert np.isnan(got[skipped]).all() and np.isnan(got[:, width:]).all()
    keep = np.setdiff1d(np.arange(n), skipped)
    want = np.concatenate([k[slots[keep]].reshape(len(keep), -1), v[slots[keep]].reshape(len(keep), -1)], 1)
    want = bf16(want) if elem == "bf16" else want.astype(np.float32)
    assert np.array_equal(got[keep, :width], want)


@pytest.mark.parametrize("T,live", [(700, 699), (2050, 2049)])
@pytest.mark.parametrize("kind", ["halves", "adjacent"])
def test_many_tokens_are_stored_as_few_are(T, live, kind):
    """Calls of many tokens take other launch shapes: the same bytes as calls of fifty."""
    import torch
    rng = np.random.default_rng(T)
    geo, Hq = (40, 64, 2, 64), 5
    n_pages, P, Hkv, D = geo
    x = torch.from_numpy(rows(rng, T, Hq + 2 * Hkv, D, "f32").reshape(T, -1)).cuda()
    width = x.shape[1]
    slots = torch.from_numpy(rng.permutation(n_pages * P)[:T].astype(np.int32)).cuda()
    pos = torch.from_numpy(rng.integers(0, 100000, (2, T)).astype(np.int32)).cuda()
    freqs = torch.from_numpy(rng.uniform(0, 1, (2, 24)).astype(np.float32)).cuda()
    got = []
    for step in (T, 50):
        pages = torch.full((n_pages * qk.qk_kv_page_bytes(P, Hkv, D),), 0x5A, dtype=torch.uint8, device="cuda")
        q = torch.full((T, Hq * D), float("nan"), device="cuda")
        for t in range(0, T, step):
            n = min(step, T - t)
            part = pos[:, t:t + n].contiguous()
            lv = torch.tensor([live - t], dtype=torch.int32, device="cuda")
            qk.qk_kv_append(qk.make_kv_cache(pages, *geo), "f32", x[t:], width, Hq, x[t:, Hq * D:], width,
                            x[t:, (Hq + Hkv) * D:], width, n, slots[t:], qk.make_rope(kind, 48, 2, part, freqs), "f32", q[t:],
                            Hq * D, lv)
            torch.cuda.synchronize()
        got.append((pages, q))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1][:live], got[1][1][:live])
    assert torch.isnan(got[0][1][live:]).all()


def test_pages_past_four_gigabytes():
    """Offsets past 32 bits: a cache of 4.5 GB, its first and last pages."""
    import torch
    D, Hkv, P = 256, 8, 4096
    per = qk.qk_kv_page_bytes(P, Hkv, D)
    n_pages = (9 << 29) // per + 1
    pd = torch.zeros((n_pages * per,), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    x = rng.normal(size=(4, 2 * Hkv, D)).astype(np.float32)
    slots = np.array([0, n_pages * P - 1, (n_pages - 1) * P, n_pages * P // 2], dtype=np.int32)
    cache = qk.make_kv_cache(pd, n_pages, P, Hkv, D)
    sd, xd = torch.from_numpy(slots).cuda(), torch.from_numpy(x.reshape(4, -1)).cuda()
    w = 2 * Hkv * D
    qk.qk_kv_append(cache, "f32", None, 0, 0, xd, w, xd[:, Hkv * D:], w, 4, sd, None, "f32", None, 0)
    out = torch.zeros((4, w), device="cuda")
    qk.qk_kv_read(cache, sd, 4, "f32", out, w)
    torch.cuda.synchronize()
    codes, d = OK.q4_block(x.reshape(4, -1, 32))
    want = ((codes - 8) * d[..., None].astype(np.float32)).astype(np.float32).reshape(4, -1)
    assert np.array_equal(out.cpu().numpy(), want)
    assert int((pd != 0).sum()) <= 4 * Hkv * 18 * D // 16
