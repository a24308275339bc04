"""Refusals of the cache's and the attention's calls: host checks, nothing is launched (the addresses are never read)."""
import ctypes as C

import pytest

from quantized_activation_q4_gb300 import binding as qk

PAGES, X, Y, S, TAB, LEN, WS, IMG, POS, FRQ, LIVE = (0x10000000 * (i + 1) for i in range(11))
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    return qk.load()


def cache(pages=PAGES, n=8, P=32, H=2, D=128):
    return qk.qk_kv_cache(pages, n, P, H, D, 0)


def append(lib, c=None, elem=0, q=X, qs=1024, Hq=4, k=X + 0x100000, ks=256, v=X + 0x200000, vs=256, T=3, slots=S, rope=None,
           qe=0, qo=Y, qos=1024, live=None):
    p = lambda a: C.c_void_p(a) if a else None
    return lib.qk_kv_append(C.byref(c or cache()), elem, p(q), qs, Hq, p(k), ks, p(v), vs, T, p(slots),
                            None if rope is None else C.byref(rope), qe, p(qo), qos, p(live), None)


def rope(kind=0, dims=128, axes=1, pos=POS, freqs=FRQ):
    return qk.qk_rope(kind, dims, axes, 0, pos, freqs)


def test_append(lib):
    n0 = lib.qk_launch_count()
    assert append(lib, cache(D=96)) == 5
    for bad in (cache(pages=None), cache(pages=PAGES + 8), cache(n=0), cache(n=1 << 27), cache(P=24), cache(P=0),
                cache(P=8192), cache(H=0), cache(H=257)):
        assert append(lib, bad) == 1
    assert append(lib, elem=2) == 1 and append(lib, qe=-1) == 1
    assert append(lib, T=-1) == 1 and append(lib, T=(1 << 24) + 1) == 1
    assert append(lib, Hq=-1) == 1 and append(lib, Hq=1025, qs=BIG, qos=BIG) == 1
    assert append(lib, q=None) == 1 and append(lib, k=None) == 1 and append(lib, v=None) == 1
    assert append(lib, slots=None) == 1 and append(lib, qo=None) == 1
    assert append(lib, q=X + 2) == 1 and append(lib, qo=Y + 2) == 1 and append(lib, slots=S + 2) == 1
    assert append(lib, qs=511) == 2 and append(lib, ks=255) == 2 and append(lib, vs=255) == 2 and append(lib, qos=511) == 2
    assert append(lib, ks=BIG) == 1
    assert append(lib, rope=rope(kind=2)) == 1 and append(lib, rope=rope(axes=0)) == 1 and append(lib, rope=rope(axes=5)) == 1
    for dims in (0, 4, 12, 136, -8):
        assert append(lib, rope=rope(dims=dims)) == 2
    assert append(lib, rope=rope(pos=None)) == 1 and append(lib, rope=rope(freqs=FRQ + 1)) == 1
    # outputs over inputs: q_out over q, k, v, slots, the tables, the live count and the cache; the cache over an input
    size = 8 * qk.qk_kv_page_bytes(32, 2, 128)
    for at in (X + 16, X + 0x100000 - 64, X + 0x200000 + 64, S + 8, LIVE, POS, FRQ + 4, PAGES + size - 4):
        assert append(lib, qo=at, live=LIVE, rope=rope()) == 3, hex(at)
    assert append(lib, k=PAGES + size - 16) == 3 and append(lib, slots=PAGES) == 3
    # nothing to do
    assert append(lib, T=0) == 0 and append(lib, T=0, q=None, k=None, v=None, slots=None, qo=None) == 0
    assert lib.qk_launch_count() == n0


def test_read(lib):
    def read(c=None, slots=S, n=3, elem=0, out=Y, stride=512, live=None):
        p = lambda a: C.c_void_p(a) if a else None
        return lib.qk_kv_read(C.byref(c or cache()), p(slots), n, elem, p(out), stride, p(live), None)
    assert read(cache(D=32)) == 5 and read(cache(P=20)) == 1
    assert read(slots=None) == 1 and read(out=None) == 1 and read(n=-1) == 1 and read(elem=7) == 1 and read(out=Y + 1) == 1
    assert read(stride=511) == 2 and read(stride=BIG) == 1
    assert read(out=PAGES) == 3 and read(slots=Y + 64) == 3 and read(live=Y) == 3
    assert read(n=0, slots=None, out=None) == 0


def attn(**over):
    f = dict(q=X, q_elem=0, n_heads=4, q_stride=512, page_table=TAB, table_stride=4, kv_lens=LEN, scale=0.1, window=0,
             sinks=None, out=Y, out_elem=0, reserved=0, out_stride=512)
    f.update(over)
    return qk.qk_attn(*(f[n] for n, _ in qk.qk_attn._fields_))


BAD = [(dict(q=None), 1), (dict(page_table=None), 1), (dict(kv_lens=None), 1), (dict(q_elem=2), 1), (dict(out_elem=-1), 1),
       (dict(n_heads=3), 5), (dict(n_heads=0), 5), (dict(n_heads=1026, q_stride=BIG), 5), (dict(scale=0.0), 1),
       (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(window=-1), 1),
       (dict(q=X + 2), 1), (dict(out=Y + 1), 1), (dict(kv_lens=LEN + 2), 1), (dict(sinks=S + 1), 1), (dict(q_stride=511), 2),
       (dict(out_stride=511), 2), (dict(q_stride=BIG), 1), (dict(table_stride=0), 1), (dict(table_stride=1 << 27), 1),
       (dict(out=X), 3), (dict(out=PAGES), 3), (dict(out=LEN), 3), (dict(out=TAB), 3), (dict(out=S, sinks=S), 3)]


@pytest.mark.parametrize("over,status", BAD)
def test_attention_descriptor(lib, over, status):
    a = attn(**over)
    assert lib.qk_attn_decode(C.byref(cache()), C.byref(a), 2, 1, None, 16, None, C.c_void_p(WS), BIG, None) == status
    assert lib.qk_attn_prefill(C.byref(cache()), C.byref(a), 2, 5, C.c_void_p(POS), 64, None, None, 16, None,
                               C.c_void_p(WS), BIG, None) == status


def test_decode(lib):
    def decode(c=None, a=None, B=2, T=1, img=None, rb=16, live=None, ws=WS, n=BIG):
        p = lambda x: C.c_void_p(x) if x else None
        return lib.qk_attn_decode(C.byref(c or cache()), C.byref(a or attn()), B, T, p(img), rb, p(live), p(ws), n, None)
    n0 = lib.qk_launch_count()
    assert decode(cache(D=80)) == 5 and decode(T=9) == 5 and decode(T=0) == 1 and decode(B=-1) == 1 and decode(B=1 << 21) == 1
    assert decode(a=attn(out=None)) == 1                                   # nothing wanted
    assert decode(img=IMG, rb=15) == 2 and decode(img=IMG + 2) == 1 and decode(img=IMG, rb=1 << 21) == 1
    assert decode(img=Y + 64) == 3 and decode(img=X) == 3 and decode(img=PAGES) == 3 and decode(img=LIVE, live=LIVE) == 3
    assert decode(ws=None) == 4 and decode(ws=WS + 8) == 4 and decode(n=0) == 4
    assert decode(ws=Y) == 3 and decode(ws=X) == 3 and decode(ws=IMG, img=IMG) == 3 and decode(ws=TAB) == 3
    many = attn(n_heads=1024, q_stride=1 << 17, out_stride=1 << 17)
    assert decode(a=many, B=1 << 20, T=8) == 5
    assert decode(B=0) == 0 and decode(B=0, a=attn(q=None, page_table=None, kv_lens=None, out=None), ws=None) == 0
    need = lib.qk_attn_decode_workspace_bytes(C.byref(cache()), 4, 2, 1)
    assert need > 0 and decode(n=need - 1) == 4
    for args in ((3, 2, 1), (4, -1, 1), (4, 2, 9), (4, 2, 0)):
        assert lib.qk_attn_decode_workspace_bytes(C.byref(cache()), *args) == 0
    assert lib.qk_launch_count() == n0


def test_prefill(lib):
    def prefill(c=None, a=None, B=2, rows=5, off=POS, kv=64, qs=None, d=None, rb=16, live=None, ws=WS, n=BIG):
        p = lambda x: C.c_void_p(x) if x else None
        return lib.qk_attn_prefill(C.byref(c or cache()), C.byref(a or attn()), B, rows, p(off), kv, p(qs), p(d), rb,
                                   p(live), p(ws), n, None)
    n0 = lib.qk_launch_count()
    assert prefill(cache(D=80)) == 5 and prefill(B=65536) == 5 and prefill(rows=(1 << 24) + 1) == 5
    assert prefill(B=-1) == 1 and prefill(rows=-1) == 1 and prefill(off=None) == 1 and prefill(off=POS + 2) == 1
    assert prefill(kv=0) == 1 and prefill(kv=4 * 32 + 1) == 1
    assert prefill(qs=IMG) == 1 and prefill(d=IMG) == 1 and prefill(qs=IMG + 4, d=S) == 1 and prefill(qs=IMG, d=S + 2) == 1
    assert prefill(a=attn(out=None)) == 1
    assert prefill(qs=IMG, d=S, rb=15) == 2
    assert prefill(qs=Y, d=S) == 3 and prefill(qs=IMG, d=IMG + 64) == 3 and prefill(qs=X, d=S) == 3
    assert prefill(qs=IMG, d=POS) == 3 and prefill(off=Y + 4) == 3
    assert prefill(ws=None) == 4 and prefill(ws=WS + 64) == 4 and prefill(n=0) == 4
    need = lib.qk_attn_prefill_workspace_bytes(C.byref(cache()), 2, 64)
    assert need > 0 and prefill(n=need - 1) == 4
    assert prefill(ws=Y) == 3 and prefill(ws=POS) == 3 and prefill(ws=PAGES) == 3
    assert prefill(B=0) == 0 and prefill(rows=0) == 0
    assert lib.qk_attn_prefill_workspace_bytes(C.byref(cache()), 2, 0) == 0
    assert lib.qk_launch_count() == n0
