"""Group-scaled weights, the routed prefill products, the Q8_0 GLU producer and the 16-bit combine:
the decoder pinned by hand, and every refusal, on the host (no pointer below is dereferenced)."""
import ctypes as C

import numpy as np
import pytest

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth

P = C.c_void_p
X, IMG, Y, W, WS, PL = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000


@pytest.fixture(scope="module")
def lib():
    return qk.load()


# ------------------------------------------------------------------ the decoder
@pytest.mark.parametrize("G", [64, 128])
def test_group_blocks_decode_by_hand(G):
    blk = np.zeros((1, 1, 4 + G // 2), dtype=np.uint8)
    blk[0, 0, 0:2] = np.array([0.5], dtype=np.float16).view(np.uint8)
    blk[0, 0, 2] = 0xF0 | 3          # zero point 3; the upper bits are not part of it
    blk[0, 0, 3] = 77                # unread
    blk[0, 0, 4] = 0x91              # run 0, byte 0: element 0 = 1, element 16 = 9
    blk[0, 0, 4 + 16 + 5] = 0x0F     # run 1, byte 5: element 32 + 5 = 15, element 32 + 21 = 0
    want = np.full((G,), (0 - 3) * 0.5)
    want[0], want[16], want[37] = (1 - 3) * 0.5, (9 - 3) * 0.5, (15 - 3) * 0.5
    assert np.array_equal(O.dequant_group(blk, 1, G)[0], want)


def test_group_blocks_with_zero_8_and_one_scale_equal_q4_0():
    N, K = 5, 256
    W0 = synth.q4_0_weight(1, N, K)
    W0[:, :, 0:2] = W0[:, :1, 0:2]                       # one scale per row
    for G in (64, 128):
        Wg = np.zeros((N, K // G, 4 + G // 2), dtype=np.uint8)
        Wg[:, :, 0:2] = W0[:, :1, 0:2]
        Wg[:, :, 2] = 8
        Wg[:, :, 4:] = W0[:, :, 2:].reshape(N, K // G, G // 2)
        assert np.array_equal(O.dequant_group(Wg, N, K), O.dequant("q4_0", W0, N, K))


# ------------------------------------------------------------------ refusals
def test_group_weight_pack_checks(lib):
    for wt, G in ((2, 64), (3, 128)):
        unit = 2048 + 128 * (128 // G)
        need = lib.qk_weight_packed_bytes(wt, 33, 128 + G)
        assert need == 2 * 2 * unit                                              # two strips x two chunks
        assert lib.qk_weight_pack(wt, P(X), 33, 128 + G, P(W), need - 1, None) == 4
        assert lib.qk_weight_pack(wt, P(X), 33, 128 + 32, P(W), 1 << 20, None) == 2   # not whole groups
        assert lib.qk_weight_pack(wt, P(X), 33, 128 + G, P(W + 8), need, None) == 1   # misaligned
        src = 33 * ((128 + G) // G) * (4 + G // 2)
        assert lib.qk_weight_pack(wt, P(X), 33, 128 + G, P(X + (src - 1) // 16 * 16), need, None) == 3
    assert lib.qk_weight_packed_bytes(4, 33, 128) == 0
    assert lib.qk_weight_pack(4, P(X), 33, 128, P(W), 1 << 20, None) == 1


def test_group_matvec_checks(lib):
    for wt, G in ((2, 64), (3, 128)):
        one = lambda **kw: (qk.qk_proj * 1)(qk.qk_proj(*{**dict(t=wt, r=0, w=W, N=64, K=256, y=Y, s=64), **kw}.values()))
        assert lib.qk_mmvq_workspace_bytes(1, one()) == 0
        assert lib.qk_mmvq(P(IMG), 8, 9, 1, one(), None, None, 0, None) == 5        # T > 8
        assert lib.qk_mmvq(P(IMG), 8, 0, 1, one(), None, None, 0, None) == 1        # T < 1
        assert lib.qk_mmvq(P(IMG), 8, 8, 1, one(K=256 + 32), None, None, 0, None) == 2    # K not whole groups
        assert lib.qk_mmvq(P(IMG), 8, 8, 1, one(K=256 + G), None, None, 0, None) == 2     # K past the image row
        assert lib.qk_mmvq(P(IMG), 8, 8, 1, one(w=W + 8), None, None, 0, None) == 1       # misaligned weights
        assert lib.qk_mmvq(P(IMG), 8, 8, 1, one(s=63), None, None, 0, None) == 2          # y_stride < N
        assert lib.qk_mmvq(P(IMG), 8, 8, 1, one(y=W + 64), None, None, 0, None) == 3      # y over the weights
        assert lib.qk_mmvq_static_ws(P(IMG), 8, 9, 1, one(), None, None) == 5
        # a mixed call still needs the Q4_0 projection's workspace
        mixed = (qk.qk_proj * 2)(one()[0], qk.qk_proj(0, 0, W, 64, 256, Y + 0x10000, 64))
        assert lib.qk_mmvq(P(IMG), 8, 8, 2, mixed, None, None, 0, None) == 4
        # the dense prefill takes Q4_0 only
        assert lib.qk_mmq(P(X), P(PL), 8, 16, 1, one(), P(WS), 1 << 20, None) == 5
        pid = (qk.qk_proj_id * 1)(qk.qk_proj_id(wt, 4, W, 64, 256 + 32, Y))
        assert lib.qk_mmvq_id(P(IMG), 10, 4, 2, 1, pid, P(PL), P(PL + 64), P(PL + 256), None) == 2
        pid = (qk.qk_proj_id * 1)(qk.qk_proj_id(wt, 4, W, 64, 256, PL))
        assert lib.qk_mmvq_id(P(IMG), 8, 4, 2, 1, pid, P(PL), P(PL + 64), P(PL + 256), None) == 3


def _mmq_id(lib, slots=False, n=1, rows=4, k=2, rb=8, ws=WS, ws_bytes=1 << 20, qs=X, d=X + 0x100000, plan=PL, second=None,
            **kw):
    f = dict(t=3, e=4, w=W, N=64, K=256, y=Y, s=64)
    f.update(kw)
    projs = [qk.qk_proj_id16(*f.values())] + ([second] if second is not None else [])
    arr = (qk.qk_proj_id16 * 8)(*projs)
    fn = lib.qk_mmq_id_slots if slots else lib.qk_mmq_id
    return fn(P(qs), P(d), rb, rows, k, n if second is None else 2, arr, P(plan), P(plan + 64), P(plan + 256), P(ws),
              ws_bytes, None)


@pytest.mark.parametrize("slots", [False, True])
def test_routed_prefill_checks(lib, slots):
    go = lambda **kw: _mmq_id(lib, slots=slots, **kw)
    need = qk.qk_mmq_id_workspace_bytes(4, 2, [qk.qk_proj_id16(3, 4, W, 64, 256, Y, 64)])
    assert need >= 4 * 2 * 256 * 2
    assert go(t=1, K=256) == 5                     # Q8_0 weights
    assert go(t=4) == 1 and go(t=-1) == 1          # no such type
    assert go(K=256 + 32) == 2                     # not whole groups
    assert go(rb=7) == 2                           # K past the image row
    assert go(N=0) == 1
    assert go(e=0) == 5 and go(e=1025) == 5
    assert go(rows=0) == 1 and go(k=0) == 1 and go(k=65) == 1 and go(rows=(1 << 24) + 1) == 1
    assert go(n=0) == 5 and go(n=9) == 5
    assert go(qs=X + 8) == 1 and go(d=X + 0x100002) == 1 and go(qs=0) == 1 and go(plan=0) == 1
    assert go(y=Y + 1) == 1 and go(y=0) == 1 and go(w=W + 8) == 1
    assert go(s=63) == 2
    assert go(y=X) == 3 and go(y=W) == 3 and go(y=PL + 256) == 3
    assert go(ws_bytes=need - 1) == 4 and go(ws=0) == 4 and go(ws=WS + 64) == 4
    assert go(ws=Y) == 3 and go(ws=X) == 3 and go(ws=W) == 3
    # two projections: different expert counts; overlapping outputs; column windows of one buffer pass
    # the output check (and are then stopped by the tiny workspace)
    other = lambda **kw: qk.qk_proj_id16(*{**dict(t=3, e=4, w=W + 0x100000, N=64, K=256, y=Y + 128, s=128), **kw}.values())
    assert go(s=128, second=other(e=5)) == 1
    assert go(s=128, second=other(y=Y + 126)) == 3
    assert go(s=128, second=other(), ws_bytes=16) == 4


def test_rows_and_columns_whose_units_pass_an_int_are_refused(lib):
    """Indices are counted in whole units of 32 or 128 rows and 128 columns, past N and K."""
    big, far = (1 << 31) - 1024, 1 << 60
    for n, k in ((big + 1, 256), (64, (1 << 31) - 128)):
        assert _mmq_id(lib, N=n, s=n, K=k, rb=1 << 26, y=far) == 1
        one = (qk.qk_proj * 1)(qk.qk_proj(3, 0, W, n, k, far, n))
        assert lib.qk_mmvq(P(IMG), 1 << 26, 1, 1, one, None, None, 0, None) == 1
        routed = (qk.qk_proj_id * 1)(qk.qk_proj_id(3, 4, W, n, k, far))
        assert lib.qk_mmvq_id(P(IMG), 1 << 26, 4, 2, 1, routed, P(PL), P(PL + 64), P(PL + 256), None) == 1
        assert lib.qk_weight_pack(3, P(X), n, k, P(far), 1 << 62, None) == 1


def test_misaligned_outputs_and_plans_are_refused(lib):
    one = lambda y: (qk.qk_proj * 1)(qk.qk_proj(3, 0, W, 64, 256, y, 64))
    assert lib.qk_mmvq(P(IMG), 8, 8, 1, one(Y + 2), None, None, 0, None) == 1
    routed = lambda y: (qk.qk_proj_id * 1)(qk.qk_proj_id(3, 4, W, 64, 256, y))
    assert lib.qk_mmvq_id(P(IMG), 8, 4, 2, 1, routed(Y + 2), P(PL), P(PL + 64), P(PL + 256), None) == 1
    assert lib.qk_mmvq_id(P(IMG), 8, 4, 2, 1, routed(Y), P(PL), P(PL + 66), P(PL + 256), None) == 1


def test_routed_prefill_outputs_stay_off_every_projections_weights(lib):
    second = qk.qk_proj_id16(3, 4, W + 0x100000, 64, 256, W + 0x40, 64)     # over the first one's weights
    assert _mmq_id(lib, second=second) == 3
    second = qk.qk_proj_id16(3, 4, Y + 0x100, 64, 256, Y + 0x100000, 64)    # the first one's output over these
    assert _mmq_id(lib, second=second) == 3


def test_routed_prefill_work_items_fit_an_int(lib):
    assert _mmq_id(lib, rows=1 << 24, k=64, N=1 << 20, s=1 << 20, K=128, y=1 << 60) == 5


def test_glu_q8_0_checks(lib):
    def go(kind=0, layout=0, elem=0, a=X, a_s=64, b=W, b_s=64, T=4, N=64, out=Y, o_s=64, qs=IMG, d=PL, rb=2, alpha=1.702,
           limit=7.0):
        return lib.qk_glu_q8_0(kind, layout, elem, P(a), a_s, P(b), b_s, T, N, P(out), o_s, P(qs), P(d), rb, alpha, limit,
                               None, None)
    assert go(kind=7) == 1 and go(kind=-1) == 1 and go(layout=3) == 1 and go(elem=2) == 1 and go(elem=-1) == 1
    assert go(N=48) == 2 and go(a_s=63) == 2 and go(b_s=63) == 2 and go(o_s=63) == 2 and go(rb=1) == 2
    assert go(layout=1, a_s=127) == 2
    assert go(T=-1) == 1 and go(N=0) == 1 and go(rb=(1 << 20) + 1) == 1
    assert go(a=0) == 1 and go(b=0) == 1 and go(qs=0) == 1 and go(d=0) == 1
    assert go(a=X + 2) == 1 and go(qs=IMG + 2) == 1 and go(d=PL + 1) == 1 and go(out=Y + 2) == 1
    assert go(elem=1, a=X + 1) == 1
    assert go(alpha=float("nan")) == 1 and go(limit=0.0) == 1 and go(limit=float("inf")) == 1
    assert go(out=X) == 3 and go(qs=X) == 3 and go(d=W) == 3 and go(qs=Y) == 3 and go(d=IMG) == 3
    # bfloat16 rows span half the bytes: an output right behind them is no alias (T = 0 launches nothing)
    assert go(T=0) == 0


def test_combine_bf16_checks(lib):
    def go(e=X, e_s=64, w=W, rows=4, k=2, N=64, y=Y, y_s=64):
        return lib.qk_moe_combine_bf16(P(e), e_s, P(w), rows, k, N, P(y), y_s, None, None)
    assert go(e=0) == 1 and go(w=0) == 1 and go(y=0) == 1
    assert go(N=62) == 1 and go(e_s=60) == 2 and go(y_s=60) == 2 and go(e_s=66) == 1 and go(y_s=66) == 1
    assert go(e=X + 4) == 1 and go(y=Y + 8) == 1 and go(w=W + 2) == 1
    assert go(k=0) == 1 and go(k=65) == 1 and go(rows=-1) == 1 and go(N=1 << 26, e_s=1 << 26, y_s=1 << 26) == 1
    assert go(y=X + 512) == 3 and go(y=W) == 3
    assert go(rows=0) == 0
