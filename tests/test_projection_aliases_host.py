"""Outputs over another projection's weights are refused, on the host (no pointer below is dereferenced): CTAs read
one projection's weights while others write another's outputs."""
import ctypes as C

import pytest

from quantized_activation_q4_gb300 import binding as qk

P = C.c_void_p
IMG, Y, W, WS, PL = 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000
N, K, T, E, ROWS, SLOTS = 64, 256, 8, 4, 4, 2
ALIAS = 3


@pytest.mark.parametrize("first,second", [(0, 0), (1, 1), (2, 2), (3, 3), (0, 3), (2, 1)])
def test_matvec_outputs_stay_off_every_projections_weights(first, second):
    lib = qk.load()
    size = [qk.qk_weight_packed_bytes(t, N, K) for t in (first, second)]
    far = W + 0x1000000

    def go(y0, y1):
        projs = (qk.qk_proj * 2)(qk.qk_proj(first, 0, W, N, K, y0, N), qk.qk_proj(second, 0, far, N, K, y1, N))
        a = lib.qk_mmvq(P(IMG), K // 32, T, 2, projs, None, P(WS), 1 << 24, None)
        b = lib.qk_mmvq_static_ws(P(IMG), K // 32, T, 2, projs, None, None)
        assert a == b
        return a

    for at in (0, 4, size[1] - 4):
        assert go(far + at, Y) == ALIAS          # the first one's output over the second one's weights
    for at in (0, 4, size[0] - 4):
        assert go(Y, W + at) == ALIAS            # and the other way round
    assert go(W + size[0] - 4, Y) == ALIAS and go(Y, far) == ALIAS


@pytest.mark.parametrize("first,second", [(0, 0), (1, 1), (2, 2), (3, 3), (0, 3), (2, 1)])
@pytest.mark.parametrize("call", ["qk_mmvq_id", "qk_mmvq_id_slots"])
def test_routed_outputs_stay_off_every_projections_weights(call, first, second):
    lib = qk.load()
    size = [E * qk.qk_weight_packed_bytes(t, N, K) for t in (first, second)]
    far = W + 0x1000000

    def go(y0, y1):
        projs = (qk.qk_proj_id * 2)(qk.qk_proj_id(first, E, W, N, K, y0), qk.qk_proj_id(second, E, far, N, K, y1))
        return getattr(lib, call)(P(IMG), K // 32, ROWS, SLOTS, 2, projs, P(PL), P(PL + 64), P(PL + 256), None)

    for at in (0, 4, size[1] - 4):               # the last expert's last bytes among them
        assert go(far + at, Y) == ALIAS
    for at in (0, 4, size[0] - 4):
        assert go(Y, W + at) == ALIAS
    assert go(W + size[0] - 4, Y) == ALIAS and go(Y, far) == ALIAS


def test_dense_prefill_outputs_stay_off_every_projections_weights():
    lib = qk.load()
    size, far = qk.qk_weight_packed_bytes(0, N, K), W + 0x1000000

    def go(y0, y1):
        projs = (qk.qk_proj * 2)(qk.qk_proj(0, 0, W, N, K, y0, N), qk.qk_proj(0, 0, far, N, K, y1, N))
        return lib.qk_mmq(P(IMG), P(PL), K // 32, T, 2, projs, P(WS), 1 << 24, None)

    for at in (0, 4, size - 4):
        assert go(far + at, Y) == ALIAS and go(Y, W + at) == ALIAS
    assert go(W + size - 4, Y) == ALIAS and go(Y, far) == ALIAS
    assert go(Y + 2, Y + 0x10000) == 1           # a misaligned output
