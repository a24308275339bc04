"""GPU: routed products at the largest numbers of experts and of slots per row that the calls take."""
import numpy as np
import pytest

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests import test_gpu_group_matvec as g
from tests import test_gpu_mmq_id as m
from tests.gpu_helpers import dev, pack_experts

pytestmark = pytest.mark.gpu

SIZES = [
    # rows, k, experts, live
    (40, 64, 1024, 37),
    (3, 64, 1023, 3),
    (70, 1, 1024, 70),
    (64, 64, 1, 63),       # one expert takes 64 slots of every row
]


@pytest.mark.parametrize("rows,k,E,live", SIZES)
@pytest.mark.parametrize("slots", [False, True])
def test_matvec(slots, rows, k, E, live):
    g.test_routed_matches_float64(slots, 64, rows, k, E, 192, (33,), live)


@pytest.mark.parametrize("rows,k,E,live", SIZES)
@pytest.mark.parametrize("wtype,K", [("q4_0", 96), ("q4_g64", 192)])
def test_prefill(wtype, K, rows, k, E, live):
    """Element by element. Not by the mean square of an expert's few outputs: one rounding to bfloat16 alone is off by
    up to 2^-8 of a value, so that mean square may reach 2^-16 = 1.5e-5."""
    N, seed = 33, 14100
    ids = synth.rng(14000 + rows + E).integers(0, E, size=(rows, k), dtype=np.int32)
    qs, dh = m.planes(seed, rows, K, None, live)
    Ws = [m.weight(wtype, seed + 10 + e, N, K) for e in range(E)]
    plan, y, packed = m.plan(ids, E, live), m.out(rows * k, N), pack_experts(Ws, wtype, N, K)
    projs = [qk.make_proj_id16(wtype, E, packed, N, K, y, N)]
    ws, n = m.workspace(rows, k, projs)
    qk.qk_mmq_id(dev(qs), dev(dh.view(np.int16)), K // 32, rows, k, projs, *plan, ws, n)
    assert qk.qk_device_faults() == 0
    got, x = m.bhost(y), O.plane_values(qs, dh, K)
    values = {e: m.dequant(wtype, Ws[e], N, K) for e in np.unique(ids[:live])}
    for p, e in enumerate(ids[:live].reshape(-1)):
        m.check(got[p:p + 1], x[p // k:p // k + 1], values[e], what=f"pair {p}, expert {e}")
    assert np.all(got[live * k:] == m.SENTINEL)
