"""GPU: routed chains over plans that leave pairs out (ids outside [0, E)). offsets[E] is then below live * k, so the
GLU between the projections is given live * k, and the combine reads what the caller put in the pairs' rows that no
projection wrote (zeros here). Every planned pair's rows equal those of the chain with no pair left out."""
import numpy as np
import pytest

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import dev, host, live_ptr, pack_experts

pytestmark = pytest.mark.gpu

ROWS, LIVE, K_SLOTS, E, K, NF = 21, 18, 4, 9, 384, 256


def left_out():
    ids = synth.rng(301).integers(0, E, size=(ROWS, K_SLOTS), dtype=np.int32)
    holes = ids.copy()
    where = synth.rng(302).random(ids.shape) < 0.3
    where[3] = True                       # a row without any expert
    where[LIVE - 1, -1] = False           # the last live pair is planned
    holes[where] = synth.rng(303).choice([-1, E, 1 << 30, -(1 << 31)], size=int(where.sum()))
    return ids, holes, where


def plan_of(ids):
    import torch
    i32 = lambda n: torch.full((n,), -3, dtype=torch.int32, device="cuda")
    plan = i32(E), i32(E + 1), i32(ROWS * K_SLOTS)
    qk.qk_moe_plan(dev(ids), ROWS, K_SLOTS, E, *plan, live_ptr(LIVE))
    return plan


def experts(seed, wtype, N, K_):
    Ws = [synth.q4_0_weight(seed + e, N, K_) if wtype == "q4_0" else synth.q4_group_weight(seed + e, N, K_, int(wtype[4:]))
          for e in range(E)]
    return pack_experts(Ws, wtype, N, K_)


def decode_chain(wtype, plan, w, pairs):
    import torch
    wg, wu, wd = w
    img = dev(O.quantize_q8_1(synth.activations(304, ROWS, K)).reshape(-1))
    g, u, h = (torch.full((ROWS * K_SLOTS, NF), float("nan"), device="cuda") for _ in range(3))
    himg = torch.zeros((ROWS * K_SLOTS * NF // 32 * 36,), dtype=torch.uint8, device="cuda")
    down = torch.zeros((ROWS * K_SLOTS, K), device="cuda")
    qk.qk_mmvq_id(img, K // 32, ROWS, K_SLOTS, [qk.make_proj_id(wtype, E, wg, NF, K, g), qk.make_proj_id(wtype, E, wu, NF, K, u)],
                  *plan)
    qk.qk_glu_q8_1("swiglu", "separate", g, NF, u, NF, ROWS * K_SLOTS, NF, h, NF, himg, NF // 32, pairs)
    qk.qk_mmvq_id_slots(himg, NF // 32, ROWS, K_SLOTS, [qk.make_proj_id(wtype, E, wd, K, NF, down)], *plan)
    return down


def prefill_chain(wtype, plan, w, pairs):
    import torch
    wg, wu, wd = w
    q, d = O.quantize_q8_0(synth.activations(304, ROWS, K))
    gu = torch.full((ROWS * K_SLOTS, 2 * NF), float("nan"), dtype=torch.bfloat16, device="cuda")
    hq = torch.zeros((ROWS * K_SLOTS, NF), dtype=torch.int8, device="cuda")
    hd = torch.zeros((ROWS * K_SLOTS, NF // 32), dtype=torch.int16, device="cuda")
    down = torch.zeros((ROWS * K_SLOTS, K), dtype=torch.bfloat16, device="cuda")
    gate_up = [qk.make_proj_id16(wtype, E, wg, NF, K, gu, 2 * NF), qk.make_proj_id16(wtype, E, wu, NF, K, gu[:, NF:], 2 * NF)]
    down_p = [qk.make_proj_id16(wtype, E, wd, K, NF, down, K)]
    n = max(qk.qk_mmq_id_workspace_bytes(ROWS, K_SLOTS, p) for p in (gate_up, down_p))
    ws = torch.empty((n,), dtype=torch.uint8, device="cuda")
    qk.qk_mmq_id(dev(q.reshape(-1)), dev(d.view(np.int16).reshape(-1)), K // 32, ROWS, K_SLOTS, gate_up, *plan, ws, n)
    qk.qk_glu_q8_0("swiglu", "packed", "bf16", gu, 2 * NF, None, 0, ROWS * K_SLOTS, NF, None, 0, hq, hd, NF // 32,
                   d_live_rows=pairs)
    qk.qk_mmq_id_slots(hq, hd, NF // 32, ROWS, K_SLOTS, down_p, *plan, ws, n)
    return down


@pytest.mark.parametrize("chain,combine,wtype", [
    (decode_chain, qk.qk_moe_combine, "q4_0"), (decode_chain, qk.qk_moe_combine, "q4_g64"),
    (prefill_chain, qk.qk_moe_combine_bf16, "q4_0"), (prefill_chain, qk.qk_moe_combine_bf16, "q4_g128")])
def test_chain_with_pairs_left_out(chain, combine, wtype):
    import torch
    ids, holes, where = left_out()
    w = [experts(310, wtype, NF, K), experts(330, wtype, NF, K), experts(350, wtype, K, NF)]
    wts = torch.rand((ROWS, K_SLOTS), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    full_plan, plan = plan_of(ids), plan_of(holes)
    assert host(full_plan[1])[E] == LIVE * K_SLOTS
    assert host(plan[1])[E] == host(plan[0]).sum() == int((~where[:LIVE]).sum()) < LIVE * K_SLOTS
    full = chain(wtype, full_plan, w, full_plan[1][E:])          # the plan's total is live * k here
    got = chain(wtype, plan, w, live_ptr(LIVE * K_SLOTS))
    assert qk.qk_device_faults() == 0
    want = full.clone()
    want.view(ROWS, K_SLOTS, K)[dev(where)] = 0
    assert torch.equal(got, want)
    assert bool((want[:LIVE * K_SLOTS].float().abs().amax(1) > 0).view(LIVE, K_SLOTS).equal(dev(~where[:LIVE])))
    sums = []
    for rows in (got, want):
        y = torch.full((ROWS, K), -7.0, device="cuda")
        combine(rows, K, wts, ROWS, K_SLOTS, K, y, K, live_ptr(LIVE))
        sums.append(host(y))
    assert np.array_equal(sums[0], sums[1]) and np.all(sums[0][3] == 0) and np.all(sums[0][LIVE:] == -7.0)
