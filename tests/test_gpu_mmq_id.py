"""GPU parity: routed prefill products (qk_mmq_id, qk_mmq_id_slots) against binary64.

Bound per element, from the roundings: each operand once to binary16 (2^-11 relative each, so
2^-10 + 2^-22 per product), the sum over K in binary32 (at most one rounding or truncation of 2^-23
per 16-term step, of partial sums no larger than S = sum |w x|), and one rounding to bfloat16
(2^-8 of the result):
    |y - ref| <= (2^-10 + 2^-22 + K / 16 * 2^-23) * S + 2^-8 * |y_before|, |y_before| <= |ref| + first term.
Whole output: the bfloat16 rounding's mean square is (2^-7)^2 / 12 of the binade's square, 2.6e-6 of
y^2 on average over mantissas, the operands add 2 (2^-11)^2 / 3: NMSE <= 6e-6 for 64 outputs or more.
"""
import numpy as np
import pytest

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import dev, host, live_ptr, pack_experts

pytestmark = pytest.mark.gpu

SENTINEL = -12352.0   # exact in bfloat16


def weight(wtype, seed, N, K):
    return synth.q4_0_weight(seed, N, K) if wtype == "q4_0" else synth.q4_group_weight(seed, N, K, int(wtype[4:]))


def dequant(wtype, W, N, K):
    return O.dequant(wtype, W, N, K).astype(np.float64) if wtype == "q4_0" else O.dequant_group(W, N, K)


def planes(seed, rows, K, rb=None, live=None):
    """Q8_0 planes of N(0, 1) rows on the host; rows past `live` hold codes 127 and NaN scales."""
    qs, dh = O.quantize_q8_0(synth.activations(seed, rows, (rb or K // 32) * 32))
    qs, dh = qs.reshape(rows, -1).copy(), dh.reshape(rows, -1).copy()
    if live is not None:
        qs[live:] = 127
        dh[live:] = 0x7E00
    return qs, dh


def plan(ids, E, live):
    import torch
    rows, k = ids.shape
    counts = torch.full((E,), -9, dtype=torch.int32, device="cuda")
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    items = torch.full((rows * k,), -3, dtype=torch.int32, device="cuda")
    qk.qk_moe_plan(dev(ids), rows, k, E, counts, offsets, items, live_ptr(live))
    return counts, offsets, items


def out(rows, width):
    import torch
    return torch.full((rows, width), SENTINEL, dtype=torch.bfloat16, device="cuda")


def bhost(t):
    return host(t.float()).astype(np.float64)


def workspace(rows, k, projs, fill=0xFF):
    import torch
    n = qk.qk_mmq_id_workspace_bytes(rows, k, projs)
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda"), n


def check(got, x, Wd, what=""):
    """Every element of got [P][N] against x [P][K] @ Wd [N][K].T within the derived bound."""
    ref, S = x @ Wd.T, np.abs(x) @ np.abs(Wd).T
    K = x.shape[1]
    acc = (2.0 ** -10 + 2.0 ** -22 + K / 16 * 2.0 ** -23) * S
    bound = acc + 2.0 ** -8 * (np.abs(ref) + acc) + 1e-30
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.max(np.abs(got - ref) / bound):.2f}x bound"
    if ref.size >= 64:
        assert O.nmse(got, ref) <= 6e-6, f"{what}: NMSE {O.nmse(got, ref):.2e}"


def run(wtype, rows, k, E, K, Ns, live, slots, ids=None, seed=12000, rb=None, pad=0, y_off=0):
    n_img = rows * k if slots else rows
    qs, dh = planes(seed, n_img, K, rb, live * k if slots else live)
    if ids is None:
        ids = synth.rng(seed + 1).integers(0, E, size=(rows, k), dtype=np.int32)
    counts, offsets, items = plan(ids, E, live)
    width = sum(Ns) + pad + y_off
    y = out(rows * k, width)
    projs, Ws, at = [], [], y_off
    for j, N in enumerate(Ns):
        ws_ = [weight(wtype, seed + 10 + 1000 * j + e, N, K) for e in range(E)]
        pw = pack_experts(ws_, wtype, N, K)
        Ws.append((ws_, pw))
        projs.append(qk.make_proj_id16(wtype, E, pw, N, K, y[:, at:], width))
        at += N
    ws, n = workspace(rows, k, projs)
    call = qk.qk_mmq_id_slots if slots else qk.qk_mmq_id
    call(dev(qs), dev(dh.view(np.int16)), qs.shape[1] // 32, rows, k, projs, counts, offsets, items, ws, n)
    assert qk.qk_device_faults() == 0
    got = bhost(y)
    flat = ids.reshape(-1)[:live * k]
    x = O.plane_values(qs, dh, K)
    planned = np.zeros(rows * k, dtype=bool)
    at = y_off
    for (ws_, _), N in zip(Ws, Ns):
        for e in np.unique(flat):
            if not 0 <= e < E:
                continue
            p = np.nonzero(flat == e)[0]
            planned[p] = True
            check(got[p, at:at + N], x[p if slots else p // k], dequant(wtype, ws_[e], N, K),
                  what=f"{wtype} {rows}x{k} E{E} K{K} N{N} expert {e}")
        at += N
    assert np.all(got[~planned] == SENTINEL), "a pair outside the plan was written"
    assert np.all(got[:, :y_off] == SENTINEL) and np.all(got[:, at:] == SENTINEL), "columns outside the windows were written"
    return got


@pytest.mark.parametrize("wtype", ["q4_0", "q4_g64", "q4_g128"])
@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("rows,k,E,K,Ns,live", [
    (1, 1, 1, 128, (1,), 1),                 # one of everything
    (5, 2, 3, 128, (64,), 5),
    (37, 2, 8, 384, (203,), 37),             # odd width, ragged counts
    (64, 4, 16, 640, (128, 130), 61),        # two projections, padding rows
    (300, 1, 2, 256, (96,), 300),            # more pairs than one tile holds
    (40, 8, 128, 1280, (160,), 33),          # a few pairs per expert
    (700, 3, 4, 512, (257,), 640),           # several tiles per expert
])
def test_matches_float64(wtype, slots, rows, k, E, K, Ns, live):
    run(wtype, rows, k, E, K, Ns, live, slots)


@pytest.mark.parametrize("wtype,K", [("q4_0", 32), ("q4_0", 96), ("q4_0", 160), ("q4_g64", 64), ("q4_g64", 192)])
@pytest.mark.parametrize("slots", [False, True])
def test_partial_chunks_and_wider_image_rows(wtype, K, slots):
    """K that ends inside a 128-column chunk, in an image whose rows continue past K."""
    run(wtype, 19, 2, 3, K, (70,), 19, slots, seed=12100, rb=K // 32 + 7)


def test_all_pairs_to_one_expert_and_one_empty_plan():
    run("q4_g128", 530, 1, 5, 256, (40,), 530, False, ids=np.full((530, 1), 3, dtype=np.int32), seed=12200)
    run("q4_0", 8, 2, 5, 256, (40,), 0, False, seed=12201)


@pytest.mark.parametrize("count", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 383, 385, 512, 513])
def test_tile_edges(count):
    """One expert with exactly `count` pairs, another with one."""
    ids = np.zeros((count + 1, 1), dtype=np.int32)
    ids[count // 2, 0] = 1
    run("q4_g64", count + 1, 1, 2, 128, (129,), count + 1, False, ids=ids, seed=12300)


def test_experts_outside_the_range_are_left_out():
    ids = synth.rng(12400).integers(-2, 7, size=(50, 3), dtype=np.int32)
    run("q4_0", 50, 3, 5, 256, (64,), 44, False, ids=ids, seed=12400)
    run("q4_0", 50, 3, 5, 256, (64,), 44, True, ids=ids, seed=12401)


@pytest.mark.parametrize("pad,off", [(0, 1), (1, 0), (3, 2), (8, 8)])
def test_strides_and_alignments_of_the_output(pad, off):
    run("q4_g128", 33, 2, 3, 256, (65, 64), 33, False, seed=12500, pad=pad, y_off=off)


def test_projections_of_different_types_and_widths_of_k():
    import torch
    rows, k, E, rb = 60, 2, 6, 20
    qs, dh = planes(12600, rows, rb * 32)
    ids = synth.rng(12601).integers(0, E, size=(rows, k), dtype=np.int32)
    p = plan(ids, E, rows)
    specs = [("q4_0", 64, 640), ("q4_g128", 100, 384), ("q4_g64", 33, 576), ("q4_0", 5, 32)]
    projs, keep, ys = [], [], []
    for i, (wt, N, K) in enumerate(specs):
        Ws = [weight(wt, 12610 + 100 * i + e, N, K) for e in range(E)]
        pw = pack_experts(Ws, wt, N, K)
        y = out(rows * k, N)
        keep.append((Ws, pw))
        ys.append(y)
        projs.append(qk.make_proj_id16(wt, E, pw, N, K, y, N))
    ws, n = workspace(rows, k, projs)
    qk.qk_mmq_id(dev(qs), dev(dh.view(np.int16)), rb, rows, k, projs, *p, ws, n)
    flat = ids.reshape(-1)
    for (wt, N, K), (Ws, _), y in zip(specs, keep, ys):
        got, x = bhost(y), O.plane_values(qs, dh, K)
        for e in range(E):
            pr = np.nonzero(flat == e)[0]
            if pr.size:
                check(got[pr], x[pr // k], dequant(wt, Ws[e], N, K), what=wt)


def test_many_experts_long_k():
    run("q4_0", 64, 8, 128, 2560, (192, 64), 64, False, seed=12700)
    run("q4_g128", 64, 8, 1024, 256, (32,), 64, True, seed=12701)


def test_deterministic_and_replayed():
    """The same bits on every call, from a captured graph on a side stream, with the plan made inside
    the graph at changing live counts."""
    import torch
    rows, k, E, K, N = 200, 4, 12, 512, 144
    qs, dh = planes(12800, rows, K)
    d_qs, d_dh = dev(qs), dev(dh.view(np.int16))
    Ws = [weight("q4_g64", 12810 + e, N, K) for e in range(E)]
    pw = pack_experts(Ws, "q4_g64", N, K)
    y = out(rows * k, N)
    projs = [qk.make_proj_id16("q4_g64", E, pw, N, K, y, N)]
    ws, n = workspace(rows, k, projs)
    logits = dev(synth.router_logits(12801, rows, E))
    ids = torch.zeros((rows, k), dtype=torch.int32, device="cuda")
    wts = torch.zeros((rows, k), device="cuda")
    counts = torch.zeros((E,), dtype=torch.int32, device="cuda")
    offsets = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
    items = torch.zeros((rows * k,), dtype=torch.int32, device="cuda")
    live = live_ptr(rows)

    def step():
        qk.qk_route_plan(logits, rows, E, k, ids, wts, counts, offsets, items, live)
        qk.qk_mmq_id(d_qs, d_dh, K // 32, rows, k, projs, counts, offsets, items, ws, n)

    step()
    full = bhost(y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
            step()
        for m in (200, 1, 77, 0, 200):
            live.fill_(m)
            y.fill_(SENTINEL)
            g.replay()
            s.synchronize()
            got = y.float().cpu().numpy()
            # a pair's bits depend neither on the other pairs nor on the live count
            assert np.array_equal(got[:m * k], full[:m * k]), m
            assert np.all(got[m * k:] == SENTINEL), m
    assert qk.qk_device_faults() == 0


def test_a_plan_from_elsewhere_reads_and_writes_inside_its_buffers():
    """Counts past the bucket, negative counts, offsets outside items, pairs outside the bucket: no
    fault, nothing written outside the rows, and the experts with a sound plan come out right."""
    import torch
    rows, k, E, K, N = 20, 2, 6, 256, 64
    qs, dh = planes(12900, rows, K)
    Ws = [weight("q4_0", 12910 + e, N, K) for e in range(E)]
    pw = pack_experts(Ws, "q4_0", N, K)
    counts = dev(np.array([5, -7, 1 << 30, 3, 2, 4], dtype=np.int32))
    offsets = dev(np.array([0, 5, 38, -(1 << 30), 1 << 30, 10, 14], dtype=np.int32))
    it = np.full((rows * k,), -1, dtype=np.int32)
    it[0:5] = [7, 39, 0, 12, 25]
    it[10:14] = [40, 1 << 30, -5, 31]          # three pairs outside the bucket
    it[38:40] = [2, 3]
    guard = torch.full((rows * k + 64, N), SENTINEL, dtype=torch.bfloat16, device="cuda")
    y = guard[32:32 + rows * k]
    projs = [qk.make_proj_id16("q4_0", E, pw, N, K, y, N)]
    ws, n = workspace(rows, k, projs)
    qk.qk_mmq_id(dev(qs), dev(dh.view(np.int16)), K // 32, rows, k, projs, counts, offsets, dev(it), ws, n)
    got, x = bhost(guard), O.plane_values(qs, dh, K)
    assert np.all(got[:32] == SENTINEL) and np.all(got[32 + rows * k:] == SENTINEL)
    sound = [7, 39, 0, 12, 25]
    check(got[32:][sound], x[np.array(sound) // k], dequant("q4_0", Ws[0], N, K), what="sound expert")
    check(got[32:][[31]], x[[15]], dequant("q4_0", Ws[5], N, K), what="the pair inside the bucket")
    left = sorted(set(range(rows * k)) - set(sound) - {31, 2, 3})
    assert np.all(got[32:][left] == SENTINEL)
    qk.qk_device_faults()
