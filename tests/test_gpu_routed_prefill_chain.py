"""GPU parity: the GLU producer of the prefill planes, the combine over bfloat16 rows, and the routed
prefill FFN as a chain.

Tolerances:
- GLU output in binary32 against binary64: |d| <= 2e-6 |y| + 3e-7 |g| (|u| + 1), as for the Q8_1
  producer (the activations' 1 + tanh and 1 + erf cancel for very negative g);
- planes: bit-identical to qk_quantize_q8_0 of the output, and to the oracle's;
- combine: each of the k fused multiply-adds rounds once, |y - ref| <= k 2^-24 sum |w e|;
- chain against the plain binary64 definition: the planes of the two quantisations leave the pages'
  5e-4 NMSE, the bfloat16 rows add 2 * 2.6e-6.
"""
import numpy as np
import pytest
from scipy.special import erf, expit

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import dev, host, live_ptr, pack_experts

pytestmark = pytest.mark.gpu

KINDS = list(qk.GLU)
S32 = np.float32(-12345.5)


def glu64(kind, g, u, alpha=1.702, limit=7.0):
    g, u = g.astype(np.float64), u.astype(np.float64)
    if kind == "swiglu":
        return g * expit(g) * u
    if kind == "geglu_tanh":
        return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))) * u
    if kind == "reglu":
        return np.maximum(g, 0) * u
    if kind == "geglu_erf":
        return 0.5 * g * (1 + erf(g / np.sqrt(2))) * u
    if kind == "geglu_quick":
        return g * expit(1.702 * g) * u
    g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    return g * expit(alpha * g) * (u + 1) if kind == "swiglu_oai" else g * expit(g) * u


def run_glu(kind, layout, elem, T, N, live, pad=0, rb=None, out=True, seed=13000, alpha=1.702, limit=7.0, off=0):
    """The call's outputs on the host and the inputs it read (binary32): (out, qs, d, g, u)."""
    import torch
    dt = torch.bfloat16 if elem == "bf16" else torch.float32
    widths = (N, N) if layout == "separate" else (2 * N, 0)
    x = [3 * synth.activations(seed + i, T, max(w, 1) + pad + off) for i, w in enumerate(widths)]
    a, b = [dev(v).to(dt) for v in x]
    rb = rb or N // 32
    o = torch.full((T, N + pad), float(S32), device="cuda") if out else None
    qs = torch.full((T, rb * 32), 99, dtype=torch.int8, device="cuda")
    dh = torch.full((T, rb), 0x1234, dtype=torch.int16, device="cuda")
    qk.qk_glu_q8_0(kind, layout, elem, a[:, off:], widths[0] + pad + off, b[:, off:] if widths[1] else None,
                   max(widths[1], 1) + pad + off, T, N, o, N + pad, qs, dh, rb, alpha, limit, live_ptr(live))
    af, bf = host(a.float())[:, off:], host(b.float())[:, off:]
    g, u = {"separate": (af[:, :N], bf[:, :N]), "packed": (af[:, :N], af[:, N:2 * N]),
            "packed_swapped": (af[:, N:2 * N], af[:, :N])}[layout]
    return (host(o) if out else None), host(qs), host(dh).view(np.uint16), g, u


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["separate", "packed", "packed_swapped"])
@pytest.mark.parametrize("elem", ["f32", "bf16"])
def test_glu_planes(kind, layout, elem):
    T, N, live, rb, pad = 9, 1120, 7, 38, 4
    o, qs, dh, g, u = run_glu(kind, layout, elem, T, N, live, pad=pad, rb=rb)
    want = glu64(kind, g, u)[:live]
    y = o[:live, :N]
    ag, au = np.abs(g[:live]).astype(np.float64), np.abs(u[:live]).astype(np.float64)
    assert np.all(np.abs(y - want) <= 2e-6 * np.abs(want) + 3e-7 * ag * (au + 1))
    oq, od = O.quantize_q8_0(np.ascontiguousarray(y), row_blocks=rb)
    assert np.array_equal(qs[:live], oq.reshape(live, -1)) and np.array_equal(dh[:live], od.reshape(live, -1))
    assert np.all(o[live:] == S32) and np.all(o[:, N:] == S32)
    assert np.all(qs[live:] == 99) and np.all(dh[live:] == 0x1234)
    # without the binary32 output the planes are the same bytes
    _, qs2, dh2, _, _ = run_glu(kind, layout, elem, T, N, live, pad=pad, rb=rb, out=False)
    assert np.array_equal(qs, qs2) and np.array_equal(dh, dh2)


@pytest.mark.parametrize("elem", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,live", [(1, 32, 1), (3, 64, 0), (2, 18944, 2), (600, 96, 599), (5, 1024, 5), (2, 1056, 1),
                                      (4100, 768, 4001)])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_glu_sizes_and_alignments(elem, T, N, live, off):
    o, qs, dh, g, u = run_glu("swiglu", "packed", elem, T, N, live, pad=off, off=off, seed=13100)
    want = glu64("swiglu", g, u)[:live]
    y = np.ascontiguousarray(o[:live, :N])
    assert np.all(np.abs(y - want) <= 2e-6 * np.abs(want) + 3e-7 * np.abs(g[:live].astype(np.float64) * u[:live]))
    if live:
        oq, od = O.quantize_q8_0(y)
        assert np.array_equal(qs[:live], oq.reshape(live, -1)) and np.array_equal(dh[:live], od.reshape(live, -1))
    assert np.all(o[live:] == S32) and np.all(qs[live:] == 99)


def test_glu_parameters_and_zero_blocks():
    o, qs, dh, g, u = run_glu("swiglu_oai", "separate", "bf16", 4, 64, 4, alpha=0.5, limit=1.25, seed=13200)
    want = glu64("swiglu_oai", g, u, 0.5, 1.25)
    assert np.all(np.abs(o - want) <= 2e-6 * np.abs(want) + 3e-7 * np.abs(g) * (np.abs(u) + 1))
    import torch
    a = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    a[:, 64:] = -1.0
    qs = torch.full((2, 64), 99, dtype=torch.int8, device="cuda")
    dh = torch.full((2, 2), 0x1234, dtype=torch.int16, device="cuda")
    qk.qk_glu_q8_0("swiglu", "packed", "bf16", a, 128, None, 0, 2, 64, None, 0, qs, dh, 2)
    assert np.all(host(qs) == 0) and np.all((host(dh) & 0x7FFF) == 0)


@pytest.mark.parametrize("elem", ["f32", "bf16"])
def test_glu_codes_at_ties_and_extremes(elem):
    """Quotients at and next to ties, scales from subnormal to near overflow, infinities and NaN: the
    planes are the bytes that qk_quantize_q8_0 makes of the output."""
    import torch
    rng = synth.rng(13250)
    N, rows = 256, 64
    g = np.zeros((rows, N), dtype=np.float32)
    for r in range(rows):
        half = rng.integers(0, 127, size=N).astype(np.float32) + 0.5
        step = np.float32(2.0) ** rng.integers(-140, 110)
        nudge = rng.integers(-2, 3, size=N, dtype=np.int32)   # up to two units in the last place off a tie
        v = (half * step).astype(np.float32)
        g[r] = (v.view(np.int32) + nudge).view(np.float32) if r % 2 else v
        g[r, ::32] = np.float32(127.0) * step                 # the block's largest: d is `step`
    g[60, 5], g[61, 7], g[62, ::3] = np.inf, np.nan, np.inf
    g[63, 64:96] = np.nan
    a = dev(g).to(torch.bfloat16 if elem == "bf16" else torch.float32)
    b = torch.ones_like(a)
    out = torch.zeros((rows, N), device="cuda")
    qs, d = torch.zeros((rows, N), dtype=torch.int8, device="cuda"), torch.zeros((rows, N // 32), dtype=torch.int16, device="cuda")
    qk.qk_glu_q8_0("reglu", "separate", elem, a, N, b, N, rows, N, out, N, qs, d, N // 32)
    q2, d2 = torch.zeros_like(qs), torch.zeros_like(d)
    qk.qk_quantize_q8_0(out, rows, N, N, q2, d2, N // 32)
    assert torch.equal(qs, q2) and torch.equal(d, d2)


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("rows,k,N,live,pad", [(1, 1, 4, 1, 0), (24, 8, 2560, 17, 0), (7, 3, 1028, 7, 4), (300, 2, 64, 0, 8),
                                               (2000, 8, 96, 1999, 0), (3, 64, 4100, 3, 12)])
def test_combine_bf16(rows, k, N, live, pad):
    import torch
    e = dev(synth.activations(13300, rows * k, N + pad)).bfloat16()
    eh = host(e.float())[:, :N].astype(np.float64).reshape(rows, k, N)
    eh_pad = e.clone()
    eh_pad[live * k:] = float("nan")
    w = dev(np.abs(synth.activations(13301, rows, k)))
    y = torch.full((rows, N + pad), float(S32), device="cuda")
    qk.qk_moe_combine_bf16(eh_pad, N + pad, w, rows, k, N, y, N + pad, live_ptr(live))
    wh = host(w).astype(np.float64)
    ref, S = (eh * wh[:, :, None]).sum(1), (np.abs(eh) * wh[:, :, None]).sum(1)
    got = host(y)
    assert np.all(np.abs(got[:live, :N] - ref[:live]) <= k * 2.0 ** -24 * S[:live] + 1e-30)
    assert np.all(got[live:] == S32) and np.all(got[:, N:] == S32)
    # the same sum as the binary32 combine of the widened rows, bit for bit
    y2 = torch.full_like(y, float(S32))
    qk.qk_moe_combine(eh_pad.float(), N + pad, w, rows, k, N, y2, N + pad, live_ptr(live))
    assert np.array_equal(got, host(y2))


# ------------------------------------------------------------------ the chain
@pytest.mark.parametrize("wtype", ["q4_0", "q4_g64", "q4_g128"])
def test_routed_prefill_ffn(wtype):
    """RMSNorm planes, routing, gate/up, SwiGLU planes, down, combine: captured once for a bucket of 150
    rows and replayed at two live counts, against the binary64 definition from the input rows."""
    import torch
    rows, k, E, K, F = 150, 4, 10, 512, 256
    gen = synth.q4_0_weight if wtype == "q4_0" else lambda s, n, kk: synth.q4_group_weight(s, n, kk, int(wtype[4:]))
    deq = (lambda W, n, kk: O.dequant("q4_0", W, n, kk).astype(np.float64)) if wtype == "q4_0" else O.dequant_group
    Wg, Wu, Wd = ([gen(13400 + 100 * j + e, n, kk) for e in range(E)] for j, (n, kk) in enumerate([(F, K), (F, K), (K, F)]))
    pg, pu, pd = pack_experts(Wg, wtype, F, K), pack_experts(Wu, wtype, F, K), pack_experts(Wd, wtype, K, F)
    x, wn = synth.activations(13410, rows, K), synth.norm_weight(13411, K)
    logits = synth.router_logits(13412, rows, E)
    dx, dw, dl = dev(x), dev(wn), dev(logits)
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
    yn, qs, d = z(rows, K), z(rows, K, dtype=torch.int8), z(rows, K // 32, dtype=torch.int16)
    ids, wts = z(rows, k, dtype=torch.int32), z(rows, k)
    counts, offsets, items = z(E, dtype=torch.int32), z(E + 1, dtype=torch.int32), z(rows * k, dtype=torch.int32)
    gu = z(rows * k, 2 * F, dtype=torch.bfloat16)
    hq, hd = z(rows * k, F, dtype=torch.int8), z(rows * k, F // 32, dtype=torch.int16)
    dn, y = z(rows * k, K, dtype=torch.bfloat16), z(rows, K)
    gate_up = [qk.make_proj_id16(wtype, E, pg, F, K, gu, 2 * F), qk.make_proj_id16(wtype, E, pu, F, K, gu[:, F:], 2 * F)]
    down = [qk.make_proj_id16(wtype, E, pd, K, F, dn, K)]
    n = max(qk.qk_mmq_id_workspace_bytes(rows, k, gate_up), qk.qk_mmq_id_workspace_bytes(rows, k, down))
    ws, live = torch.empty((n,), dtype=torch.uint8, device="cuda"), live_ptr(rows)

    def ffn():
        qk.qk_rmsnorm_q8_0(dx, rows, K, K, "mul", dw, None, 1.0, 1e-6, yn, K, qs, d, K // 32, live)
        qk.qk_route_plan(dl, rows, E, k, ids, wts, counts, offsets, items, live)
        qk.qk_mmq_id(qs, d, K // 32, rows, k, gate_up, counts, offsets, items, ws, n)
        qk.qk_glu_q8_0("swiglu", "packed", "bf16", gu, 2 * F, None, 0, rows * k, F, None, 0, hq, hd, F // 32,
                       d_live_rows=offsets[E:])
        qk.qk_mmq_id_slots(hq, hd, F // 32, rows, k, down, counts, offsets, items, ws, n)
        qk.qk_moe_combine_bf16(dn, K, wts, rows, k, K, y, K, live)

    ffn()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            ffn()
    xn = O.rmsnorm(x, "mul", w=wn, eps=1e-6).astype(np.float64)
    ri, rw = O.topk_route(logits, k)
    want = np.zeros((rows, K))
    for e in range(E):
        r, sl = np.nonzero(ri == e)
        if r.size:
            h = glu64("swiglu", xn[r] @ deq(Wg[e], F, K).T, xn[r] @ deq(Wu[e], F, K).T)
            np.add.at(want, r, rw[r, sl][:, None] * (h @ deq(Wd[e], K, F).T))
    for m in (rows, 83):
        live.fill_(m)
        y.fill_(float(S32))
        torch.cuda.synchronize()
        graph.replay()
        got = host(y)
        assert O.nmse(got[:m], want[:m]) <= 5e-4 + 6e-6, m
        assert np.all(got[m:] == S32), m
    assert qk.qk_device_faults() == 0
