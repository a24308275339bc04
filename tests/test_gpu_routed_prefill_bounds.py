"""Guard bands, far offsets, unsound plans, concurrent streams: group-scaled matvecs, routed prefill
products, the Q8_0 GLU producer and the bfloat16 combine.

Results are compared with the binary64 product of the decoded operands where a tolerance is needed:
binary32 outputs within 1e-5 of the largest (see assert_exact_path), bfloat16 ones within 2^-8 of the
result plus 2^-9 of sum |w x| (a rounding to bfloat16 and two to binary16 per product, doubled)."""
import numpy as np
import pytest

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import assert_exact_path, dev, host, live_ptr, pack_experts, pack_weight

pytestmark = pytest.mark.gpu

CANARY = 0xC3


class Guarded:
    """`rows` rows of `width` elements with `pad` elements between them, in a buffer of canary bytes."""

    def __init__(self, rows, width, pad, dtype):
        import torch
        self.rows, self.width, self.stride = rows, width, width + pad
        self.es = torch.empty((), dtype=dtype).element_size()
        self.front = 4096
        self.buf = torch.full((2 * self.front + rows * self.stride * self.es,), CANARY, dtype=torch.uint8, device="cuda")
        self.t = self.buf[self.front:-self.front].view(dtype).view(rows, self.stride)

    def check(self, written_rows, what):
        b = host(self.buf)
        assert (b[:self.front] == CANARY).all() and (b[-self.front:] == CANARY).all(), f"{what}: outside the buffer"
        r = b[self.front:-self.front].reshape(self.rows, self.stride * self.es)
        assert (r[:, self.width * self.es:] == CANARY).all(), f"{what}: past a row's width"
        keep = np.ones(self.rows, dtype=bool)
        keep[list(written_rows)] = False
        assert (r[keep] == CANARY).all(), f"{what}: a row that is none of the call's"


def plan(ids, E, live):
    import torch
    rows, k = ids.shape
    c, o, i = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (E, E + 1, rows * k))
    qk.qk_moe_plan(dev(ids), rows, k, E, c, o, i, live_ptr(live))
    return c, o, i


# ------------------------------------------------------------------ guard bands
@pytest.mark.parametrize("G", [64, 128])
@pytest.mark.parametrize("N", [1, 31, 33, 97])
def test_matvec_guard_bands(G, N):
    import torch
    T, K, live = 7, 384, 5
    img = dev(O.quantize_q8_1(synth.activations(14000, T, K)).reshape(-1))
    y = Guarded(T, N, 3, torch.float32)
    W = pack_weight(synth.q4_group_weight(14001, N, K, G), f"q4_g{G}", N, K)
    qk.qk_mmvq(img, K // 32, T, [qk.make_proj(f"q4_g{G}", W, N, K, y.t, y.stride)], None, 0, live_ptr(live))
    y.check(range(live), "mmvq")
    rows, k, E = 5, 2, 3
    ids = synth.rng(14002).integers(0, E, size=(rows, k), dtype=np.int32)
    img = dev(O.quantize_q8_1(synth.activations(14003, rows, K)).reshape(-1))
    yi = Guarded(rows * k, N, 0, torch.float32)
    pw = pack_experts([synth.q4_group_weight(14010 + e, N, K, G) for e in range(E)], f"q4_g{G}", N, K)
    qk.qk_mmvq_id(img, K // 32, rows, k, [qk.make_proj_id(f"q4_g{G}", E, pw, N, K, yi.t)], *plan(ids, E, 4))
    yi.check(range(4 * k), "mmvq_id")


@pytest.mark.parametrize("wtype", ["q4_0", "q4_g64", "q4_g128"])
@pytest.mark.parametrize("N,pad", [(1, 0), (7, 1), (129, 0), (136, 8), (260, 2)])
def test_routed_prefill_guard_bands(wtype, N, pad):
    import torch
    rows, k, E, K, live = 45, 2, 3, 256, 41
    qs, dh = O.quantize_q8_0(synth.activations(14100, rows, K))
    ids = synth.rng(14101).integers(0, E, size=(rows, k), dtype=np.int32)
    gen = synth.q4_0_weight if wtype == "q4_0" else lambda s, n, kk: synth.q4_group_weight(s, n, kk, int(wtype[4:]))
    pw = pack_experts([gen(14110 + e, N, K) for e in range(E)], wtype, N, K)
    y = Guarded(rows * k, N, pad, torch.bfloat16)
    projs = [qk.make_proj_id16(wtype, E, pw, N, K, y.t, y.stride)]
    n = qk.qk_mmq_id_workspace_bytes(rows, k, projs)
    ws = Guarded(1, n, 0, torch.uint8)
    qk.qk_mmq_id(dev(qs), dev(dh.view(np.int16)), K // 32, rows, k, projs, *plan(ids, E, live), ws.t, n)
    y.check(range(live * k), "mmq_id")
    ws.check([0], "workspace")


@pytest.mark.parametrize("elem", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,rb", [(11, 32, 1), (5, 4128, 129), (13, 96, 7), (3, 8192, 256)])
def test_glu_guard_bands(elem, T, N, rb):
    import torch
    dt = torch.bfloat16 if elem == "bf16" else torch.float32
    live = T - 2
    a = dev(synth.activations(14200, T, 2 * N)).to(dt)
    out, qs, d = Guarded(T, N, 4, torch.float32), Guarded(T, rb * 32, 0, torch.int8), Guarded(T, rb, 0, torch.int16)
    qk.qk_glu_q8_0("swiglu", "packed", elem, a, 2 * N, None, 0, T, N, out.t, out.stride, qs.t, d.t, rb,
                   d_live_rows=live_ptr(live))
    out.check(range(live), "out")
    qs.check(range(live), "qs")
    d.check(range(live), "d")


def test_combine_guard_bands():
    import torch
    for N in (4, 1028, 2056):
        e = dev(synth.activations(14300, 15, N)).bfloat16()
        y = Guarded(5, N, 4, torch.float32)
        qk.qk_moe_combine_bf16(e, N, dev(synth.activations(14301, 5, 3)), 5, 3, N, y.t, y.stride, live_ptr(3))
        y.check(range(3), f"combine {N}")


# ------------------------------------------------------------------ far offsets
def test_rows_more_than_four_gib_apart():
    """Strides at which rows start past 2^31 and 2^32 bytes, outputs and inputs."""
    import torch
    far = (1 << 29) + 8                                      # elements between rows
    K, N, T = 256, 40, 5
    W = synth.q4_group_weight(14400, N, K, 64)
    x = synth.activations(14401, T, K)
    img = O.quantize_q8_1(x)
    y = torch.empty(((T - 1) * far + 128,), device="cuda")      # a row of 128 as bfloat16 fits too
    qk.qk_mmvq(dev(img.reshape(-1)), K // 32, T, [qk.make_proj("q4_g64", pack_weight(W, "q4_g64", N, K), N, K, y, far)],
               None, 0)
    got = np.stack([host(y[t * far:t * far + N]) for t in range(T)])
    assert_exact_path(got, O.image_values(img, K) @ O.dequant_group(W, N, K).T)
    # GLU input rows and combine rows out of the same buffer, seen as bfloat16
    b = y.view(torch.bfloat16)
    g = synth.activations(14402, T, 128)
    for t in range(T):
        b[t * 2 * far:t * 2 * far + 128] = dev(g[t]).bfloat16()
    qs, d = torch.empty((T, 64), dtype=torch.int8, device="cuda"), torch.empty((T, 2), dtype=torch.int16, device="cuda")
    qk.qk_glu_q8_0("reglu", "packed", "bf16", b, 2 * far, None, 0, T, 64, None, 0, qs, d, 2)
    gr = host(dev(g).bfloat16().float())
    oq, od = O.quantize_q8_0(np.maximum(gr[:, :64], 0) * gr[:, 64:])
    assert np.array_equal(host(qs), oq.reshape(T, -1)) and np.array_equal(host(d).view(np.uint16), od.reshape(T, -1))
    z = torch.empty((1, 128), device="cuda")
    qk.qk_moe_combine_bf16(b, 2 * far, dev(np.ones((1, T), dtype=np.float32)), 1, T, 128, z, 128)
    assert np.allclose(host(z)[0], gr.sum(0), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("wtype", ["q4_g128", "q4_0"])
def test_weights_past_four_gib(wtype):
    """The last expert's weights start past 2^32 bytes."""
    import torch
    E, N, K, rows = 9, 16384, 65536, 3
    block = 18 if wtype == "q4_0" else 68
    G = 32 if wtype == "q4_0" else 128
    gen = torch.Generator(device="cuda")
    gen.manual_seed(14500)
    per = qk.qk_weight_packed_bytes(wtype, N, K)
    assert per * (E - 1) > 1 << 32
    packed = torch.zeros((E * per,), dtype=torch.uint8, device="cuda")
    w = torch.randint(0, 256, (N, K // G, block), dtype=torch.uint8, device="cuda", generator=gen)
    scale = torch.full((N, K // G, 1), 0.01, dtype=torch.float16, device="cuda")
    w[..., 0:2] = scale.view(torch.uint8)
    qk.qk_weight_pack(wtype, w, N, K, packed[(E - 1) * per:], per)
    ids = np.full((rows, 1), E - 1, dtype=np.int32)
    p = plan(ids, E, rows)
    x = synth.activations(14501, rows, K)
    sel = np.array([0, 1, 127, 8191, N - 2, N - 1])
    Wd = (O.dequant("q4_0", host(w[sel]), len(sel), K) if wtype == "q4_0" else O.dequant_group(host(w[sel]), len(sel), K))
    if wtype != "q4_0":
        img = O.quantize_q8_1(x)
        y = torch.zeros((rows, N), device="cuda")
        qk.qk_mmvq_id(dev(img.reshape(-1)), K // 32, rows, 1, [qk.make_proj_id(wtype, E, packed, N, K, y)], *p)
        assert_exact_path(host(y)[:, sel], O.image_values(img, K) @ Wd.T, what="mmvq_id")
    qs, dh = O.quantize_q8_0(x)
    yb = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    projs = [qk.make_proj_id16(wtype, E, packed, N, K, yb, N)]
    n = qk.qk_mmq_id_workspace_bytes(rows, 1, projs)
    ws = torch.empty((n,), dtype=torch.uint8, device="cuda")
    qk.qk_mmq_id(dev(qs), dev(dh.view(np.int16)), K // 32, rows, 1, projs, *p, ws, n)
    xv = O.plane_values(qs.reshape(rows, -1), dh.reshape(rows, -1), K)
    ref, S = xv @ Wd.T, np.abs(xv) @ np.abs(Wd).T
    got = host(yb.float())[:, sel]
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * S)
    assert qk.qk_device_faults() == 0


# ------------------------------------------------------------------ plans from elsewhere
def test_counts_that_no_plan_has_do_no_work():
    """Every expert claims every pair: more passes than any plan of the bucket. Nothing is written and
    bit 1 of the fault word is set; the next sound call works."""
    import torch
    rows, k, E, K, N = 200, 2, 16, 128, 40
    qs, dh = O.quantize_q8_0(synth.activations(14600, rows, K))
    img = dev(O.quantize_q8_1(synth.activations(14600, rows, K)).reshape(-1))
    pw = pack_experts([synth.q4_group_weight(14610 + e, N, K, 128) for e in range(E)], "q4_g128", N, K)
    counts = torch.full((E,), rows * k, dtype=torch.int32, device="cuda")
    offsets = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
    items = torch.arange(rows * k, dtype=torch.int32, device="cuda")
    qk.qk_device_faults()
    y = torch.full((rows * k, N), 7.0, device="cuda")
    qk.qk_mmvq_id(img, K // 32, rows, k, [qk.make_proj_id("q4_g128", E, pw, N, K, y)], counts, offsets, items)
    assert qk.qk_device_faults() == 2 and bool((y == 7.0).all())
    yb = torch.full((rows * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    projs = [qk.make_proj_id16("q4_g128", E, pw, N, K, yb, N)]
    n = qk.qk_mmq_id_workspace_bytes(rows, k, projs)
    ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")
    args = (dev(qs), dev(dh.view(np.int16)), K // 32, rows, k, projs)
    qk.qk_mmq_id(*args, counts, offsets, items, ws, n)
    assert qk.qk_device_faults() == 2 and bool((yb == 7.0).all())
    ids = synth.rng(14601).integers(0, E, size=(rows, k), dtype=np.int32)
    qk.qk_mmq_id(*args, *plan(ids, E, rows), ws, n)
    assert qk.qk_device_faults() == 0 and not bool((yb == 7.0).any())


def test_matvec_of_a_plan_from_elsewhere_stays_in_bounds():
    import torch
    rows, k, E, K, N = 20, 2, 6, 256, 64
    img_h = O.quantize_q8_1(synth.activations(14700, rows, K))
    Ws = [synth.q4_group_weight(14710 + e, N, K, 64) for e in range(E)]
    pw = pack_experts(Ws, "q4_g64", N, K)
    counts = dev(np.array([5, -7, 1 << 30, 3, 2, 4], dtype=np.int32))
    offsets = dev(np.array([0, 5, 38, -(1 << 30), 1 << 30, 10, 14], dtype=np.int32))
    it = np.full((rows * k,), -1, dtype=np.int32)
    it[0:5] = [7, 39, 0, 12, 25]
    it[10:14] = [40, 1 << 30, -5, 31]
    y = Guarded(rows * k, N, 0, torch.float32)
    qk.qk_mmvq_id(dev(img_h.reshape(-1)), K // 32, rows, k, [qk.make_proj_id("q4_g64", E, pw, N, K, y.t)], counts, offsets,
                  dev(it))
    sound = [7, 39, 0, 12, 25]
    y.check(sound + [31], "mmvq_id")
    x = O.image_values(img_h, K)
    assert_exact_path(host(y.t)[sound], x[np.array(sound) // k] @ O.dequant_group(Ws[0], N, K).T)
    assert_exact_path(host(y.t)[[31]], x[[15]] @ O.dequant_group(Ws[5], N, K).T)
    qk.qk_device_faults()


# ------------------------------------------------------------------ streams
def test_calls_on_two_streams_at_once():
    """The same projections enqueued on two streams without any order between them, each with its own
    outputs and workspace: every result is the lone call's."""
    import torch
    rows, k, E, K, N = 150, 2, 5, 512, 200
    qs, dh = O.quantize_q8_0(synth.activations(14800, rows, K))
    d_qs, d_dh = dev(qs), dev(dh.view(np.int16))
    img = dev(O.quantize_q8_1(synth.activations(14801, 8, K)).reshape(-1))
    ids = synth.rng(14802).integers(0, E, size=(rows, k), dtype=np.int32)
    p = plan(ids, E, rows)
    pw = pack_experts([synth.q4_group_weight(14810 + e, N, K, 64) for e in range(E)], "q4_g64", N, K)
    pm = pack_weight(synth.q4_group_weight(14820, 4096, K, 128), "q4_g128", 4096, K)

    def call(stream):
        yb = torch.zeros((rows * k, N), dtype=torch.bfloat16, device="cuda")
        ym = torch.zeros((8, 4096), device="cuda")
        projs = [qk.make_proj_id16("q4_g64", E, pw, N, K, yb, N)]
        n = qk.qk_mmq_id_workspace_bytes(rows, k, projs)
        ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

        def go():
            qk.qk_mmq_id(d_qs, d_dh, K // 32, rows, k, projs, *p, ws, n, stream=stream)
            qk.qk_mmvq(img, K // 32, 8, [qk.make_proj("q4_g128", pm, 4096, K, ym, 4096)], None, 0, stream=stream)
        return go, yb, ym, ws

    lone, yb0, ym0, _ = call(None)
    lone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = call(s1), call(s2)
    for _ in range(20):
        a[0]()
        b[0]()
    torch.cuda.synchronize()
    for _, yb, ym, _ in (a, b):
        assert torch.equal(yb, yb0) and torch.equal(ym, ym0)
    assert qk.qk_device_faults() == 0


def test_plans_rewritten_between_calls():
    """Plan, products, another plan into the same buffers, products .. without a wait in between: the products
    read the plan early, so every result has to be that of its own plan, also in one captured graph."""
    import torch
    rows, k, E, K, N = 96, 2, 12, 128, 136
    qs, dh = O.quantize_q8_0(synth.activations(14900, rows, K))
    d_qs, d_dh = dev(qs), dev(dh.view(np.int16))
    img = dev(O.quantize_q8_1(synth.activations(14901, rows, K)).reshape(-1))
    Ws = [synth.q4_group_weight(14910 + e, N, K, 64) for e in range(E)]
    pw = pack_experts(Ws, "q4_g64", N, K)
    g = synth.rng(14902)
    ids = [g.integers(0, E, size=(rows, k), dtype=np.int32) for _ in range(4)]
    ids[1][:] = 7                                                            # one expert has everything
    d_ids = [dev(i) for i in ids]
    c, o, it = (torch.zeros((n,), dtype=torch.int32, device="cuda") for n in (E, E + 1, rows * k))
    yb = [torch.zeros((rows * k, N), dtype=torch.bfloat16, device="cuda") for _ in ids]
    ym = [torch.zeros((rows * k, N), device="cuda") for _ in ids]
    n = qk.qk_mmq_id_workspace_bytes(rows, k, [qk.make_proj_id16("q4_g64", E, pw, N, K, yb[0], N)])
    ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")

    def step(i, wait):
        qk.qk_moe_plan(d_ids[i], rows, k, E, c, o, it)
        qk.qk_mmq_id(d_qs, d_dh, K // 32, rows, k, [qk.make_proj_id16("q4_g64", E, pw, N, K, yb[i], N)], c, o, it, ws, n)
        qk.qk_mmvq_id(img, K // 32, rows, k, [qk.make_proj_id("q4_g64", E, pw, N, K, ym[i])], c, o, it)
        if wait:
            torch.cuda.synchronize()

    for i in range(4):
        step(i, True)
    want = [(a.clone(), b.clone()) for a, b in zip(yb, ym)]
    x = O.plane_values(qs.reshape(rows, -1), dh.reshape(rows, -1), K)
    Wd = [O.dequant_group(W, N, K) for W in Ws]
    for i, (a, _) in enumerate(want):
        ref = np.stack([x[p // k] @ Wd[e].T for p, e in enumerate(ids[i].reshape(-1))])
        S = np.stack([np.abs(x[p // k]) @ np.abs(Wd[e]).T for p, e in enumerate(ids[i].reshape(-1))])
        assert np.all(np.abs(host(a.float()) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * S)

    def check(what):
        torch.cuda.synchronize()
        for i in range(4):
            assert torch.equal(yb[i], want[i][0]) and torch.equal(ym[i], want[i][1]), (what, i)
            yb[i].zero_()
            ym[i].zero_()

    for rep in range(25):
        for i in range(4):
            step(i, False)
        check(f"run {rep}")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            for i in range(4):
                step(i, False)
    for rep in range(25):
        graph.replay()
        check(f"replay {rep}")
    assert qk.qk_device_faults() == 0
