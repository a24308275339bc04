"""GPU: in a captured graph every kernel of a chain reads what the kernel before it wrote in this replay.

A kernel of the library starts while its predecessor still runs and then waits for it; a read of the predecessor's
outputs that is made before that wait gets the bytes of the replay before. Every chain is captured once and replayed
with new inputs, live counts and routes; each of its buffers has to equal, byte for byte, those of calls made one at a
time with the device idle in between.
"""
import numpy as np
import pytest

from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import dev, live_ptr

pytestmark = pytest.mark.gpu


def weights(seed, wtype, E, N, K):
    """E packed random matrices, made on the device."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    G, head = {"q4_0": (32, 2), "q8_0": (32, 2), "q4_g64": (64, 4), "q4_g128": (128, 4)}[wtype]
    per = qk.qk_weight_packed_bytes(wtype, N, K)
    out = torch.empty((E * per,), dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.randint(0, 256, (N, K // G, head + (32 if wtype == "q8_0" else G // 2)), dtype=torch.uint8, device="cuda",
                          generator=gen)
        w[..., 0:2] = (torch.rand((N, K // G, 1), device="cuda", generator=gen) * 0.02 + 0.001).half().view(torch.uint8)
        qk.qk_weight_pack(wtype, w, N, K, out[e * per:], per)
    return out


class Chain:
    """Calls in order over named buffers. A subclass fills `buf` and `steps`; `fresh(i)` gives the inputs of pass i."""

    def __init__(self):
        self.buf, self.steps, self.keep = {}, [], []

    def new(self, name, shape, dtype="float32"):
        import torch
        self.buf[name] = torch.zeros(shape, dtype=getattr(torch, dtype), device="cuda")
        return self.buf[name]

    def snapshot(self):
        import torch
        torch.cuda.synchronize()
        return {n: t.view(torch.uint8).cpu().numpy().copy() for n, t in self.buf.items()}

    def load(self, inputs):
        import torch
        for n, v in inputs.items():
            self.buf[n].copy_(dev(np.asarray(v)))
        torch.cuda.synchronize()

    def one_at_a_time(self):
        import torch
        for step in self.steps:
            step()
            torch.cuda.synchronize()


class RoutedDecode(Chain):
    def __init__(self, wtype, rows, E, k, K, NF, fused_plan):
        super().__init__()
        self.rows, self.E, self.K = rows, E, K
        new, b = self.new, self.buf
        x, norm, logits = new("x", (rows, K)), new("norm", (K,)), new("logits", (rows, E))
        y, img = new("y", (rows, K)), new("img", (rows * K // 32 * 36,), "uint8")
        ids, wts, live = new("ids", (rows, k), "int32"), new("wts", (rows, k)), new("live", (1,), "int32")
        plan = new("counts", (E,), "int32"), new("offsets", (E + 1,), "int32"), new("items", (rows * k,), "int32")
        g, u, h = (new(n, (rows * k, NF)) for n in ("gate", "up", "h"))
        himg, down, out = new("himg", (rows * k * NF // 32 * 36,), "uint8"), new("down", (rows * k, K)), new("out", (rows, K))
        w = [weights(61, wtype, E, NF, K), weights(62, wtype, E, NF, K), weights(63, wtype, E, K, NF)]
        gate_up = [qk.make_proj_id(wtype, E, w[0], NF, K, g), qk.make_proj_id(wtype, E, w[1], NF, K, u)]
        down_p = [qk.make_proj_id(wtype, E, w[2], K, NF, down)]
        self.keep = w
        self.steps = [lambda: qk.qk_rmsnorm_q8_1(x, rows, K, K, "mul", norm, None, 0.0, 1e-5, y, K, img, K // 32, live)]
        if fused_plan:
            self.steps += [lambda: qk.qk_route_plan(logits, rows, E, k, ids, wts, *plan, live)]
        else:
            self.steps += [lambda: qk.qk_topk_route(logits, rows, E, k, ids, wts, live),
                           lambda: qk.qk_moe_plan(ids, rows, k, E, *plan, live)]
        self.steps += [
            lambda: qk.qk_mmvq_id(img, K // 32, rows, k, gate_up, *plan),
            lambda: qk.qk_glu_q8_1("swiglu", "separate", g, NF, u, NF, rows * k, NF, h, NF, himg, NF // 32, plan[1][E:]),
            lambda: qk.qk_mmvq_id_slots(himg, NF // 32, rows, k, down_p, *plan),
            lambda: qk.qk_moe_combine(down, K, wts, rows, k, K, out, K, live)]

    def fresh(self, i):
        return dict(x=synth.activations(70 + i, self.rows, self.K) * (1 + i), norm=synth.norm_weight(71 + i, self.K),
                    logits=synth.router_logits(72 + i, self.rows, self.E), live=[max(1, self.rows * (3 * i % 4 + 1) // 4)])


class RoutedPrefill(Chain):
    def __init__(self, wtype, rows, E, k, K, NF):
        super().__init__()
        self.rows, self.E, self.K = rows, E, K
        new = self.new
        x, norm, logits, y = new("x", (rows, K)), new("norm", (K,)), new("logits", (rows, E)), new("y", (rows, K))
        q, d = new("q", (rows, K), "int8"), new("d", (rows, K // 32), "int16")
        ids, wts, live = new("ids", (rows, k), "int32"), new("wts", (rows, k)), new("live", (1,), "int32")
        plan = new("counts", (E,), "int32"), new("offsets", (E + 1,), "int32"), new("items", (rows * k,), "int32")
        gu, down, out = new("gu", (rows * k, 2 * NF), "bfloat16"), new("down", (rows * k, K), "bfloat16"), new("out", (rows, K))
        hq, hd = new("hq", (rows * k, NF), "int8"), new("hd", (rows * k, NF // 32), "int16")
        w = [weights(64, wtype, E, NF, K), weights(65, wtype, E, NF, K), weights(66, wtype, E, K, NF)]
        gate_up = [qk.make_proj_id16(wtype, E, w[0], NF, K, gu, 2 * NF), qk.make_proj_id16(wtype, E, w[1], NF, K, gu[:, NF:], 2 * NF)]
        down_p = [qk.make_proj_id16(wtype, E, w[2], K, NF, down, K)]
        n = max(qk.qk_mmq_id_workspace_bytes(rows, k, gate_up), qk.qk_mmq_id_workspace_bytes(rows, k, down_p))
        import torch
        ws = torch.empty((n,), dtype=torch.uint8, device="cuda")   # scratch: not compared
        self.keep = w + [ws]
        self.steps = [
            lambda: qk.qk_rmsnorm_q8_0(x, rows, K, K, "mul", norm, None, 0.0, 1e-5, y, K, q, d, K // 32, live),
            lambda: qk.qk_topk_route(logits, rows, E, k, ids, wts, live),
            lambda: qk.qk_moe_plan(ids, rows, k, E, *plan, live),
            lambda: qk.qk_mmq_id(q, d, K // 32, rows, k, gate_up, *plan, ws, n),
            lambda: qk.qk_glu_q8_0("swiglu", "packed", "bf16", gu, 2 * NF, None, 0, rows * k, NF, None, 0, hq, hd, NF // 32,
                                   d_live_rows=plan[1][E:]),
            lambda: qk.qk_mmq_id_slots(hq, hd, NF // 32, rows, k, down_p, *plan, ws, n),
            lambda: qk.qk_moe_combine_bf16(down, K, wts, rows, k, K, out, K, live)]

    fresh = RoutedDecode.fresh


class DenseDecode(Chain):
    """A norm, projections of every weight type, a GLU, a down projection and a quantiser."""

    def __init__(self, T, K, N):
        super().__init__()
        import torch
        self.T, self.K = T, K
        new = self.new
        x, norm, live = new("x", (T, K)), new("norm", (K,)), new("live", (1,), "int32")
        y, img = new("y", (T, K)), new("img", (T * K // 32 * 36,), "uint8")
        types = ("q4_0", "q8_0", "q4_g64", "q4_g128")
        ys = [new("y_" + t, (T, N)) for t in types]
        h, himg, down = new("h", (T, N)), new("himg", (T * N // 32 * 36,), "uint8"), new("down", (T, K))
        dimg, last = new("dimg", (T * K // 32 * 36,), "uint8"), new("last", (T, N))
        w = [weights(80 + i, t, 1, N, K) for i, t in enumerate(types)]
        wd = weights(85, "q4_g128", 1, K, N)
        projs = [qk.make_proj(t, wi, N, K, yi, N) for t, wi, yi in zip(types, w, ys)]
        down_p, last_p = [qk.make_proj("q4_g128", wd, K, N, down, K)], [qk.make_proj("q4_g64", w[2], N, K, last, N)]
        n = qk.qk_mmvq_workspace_bytes(projs)
        ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")
        self.keep = w + [wd, ws]
        self.steps = [
            lambda: qk.qk_rmsnorm_q8_1(x, T, K, K, "mul", norm, None, 0.0, 1e-5, y, K, img, K // 32, live),
            lambda: qk.qk_mmvq(img, K // 32, T, projs, ws, n, live),
            lambda: qk.qk_glu_q8_1("geglu_tanh", "separate", ys[2], N, ys[3], N, T, N, h, N, himg, N // 32, live),
            lambda: qk.qk_mmvq(himg, N // 32, T, down_p, None, 0, live),
            lambda: qk.qk_quantize_q8_1(down, T, K, K, dimg, K // 32, live),
            lambda: qk.qk_mmvq(dimg, K // 32, T, last_p, None, 0, live)]

    def fresh(self, i):
        return dict(x=synth.activations(90 + i, self.T, self.K) * (1 + i), norm=synth.norm_weight(91 + i, self.K),
                    live=[max(1, self.T * (3 * i % 4 + 1) // 4)])


class DensePrefill(Chain):
    def __init__(self, T, K, N):
        super().__init__()
        import torch
        self.T, self.K = T, K
        new = self.new
        x, norm, y = new("x", (T, K)), new("norm", (K,)), new("y", (T, K))
        q, d = new("q", (T, K), "int8"), new("d", (T, K // 32), "int16")
        g, u = new("gate", (T, N)), new("up", (T, N))
        hq, hd, down = new("hq", (T, N), "int8"), new("hd", (T, N // 32), "int16"), new("down", (T, K))
        dq, dd = new("dq", (T, K), "int8"), new("dd", (T, K // 32), "int16")
        w = [weights(86, "q4_0", 1, N, K), weights(87, "q4_0", 1, N, K), weights(88, "q4_0", 1, K, N)]
        gate_up = [qk.make_proj("q4_0", w[0], N, K, g, N), qk.make_proj("q4_0", w[1], N, K, u, N)]
        down_p = [qk.make_proj("q4_0", w[2], K, N, down, K)]
        n = max(qk.qk_mmq_workspace_bytes(T, gate_up), qk.qk_mmq_workspace_bytes(T, down_p))
        ws = torch.empty((n,), dtype=torch.uint8, device="cuda")
        self.keep = w + [ws]
        self.steps = [
            lambda: qk.qk_rmsnorm_q8_0(x, T, K, K, "mul", norm, None, 0.0, 1e-5, y, K, q, d, K // 32),
            lambda: qk.qk_mmq(q, d, K // 32, T, gate_up, ws, n),
            lambda: qk.qk_glu_q8_0("swiglu", "separate", "f32", g, N, u, N, T, N, None, 0, hq, hd, N // 32),
            lambda: qk.qk_mmq(hq, hd, N // 32, T, down_p, ws, n),
            lambda: qk.qk_quantize_q8_0(down, T, K, K, dq, dd, K // 32)]

    def fresh(self, i):
        return dict(x=synth.activations(95 + i, self.T, self.K) * (1 + i), norm=synth.norm_weight(96 + i, self.K))


CHAINS = {
    **{f"decode-{wt}-{rows}-{'fused' if fused else 'two'}": (lambda wt=wt, rows=rows, fused=fused:
       RoutedDecode(wt, rows, 128, 8, 512, 256, fused))
       for wt in ("q4_0", "q8_0", "q4_g64", "q4_g128") for rows, fused in ((4, True), (16, True), (16, False), (64, False))},
    "decode-long-q4_g64": lambda: RoutedDecode("q4_g64", 8, 6, 2, 4096, 2752, True),
    **{f"prefill-{wt}-{rows}": (lambda wt=wt, rows=rows: RoutedPrefill(wt, rows, 64, 8, 512, 256))
       for wt in ("q4_0", "q4_g64", "q4_g128") for rows in (20, 300)},
    "dense-decode-1": lambda: DenseDecode(1, 512, 256),
    "dense-decode-8": lambda: DenseDecode(8, 3584, 2048),
    "dense-prefill-40": lambda: DensePrefill(40, 512, 256),
    "dense-prefill-700": lambda: DensePrefill(700, 1024, 2048),
}


@pytest.mark.parametrize("name", CHAINS)
def test_back_to_back_calls_read_each_others_outputs(name):
    import torch
    chain, passes = CHAINS[name](), 6
    chain.load(chain.fresh(passes))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for step in chain.steps:
            step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for step in chain.steps:
            step()

    def queued():
        torch.cuda._sleep(300000)   # the calls are all in the stream before the first of them starts
        for step in chain.steps:
            step()

    start = {n: t.clone() for n, t in chain.buf.items()}
    runs = {}
    for how, go in (("one at a time", chain.one_at_a_time), ("replayed", graph.replay), ("queued", queued)):
        for n, t in start.items():
            chain.buf[n].copy_(t)
        runs[how] = []
        for i in range(passes):
            chain.load(chain.fresh(i))
            go()
            runs[how].append(chain.snapshot())
    assert qk.qk_device_faults() == 0
    for how in ("replayed", "queued"):
        for i, (got, want) in enumerate(zip(runs[how], runs["one at a time"])):
            wrong = [n for n in got if not np.array_equal(got[n], want[n])]
            assert not wrong, f"{how}, pass {i}: {wrong}"
