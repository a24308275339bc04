"""The cache and its attention as they are used: a prompt through RMSNorm, q/k/v, append, attention and the output
projection, then decode steps over the same cache, eager and as a captured graph replayed with new contents."""
import numpy as np
import pytest

from oracle import kv as OK
from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import pack_weight
from tests.kv_helpers import HB16, bf16, decode_error, random_pages

pytestmark = pytest.mark.gpu

D, HQ, HKV, P, K = 64, 6, 2, 16, 256
WIDTH = (HQ + 2 * HKV) * D
SCALE = D ** -0.5


class Layer:
    """Buffers and descriptors of one layer for `rows` rows of B sequences."""

    def __init__(self, seed, pages, geo, B, rows, weights):
        import torch
        f = lambda *s: torch.zeros(s, device="cuda")
        u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        self.B, self.rows, self.geo, self.pages = B, rows, geo, pages
        self.x, self.y, self.qkv, self.o = f(rows, K), f(rows, K), f(rows, WIDTH), f(rows, K)
        self.q = torch.zeros((rows, HQ * D), dtype=torch.bfloat16, device="cuda")
        self.out = f(rows, HQ * D)
        self.img, self.oimg = u8(rows, K // 32, 36), u8(rows, HQ * D // 32, 36)
        self.qs, self.d = u8(rows, K).view(torch.int8), i32(rows, K // 64).view(torch.int16)
        self.oqs, self.od = u8(rows, HQ * D).view(torch.int8), i32(rows, HQ * D // 64).view(torch.int16)
        self.pos, self.slots, self.lens, self.first = i32(1, rows), i32(rows), i32(B), i32(B + 1)
        self.table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
        self.norm = torch.from_numpy(synth.norm_weight(seed, K)).cuda()
        self.freqs = torch.from_numpy((1000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)).cuda()
        self.cache = qk.make_kv_cache(pages, *geo)
        self.rope = qk.make_rope("halves", D, 1, self.pos, self.freqs)
        self.attn = qk.make_attn(self.q, "bf16", HQ * D, HQ, self.table, 12, self.lens, SCALE, 0, None, self.out, "f32",
                                 HQ * D)
        w_qkv, w_o = weights
        self.p_qkv = [qk.make_proj("q4_0", w_qkv, WIDTH, K, self.qkv, WIDTH)]
        self.p_o = [qk.make_proj("q4_0", w_o, K, HQ * D, self.o, K)]
        n = max(qk.qk_mmvq_workspace_bytes(self.p_qkv), qk.qk_mmvq_workspace_bytes(self.p_o), 16)
        self.ws = u8(n)
        n = max(qk.qk_mmq_workspace_bytes(rows, self.p_qkv), qk.qk_mmq_workspace_bytes(rows, self.p_o))
        self.wsm = u8(n)
        self.max_kv = 12 * P
        self.wsp = u8(qk.qk_attn_prefill_workspace_bytes(self.cache, B, self.max_kv))
        if rows <= 8 * B:
            self.wsd = u8(qk.qk_attn_decode_workspace_bytes(self.cache, HQ, B, max(1, rows // B)))

    def _append(self, live=None):
        q = self.qkv
        qk.qk_kv_append(self.cache, "f32", q, WIDTH, HQ, q[:, HQ * D:], WIDTH, q[:, (HQ + HKV) * D:], WIDTH, self.rows,
                        self.slots, self.rope, "bf16", self.q, HQ * D, live)

    def prompt(self):
        r = self.rows
        qk.qk_rmsnorm_q8_0(self.x, r, K, K, "mul", self.norm, None, 1.0, 1e-6, self.y, K, self.qs, self.d, K // 32)
        qk.qk_mmq(self.qs, self.d, K // 32, r, self.p_qkv, self.wsm, self.wsm.numel())
        self._append()
        qk.qk_attn_prefill(self.cache, self.attn, self.B, r, self.first, self.max_kv, self.oqs, self.od, HQ * D // 32,
                           self.wsp, self.wsp.numel())
        qk.qk_mmq(self.oqs, self.od, HQ * D // 32, r, self.p_o, self.wsm, self.wsm.numel())

    def step(self):
        r = self.rows
        qk.qk_rmsnorm_q8_1(self.x, r, K, K, "mul", self.norm, None, 1.0, 1e-6, self.y, K, self.img, K // 32)
        qk.qk_mmvq(self.img, K // 32, r, self.p_qkv, self.ws, self.ws.numel())
        self._append()
        qk.qk_attn_decode(self.cache, self.attn, self.B, r // self.B, self.oimg, HQ * D // 32, self.wsd, self.wsd.numel())
        qk.qk_mmvq(self.oimg, HQ * D // 32, r, self.p_o, self.ws, self.ws.numel())

    def feed(self, seed, n_rows, lens, table):
        """Contents of one call: n_rows[b] new rows of sequence b, whose length becomes lens[b]."""
        import torch
        pos = np.concatenate([np.arange(L - n, L) for n, L in zip(n_rows, lens)])
        slot = np.concatenate([table[b, np.arange(L - n, L) // P] * P + np.arange(L - n, L) % P
                               for b, (n, L) in enumerate(zip(n_rows, lens))])
        put = lambda t, a: t.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(t.dtype).view(t.shape))
        put(self.x, synth.activations(seed, self.rows, K))
        put(self.pos, pos), put(self.slots, slot), put(self.lens, lens), put(self.table, table)
        put(self.first, np.concatenate([[0], np.cumsum(n_rows)]))


def check_attention(L, n_rows, lens, table, prefill):
    """The attention stage against binary64, from the rotated rows and the pages that the GPU has."""
    import torch
    torch.cuda.synchronize()
    k, v = OK.values(L.pages.cpu().numpy(), L.geo)
    q = L.q.float().cpu().numpy().reshape(L.rows, HQ, D)
    got = L.out.cpu().numpy().reshape(L.rows, HQ, D)
    at = 0
    for b, (n, length) in enumerate(zip(n_rows, lens)):
        j = np.arange(length)
        slot = table[b, j // P] * P + j % P
        want, parts = OK.attention(q[at:at + n].astype(np.float64), k[slot], v[slot], np.ones(length, bool), n, SCALE)
        tol = decode_error(v[slot], want, parts, HQ // HKV, prefill) + 2.0 ** -24 * np.abs(want)
        assert (np.abs(got[at:at + n] - want) <= tol).all()
        at += n


def test_prompt_then_decode_steps_eager_and_captured():
    import torch
    W = synth.q4_0_weight(71, WIDTH, K)
    weights = pack_weight(W, "q4_0", WIDTH, K), pack_weight(synth.q4_0_weight(72, K, HQ * D), "q4_0", K, HQ * D)
    geo = (30, P, HKV, D)
    pages = torch.full((30 * qk.qk_kv_page_bytes(P, HKV, D),), 0xFF, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)
    table = rng.permutation(24).reshape(2, 12)
    # prompts of 61 and 40 tokens
    rows = [61, 40]
    pre = Layer(70, pages, geo, 2, sum(rows), weights)
    pre.feed(1, rows, rows, table)
    pre.prompt()
    check_attention(pre, rows, rows, table, True)
    x = pre.x.cpu().numpy()
    y = O.rmsnorm(x, "mul", w=synth.norm_weight(70, K), eps=1e-6)
    qkv = y.astype(np.float64) @ O.dequant("q4_0", W, WIDTH, K).T
    assert O.nmse(pre.qkv.cpu().numpy(), qkv) <= 5e-4
    pos = np.concatenate([np.arange(n) for n in rows])
    rot = OK.rotate(pre.qkv.cpu().numpy().reshape(-1, HQ + 2 * HKV, D)[:, :HQ], "halves", D, pos[None],
                    pre.freqs.cpu().numpy()[None])
    assert (np.abs(pre.q.float().cpu().numpy().reshape(rot.shape) - rot) <= HB16 * np.abs(rot) + 1e-5 * np.abs(rot).max()).all()
    oq = O.quantize_q8_0(pre.out.cpu().numpy())
    assert np.array_equal(pre.oqs.cpu().numpy().reshape(101, -1), oq[0].reshape(101, -1))
    # decode: two tokens a sequence and step; the same steps eager and replayed
    lens = np.array(rows)
    dec = Layer(70, pages, geo, 2, 4, weights)
    kept = []
    start = pages.clone()
    for step in range(4):
        lens = lens + 2
        dec.feed(100 + step, [2, 2], lens, table)
        dec.step()
        check_attention(dec, [2, 2], lens, table, False)
        kept.append((dec.out.clone(), dec.oimg.clone(), dec.o.clone(), pages.clone()))
    pages.copy_(start)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            dec.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(pages, start)      # capturing runs nothing
    lens = np.array(rows)
    for step in range(4):
        lens = lens + 2
        dec.feed(100 + step, [2, 2], lens, table)
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip((dec.out, dec.oimg, dec.o, pages), kept[step]):
            assert torch.equal(got, want)
    # one more prompt chunk behind the past, then both calls on the same rows agree within their bounds
    more = Layer(70, pages, geo, 2, 4, weights)
    lens = lens + 2
    more.feed(300, [2, 2], lens, table)
    more.step()
    a = more.out.clone()
    qk.qk_attn_prefill(more.cache, more.attn, 2, 4, more.first, more.max_kv, None, None, 0, more.wsp, more.wsp.numel())
    torch.cuda.synchronize()
    check_attention(more, [2, 2], lens, table, True)
    assert (a - more.out).abs().max() <= 0.01 * a.abs().max()
    assert qk.qk_device_faults() == 0


def test_two_streams_with_their_own_workspaces():
    import torch
    weights = (pack_weight(synth.q4_0_weight(71, WIDTH, K), "q4_0", WIDTH, K),
               pack_weight(synth.q4_0_weight(72, K, HQ * D), "q4_0", K, HQ * D))
    geo = (24, P, HKV, D)
    layers, alone = [], []
    for s in range(2):
        pages = torch.full((24 * qk.qk_kv_page_bytes(P, HKV, D),), 0xFF, dtype=torch.uint8, device="cuda")
        table = np.arange(24).reshape(2, 12)[:, ::-1].copy()
        pre = Layer(70, pages, geo, 2, 100, weights)
        pre.feed(s, [60, 40], [60, 40], table)
        pre.prompt()
        dec = Layer(70, pages, geo, 2, 2, weights)
        dec.feed(10 + s, [1, 1], [61, 41], table)
        dec.step()
        torch.cuda.synchronize()
        layers.append((pre, dec))
        alone.append([t.clone() for t in (pre.out, pre.oqs, pre.o, dec.out, dec.oimg, dec.o)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for (pre, dec), s in zip(layers, streams):
            with torch.cuda.stream(s):
                pre.prompt()
                dec.step()
    torch.cuda.synchronize()
    for (pre, dec), want in zip(layers, alone):
        for got, w in zip((pre.out, pre.oqs, pre.o, dec.out, dec.oimg, dec.o), want):
            assert torch.equal(got, w)


def test_a_captured_prompt_replayed_with_other_splits_of_its_rows():
    """One captured prefill of a bucket of rows: the sequences' rows and lengths change between replays."""
    import torch
    weights = (pack_weight(synth.q4_0_weight(71, WIDTH, K), "q4_0", WIDTH, K),
               pack_weight(synth.q4_0_weight(72, K, HQ * D), "q4_0", K, HQ * D))
    geo = (24, P, HKV, D)
    # some of the splits have pasts that no row of theirs stored: what the pages hold then
    start = torch.from_numpy(random_pages(np.random.default_rng(9), geo).reshape(-1)).cuda()
    pages = start.clone()
    table = np.random.default_rng(3).permutation(24).reshape(2, 12)
    L = Layer(70, pages, geo, 2, 90, weights)
    splits = [([60, 30], [60, 30]), ([1, 89], [1, 150]), ([45, 45], [180, 45]), ([90, 0], [192, 0])]
    kept = []
    for i, (rows, lens) in enumerate(splits):
        L.feed(i, rows, lens, table)
        L.prompt()
        check_attention(L, rows, lens, table, True)
        kept.append((L.out.clone(), L.oqs.clone(), L.od.clone(), L.o.clone(), pages.clone()))
    pages.copy_(start)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            L.prompt()
    torch.cuda.current_stream().wait_stream(side)
    for i, (rows, lens) in enumerate(splits):
        L.feed(i, rows, lens, table)
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip((L.out, L.oqs, L.od, L.o, pages), kept[i]):
            assert torch.equal(got, want)
    assert qk.qk_device_faults() == 0
