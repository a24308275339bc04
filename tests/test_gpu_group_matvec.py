"""GPU parity: projections of a Q8_1 image through group-scaled 4-bit weights, ordinary and routed.

The reference is the product of the decoded operands in binary64 (image values d_a * q, weights
(nibble - z) * d). Block sums are exact integers; binary32 sums over at most K / 32 blocks separate
the two, so assert_exact_path's derivation holds here as well: the correction for the zero point adds
(z - 8) * d * sum(x) per group, of the size of the group's own part and summed in the same binary32.
"""
import numpy as np
import pytest

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import assert_exact_path, dev, host, live_ptr, pack_experts, pack_weight

pytestmark = pytest.mark.gpu

SENTINEL = np.float32(-12345.5)


def image(seed, rows, K, rb=None):
    """A Q8_1 image of N(0, 1) rows, bytes on the host (uint8 [rows][rb * 36])."""
    return O.quantize_q8_1(synth.activations(seed, rows, K), row_blocks=rb or K // 32)


def out(rows, N):
    import torch
    return torch.full((rows, N), float(SENTINEL), dtype=torch.float32, device="cuda")


def ref(img, W, N, K):
    return O.image_values(img, K) @ O.dequant_group(W, N, K).T


# ------------------------------------------------------------------ ordinary
@pytest.mark.parametrize("G", [64, 128])
@pytest.mark.parametrize("T,N,K", [
    (1, 1, 128), (1, 256, 256), (8, 33, 128), (3, 31, 384), (2, 100, 640), (7, 300, 1152), (8, 512, 3584),
    (5, 129, 8192), (8, 64, 18944), (1, 3000, 256), (4, 2100, 2560), (8, 40, 65536),
])
def test_matvec_matches_float64(G, T, N, K):
    seed = 11000 + N + K + T
    img = image(seed, T, K)
    W = synth.q4_group_weight(seed + 1, N, K, G)
    y = out(T, N)
    qk.qk_mmvq(dev(img.reshape(-1)), K // 32, T, [qk.make_proj(f"q4_g{G}", pack_weight(W, f"q4_g{G}", N, K), N, K, y, N)],
               None, 0)
    assert_exact_path(host(y), ref(img, W, N, K), what=f"g{G} {T}x{N}x{K}")
    assert qk.qk_device_faults() == 0


def test_matvec_of_half_a_chunk():
    """K = 64 and K = 192 (groups of 64): the last 128-column chunk is half empty, and the image row
    continues past K with blocks that must not be read into the sums."""
    for K in (64, 192):
        T, N, rb = 4, 70, 9
        img = image(11100 + K, T, rb * 32)
        W = synth.q4_group_weight(11101, N, K, 64)
        y = out(T, N)
        qk.qk_mmvq(dev(img.reshape(-1)), rb, T, [qk.make_proj("q4_g64", pack_weight(W, "q4_g64", N, K), N, K, y, N)],
                   None, 0)
        assert_exact_path(host(y), ref(img, W, N, K), what=f"K={K}")


def test_extreme_zero_points_and_codes():
    """z = 0 and z = 15 with one-signed codes of +-127: the largest sums that the integer path meets."""
    T, N, K = 8, 64, 1024
    for G in (64, 128):
        W = synth.q4_group_weight(11200, N, K, G)
        W[:32, :, 2] = 0
        W[32:, :, 2] = 15
        W[:16, :, 4:] = 0xFF
        W[48:, :, 4:] = 0x00
        x = np.full((T, K), 3.0, dtype=np.float32)
        x[1::2] = -3.0
        img = O.quantize_q8_1(x)
        y = out(T, N)
        qk.qk_mmvq(dev(img.reshape(-1)), K // 32, T,
                   [qk.make_proj(f"q4_g{G}", pack_weight(W, f"q4_g{G}", N, K), N, K, y, N)], None, 0)
        r = ref(img, W, N, K)
        got = host(y)
        # every partial sum is bounded by 15 * 127 * K * d * d_a; K / 32 binary32 roundings of it
        bound = 2.0 ** -24 * (K / 32 + 8) * 15 * np.abs(O.image_values(img, K)).sum(1)[:, None] * 0.02
        assert np.all(np.abs(got - r) <= bound)


def test_projections_of_several_types_share_one_image():
    """Every weight type in one call, each with its own K, over column windows of one output."""
    import torch
    T, live, rb = 6, 5, 40
    img = image(11300, T, rb * 32)
    specs = [("q4_0", 96, 1280), ("q4_g64", 130, 1216), ("q8_0", 40, 1280), ("q4_g128", 1, 128), ("q4_g128", 200, 1280),
             ("q4_g64", 64, 64)]
    width = sum(n for _, n, _ in specs) + 5
    y = out(T, width)
    projs, keep, at = [], [], 0
    for i, (wt, N, K) in enumerate(specs):
        W = (synth.q4_0_weight(11310 + i, N, K) if wt == "q4_0" else synth.q8_0_weight(11310 + i, N, K) if wt == "q8_0"
             else synth.q4_group_weight(11310 + i, N, K, int(wt[4:])))
        p = pack_weight(W, wt, N, K)
        keep.append((W, p))
        projs.append(qk.make_proj(wt, p, N, K, y[:, at:], width))
        at += N
    n = qk.qk_mmvq_workspace_bytes(projs)
    ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")
    d_img = dev(img.reshape(-1))
    qk.qk_mmvq(d_img, rb, T, projs, ws, n, live_ptr(live))
    got = host(y)
    at = 0
    for (wt, N, K), (W, _) in zip(specs, keep):
        r = (ref(img, W, N, K) if wt.startswith("q4_g") else
             O.proj_q8_1(wt, W, N, K, img, rb))
        assert_exact_path(got[:live, at:at + N], r[:live], what=wt)
        at += N
    assert np.all(got[live:] == SENTINEL) and np.all(got[:, at:] == SENTINEL)
    y.fill_(float(SENTINEL))
    qk.qk_mmvq_static_ws(d_img, rb, T, projs, live_ptr(live))
    assert np.array_equal(host(y), got)


@pytest.mark.parametrize("live", [0, 1, 3, 8, 99, -4])
def test_rows_past_the_live_count_stay(live):
    import torch
    T, N, K = 8, 90, 512
    x = synth.poison_rows(synth.activations(11400, T, K), min(max(live, 0), T))
    img = O.quantize_q8_1(np.nan_to_num(x, nan=3.0))
    img = img.reshape(T, -1).copy()
    img[min(max(live, 0), T):] = 0xFF                    # NaN scales in the padding rows
    W = synth.q4_group_weight(11401, N, K, 128)
    y = out(T, N)
    qk.qk_mmvq(dev(img.reshape(-1)), K // 32, T, [qk.make_proj("q4_g128", pack_weight(W, "q4_g128", N, K), N, K, y, N)],
               None, 0, live_ptr(live))
    n = min(max(live, 0), T)
    got = host(y)
    assert_exact_path(got[:n], ref(img[:n], W, N, K), what=f"live {live}") if n else None
    assert np.all(got[n:] == SENTINEL)


def test_deterministic_and_independent_of_the_batch():
    """The same bits on every call; and a row's bits do not depend on the other rows of the batch."""
    T, N, K = 8, 777, 2560
    img = image(11500, T, K)
    W = synth.q4_group_weight(11501, N, K, 64)
    p = pack_weight(W, "q4_g64", N, K)
    y = out(T, N)
    runs = []
    for _ in range(3):
        qk.qk_mmvq(dev(img.reshape(-1)), K // 32, T, [qk.make_proj("q4_g64", p, N, K, y, N)], None, 0)
        runs.append(host(y).copy())
    assert np.array_equal(runs[0], runs[1]) and np.array_equal(runs[0], runs[2])
    y1 = out(1, N)
    qk.qk_mmvq(dev(img[5].copy()), K // 32, 1, [qk.make_proj("q4_g64", p, N, K, y1, N)], None, 0)
    assert np.array_equal(host(y1)[0], runs[0][5])


def test_captured_call_replays_with_new_inputs_on_a_side_stream():
    import torch
    T, N, K = 8, 520, 1024
    W = synth.q4_group_weight(11600, N, K, 128)
    p = pack_weight(W, "q4_g128", N, K)
    x = torch.zeros((T, K), device="cuda")
    img = torch.zeros((T * (K // 32) * 36,), dtype=torch.uint8, device="cuda")
    y, live = out(T, N), live_ptr(T)
    proj = [qk.make_proj("q4_g128", p, N, K, y, N)]

    def step():
        qk.qk_quantize_q8_1(x, T, K, K, img, K // 32, live)
        qk.qk_mmvq(img, K // 32, T, proj, None, 0, live)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                step()
        for i, n in enumerate((8, 2, 5)):
            xs = synth.activations(11610 + i, T, K)
            x.copy_(dev(xs))
            live.fill_(n)
            y.fill_(float(SENTINEL))
            g.replay()
            s.synchronize()
            got = y.cpu().numpy()
            assert_exact_path(got[:n], ref(O.quantize_q8_1(xs), W, N, K)[:n], what=f"replay {i}")
            assert np.all(got[n:] == SENTINEL)


# ------------------------------------------------------------------ routed
def plan(ids, E, live):
    import torch
    rows, k = ids.shape
    counts = torch.full((E,), -9, dtype=torch.int32, device="cuda")
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    items = torch.full((rows * k,), -3, dtype=torch.int32, device="cuda")
    qk.qk_moe_plan(dev(ids), rows, k, E, counts, offsets, items, live_ptr(live))
    return counts, offsets, items


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("G,rows,k,E,K,Ns,live", [
    (64, 1, 1, 1, 64, (1,), 1),
    (128, 16, 8, 128, 2560, (768, 768), 13),
    (64, 24, 2, 3, 320, (203, 77), 24),       # several passes of eight pairs per expert
    (128, 9, 4, 300, 256, (33,), 9),          # most experts have no pair
    (64, 40, 1, 1, 1024, (64,), 37),          # one expert takes everything: five passes
    (128, 32, 6, 7, 768, (129,), 0),          # no live row
])
def test_routed_matches_float64(slots, G, rows, k, E, K, Ns, live):
    import torch
    seed = 11700 + rows + K + E
    n_img = rows * k if slots else rows
    img = image(seed, n_img, K)
    ids = synth.rng(seed + 1).integers(0, E, size=(rows, k), dtype=np.int32)
    counts, offsets, items = plan(ids, E, live)
    ys, projs, keep = [], [], []
    for j, N in enumerate(Ns):
        Ws = [synth.q4_group_weight(seed + 10 + 1000 * j + e, N, K, G) for e in range(E)]
        pw = pack_experts(Ws, f"q4_g{G}", N, K)
        y = out(rows * k, N)
        keep.append((Ws, pw))
        ys.append(y)
        projs.append(qk.make_proj_id(f"q4_g{G}", E, pw, N, K, y))
    call = qk.qk_mmvq_id_slots if slots else qk.qk_mmvq_id
    call(dev(img.reshape(-1)), K // 32, rows, k, projs, counts, offsets, items)
    assert qk.qk_device_faults() == 0
    x = O.image_values(img, K)
    flat = ids.reshape(-1)
    for (Ws, _), y, N in zip(keep, ys, Ns):
        got = host(y)
        if live:
            want = np.zeros((live * k, N))
            for e in np.unique(flat[:live * k]):
                p = np.nonzero(flat[:live * k] == e)[0]
                want[p] = x[p if slots else p // k] @ O.dequant_group(Ws[e], N, K).T
            assert_exact_path(got[:live * k], want, what=f"routed N={N}")
        assert np.all(got[live * k:] == SENTINEL)


def test_routed_row_equals_the_ordinary_matvec_of_its_expert():
    """One token, every expert picked once: each pair's row is qk_mmvq's of that expert (binary32 sums
    in another order)."""
    rows, k, E, N, K = 1, 8, 8, 200, 640
    img = image(11800, rows, K)
    ids = np.array([[3, 1, 7, 0, 2, 6, 5, 4]], dtype=np.int32)
    Ws = [synth.q4_group_weight(11801 + e, N, K, 128) for e in range(E)]
    pw = pack_experts(Ws, "q4_g128", N, K)
    y = out(rows * k, N)
    qk.qk_mmvq_id(dev(img.reshape(-1)), K // 32, rows, k, [qk.make_proj_id("q4_g128", E, pw, N, K, y)],
                  *plan(ids, E, rows))
    got = host(y)
    for p, e in enumerate(ids[0]):
        y1 = out(1, N)
        qk.qk_mmvq(dev(img.reshape(-1)), K // 32, 1,
                   [qk.make_proj("q4_g128", pack_weight(Ws[e], "q4_g128", N, K), N, K, y1, N)], None, 0)
        assert_exact_path(got[p:p + 1], host(y1), nmse_max=1e-12, rel_max=1e-6, what=f"expert {e}")


@pytest.mark.parametrize("G,Ks", [(64, (64, 1024)), (128, (2048, 128)), (64, (1088, 64, 192))])
def test_routed_projections_of_different_inner_sizes(G, Ks):
    """K of one or two chunks beside a long one: the CTAs that share the long K have nothing of the short one,
    which comes first in every pass of some of them."""
    import torch
    rows, k, E, N = 64, 2, 4, 96
    rb = max(Ks) // 32
    img = image(11900, rows, rb * 32)
    ids = synth.rng(11901).integers(0, E, size=(rows, k), dtype=np.int32)
    p = plan(ids, E, rows)
    Ws = [[synth.q4_group_weight(11910 + 100 * j + e, N, K, G) for e in range(E)] for j, K in enumerate(Ks)]
    pw = [pack_experts(w, f"q4_g{G}", N, K) for w, K in zip(Ws, Ks)]
    ys = [out(rows * k, N) for _ in Ks]
    qk.qk_mmvq_id(dev(img.reshape(-1)), rb, rows, k,
                  [qk.make_proj_id(f"q4_g{G}", E, w, N, K, y) for w, K, y in zip(pw, Ks, ys)], *p)
    assert qk.qk_device_faults() == 0
    flat = ids.reshape(-1)
    for w, K, y in zip(Ws, Ks, ys):
        x = O.image_values(img, K)
        want = np.stack([x[i // k] @ O.dequant_group(w[e], N, K).T for i, e in enumerate(flat)])
        assert_exact_path(host(y), want, what=f"K={K}")


@pytest.mark.parametrize("G,T,K,Ns", [
    (64, 8, 256, (120000,)),             # short K: eight warps, items for every CTA several times over
    (128, 3, 2560, (20000, 19003, 33)),  # the longest of that form
    (64, 5, 2624, (40000,)),             # one chunk more: sixteen warps
    (128, 8, 9216, (25001, 15000)),      # the longest K whose fragments a CTA holds
    (64, 2, 9280, (20000,)),             # shared by two CTAs of sixteen warps
    (128, 4, 18944, (9000, 40)),         # by three
    (64, 3, 75776, (1000,)),             # by eight, with two pieces each
    (128, 3, 4352, (20000, 19003, 33)),
    (64, 5, 4416, (40000,)),
])
def test_matvec_with_many_rows(G, T, K, Ns):
    import torch
    img = image(12000 + K, T, K)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(12001)
    x = dev(O.image_values(img, K))
    projs, keep = [], []
    for N in Ns:
        w = torch.randint(0, 256, (N, K // G, 4 + G // 2), dtype=torch.uint8, device="cuda", generator=gen)
        d = (torch.rand((N, K // G, 1), device="cuda", generator=gen) * 0.02 + 0.001).half()
        w[..., 0:2] = d.view(torch.uint8)
        n = qk.qk_weight_packed_bytes(f"q4_g{G}", N, K)
        p = torch.empty((n,), dtype=torch.uint8, device="cuda")
        qk.qk_weight_pack(f"q4_g{G}", w, N, K, p, n)
        nib = w[..., 4:].reshape(N, K // G, G // 32, 16)
        v = torch.stack([nib & 15, nib >> 4], dim=3).reshape(N, K // G, G).double()
        W = ((v - (w[..., 2:3] & 15).double()) * d.double()).reshape(N, K)
        y = out(T, N)
        keep.append((p, x @ W.T, y))
        projs.append(qk.make_proj(f"q4_g{G}", p, N, K, y, N))
        del nib, v, W, w
    qk.qk_mmvq(dev(img.reshape(-1)), K // 32, T, projs, None, 0)
    assert qk.qk_device_faults() == 0
    for _, want, y in keep:
        assert_exact_path(host(y), host(want), what=f"{K} -> {y.shape[1]}")


@pytest.mark.parametrize("slots", [False, True])
def test_routed_with_long_rows_and_many_passes(slots):
    """K beyond the eight-warp form and items for every CTA several times over: the sixteen-warp routed form."""
    import torch
    rows, k, E, K, N, live = 300, 2, 5, 4608, 2400, 287
    img = image(12100, rows * k if slots else rows, K)
    ids = synth.rng(12101).integers(0, E, size=(rows, k), dtype=np.int32)
    Ws = [synth.q4_group_weight(12110 + e, N, K, 64) for e in range(E)]
    y = out(rows * k, N)
    pw = pack_experts(Ws, "q4_g64", N, K)
    call = qk.qk_mmvq_id_slots if slots else qk.qk_mmvq_id
    call(dev(img.reshape(-1)), K // 32, rows, k, [qk.make_proj_id("q4_g64", E, pw, N, K, y)], *plan(ids, E, live))
    assert qk.qk_device_faults() == 0
    x, flat, got = O.image_values(img, K), ids.reshape(-1), host(y)
    want = np.zeros((live * k, N))
    for e in range(E):
        p = np.nonzero(flat[:live * k] == e)[0]
        want[p] = x[p if slots else p // k] @ O.dequant_group(Ws[e], N, K).T
    assert_exact_path(got[:live * k], want)
    assert np.all(got[live * k:] == SENTINEL)


def test_static_workspace_call_takes_group_scaled_projections():
    T, N, K = 3, 200, 512
    img = image(12200, T, K)
    W = synth.q4_group_weight(12201, N, K, 128)
    y = out(T, N)
    qk.qk_mmvq_static_ws(dev(img.reshape(-1)), K // 32, T,
                         [qk.make_proj("q4_g128", pack_weight(W, "q4_g128", N, K), N, K, y, N)])
    assert_exact_path(host(y), ref(img, W, N, K))
