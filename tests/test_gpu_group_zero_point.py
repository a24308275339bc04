"""GPU: the zero point of group-scaled weights against its documented arithmetic: exact block sums of nibble - 8 and of
the codes, binary32 from there on, with the error bound that follows, where the two parts cancel and at outliers."""
import numpy as np
import pytest

from oracle import oracle as O
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import dev, host, pack_experts, pack_weight

pytestmark = pytest.mark.gpu


def outlier_image(seed, T, K):
    """N(0, 1) rows with a one-signed block a thousand times larger in every row."""
    x = synth.activations(seed, T, K)
    for t in range(T):
        b = (5 * t + 3) % (K // 32)
        x[t, 32 * b:32 * b + 32] = 1000.0 + np.arange(32)
    return O.quantize_q8_1(x).reshape(T, -1)


def zero_groups(W, G, which):
    """In place: the groups where `which` is true get nibbles equal to their zero point."""
    z = W[:, :, 2] & 15
    W[:, :, 4:][which] = np.repeat((z * 17)[which][:, None], G // 2, axis=1)
    return W


def products(img, Ws, G, N, K):
    """Every row of `img` through every matrix of Ws: by the ordinary call and by the routed one."""
    import torch
    T, E, wt = img.shape[0], len(Ws), f"q4_g{G}"
    img_d = dev(img.reshape(-1))
    plain = []
    for W in Ws:
        y = torch.full((T, N), 7.0, device="cuda")
        qk.qk_mmvq(img_d, K // 32, T, [qk.make_proj(wt, pack_weight(W, wt, N, K), N, K, y, N)], None, 0)
        plain.append(host(y))
    ids = dev(np.tile(np.arange(E, dtype=np.int32), (T, 1)))
    i32 = lambda n: torch.zeros((n,), dtype=torch.int32, device="cuda")
    plan = i32(E), i32(E + 1), i32(T * E)
    qk.qk_moe_plan(ids, T, E, E, *plan)
    y = torch.full((T * E, N), 7.0, device="cuda")
    qk.qk_mmvq_id(img_d, K // 32, T, E, [qk.make_proj_id(wt, E, pack_experts(Ws, wt, N, K), N, K, y)], *plan)
    assert qk.qk_device_faults() == 0
    return np.stack(plain, axis=1), host(y).reshape(T, E, N)


def bound(img, W, G, N, K):
    """A block's two parts d_g d_a D_b and d_g d_a (z_g - 8) S_b are rounded in at most G / 32 sums of the group, three
    steps of the code sums, the group's difference, K / G sums of groups, 16 of warps and 8 of CTAs: each by 2^-24 of a
    partial sum that the parts' absolute values bound."""
    blocks = img.reshape(img.shape[0], -1, 36)
    q = blocks[:, :, 4:].view(np.int8).astype(np.float64)
    da = np.ascontiguousarray(blocks[:, :, 0:2]).view(np.float16)[..., 0].astype(np.float64)
    dg = np.ascontiguousarray(W[:, :, 0:2]).view(np.float16)[..., 0].astype(np.float64)
    z = (W[:, :, 2] & 15).astype(np.float64) - 8
    runs = W[:, :, 4:].reshape(N, K // 32, 16)
    c = np.concatenate([runs & 15, runs >> 4], axis=-1).astype(np.float64) - 8
    D = np.abs(np.einsum("tbi,nbi->tnb", q, c))
    S = np.abs(q.sum(-1))[:, None, :]
    per = lambda v: np.repeat(v, G // 32, axis=1)[None]          # of a group, for each of its blocks
    return 2.0 ** -24 * (K / G + G / 32 + 32) * (per(dg) * np.abs(da)[:, None] * (D + np.abs(per(z)) * S)).sum(-1)


@pytest.mark.parametrize("G", [64, 128])
@pytest.mark.parametrize("K", [128, 1024, 2688])
def test_weights_equal_to_their_zero_point(G, K):
    T, N, E = 8, 48, 3
    img = outlier_image(41 + K, T, K)
    Ws = [synth.q4_group_weight(42 + e, N, K, G) for e in range(E)]
    for e, W in enumerate(Ws):
        W[:, :, 2] = (np.arange(N)[:, None] + np.arange(K // G)[None] + e) % 16 if e else 8     # every zero point; 8 alone
        zero_groups(W, G, np.ones(W.shape[:2], dtype=bool))
    for y in products(img, Ws, G, N, K):
        assert np.all(y[:, 0] == 0.0)
        for e, W in enumerate(Ws):
            assert np.all(np.abs(y[:, e]) <= bound(img, W, G, N, K))


@pytest.mark.parametrize("G", [64, 128])
@pytest.mark.parametrize("K", [256, 2560, 4096, 9472])
def test_error_bound_where_the_parts_cancel(G, K):
    """Nibbles within one of their zero point, half the groups zero."""
    T, N, E = 8, 64, 2
    img = outlier_image(51 + K, T, K)
    g = synth.rng(52 + K + G)
    Ws = []
    for e in range(E):
        W = synth.q4_group_weight(53 + e, N, K, G)
        W[:, :, 2] = g.choice([0, 1, 14, 15], size=W.shape[:2])
        z = W[:, :, 2].astype(np.int64)[:, :, None]
        lo, hi = (np.clip(z + g.integers(-1, 2, size=(N, K // G, G // 2)), 0, 15) for _ in range(2))
        W[:, :, 4:] = (lo + 16 * hi).astype(np.uint8)
        Ws.append(zero_groups(W, G, g.random(W.shape[:2]) < 0.5))
    x = O.image_values(img, K)
    for y in products(img, Ws, G, N, K):
        for e, W in enumerate(Ws):
            assert np.all(np.abs(y[:, e] - x @ O.dequant_group(W, N, K).T) <= bound(img, W, G, N, K))
