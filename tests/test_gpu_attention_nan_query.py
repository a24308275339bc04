"""A NaN in a query row and head makes that row and head NaN, whatever the sinks, in rows, image and planes."""
import numpy as np
import pytest

from quantized_activation_q4_gb300 import binding as qk
from tests.kv_helpers import run_attention
from tests.test_gpu_attention import case, queries

pytestmark = pytest.mark.gpu

SHAPES = [(64, 1, 2, [40, 300, 0], 3), (128, 2, 4, [333, 70], 5), (256, 1, 3, [90, 200], 2)]


def inputs(D, Hkv, G, lens, n, kind):
    rng = np.random.default_rng(D + n)
    geo, pages, table = case(rng, D, Hkv, 32, lens)
    q = queries(rng, n * len(lens), Hkv * G, D, "f32")
    sink = {"none": None, "finite": rng.standard_normal(Hkv * G), "large": np.full(Hkv * G, 80.0),
            "minus infinity": np.full(Hkv * G, -np.inf)}[kind]
    return geo, pages, table, q, None if sink is None else sink.astype(np.float32)


@pytest.mark.parametrize("call", ["decode", "prefill"])
@pytest.mark.parametrize("kind", ["finite", "large", "minus infinity"])
@pytest.mark.parametrize("D,Hkv,G,lens,n", SHAPES)
def test_with_sinks(call, kind, D, Hkv, G, lens, n):
    geo, pages, table, q, sink = inputs(D, Hkv, G, lens, n, kind)
    run = lambda: run_attention(geo, pages, table, lens, q, [n] * len(lens), "f32", 0.1, 0, sink, "f32", False, call)[0]
    clean = run()
    assert np.isfinite(clean).all()
    at = [(0, Hkv * G - 1), (n - 1, 0), (n, 1)]
    for i, h in at:
        q[i, h, 33] = np.nan
    got = run()
    for i, h in at:
        assert np.isnan(got[i, h]).all()
        got[i, h] = clean[i, h]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("call", ["decode", "prefill"])
@pytest.mark.parametrize("kind", ["none", "finite"])
@pytest.mark.parametrize("long", [False, True])   # long: the prefill's keys are shared out and joined
@pytest.mark.parametrize("D,Hkv,G,lens,n", SHAPES)
def test_image_is_the_quantisers_of_a_nan_row(call, kind, long, D, Hkv, G, lens, n):
    """The image or planes alone (no rows wanted) are what the library's quantiser makes of the rows, NaN ones among them."""
    import torch
    lens = [x + 2100 if long and x else x for x in lens]
    geo, pages, table, q, sink = inputs(D, Hkv, G, lens, n, kind)
    q[0, 0, 5], q[n, 1, D - 1] = np.nan, np.nan
    run = lambda out_elem, image: run_attention(geo, pages, table, lens, q, [n] * len(lens), "f32", 0.1, 0, sink, out_elem,
                                                image, call, spare_blocks=1)
    out, _ = run("f32", False)
    assert np.isnan(out[0, 0]).all() and np.isnan(out[n, 1]).all()
    _, img = run(None, True)
    rows, K = out.shape[0], out.shape[1] * D
    blocks = K // 32 + 1
    x = torch.from_numpy(out.reshape(rows, K)).cuda()
    if call == "decode":
        want = torch.zeros((rows, blocks, 36), dtype=torch.uint8, device="cuda")
        qk.qk_quantize_q8_1(x, rows, K, K, want, blocks)
        torch.cuda.synchronize()
        assert np.array_equal(img, want.cpu().numpy())
    else:
        qs = torch.zeros((rows, blocks * 32), dtype=torch.int8, device="cuda")
        d = torch.zeros((rows, blocks), dtype=torch.int16, device="cuda")
        qk.qk_quantize_q8_0(x, rows, K, K, qs, d, blocks)
        torch.cuda.synchronize()
        assert np.array_equal(img[0], qs.cpu().numpy()) and np.array_equal(img[1], d.cpu().numpy().view(np.uint16))
        nan = np.isnan(img[1].view(np.float16))
        assert nan[0, :D // 32].all() and nan[n, D // 32:2 * D // 32].all() and nan.sum() == 2 * D // 32
