"""GPU: a wait for other warps' partial sums that runs out in a group-scaled matvec sets bit 0 of the fault word, stops
the kernel's stores and lets it end: what is in the outputs is the right sum or what was there before."""
import os
import subprocess
import sys
import time

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SCRIPT = r"""
import sys
sys.path.insert(0, sys.argv[1])
import numpy as np, torch
from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from oracle import oracle as O
from tests.gpu_helpers import dev, host
out, seed = {}, 0

def weights(G, E, N, K):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    per = qk.qk_weight_packed_bytes(f"q4_g{G}", N, K)
    buf = torch.empty((E * per,), dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.randint(0, 256, (N, K // G, 4 + G // 2), dtype=torch.uint8, device="cuda", generator=gen)
        w[..., 0:2] = (torch.rand((N, K // G, 1), device="cuda", generator=gen) * 0.02 + 0.001).half().view(torch.uint8)
        qk.qk_weight_pack(f"q4_g{G}", w, N, K, buf[e * per:], per)
    return buf

image = lambda rows, K: dev(O.quantize_q8_1(synth.activations(K, rows, K)).reshape(-1))
# (group, N, K): eight warps with one item and with many a CTA, sixteen warps; the last in clusters (no such wait)
for G, N, K in ((64, 96, 256), (128, 60000, 1024), (64, 40000, 2688), (128, 64, 4096)):
    y = torch.full((5, N), -7.0, device="cuda")
    qk.qk_mmvq(image(5, K), K // 32, 5, [qk.make_proj(f"q4_g{G}", weights(G, 1, N, K), N, K, y, N)], None, 0)
    out[f"plain{N}"] = host(y)
    out[f"plain{N}_faults"] = qk.qk_device_faults()
for G, N, K, rows, k, E in ((64, 768, 2560, 16, 8, 32), (128, 2400, 4608, 40, 2, 5)):
    ids = dev(np.stack([synth.rng(r).permutation(E)[:k] for r in range(rows)]).astype(np.int32))
    plan = [torch.zeros((n,), dtype=torch.int32, device="cuda") for n in (E, E + 1, rows * k)]
    qk.qk_moe_plan(ids, rows, k, E, *plan)
    y = torch.full((rows * k, N), -7.0, device="cuda")
    qk.qk_mmvq_id(image(rows, K), K // 32, rows, k, [qk.make_proj_id(f"q4_g{G}", E, weights(G, E, N, K), N, K, y)], *plan)
    out[f"routed{N}"] = host(y)
    out[f"routed{N}_faults"] = qk.qk_device_faults()
np.savez(sys.argv[2], **out)
"""


def test_waits_that_run_out_leave_no_wrong_output(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    runs = {}
    for tries in (None, "1", "0"):   # 0: every wait runs out at once; 1: one look of 20 us at most
        env = dict(os.environ)
        env.pop("QK_MMVQ_G_WAIT_TRIES", None)
        if tries is not None:
            env["QK_MMVQ_G_WAIT_TRIES"] = tries
        path, t0 = str(tmp_path / f"y_{tries}.npz"), time.perf_counter()
        subprocess.run([sys.executable, "-c", SCRIPT, root, path], env=env, check=True, timeout=300)
        assert time.perf_counter() - t0 < 120
        runs[tries] = dict(np.load(path))
    for name, want in runs[None].items():
        if name.endswith("_faults"):
            assert want == 0
            assert runs["0"][name] == (0 if name == "plain64_faults" else 1), name
            continue
        assert np.all(want != -7.0) and np.all(np.isfinite(want)), name
        for tries in ("0", "1"):
            got = runs[tries][name]
            assert np.all((got == -7.0) | (got.view(np.uint32) == want.view(np.uint32))), (name, tries)
            if runs[tries][name + "_faults"] == 0:
                assert np.array_equal(got.view(np.uint32), want.view(np.uint32)), (name, tries)
        if name != "plain64":
            assert np.all(runs["0"][name] == -7.0), name
