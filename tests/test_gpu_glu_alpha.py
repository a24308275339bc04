"""GPU: SwiGLU-OAI's Q8_0 producer at the ends of alpha's range (any finite value), against the Q8_1 producer."""
import numpy as np
import pytest

from quantized_activation_q4_gb300 import binding as qk
from quantized_activation_q4_gb300 import synth
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("alpha", [3.4e38, -3.4e38, 2.4e38, 1.0, 0.0, 1e-30])
def test_gates_of_zero_and_alpha_at_its_ends(alpha):
    import torch
    T, N = 3, 64
    g = synth.activations(401, T, N)
    g[:, ::4] = 0.0
    g[1, ::8] = -0.0
    g[2] = 0.0
    u = synth.activations(402, T, N)
    outs = []
    for q8_0 in (True, False):
        out = torch.full((T, N), float("nan"), device="cuda")
        qs, d = torch.zeros((T, N), dtype=torch.int8, device="cuda"), torch.zeros((T, N // 32), dtype=torch.int16, device="cuda")
        img = torch.zeros((T * N // 32 * 36,), dtype=torch.uint8, device="cuda")
        if q8_0:
            qk.qk_glu_q8_0("swiglu_oai", "separate", "f32", dev(g), N, dev(u), N, T, N, out, N, qs, d, N // 32, alpha, 7.0)
        else:
            qk.qk_glu_q8_1_ex("swiglu_oai", "separate", dev(g), N, dev(u), N, T, N, out, N, img, N // 32, alpha, 7.0)
        outs.append(host(out).astype(np.float64))
    assert np.all(np.isfinite(outs[0])) and np.all(outs[0][g == 0] == 0)
    # either is within 3e-7 |g| (|u| + 1) of the definition
    assert np.all(np.abs(outs[0] - outs[1]) <= 6e-7 * np.abs(g) * (np.abs(u) + 1))
