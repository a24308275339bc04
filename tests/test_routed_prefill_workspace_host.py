"""qk_mmq_id_workspace_bytes is 0 for arguments out of range, the projections' K among them."""
import pytest

from quantized_activation_q4_gb300 import binding as qk


@pytest.mark.parametrize("K", [-64, 0, 31, (1 << 31) - 128, 1 << 62, -(1 << 63)])
def test_workspace_of_an_inner_size_out_of_range(K):
    proj = lambda k: qk.qk_proj_id16(2, 4, 0x1000, 64, k, 0x2000, 64)
    assert qk.qk_mmq_id_workspace_bytes(4, 2, [proj(256)]) >= 4 * 2 * 256 * 2
    assert qk.qk_mmq_id_workspace_bytes(4, 2, [proj(K)]) == 0
    assert qk.qk_mmq_id_workspace_bytes(4, 2, [proj(256), proj(K)]) == 0
