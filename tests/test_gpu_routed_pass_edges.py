"""GPU: routed prefill products of experts whose pairs fill several passes and end in a ragged one."""
import numpy as np
import pytest

from tests.test_gpu_mmq_id import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [143, 641, 897, 1009, 1025, 1153, 2049])
def test_several_passes_of_one_expert(count):
    ids = np.zeros((count + 1, 1), dtype=np.int32)
    ids[count // 2, 0] = 1
    run("q4_g64", count + 1, 1, 2, 128, (129,), count + 1, False, ids=ids, seed=13300)
