"""kvq_prompt_attention: what its waits count, and values that are not finite in batches whose
CTAs go on to other sequences."""
import numpy as np
import pytest
import torch

from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, bits, ints
from test_gpu_prompt import attend, offsets, projection

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_ordinary_waits_need_few_polls(d):
    """A poll sleeps for up to 3.7 us, so four of them cover what a tile or a first load takes; the
    issuing warp's, too."""
    cu = offsets([300, 200, 77])
    q, k, v = projection(int(cu[-1]), 8, 2, d)
    ref = attend(q, k, v, cu)
    assert kvq.kvq_get_device_error() == 0
    for _ in range(5):
        kvq.kvq_debug_arm_wait_timeout(4, 0, -1)
        out = attend(q, k, v, cu)
        assert kvq.kvq_get_device_error() == 0
        assert torch.equal(bits(out), bits(ref))
