"""The chunk attention's bounded pipeline waits, made to run out on purpose.

Every mbarrier wait of the kernel polls a bounded number of times; the first that runs
out raises KVQ_DEVERR_TIMEOUT and its CTA returns once no copy or product is in flight.
The test hook kvq_debug_arm_wait_timeout makes one CTA's products wait for what nothing
signals in place of a K tile (nothing faults): that wait runs out, the launch ends by itself, the error word says so, and the next launch on the same context gives
the same bits as before."""
import time

import numpy as np
import pytest
import torch

from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, Paged, bits, garbage, ints, random_query

pytestmark = pytest.mark.gpu

POLLS = 1 << 12
# sequences, keys, rows a sequence, query heads a kv-head: the form they take
SHAPES = {"64_rows": (40, 900, 3, 4), "128_rows": (40, 900, 30, 4), "256_rows": (24, 900, 100, 4), "parts": (1, 5000, 2, 8),
          "ahead": (3, 1100, 700, 8)}


@pytest.mark.parametrize("tile", [0, 1, 2, 5])
@pytest.mark.parametrize("shape,fmt", [("64_rows", "int8"), ("64_rows", "kvarn"), ("64_rows", "bf16"), ("128_rows", "uint8"),
                                       ("128_rows", "e5m2"), ("256_rows", "int8"), ("256_rows", "kvarn"),
                                       ("256_rows", "bf16"), ("parts", "int4"), ("ahead", "int8"), ("ahead", "kvarn")])
def test_a_wait_that_runs_out_ends_the_launch(shape, fmt, tile):
    seqs, n, rows, g = SHAPES[shape]
    if shape == "parts" and tile > 1:
        pytest.skip("a part has two tiles")
    p = Paged(fmt, [n] * seqs, 2, 64, 16)
    q = random_query(seqs * rows, 2 * g, 64)
    cu = ints(np.arange(seqs + 1) * rows)
    out = torch.empty_like(q)
    ws = garbage(kvq.kvq_prefill_workspace_size(p.cache, seqs, 2 * g, seqs * rows, rows, n))
    call = lambda: kvq.kvq_paged_prefill(p.cache, q, out, cu, p.block_table, p.context_lens, rows, n, 0.125, 0, 0, ws)
    call()
    assert kvq.kvq_get_device_error() == 0
    ref = out.clone()
    kvq.kvq_debug_arm_wait_timeout(POLLS, 0, tile)
    t0 = time.perf_counter()
    call()
    found = kvq.kvq_get_device_error()  # synchronizes with the launch
    elapsed = time.perf_counter() - t0
    assert found & kvq.DEVERR_TIMEOUT, f"no timeout reported (bits {found})"
    assert elapsed < 5.0, f"the launch took {elapsed:.2f} s to give up"
    out.fill_(7.0)
    call()  # the hook disarmed itself and the context is still usable
    assert kvq.kvq_get_device_error() == 0
    assert torch.equal(bits(out), bits(ref))
