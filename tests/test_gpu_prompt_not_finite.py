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


def batch_with_a_bad_sequence(d, window, sinks, where, n=9000):
    """Two prompts whose items are more than the SMs: the first one's values at `where` are not
    finite; and the same with zeros there."""
    cu = offsets([n, n])
    q, k, v = projection(2 * n, 16, 4, d)
    clean, v = v.clone(), v.clone()
    clean[where], v[where] = 0.0, float("nan")
    run = lambda x: attend(q, k, x, cu, None, window, sinks)
    return run, clean, v


def event_ms(call):
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    call()
    b.record()
    b.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (8192, 4), (2000, 300)])
def test_a_sequence_of_nan_costs_the_others_nothing(d, window, sinks):
    n = 9000
    run, clean, v = batch_with_a_bad_sequence(d, window, sinks, slice(0, n))
    ref, out = run(clean), run(v)
    assert kvq.kvq_get_device_error() == 0
    assert torch.equal(bits(out[n:]), bits(ref[n:]))
    assert torch.isnan(out[:n]).all()
    good, bad = (min(event_ms(lambda: run(x)) for _ in range(3)) for x in (clean, v))
    assert bad < 5 * good + 1, f"{bad:.2f} ms with NaN, {good:.2f} without"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_not_finite_at_both_ends_of_a_wide_window(d, value):
    """A kept key, one at a window's edge and one near the diagonal: the rows that see one of them
    get it in its element, everything else keeps its bits; and in reasonable time when all of a
    sequence's values are infinities of one sign, of which each row has to look at all."""
    n, window, sinks = 9000, 4096, 4
    run, clean, v = batch_with_a_bad_sequence(d, window, sinks, slice(0, 0))
    at = {1: 3, 2000: 17, 2050: d - 1, 6000: 40, 8999: 5}  # key: element
    for t, e in at.items():
        clean[t, 0, e], v[t, 0, e] = 0.0, value
    ref, out = run(clean), run(v)
    assert kvq.kvq_get_device_error() == 0
    p = torch.arange(n, device=DEV)
    want = ref.clone()
    for t, e in at.items():
        sees = (p >= t) & ((p < t + window) | (t < sinks))
        want[:n][sees, :4, e] = value
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(bits(out)[keep], bits(want)[keep])
    good = min(event_ms(lambda: run(clean)) for _ in range(3))
    v[:n] = value
    out = run(v)
    assert kvq.kvq_get_device_error() == 0
    assert torch.equal(bits(out[n:]), bits(ref[n:])) and not torch.isfinite(out[:n]).any()
    bad = min(event_ms(lambda: run(v)) for _ in range(3))
    assert bad < 30 * good + 1, f"{bad:.2f} ms, {good:.2f} with finite values"


@pytest.mark.parametrize("d,g", [(64, 1), (128, 4)])
@pytest.mark.parametrize("a,b,window,sinks", [(500, 1000, 700, 0), (1000, 500, 700, 0), (2, 900, 300, 4), (1200, 1210, 0, 0)])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinities_of_both_signs_make_nan(d, g, a, b, window, sinks, sign):
    """One in a tile that every row of an item sees, the other in one that only some see."""
    n, inf = 2000, sign * float("inf")
    q, k, v = projection(n, g, 1, d)
    clean, v = v.clone(), v.clone()
    clean[[a, b], 0, 3] = 0.0
    v[a, 0, 3], v[b, 0, 3] = -inf, inf
    cu = np.array([0, n])
    ref, out = (attend(q, k, x, cu, None, window, sinks) for x in (clean, v))
    p = torch.arange(n, device=DEV)
    sees = [(p >= t) & ((window == 0) | (p < t + window) | (t < sinks)) for t in (a, b)]
    want = ref.clone()
    want[sees[0], :, 3] = -inf
    want[sees[1], :, 3] = inf
    want[sees[0] & sees[1], :, 3] = float("nan")
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(bits(out)[keep], bits(want)[keep])
