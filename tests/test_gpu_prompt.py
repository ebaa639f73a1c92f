"""kvq_prompt_attention against float64."""
import time

import numpy as np
import pytest
import torch

from oracle import blocks as B
from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, bits, check_close, ints

pytestmark = pytest.mark.gpu


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)])


def projection(total, hq, hkv, d, seed=0, scale=1.0):
    """Queries, keys and values as slices of one projection."""
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn((total, (hq + 2 * hkv) * d), device=DEV, generator=g)
    x[:, :(hq + hkv) * d] *= scale
    x = x.to(torch.bfloat16)
    return tuple(x[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))


def expect(q, k, v, cu, sm, window=0, sinks=0):
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    out, tol = np.zeros(q.shape), np.full(q.shape, 1e-30)
    for a, b in zip(cu[:-1], cu[1:]):
        out[a:b], tol[a:b] = B.attention(q[a:b], k[a:b], v[a:b], sm, 0, window, sinks)
    return out, tol


def attend(q, k, v, cu, sm=None, window=0, sinks=0, out=None, max_len=None):
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    max_len = int(np.diff(cu).max(initial=0)) if max_len is None else max_len
    return kvq.kvq_prompt_attention(q, k, v, out, ints(cu), max_len, q.shape[-1] ** -0.5 if sm is None else sm, window, sinks)


def check(lens, hkv, g, d, window=0, sinks=0, seed=0, scale=1.0, sm=None):
    cu = offsets(lens)
    q, k, v = projection(int(cu[-1]), hkv * g, hkv, d, seed, scale)
    ref, tol = expect(q, k, v, cu, d ** -0.5 if sm is None else sm, window, sinks)
    check_close(attend(q, k, v, cu, sm, window, sinks), ref, tol)
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("hkv,g,d", [(2, 4, 128), (2, 3, 64), (1, 8, 128), (4, 1, 64), (3, 1, 128), (8, 4, 128)])
def test_ragged_batches(hkv, g, d):
    check([40, 130, 1, 300, 0, 129, 7], hkv, g, d)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385, 513])
def test_tile_edges(n):
    check([n], 1, 4, 128)
    check([n], 2, 8, 64)
    check([n], 1, 1, 64)


@pytest.mark.parametrize("g", range(1, 9))
def test_every_head_ratio(g):
    check([150, 261, 1], 2, g, 64)
    check([333], 1, g, 128)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 0), (64, 5), (128, 130), (129, 4), (200, 300), (5000, 9)])
def test_windows(window, sinks):
    check([300, 1, 33, 700], 2, 4, 128, window, sinks)
    check([500, 18], 2, 2, 64, window, sinks)
    check([600], 1, 1, 128, window, sinks)


def test_more_tiles_than_the_device_holds_at_once():
    check(np.random.default_rng(3).integers(1, 600, 40), 8, 4, 64)


@pytest.mark.parametrize("count", [128, 129, 641, 1500])
def test_many_sequences(count):
    """The order by length, and more sequences than a CTA has threads."""
    lens = np.random.default_rng(count).integers(0, 30, count)
    lens[count - 2] = 300
    check(lens, 1, 2, 64)
    check(lens[::-1].copy(), 2, 1, 64, 20, 3)


def test_a_long_prompt():
    check([3001], 1, 2, 128)
    check([2500], 1, 7, 64, 1000, 4)


@pytest.mark.parametrize("sm", [-0.125, 0.0, 1.0, -1.0])
def test_scales(sm):
    check([140, 300], 2, 4, 64, sm=sm)
    check([270], 1, 2, 128, 60, 3, sm=sm)


def test_large_logits():
    """Logits that span hundreds, and a new maximum in every tile."""
    check([400, 1000], 1, 4, 128, scale=5.0)
    n = 1100
    q = torch.ones((n, 2, 64), dtype=torch.bfloat16, device=DEV)
    v = projection(n, 1, 1, 64)[2]
    for slope in (8, -8):
        k = (torch.ones((n, 1, 64), device=DEV) * torch.linspace(-slope, slope, n, device=DEV)[:, None, None]).to(torch.bfloat16)
        for sm in (1.0, -1.0):
            ref, tol = expect(q, k, v, [0, n], sm)
            check_close(attend(q, k, v, np.array([0, n]), sm), ref, tol)


def test_strides_and_rows_outside_the_batch():
    """Contiguous and strided rows give the same bits; rows outside the offsets stay."""
    q, k, v = projection(333, 8, 2, 128)
    cu = np.array([3, 103, 103, 320])
    one = attend(q, k, v, cu)
    assert torch.equal(bits(attend(q.contiguous(), k.contiguous(), v.contiguous(), cu)), bits(one))
    wide = torch.full((333, 11, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(bits(attend(q, k, v, cu, out=wide[:, 2:10])), bits(one))
    assert (wide[:, :2] == 7).all() and (wide[:, 10:] == 7).all()
    assert (one[:3] == 7).all() and (one[320:] == 7).all()
    ref, tol = expect(q, k, v, cu, 128 ** -0.5)
    check_close(one[3:320], ref[3:320], tol[3:320])
    assert kvq.kvq_get_device_error() == 0


def test_rows_past_4_gib():
    """Tokens 32 MB apart: offsets of elements and bytes past 2^31 and 2^32."""
    q, k, v = projection(150, 4, 2, 64)
    cu = np.array([0, 100, 150])
    one = attend(q, k, v, cu)
    flat = torch.empty(150 << 24, dtype=torch.bfloat16, device=DEV)
    far = [torch.as_strided(flat, x.shape, (1 << 24, 64, 1), 1024 * i) for i, x in enumerate((q, k, v, q))]
    for x, y in zip(far, (q, k, v)):
        x.copy_(y)
    attend(*far[:3], cu, out=far[3])
    assert torch.equal(bits(far[3]), bits(one))
    # and written to and read back from a cache so
    cache = kvq.alloc_kv_cache("bf16", "bf16", 10, 16, 2, 64, device=DEV)
    slots = ints(np.arange(150), torch.int64)
    kvq.kvq_write_cache(cache, far[1], far[2], slots)
    outs = [torch.as_strided(flat, k.shape, (1 << 24, 64, 1), 8192 + 1024 * i) for i in range(2)]
    kvq.kvq_read_cache(cache, slots, *outs)
    assert torch.equal(bits(outs[0]), bits(k)) and torch.equal(bits(outs[1]), bits(v))
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_that_are_16_byte_aligned_only(d):
    """Rows that begin in the middle of a 32-byte sector, in either way, give the same bits."""
    q, k, v = projection(150, 4, 2, d)
    cu = np.array([0, 100, 150])
    one = attend(q, k, v, cu)
    for off, stride in ((8, 4 * d + 16), (0, 4 * d + 8), (8, 4 * d + 8)):
        flat = torch.full((160 * (4 * d + 16),), 7.0, dtype=torch.bfloat16, device=DEV)
        out = torch.as_strided(flat[off:], (150, 4, d), (stride, d, 1))
        attend(q, k, v, cu, out=out)
        assert torch.equal(bits(out), bits(one))
        out.fill_(7.0)
        assert (flat == 7).all()


def test_bad_offsets_are_flagged_and_cut():
    q, k, v = projection(30, 4, 2, 64)
    for cu, most in (([0, 40, 50], 30), ([0, 10, 5], 20), ([-4, 10, 20], 20), ([0, 20, 30], 12)):
        out = torch.full((40, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        attend(q, k, v, np.array(cu), out=out[:30], max_len=most)
        assert kvq.kvq_get_device_error() & kvq.DEVERR_TOKENS
        assert (out[30:] == 7).all()
    out = attend(q, k, v, np.array([0, 20, 30]), max_len=12)
    ref, tol = expect(q, k, v, [0, 12], 0.125)
    check_close(out[:12], ref[:12], tol[:12])
    assert (out[12:20] == 7).all() and kvq.kvq_get_device_error() == kvq.DEVERR_TOKENS


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 60, 128, 299])
def test_values_not_finite_reach_the_rows_that_see_them(d, at):
    q, k, v = projection(700, 4, 2, d)
    v = v.clone()
    v[at, 0, 5], v[at, 0, d - 3], v[at, 0, 9] = float("inf"), float("-inf"), float("nan")
    out = attend(q, k, v, np.array([0, 300, 700]))
    good = torch.isfinite(out)
    assert good[:at].all() and good[300:].all() and good[:, 2:].all()
    assert (out[at:300, :2, 5] == float("inf")).all() and (out[at:300, :2, d - 3] == float("-inf")).all()
    assert torch.isnan(out[at:300, :2, 9]).all()
    good[at:300, :2, [5, d - 3, 9]] = True
    assert good.all()


def test_nan_where_no_row_looks():
    """Between the kept tokens and the window, in other sequences and behind the last one."""
    q, k, v = projection(900, 8, 2, 64)
    k, v, q = k.clone(), v.clone(), q.clone()
    cu = np.array([10, 410, 850])
    ref, tol = expect(q, k, v, cu, 0.125)
    for x in (q, k, v):
        x[:10] = x[850:] = float("nan")
    check_close(attend(q, k, v, cu)[10:850], ref[10:850], tol[10:850])
    k[410:], v[410:] = float("nan"), float("nan")
    check_close(attend(q, k, v, cu)[10:410], ref[10:410], tol[10:410])
    # keys 20..149 of the second sequence: out of sight from position 250 on
    q, k, v = projection(600, 4, 1, 128)
    k, v = k.clone(), v.clone()
    k[20:150], v[20:150] = float("nan"), float("nan")
    out = attend(q, k, v, np.array([0, 600]), window=100, sinks=20)
    clean = np.nan_to_num(k.double().cpu().numpy()), np.nan_to_num(v.double().cpu().numpy())
    ref, tol = B.attention(q.double().cpu().numpy(), *clean, 128 ** -0.5, 0, 100, 20)
    check_close(out[:20], ref[:20], tol[:20])
    check_close(out[249:], ref[249:], tol[249:])
    assert torch.isnan(out[20:249]).all()


def test_queries_not_finite_stay_in_their_rows():
    q, k, v = projection(200, 4, 2, 64)
    q = q.clone()
    ref, tol = expect(q, k, v, [0, 200], 0.125)
    q[77, 1, 3], q[150, 3] = float("nan"), float("inf")
    out = attend(q, k, v, np.array([0, 200]))
    keep = np.ones((200, 4), bool)
    keep[77, 1] = keep[150, 3] = False
    assert not torch.isfinite(out[77, 1]).any()
    check_close(out[torch.from_numpy(keep).to(DEV)], ref[keep], tol[keep])


def test_repeats_streams_and_graphs():
    cu = np.array([0, 700, 750, 1400])
    q, k, v = projection(1400, 8, 2, 128)
    one = attend(q, k, v, cu)
    assert torch.equal(bits(attend(q, k, v, cu)), bits(one))  # no order of sums varies
    out, cut = torch.empty_like(one), ints(cu)
    call = lambda: kvq.kvq_prompt_attention(q, k, v, out, cut, 700, 128 ** -0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(bits(out), bits(one))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for i in range(3):
        for x, y in zip((q, k, v), projection(1400, 8, 2, 128, seed=30 + i)):
            x.copy_(y)
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(attend(q, k, v, cu)))


def test_two_calls_at_once():
    """Calls on two streams share nothing."""
    cu = np.array([0, 900, 1400])
    sets = [projection(1400, 8, 2, 128, seed=s) for s in (1, 2)]
    ref = [attend(*x, cu) for x in sets]
    streams, cut = [torch.cuda.Stream() for _ in sets], ints(cu)
    outs = [torch.empty_like(r) for r in ref]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, out in zip(streams, sets, outs):
            kvq.kvq_prompt_attention(*x, out, cut, 900, 128 ** -0.5, stream=s)
    torch.cuda.synchronize()
    for out, r in zip(outs, ref):
        assert torch.equal(bits(out), bits(r))


def test_nothing_to_do():
    q, k, v = projection(5, 4, 2, 64)
    out = attend(q, k, v, np.array([0]))
    assert (out == 7).all()
    out = attend(q, k, v, np.array([0, 0, 0]))
    assert (out == 7).all()
    assert attend(q[:0], k[:0], v[:0], np.array([0, 0])).numel() == 0
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("tile", [0, 1, 2, 5])
@pytest.mark.parametrize("lens,g,d", [([900] * 40, 4, 128), ([700], 8, 64)])
def test_a_wait_that_runs_out_ends_the_launch(lens, g, d, tile):
    """The products of one CTA wait for what nothing signals in place of a K tile."""
    cu = offsets(lens)
    q, k, v = projection(int(cu[-1]), 2 * g, 2, d)
    ref = attend(q, k, v, cu)
    assert kvq.kvq_get_device_error() == 0
    kvq.kvq_debug_arm_wait_timeout(1 << 12, 0, tile)
    t0 = time.perf_counter()
    attend(q, k, v, cu)
    found = kvq.kvq_get_device_error()  # synchronizes with the launch
    elapsed = time.perf_counter() - t0
    assert found & kvq.DEVERR_TIMEOUT, f"no timeout reported (bits {found})"
    assert elapsed < 5.0, f"the launch took {elapsed:.2f} s to give up"
    assert torch.equal(bits(attend(q, k, v, cu)), bits(ref))
    assert kvq.kvq_get_device_error() == 0
