"""kvq_decode_window against the oracle: windows and kept tokens at every edge."""
import numpy as np
import pytest
import torch

from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, FORMATS, Paged, bits, check_close, garbage, random_query

pytestmark = pytest.mark.gpu


def decode(p, q, window, sinks, num_ctas=0, **kw):
    out = torch.full_like(q, 7.0)
    ws = garbage(kvq.kvq_decode_workspace_size(p.cache, len(p.lens), q.shape[1], p.max_len, num_ctas))
    return kvq.kvq_decode_window(p.cache, q, out, p.block_table, p.context_lens, p.max_len, p.d ** -0.5, window,
                                 sinks, ws, num_ctas, **kw)


def seen(p, window, sinks):
    return lambda s, t: t >= p[s] - window or t < sinks


LENS = [0, 1, 5, 16, 17, 33, 64, 100, 257, 400]


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("bs,hkv,g,d", [(16, 2, 4, 64), (8, 2, 3, 128), (64, 8, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (20, 4), (33, 17), (100, 40), (1000, 4), (3, 500)])
def test_against_the_oracle(fmt, bs, hkv, g, d, window, sinks):
    # pages out of view are gone from the block table, and what is not written is NaN
    p = Paged(fmt, LENS, hkv, d, bs, seed=window, keep=seen(LENS, window, sinks))
    q = random_query(len(LENS), hkv * g, d)
    ref, tol = p.expect(q, np.arange(len(LENS) + 1), p.d ** -0.5, window, sinks)
    for ctas in (0, 1, 5):
        check_close(decode(p, q, window, sinks, ctas), ref, tol, f"{ctas} ctas")
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "kvarn", "bf16"])
def test_a_wide_window_is_the_decode(fmt):
    p = Paged(fmt, [300, 17, 0, 512], 4, 128, 16)
    q = random_query(4, 16, 128)
    out = torch.empty_like(q)
    kvq.kvq_paged_decode(p.cache, q, out, p.block_table, p.context_lens, p.max_len, p.d ** -0.5, garbage(1 << 22), 6)
    assert torch.equal(bits(decode(p, q, 512, 0, 6)), bits(out))
    assert torch.equal(bits(decode(p, q, 1 << 30, 1 << 30, 6)), bits(out))


@pytest.mark.parametrize("fmt", ["e5m2", "bf16", "uint8"])
def test_nan_out_of_view(fmt):
    """NaN codes and fields at positions that the window leaves out of a page that is read."""
    p = Paged(fmt, [200], 2, 64, 128)
    for t in list(range(3, 90)):
        blk = p.table[0, t // 128]
        p.cache.k_cache[blk, t % 128] = 0xFF
        p.cache.v_cache[blk, t % 128] = 0xFF
        if p.cache.k_meta is not None:
            for m in (p.cache.k_meta, p.cache.v_meta):
                m[blk, :, :, t % 128] = float("nan")
    q = random_query(1, 4, 64)
    ref, tol = p.expect(q, [0, 1], 0.125, 110, 3)
    check_close(decode(p, q, 110, 3, 4), ref, tol)


@pytest.mark.parametrize("fmt", ["int8", "int4", "kvarn"])
def test_append_through_a_window(fmt):
    """The new token's row is stored as kvq_decode_append stores it, then seen."""
    lens = [1, 16, 17, 90, 0, 300]
    p, r = Paged(fmt, lens, 2, 128, 16), Paged(fmt, lens, 2, 128, 16)
    q = random_query(len(lens), 8, 128)
    g = torch.Generator(DEV).manual_seed(4)
    nk, nv = torch.randn((2, len(lens), 2, 128), device=DEV, generator=g).to(torch.bfloat16)
    kvq.kvq_decode_append(r.cache, nk, nv, q, torch.empty_like(q), r.block_table, r.context_lens, r.max_len, 0.1, garbage(1 << 22), 3)
    out = decode(p, q, 20, 2, 3, new_key=nk, new_value=nv)
    assert torch.equal(p.cache.k_cache, r.cache.k_cache) and torch.equal(p.cache.v_cache, r.cache.v_cache)
    ref, tol = p.expect(q, np.arange(len(lens) + 1), p.d ** -0.5, 20, 2)
    check_close(out, ref, tol)
    assert kvq.kvq_get_device_error() == 0


def test_long_context_and_many_sequences():
    p = Paged("int8", [20000, 3, 9000], 1, 64, 32, keep=seen([20000, 3, 9000], 3000, 100))
    q = random_query(3, 8, 64)
    ref, tol = p.expect(q, [0, 1, 2, 3], 0.125, 3000, 100)
    check_close(decode(p, q, 3000, 100), ref, tol)
    lens = np.random.default_rng(2).integers(0, 60, 300)
    p = Paged("e5m2", lens, 2, 64, 16)
    q = random_query(300, 2, 64)
    ref, tol = p.expect(q, np.arange(301), 0.125, 11, 3)
    check_close(decode(p, q, 11, 3), ref, tol)


def test_replayed_from_a_graph():
    p = Paged("int8", [700, 40], 2, 128, 16)
    q = random_query(2, 8, 128)
    out, ws = torch.empty_like(q), garbage(1 << 22)
    call = lambda o, w: kvq.kvq_decode_window(p.cache, q, o, p.block_table, p.context_lens, p.max_len, 0.1, 300, 4, w, 7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(out, ws)
    for i in range(3):
        q.copy_(random_query(2, 8, 128, seed=20 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(call(torch.empty_like(q), garbage(1 << 22))))
