"""The cache with a scale per (page, kv-head): store, decode, the decode step's own token."""
import numpy as np
import pytest
import torch

from oracle import blocks as B
from quantized_paged_kv_kvq_gb300 import kvq

from block_testing import PAIRS, Blocked
from step_testing import DEV, bits, check_close, garbage, ints, random_query

pytestmark = pytest.mark.gpu


# ---- store -------------------------------------------------------------------
@pytest.mark.parametrize("pair", sorted(PAIRS))
@pytest.mark.parametrize("hkv,d,bs", [(8, 128, 16), (2, 64, 8), (1, 128, 32), (3, 64, 64), (5, 128, 128), (16, 64, 16)])
def test_codes_and_scales_step_by_step(pair, hkv, d, bs):
    """Prompts, chunks and single tokens behind what is there: bit-equal after all of them."""
    p = Blocked(pair, [300, 1, 0, 130, 17, 128, 77], hkv, d, bs, seed=bs + d)
    p.fill()
    p.same()
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("pair", ["int8", "e4m3"])
@pytest.mark.parametrize("bs", [8, 16, 128])
def test_tokens_that_grow(pair, bs):
    """One token after another, each larger: the scale doubles, the codes in front shrink."""
    p = Blocked(pair, [bs + 3], 2, 64, bs, seed=5)
    for t in range(bs + 3):
        p.store(*p.rows(1, 1.4 ** t), p.slots(0, [t]))
        p.same()


@pytest.mark.parametrize("pair", ["int8", "e4m3"])
def test_rows_at_the_ends_of_the_range(pair):
    p = Blocked(pair, [64] * 5, 2, 64, 16)
    k, v = p.rows(64)
    zero = torch.zeros_like(k)
    p.store(zero[:5], zero[:5], p.slots(0, np.arange(5)))  # scale 0, then the first that is not
    p.store(k[:3], v[:3], p.slots(0, np.arange(5, 8)))
    for s, f in ((1, 1e-39), (2, 3e38), (3, 1e-30)):
        p.store((k[:16].float() * f).to(torch.bfloat16), (v[:16].float() * f).to(torch.bfloat16), p.slots(s, np.arange(16)))
    p.store((k[:2].float() * 1e30).to(torch.bfloat16), v[:2], p.slots(3, [16, 17]))
    p.store((k[:2].float() * 1e36).to(torch.bfloat16), v[:2], p.slots(3, [18, 19]))
    p.same()
    x = k.clone()
    x[0, 0, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    x[20] = float("nan")
    p.store(x[:40], x[:40], p.slots(4, np.arange(40)))  # not finite: not counted
    p.same()
    assert torch.isfinite(p.cache.k_meta[torch.from_numpy(p.table[4, :3]).to(DEV), :2]).all()


@pytest.mark.parametrize("bs", [8, 16, 64])
def test_slots_that_are_skipped_bad_or_out_of_order(bs):
    p = Blocked("int8", [90, 40], 4, 128, bs)
    slots = np.concatenate([p.slots(0, np.arange(90)), p.slots(1, np.arange(40))])
    slots[[0, 7, 100, 129]] = -1
    slots[50] = p.nb * bs
    slots[51] = 1 << 40
    k, v = p.rows(len(slots))
    p.store(k, v, slots)
    p.same()
    assert kvq.kvq_get_device_error() == kvq.DEVERR_SLOT_RANGE
    p = Blocked("e4m3", [bs], 2, 64, bs)  # any order within the page
    order = p.rng.permutation(bs)
    p.store(*p.rows(bs), p.slots(0, order))
    p.same()


def test_skipped_tokens_between_those_of_a_page():
    """Up to 31 in a row do not part a page's tokens, wherever they lie among the call's."""
    rng = np.random.default_rng(8)
    for bs in (8, 16, 128):
        p = Blocked("e4m3_int8", [400, 130, 64], 2, 64, bs)
        slots = []
        for s, n in enumerate(p.lens):
            for t in range(n):
                slots += [-1] * int(rng.choice((0, 0, 0, 1, 5, 31))) + [int(p.slots(s, [t])[0])]
        slots += [-1] * 500
        p.store(*p.rows(len(slots), np.exp(rng.standard_normal((2, len(slots), 1, 1)))), np.array(slots))
        p.same()


@pytest.mark.parametrize("bs,front", [(16, 0), (32, 5), (64, 0), (128, 0), (128, 37)])
def test_one_jump_among_offsets_in_a_row(bs, front):
    """Two neighbours swapped, or one left out, anywhere in the page; the rest in order."""
    p = Blocked("e4m3_int8", [bs] * (2 * bs), 1, 64, bs)
    for s in range(2 * bs):  # where the pages begin within the call moves by `front`
        at = np.arange(front, bs)
        if s % 2:
            at = np.delete(at, (s // 2) % len(at))
        else:
            i = (s // 2) % (len(at) - 1)
            at[[i, i + 1]] = at[[i + 1, i]]
        slots = np.concatenate([np.full(s % 3, -1), p.slots(s, at), p.slots((s + 1) % (2 * bs), [0])]) if s % 4 == 3 else p.slots(s, at)
        if front:
            p.store(*p.rows(front), p.slots(s, np.arange(front)))
        p.store(*p.rows(len(slots)), slots)
    p.same()
    assert kvq.kvq_get_device_error() == 0


def test_a_slot_named_twice_spoils_no_other_row():
    p = Blocked("int8", [16], 2, 64, 16)
    k, v = p.rows(40)
    pos = np.concatenate([np.arange(16), np.full(24, 9)])  # a run longer than its page
    kvq.kvq_write_cache(p.cache, k, v, ints(p.slots(0, pos), torch.int64))
    p.record(k, v, p.slots(0, pos))
    page, keep = p.table[0, 0], np.arange(16) != 9
    assert np.array_equal(p.cache.k_cache.cpu().numpy()[page, keep], p.kc[page, keep])
    assert np.array_equal(p.cache.k_meta.cpu().numpy()[page, :2], p.ks[page, :2])


def test_strided_rows_and_an_empty_call():
    p, q = Blocked("e4m3_int8", [70], 8, 128, 16), Blocked("e4m3_int8", [70], 8, 128, 16)
    wide = torch.randn((70, 20, 128), device=DEV).to(torch.bfloat16)
    p.store(wide[:, :8], wide[:, 12:], p.slots(0, np.arange(70)))
    p.same()
    kvq.kvq_write_cache(q.cache, wide[:0, :8], wide[:0, 12:], ints([], torch.int64))
    q.same()


def test_many_tokens():
    """More runs than CTAs at once, and windows of tokens that end inside a page."""
    for bs, n in ((16, 9001), (128, 5003), (8, 3001)):
        p = Blocked("e4m3", [n, 3, n // 2], 8, 64, bs)
        slots = np.concatenate([p.slots(s, np.arange(m)) for s, m in enumerate(p.lens)])
        p.store(*p.rows(len(slots), np.exp(p.rng.standard_normal((2, len(slots), 8, 1)))), slots)
        p.same()


def test_pools_past_4_gib():
    """Slots whose bytes lie past 2^32."""
    nb, bs, hkv, d = (1 << 32) // (16 * 8 * 128) + 100, 16, 8, 128
    cache = kvq.alloc_kv_cache("int8_block", "int8_block", nb, bs, hkv, d, device=DEV)
    g = torch.Generator(DEV).manual_seed(1)
    k, v = torch.randn((2, 40, hkv, d), device=DEV, generator=g).to(torch.bfloat16)
    slots = ints((nb - 3) * bs + np.arange(40), torch.int64)
    kvq.kvq_write_cache(cache, k, v, slots)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    kvq.kvq_read_cache(cache, slots, ko, vo)
    step = k.float().abs().amax() / 127
    assert (ko.float() - k.float()).abs().max() <= 0.5 * step + 2.0 ** -8 * k.float().abs().max()
    table, lens = ints(np.arange(nb - 3, nb)[None]), ints([40])
    q = random_query(1, 32, d)
    out = torch.empty_like(q)
    ws = garbage(kvq.kvq_decode_workspace_size(cache, 1, 32, 40))
    kvq.kvq_paged_decode(cache, q, out, table, lens, 40, d ** -0.5, ws)
    logit = torch.einsum("hgd,thd->hgt", q[0].float().view(hkv, 4, d), ko.float()) * d ** -0.5
    ref = torch.einsum("hgt,thd->hgd", torch.softmax(logit, -1), vo.float()).view(32, d)
    assert (out[0].float() - ref).abs().max() < 2e-2
    assert kvq.kvq_get_device_error() == 0


# ---- decode -------------------------------------------------------------------
def check_decode(p, g, window=0, sinks=0, num_ctas=0, sm=None):
    s = len(p.lens)
    q = random_query(s, p.hkv * g, p.d)
    ref, tol = p.expect(q, np.arange(s + 1), p.d ** -0.5 if sm is None else sm, window, sinks)
    check_close(p.decode(q, None, window, sinks, num_ctas, sm), ref, tol)
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("pair", sorted(PAIRS))
@pytest.mark.parametrize("hkv,g,d,bs", [(8, 4, 128, 16), (2, 4, 64, 8), (1, 8, 128, 32), (3, 3, 64, 64), (5, 1, 128, 128),
                                        (16, 2, 64, 16), (4, 7, 128, 8)])
def test_decode(pair, hkv, g, d, bs):
    p = Blocked(pair, [300, 1, 0, 130, 17, 128, 8, 9], hkv, d, bs, seed=3)
    p.fill()
    for num_ctas in (0, 1, 7):
        check_decode(p, g, num_ctas=num_ctas)


@pytest.mark.parametrize("bs", [8, 16, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (17, 0), (100, 20), (128, 130), (5000, 4)])
def test_decode_through_a_window(bs, window, sinks):
    p = Blocked("e4m3_int8", [300, 1, 0, 130, 257], 2, 128, bs)
    p.fill()
    for s, n in enumerate(p.lens):  # pages out of sight are gone
        for page in range(-(-int(n) // bs)):
            t = np.arange(page * bs, min((page + 1) * bs, n))
            if not ((t >= n - window) | (t < sinks)).any():
                p.table[s, page] = 999999
    p.block_table = ints(p.table)
    check_decode(p, 4, window, sinks)
    check_decode(p, 4, window, sinks, num_ctas=5)


def test_decode_of_a_long_context():
    """Over more than 32 ranges (merged in two levels), and 300 sequences."""
    p = Blocked("int8", [9000, 1200], 2, 128, 16)
    p.fill()
    check_decode(p, 4, num_ctas=64)
    check_decode(p, 4)
    p = Blocked("e4m3", np.random.default_rng(0).integers(0, 60, 300), 2, 64, 32)
    p.fill()
    check_decode(p, 2)


@pytest.mark.parametrize("f", [1e-30, 1e-20, 1e-6, 1e5, 1e15, 1e30])
@pytest.mark.parametrize("bs", [8, 16])
def test_values_of_any_size(f, bs):
    """Page scales far outside fp16's range, the whole cache's and one page's beside others."""
    p = Blocked("int8", [100, 100], 2, 64, bs)
    p.fill()
    k, v = p.rows(100)
    v = (v.float() * f).to(torch.bfloat16)
    p.store(k, v, p.slots(0, np.arange(100)))
    p.store(k[:bs], v[:bs], p.slots(1, np.arange(bs)))
    q = random_query(2, 8, 64)
    ref, tol = p.expect(q, [0, 1, 2], 0.125)
    got = p.decode(q).double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()


def test_light_keys_count_beside_one_that_dominates():
    """Thousands of keys of 2^-20 of the largest probability, small values beside a large page."""
    n, d = 8192, 64
    p = Blocked("int8", [n], 1, d, 16)
    q = torch.ones((1, 1, d), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((n, 1, d), device=DEV)
    k[0] = 20 * np.log(2) / (d * 0.125)
    v = torch.ones((n, 1, d), device=DEV)
    v[0] = 0.0
    p.store(k.to(torch.bfloat16), v.to(torch.bfloat16), p.slots(0, np.arange(n)))
    ref, tol = p.expect(q, [0, 1], 0.125)
    assert ref.min() > 1e-3
    check_close(p.decode(q), ref, np.maximum(tol, 2.0 ** -8 * np.abs(ref)))


def test_bad_pages_are_flagged():
    p = Blocked("int8", [100], 2, 64, 16)
    p.fill()
    p.block_table[0, 2] = -1
    p.block_table[0, 3] = p.nb
    q = random_query(1, 4, 64)
    p.cache.k_meta.nan_to_num_(1.0)
    p.cache.v_meta.nan_to_num_(1.0)
    p.decode(q)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_BLOCK_RANGE


def test_static_scratch_graphs_and_repeats():
    p = Blocked("e4m3", [700, 33, 1500], 8, 128, 16)
    p.fill()
    q = random_query(3, 32, 128)
    one = p.decode(q, num_ctas=16)
    assert torch.equal(bits(p.decode(q, num_ctas=16)), bits(one))
    out = torch.full_like(q, 7.0)
    kvq.kvq_paged_decode_static(p.cache, q, out, p.block_table, p.context_lens, p.max_len, 128 ** -0.5, 16)
    assert torch.equal(bits(out), bits(one))
    ws = garbage(kvq.kvq_decode_workspace_size(p.cache, 3, 32, p.max_len, 16))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kvq.kvq_paged_decode(p.cache, q, out, p.block_table, p.context_lens, p.max_len, 128 ** -0.5, ws, 16)
    for i in range(3):
        q.copy_(random_query(3, 32, 128, seed=50 + i))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(p.decode(q, num_ctas=16)))


# ---- the decode step's own token -------------------------------------------------
@pytest.mark.parametrize("pair", sorted(PAIRS))
@pytest.mark.parametrize("hkv,g,d,bs", [(8, 4, 128, 16), (2, 4, 64, 8), (1, 8, 128, 128), (3, 1, 64, 32)])
@pytest.mark.parametrize("window", [0, 50])
def test_append(pair, hkv, g, d, bs, window):
    """Codes and scales bit-equal to the oracle's store, the output to a store and a decode."""
    lens = np.array([300, 1, 0, 130, 16, 128, 8, 9])
    p = Blocked(pair, lens, hkv, d, bs)
    p.lens = np.maximum(lens - 1, 0)
    p.fill()
    p.lens = lens
    k, v = p.rows(8, np.exp(p.rng.standard_normal((2, 8, 1, 1)) * 2))  # some make their page's scale grow
    q = random_query(8, hkv * g, d)
    out = p.decode(q, None, window, 4, new=(k, v))
    at = np.array([p.slots(s, [n - 1])[0] if n else -1 for s, n in enumerate(lens)])
    p.record(k, v, at)
    p.same()
    assert torch.equal(bits(out), bits(p.decode(q, None, window, 4)))
    ref, tol = p.expect(q, np.arange(9), d ** -0.5, window, 4 if window else 0)
    check_close(out, ref, tol)
    assert kvq.kvq_get_device_error() == 0


def test_append_with_a_bad_page_writes_nothing():
    p = Blocked("int8", [20, 20], 2, 64, 16)
    p.fill()
    p.cache.k_meta.nan_to_num_(1.0)
    p.cache.v_meta.nan_to_num_(1.0)
    before = [x.clone() for x in (p.cache.k_cache, p.cache.v_cache, p.cache.k_meta, p.cache.v_meta)]
    p.block_table[0, 1] = p.nb
    p.block_table[1, 1] = -3
    p.decode(random_query(2, 4, 64), new=p.rows(2))
    assert kvq.kvq_get_device_error() == kvq.DEVERR_BLOCK_RANGE
    for x, y in zip(before, (p.cache.k_cache, p.cache.v_cache, p.cache.k_meta, p.cache.v_meta)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_a_captured_step_grows_its_pages_at_every_replay():
    p = Blocked("int8", [25, 40], 2, 64, 16)
    p.fill()
    k, v = p.rows(2)
    q, out = random_query(2, 4, 64), torch.empty((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    ws = garbage(kvq.kvq_decode_workspace_size(p.cache, 2, 4, p.max_len))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kvq.kvq_decode_append(p.cache, k, v, q, out, p.block_table, p.context_lens, p.max_len, 0.125, ws)
    at = np.array([p.slots(s, [n - 1])[0] for s, n in enumerate(p.lens)])
    for i in range(4):
        for x, y in zip((k, v), p.rows(2, 3.0 ** i)):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        p.record(k, v, at)
        p.same()
        ref, tol = p.expect(q, [0, 1, 2], 0.125)
        # the element bound alone: new values of size 27 put |out| at some units, whose rounding
        # to bf16 is off by |out| 2^-10 on average (a quarter step), past a mean of 2e-3
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


# ---- chunk attention -------------------------------------------------------------
def check_chunks(p, counts, g, window=0, sinks=0):
    cu = np.concatenate([[0], np.cumsum(counts)])
    q = random_query(int(cu[-1]), p.hkv * g, p.d)
    ref, tol = p.expect(q, cu, p.d ** -0.5, window, sinks, key=2.0 ** -11)
    most = int(np.max(counts, initial=0))
    ws = garbage(kvq.kvq_prefill_workspace_size(p.cache, len(p.lens), q.shape[1], q.shape[0], most, p.max_len))
    out = torch.full_like(q, 7.0)
    kvq.kvq_paged_prefill(p.cache, q, out, ints(cu), p.block_table, p.context_lens, most, p.max_len, p.d ** -0.5, window, sinks, ws)
    check_close(out, ref, tol)
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("pair", sorted(PAIRS))
@pytest.mark.parametrize("hkv,g,d,bs", [(2, 4, 128, 16), (2, 3, 64, 8), (1, 8, 128, 128), (5, 1, 64, 32), (3, 2, 64, 64)])
def test_chunks(pair, hkv, g, d, bs):
    """Prompts from nothing, chunks behind cached tokens, single tokens, no tokens."""
    p = Blocked(pair, [40, 130, 1, 300, 200, 0, 129], hkv, d, bs)
    p.fill()
    check_chunks(p, [40, 7, 1, 1, 70, 0, 128], g)
    check_chunks(p, [40, 7, 1, 9, 70, 0, 12], g, 50, 20)


@pytest.mark.parametrize("pair", ["int8", "e4m3"])
def test_chunks_dequantized_ahead_and_keys_in_parts(pair):
    p = Blocked(pair, [620, 700], 2, 128, 16)
    p.fill()
    check_chunks(p, [600, 500], 4)
    check_chunks(p, [600, 500], 8, 100, 20)
    p = Blocked(pair, [3000], 1, 64, 8)
    p.fill()
    check_chunks(p, [3], 8)


def test_chunks_with_values_that_are_not_finite():
    """A NaN value, an infinite scale: the rows that see them and no others."""
    for rows in (100, 600):  # dequantized by each CTA, and ahead
        p = Blocked("e4m3", [rows], 2, 64, 8)
        p.fill()
        blk, off = p.table[0, 60 // 8], 60 % 8
        p.cache.v_cache[blk, off, 0, 9] = 0x7F
        p.cache.v_meta[p.table[0, 80 // 8], 1] = float("inf")
        cu = ints([0, rows])
        q, out = random_query(rows, 4, 64), torch.empty((rows, 4, 64), dtype=torch.bfloat16, device=DEV)
        ws = garbage(kvq.kvq_prefill_workspace_size(p.cache, 1, 4, rows, rows, rows))
        kvq.kvq_paged_prefill(p.cache, q, out, cu, p.block_table, p.context_lens, rows, rows, 0.125, 0, 0, ws)
        good = torch.isfinite(out)
        assert good[:60].all() and good[60:, :2, :9].all() and good[60:, :2, 10:].all() and not good[60:, :2, 9].any()
        assert good[:80, 2:].all() and not good[88:, 2:].any(-1).any()


# ---- the operators together ------------------------------------------------------
@pytest.mark.parametrize("pair,bs", [("e4m3", 16), ("int8", 32)])
def test_a_serving_loop(pair, bs):
    """Prompts attend in 16 bits while they are stored; further chunks and single tokens attend to
    the pages; what was stored is read back.  Nothing comes back to the host in between."""
    hq, hkv, d, nb = 8, 2, 64, 60
    p = Blocked(pair, [0, 0, 0], hkv, d, bs)
    p.nb, p.cache = nb, kvq.alloc_kv_cache(p.k_fmt, p.v_fmt, nb, bs, hkv, d, device=DEV, fill=0xFF)
    p.kc, p.vc = (np.full((nb, bs, hkv, d), 0xFF, np.uint8) for _ in range(2))
    p.ks, p.vs = (np.full((nb, 4), 0xFFFFFFFF, np.uint32).view(np.float32) for _ in range(2))
    rope_table = torch.empty((512, d // 2, 2), device=DEV)
    kvq.kvq_rope_table(rope_table, 10000.0)
    rope = kvq.Rope(rope_table)
    lens, rng = ints([0, 0, 0]), ints([0, nb])
    table, free = torch.full((3, 20), -1, dtype=torch.int32, device=DEV), ints(np.random.default_rng(0).permutation(nb))
    new_lens, total = torch.empty(3, dtype=torch.int32, device=DEV), 0
    for step, new in enumerate(([130, 7, 64], [1, 40, 0], [1, 1, 1], [1, 1, 1], [3, 0, 200])):
        n = sum(new) + 5
        new_lens.copy_(ints(new))
        slots, pos = torch.empty(n, dtype=torch.int64, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV)
        after, cu, rest = torch.empty_like(lens), torch.empty(4, dtype=torch.int32, device=DEV), torch.empty_like(rng)
        kvq.kvq_plan_step(lens, new_lens, table, free, rng, bs, nb, slots, pos, after, cu, rest)
        qkv = random_query(n, hq + 2 * hkv, d, seed=step)
        qkv = (qkv.float() * 1.5 ** step).to(torch.bfloat16)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        kvq.kvq_norm_rope(rope, q, k, pos, q, k)
        out = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        query = q.contiguous()
        if step == 0:
            kvq.kvq_prompt_attention(q, k, v, out, cu, 130, d ** -0.5)
            kvq.kvq_write_cache(p.cache, k, v, slots)
        elif max(new) == 1:
            ws = garbage(kvq.kvq_decode_workspace_size(p.cache, 3, hq, 320))
            kvq.kvq_decode_append(p.cache, k[:3], v[:3], query[:3], out[:3], table, after, 320, d ** -0.5, ws)
        else:
            kvq.kvq_write_cache(p.cache, k, v, slots)
            ws = garbage(kvq.kvq_prefill_workspace_size(p.cache, 3, hq, n, max(new), 320))
            kvq.kvq_paged_prefill(p.cache, query, out, cu, table, after, max(new), 320, d ** -0.5, 0, 0, ws)
        lens, rng = after, rest
        # the oracle, from the same rotated rows
        p.table, p.lens, at = table.cpu().numpy(), after.cpu().numpy(), cu.tolist()
        p.record(k, v, slots.cpu().numpy())
        p.same()
        if step == 0:
            for s in range(3):
                a, b = at[s], at[s + 1]
                ref, tol = B.attention(*(x[a:b].double().cpu().numpy() for x in (query, k, v)), d ** -0.5)
                assert (np.abs(out[a:b].double().cpu().numpy() - ref) <= tol).all()
        else:
            ref, tol = p.expect(query, at, d ** -0.5, key=2.0 ** -11)
            assert (np.abs(out.double().cpu().numpy() - ref) <= tol)[:at[-1]].all()
        assert (out[at[-1]:] == 7).all()
    assert kvq.kvq_get_device_error() == 0
    for s in range(3):
        n = int(p.lens[s])
        ko, vo = (torch.empty((n, hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kvq.kvq_read_cache(p.cache, ints(p.slots(s, np.arange(n)), torch.int64), ko, vo)
        for got, want in zip((ko, vo), p.sequence(s, n)):
            assert (np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) + 1e-30).all()
