"""kvq_paged_prefill against the oracle."""
import numpy as np
import pytest
import torch

from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, FORMATS, Paged, bits, check_close, garbage, ints, random_query

pytestmark = pytest.mark.gpu


def prefill(p, q, cu, window=0, sinks=0, sm=None, max_q=None, out=None):
    out = torch.full_like(q, 7.0) if out is None else out
    counts = np.diff(cu)
    max_q = int(counts.max(initial=0)) if max_q is None else max_q
    ws = garbage(kvq.kvq_prefill_workspace_size(p.cache, len(p.lens), q.shape[1], q.shape[0], max_q, p.max_len))
    return kvq.kvq_paged_prefill(p.cache, q, out, ints(cu), p.block_table, p.context_lens, max_q, p.max_len,
                                 p.d ** -0.5 if sm is None else sm, window, sinks, ws)


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)])


def check(fmt, lens, counts, hkv, g, d, bs, window=0, sinks=0, **kw):
    lens, counts = np.asarray(lens), np.asarray(counts)
    keep = None
    if window:
        keep = lambda s, t: counts[s] > 0 and (t > lens[s] - counts[s] - window or t < sinks)
    p = Paged(fmt, lens, hkv, d, bs, seed=d + bs, keep=keep, **kw)
    cu = offsets(counts)
    q = random_query(int(cu[-1]), hkv * g, d)
    ref, tol = p.expect(q, cu, d ** -0.5, window, sinks)
    check_close(prefill(p, q, cu, window, sinks), ref, tol, fmt)
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("hkv,g,d,bs", [(2, 4, 128, 16), (2, 3, 64, 8), (1, 8, 128, 128), (4, 1, 64, 32)])
def test_ragged_batches(fmt, hkv, g, d, bs):
    # prompts from nothing, chunks behind cached tokens, single tokens, no tokens
    check(fmt, [40, 130, 1, 300, 200, 0, 129], [40, 7, 1, 1, 70, 0, 128], hkv, g, d, bs)


@pytest.mark.parametrize("fmt", ["int8", "kvarn", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 0), (64, 5), (128, 130), (129, 4), (5000, 9)])
def test_windows(fmt, window, sinks):
    check(fmt, [300, 257, 33, 600], [300, 1, 33, 90], 2, 4, 128, 16, window, sinks)
    check(fmt, [500, 18], [200, 9], 2, 2, 64, 8, window, sinks)


@pytest.mark.parametrize("g", range(1, 9))
def test_every_head_ratio(g):
    check("int8", [150, 261], [35, 64], 2, g, 64, 16)


@pytest.mark.parametrize("n,q", [(127, 127), (128, 128), (129, 129), (255, 32), (256, 33), (257, 64), (385, 63), (1, 1), (16, 16)])
def test_tile_edges(n, q):
    check("e4m3_int8", [n], [q], 1, 4, 128, 16)
    check("bf16", [n], [q], 2, 8, 64, 64)


@pytest.mark.parametrize("fmt", ["int8", "e4m3_int8", "e5m2"])
def test_head_scales(fmt):
    check(fmt, [200, 50], [20, 50], 3, 2, 128, 16, head_scales=True)


@pytest.mark.parametrize("fmt", ["int8", "kvarn"])
def test_long_contexts(fmt):
    """Few rows and many keys (the keys are split), and many rows."""
    check(fmt, [9000], [3], 1, 8, 128, 32)
    check(fmt, [2500, 30], [1, 1], 2, 4, 64, 16)
    check(fmt, [1500], [700], 1, 4, 128, 16)


def test_more_tiles_than_the_device_holds_at_once():
    """Short chunks over long contexts, several waves of CTAs: every warp's pace differs."""
    lens = np.random.default_rng(3).integers(600, 1500, 48)
    check("int8", lens, np.random.default_rng(4).integers(1, 4, 48), 8, 2, 64, 16)


@pytest.mark.parametrize("count", [513, 1100])
def test_many_sequences(count):
    """More sequences than a CTA has threads: the row tiles are found over several chunks."""
    rng = np.random.default_rng(count)
    lens, new = rng.integers(0, 40, count), rng.integers(0, 4, count)
    check("e5m2", lens, np.minimum(lens, new), 2, 1, 64, 16)
    lens[count - 2], new[count - 2] = 300, 140  # one long chunk near the end
    check("int8", lens, np.minimum(lens, new), 1, 2, 64, 16, 30, 3)


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("g,q", [(1, 64), (8, 8), (8, 9), (5, 13), (3, 21), (4, 1)])
def test_few_rows(fmt, g, q):
    """63, 64, 65 and fewer rows of the longest chunk, on contexts of one tile and of several."""
    check(fmt, [q, 128, 700, 1300], [q, 1, q, q // 2], 1, g, 128, 16)
    check(fmt, [2000 + q], [q], 2, g, 64, 8)  # cut into parts
    check(fmt, [900, 385], [q, q], 1, g, 128, 32, 200, 40)


@pytest.mark.parametrize("count", [2, 63, 128, 129])
def test_sequences_of_one_order(count):
    """Equal, rising and falling lengths, rows of no tokens between: each row is its own sequence's."""
    lens = np.full(count, 37)
    check("int8", lens, np.ones(count, int), 1, 4, 64, 16)
    lens = np.arange(count) * 3 % 200 + 1
    new = np.minimum(np.arange(count) % 4, lens)
    check("bf16", lens, new, 2, 2, 64, 16)
    check("int4", lens[::-1].copy(), new[::-1].copy(), 1, 1, 128, 32, 40, 2)


def test_large_logits():
    """Keys whose logits span hundreds: the running maximum moves by more than any fixed range."""
    check("bf16", [400], [130], 1, 4, 128, 16, k_std=20.0)
    check("int8", [400, 1000], [130, 2], 1, 4, 128, 16)
    p = Paged("bf16", [640], 1, 64, 16)
    # keys that grow along the sequence, all in the queries' direction: a new maximum in every tile
    q = torch.ones((300, 4, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.ones((640, 1, 64), device=DEV) * torch.linspace(-8, 8, 640, device=DEV)[:, None, None]
    v = torch.randn((640, 1, 64), device=DEV).to(torch.bfloat16)
    slots = ints([p.table[0, t // 16] * 16 + t % 16 for t in range(640)], torch.int64)
    kvq.kvq_write_cache(p.cache, k.to(torch.bfloat16), v, slots)
    for keys in (k, k.flip(0)):
        kvq.kvq_write_cache(p.cache, keys.to(torch.bfloat16).contiguous(), v, slots)
        ref, tol = p.expect(q, [0, 300], 1.0)
        check_close(prefill(p, q, np.array([0, 300]), sm=1.0), ref, tol)
        ref, tol = p.expect(q, [0, 300], -1.0)
        check_close(prefill(p, q, np.array([0, 300]), sm=-1.0), ref, tol)


def test_rows_outside_the_batch_stay():
    p = Paged("int8", [50, 20], 2, 64, 16)
    q = random_query(40, 4, 64)
    cu = np.array([3, 13, 30])
    out = torch.full_like(q, 7.0)
    prefill(p, q, cu, out=out)
    ref, tol = p.expect(q, cu, 0.125)
    check_close(out[3:30], ref[3:30], tol[3:30])
    assert (out[:3] == 7).all() and (out[30:] == 7).all()
    assert kvq.kvq_get_device_error() == 0


def test_more_rows_than_context():
    """Rows before the first position see nothing: zero, and flagged."""
    p = Paged("int8", [5, 40, 0], 2, 64, 16)
    q = random_query(21, 4, 64)
    cu = np.array([0, 9, 19, 21])
    out = prefill(p, q, cu)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_CONTEXT_RANGE
    ref, tol = p.expect(q, cu, 0.125)
    assert (ref[:4] == 0).all()
    check_close(out, ref, tol)
    assert (out[:4] == 0).all() and (out[19:] == 0).all()


def test_bad_offsets_are_flagged_and_cut():
    p = Paged("int8", [50, 20], 2, 64, 16)
    q = random_query(30, 4, 64)
    for cu, max_q in (([0, 40, 50], 30), ([0, 10, 5], 20), ([-4, 10, 20], 20), ([0, 20, 30], 12)):
        out = torch.full((40, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        prefill(p, q, np.array(cu), max_q=max_q, out=out[:30])
        assert kvq.kvq_get_device_error() & kvq.DEVERR_TOKENS
        assert (out[30:] == 7).all()


def test_bad_pages_and_queries_are_flagged():
    p = Paged("int8", [50], 2, 64, 16)
    p.block_table[0, 1] = -1
    q = random_query(3, 4, 64)
    out = prefill(p, q, np.array([0, 3]))
    assert kvq.kvq_get_device_error() == kvq.DEVERR_BLOCK_RANGE and torch.isfinite(out).all()
    p = Paged("int8", [50], 2, 64, 16)
    q[1, 2, 3] = 1e30
    out = prefill(p, q, np.array([0, 3]))
    assert kvq.kvq_get_device_error() == kvq.DEVERR_QUERY_RANGE
    ref, tol = p.expect(q[:1], [0, 1], 0.125)  # rows 0 and 2 are untouched by it
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("g,d,bs", [(4, 128, 16), (5, 64, 8), (8, 128, 128)])
def test_contexts_dequantized_ahead(fmt, g, d, bs):
    """Enough rows a sequence that the keys are dequantized once, ahead of the attention."""
    check(fmt, [620, 700], [600, 500], 2, g, d, bs)
    check(fmt, [720], [520], 1, g, d, bs, 100, 20)
    check(fmt, [1000], [515], 1, g, d, bs, 300, 130)


@pytest.mark.parametrize("n,q", [(512, 512), (640, 513), (769, 576), (1025, 700)])
def test_ahead_at_tile_edges(n, q):
    check("int8", [n], [q], 1, 4, 64, 32)
    check("uint8", [n], [q], 2, 8, 128, 16, 129, 1)
    check("e4m3_int8", [n, 7], [q, 0], 1, 8, 64, 16, head_scales=True)


@pytest.mark.parametrize("q", [100, 1100])  # dequantized by each CTA, and ahead
@pytest.mark.parametrize("fmt", ["e5m2", "bf16"])
def test_values_not_finite(fmt, q):
    """A value that is not finite reaches the rows that see it and no others."""
    p = Paged(fmt, [q], 2, 64, 16)
    b = p.table[0, 60 // 16]
    if fmt == "bf16":
        p.cache.v_cache.view(torch.bfloat16)[b, 60 % 16, 0, 5] = float("inf")
        p.cache.v_cache.view(torch.bfloat16)[b, 60 % 16, 0, 9] = float("nan")
    else:
        p.cache.v_cache[b, 60 % 16, 0, 5] = 0x7C  # inf
        p.cache.v_cache[b, 60 % 16, 0, 9] = 0x7F  # NaN
    out = prefill(p, random_query(q, 4, 64), np.array([0, q]))
    good = torch.isfinite(out)
    assert good[:60].all() and good[:, 2:].all()
    assert not good[60:, :2, 5].any() and not good[60:, :2, 9].any()
    good[60:, :2, 5] = good[60:, :2, 9] = True
    assert good.all()


@pytest.mark.parametrize("fmt", ["e5m2", "bf16", "uint8"])
def test_nan_where_no_row_looks(fmt):
    """NaN beyond the context and between the kept tokens and the window."""
    p = Paged(fmt, [200], 2, 64, 128)
    for t in range(3, 90):
        blk = p.table[0, t // 128]
        p.cache.k_cache[blk, t % 128] = 0xFF
        p.cache.v_cache[blk, t % 128] = 0xFF
        if p.cache.k_meta is not None:
            for m in (p.cache.k_meta, p.cache.v_meta):
                m[blk, :, :, t % 128] = float("nan")
    q = random_query(10, 4, 64)
    ref, tol = p.expect(q, [0, 10], 0.125, 100, 3)
    check_close(prefill(p, q, np.array([0, 10]), 100, 3), ref, tol)
    p = Paged(fmt, [1400], 2, 64, 16)  # and ahead: rows 300 on, a window of 150 behind 20 kept
    for t in range(20, 151):
        blk = p.table[0, t // 16]
        p.cache.k_cache[blk, t % 16] = 0xFF
        p.cache.v_cache[blk, t % 16] = 0xFF
        if p.cache.k_meta is not None:
            for m in (p.cache.k_meta, p.cache.v_meta):
                m[blk, :, :, t % 16] = float("nan")
    q = random_query(1100, 4, 64)
    ref, tol = p.expect(q, [0, 1100], 0.125, 150, 20)
    check_close(prefill(p, q, np.array([0, 1100]), 150, 20), ref, tol)


@pytest.mark.parametrize("lens,counts", [([260, 1000], [100, 3]), ([700, 800], [500, 300])])
def test_rows_repeat_and_streams_and_graphs(lens, counts):
    p = Paged("kvarn", lens, 2, 128, 16)
    cu = offsets(counts)
    rows, most = sum(counts), max(counts)
    q = random_query(rows, 8, 128)
    one = prefill(p, q, cu)
    assert torch.equal(bits(prefill(p, q, cu)), bits(one))  # no order of sums varies
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = kvq.kvq_prefill_workspace_size(p.cache, 2, 8, rows, most, p.max_len)
    ws, out, cut = garbage(n), torch.empty_like(q), ints(cu)
    call = lambda: kvq.kvq_paged_prefill(p.cache, q, out, cut, p.block_table, p.context_lens, most, p.max_len,
                                         p.d ** -0.5, 0, 0, ws)
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(bits(out), bits(one))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for i in range(3):
        q.copy_(random_query(rows, 8, 128, seed=30 + i))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(prefill(p, q, cu)))


def test_matches_the_decode_for_single_tokens():
    p = Paged("int8", [77, 300, 1], 4, 128, 16)
    q = random_query(3, 16, 128)
    out = torch.empty_like(q)
    kvq.kvq_paged_decode(p.cache, q, out, p.block_table, p.context_lens, p.max_len, p.d ** -0.5, garbage(1 << 22))
    ref, tol = p.expect(q, [0, 1, 2, 3], p.d ** -0.5)
    check_close(out, ref, tol)
    check_close(prefill(p, q, np.array([0, 1, 2, 3])), ref, tol)


@pytest.mark.parametrize("lens,counts", [([3000], [2]), ([700], [600])])  # keys cut into parts; dequantized ahead
def test_workspaces_that_do_not_serve_are_refused(lens, counts):
    p = Paged("int8", lens, 2, 64, 16)
    cu = offsets(counts)
    rows, most = sum(counts), max(counts)
    q = random_query(rows, 8, 64)
    out = torch.full_like(q, 7.0)
    n = kvq.kvq_prefill_workspace_size(p.cache, 1, 8, rows, most, p.max_len)
    assert n > 0
    ws = torch.zeros(n + 64, dtype=torch.uint8, device=DEV)
    call = lambda w: kvq.kvq_paged_prefill(p.cache, q, out, ints(cu), p.block_table, p.context_lens, most, p.max_len,
                                           0.125, 0, 0, w)
    for bad, status in ((None, 3), (ws[:0], 3), (ws[:16], 3), (ws[8:n + 8], 1), (ws[4:n + 4], 1)):
        with pytest.raises(kvq.KvqError) as e:
            call(bad)
        assert e.value.status == status
    torch.cuda.synchronize()
    assert (out == 7).all() and not ws.any()
    ref, tol = p.expect(q, cu, 0.125)
    check_close(call(ws[:n]), ref, tol)
    assert not ws[n:].any() and kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "kvarn", "bf16"])
@pytest.mark.parametrize("hkv,g,d", [(8, 4, 128), (1, 1, 64), (2, 8, 128), (16, 1, 64), (3, 5, 64), (96, 1, 64)])
def test_a_workspace_for_limits_serves_every_batch_within_them(fmt, hkv, g, d):
    """The size never grows when a limit shrinks."""
    kf, vf, kvarn = FORMATS[fmt]
    cache = kvq.alloc_kv_cache(kf, vf, 2, 16, hkv, d, 0.1, 0.1, kvarn, device=DEV)
    size = lambda s, t, q, c: kvq.kvq_prefill_workspace_size(cache, s, hkv * g, t, q, c)
    rng = np.random.default_rng(hkv * g)
    for _ in range(300):
        s, q, c = (int(np.exp(rng.uniform(0, np.log(hi)))) for hi in (300, 9000, 140000))
        t = int(rng.integers(q, s * q + 1))
        most = size(s, t, q, c)
        for _ in range(8):
            s2, q2, c2 = (int(rng.integers(1, x + 1)) if rng.random() < 0.6 else x for x in (s, q, c))
            assert size(s2, min(t, s2 * q2), q2, c2) <= most
            assert size(s2, int(rng.integers(0, t + 1)), q2, c2) <= most


@pytest.mark.parametrize("fmt", ["int8", "kvarn"])
def test_one_workspace_for_every_step_of_a_server(fmt):
    """A buffer of the largest step's size serves smaller steps, whose keys are cut into
    parts or dequantized ahead where the largest step's are not."""
    p = Paged(fmt, [1300, 700, 64, 900] + [300] * 60, 8, 64, 16)
    n, most, g = len(p.lens), 600, 4
    counts = np.full(n, 30)
    counts[0] = most
    ws = garbage(kvq.kvq_prefill_workspace_size(p.cache, n, 8 * g, int(counts.sum()), most, p.max_len))
    for seqs, new in ((range(n), counts), ([0], [1]), ([0], [most]), ([1, 3], [40, 8]), ([2], [64]), (range(4), [1] * 4)):
        seqs = list(seqs)
        cu = offsets(np.asarray(new))
        q = random_query(int(cu[-1]), 8 * g, 64)
        ids = ints(seqs, torch.int64)
        out = kvq.kvq_paged_prefill(p.cache, q, torch.empty_like(q), ints(cu), p.block_table[ids].contiguous(),
                                    p.context_lens[ids].contiguous(), int(max(new)), p.max_len, 0.125, 0, 0, ws)
        own = garbage(kvq.kvq_prefill_workspace_size(p.cache, len(seqs), 8 * g, int(cu[-1]), int(max(new)), p.max_len))
        ref = kvq.kvq_paged_prefill(p.cache, q, torch.empty_like(q), ints(cu), p.block_table[ids].contiguous(),
                                    p.context_lens[ids].contiguous(), int(max(new)), p.max_len, 0.125, 0, 0, own)
        assert torch.equal(bits(out), bits(ref))
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("q", [3, 100, 700])  # keys cut into parts, by each CTA, and ahead
@pytest.mark.parametrize("which", ["k", "v"])
def test_rotated_rows_whose_deviation_brings_them_into_range(which, q):
    """code * scale + zero point past 65,504, times a small deviation: some hundred at most."""
    p = Paged("kvarn", [q + 700], 2, 64, 16, seed=q)
    meta = getattr(p.cache, which + "_meta")
    for t in (5, 400, 640):  # seen by every row
        b, off = p.table[0, t // 16], t % 16
        meta[b, 0, :, off] = torch.tensor([6000.0 if which == "k" else 400.0, 30000.0, 1e-4], dtype=torch.float16, device=DEV)
    cu = np.array([0, q])
    x = random_query(q, 8, 64)
    ref, tol = p.expect(x, cu, 0.125)
    check_close(prefill(p, x, cu), ref, tol)
    assert kvq.kvq_get_device_error() == 0


NOT_FINITE = {"parts": (1500, 3, 1498), "by_each_cta": (100, 100, 60), "ahead": (1100, 1100, 60)}  # keys, rows, the key


@pytest.mark.parametrize("way", sorted(NOT_FINITE))
@pytest.mark.parametrize("fmt", ["uint8", "int4", "kvarn", "e4m3", "e5m2", "bf16"])
def test_one_value_row_not_finite(fmt, way, monkeypatch):
    """Rows that see it are not finite in the elements that its dequantized row is not
    (rotated rows: in all); everything else is what it is without it."""
    n, rows, key = NOT_FINITE[way]
    monkeypatch.setitem(FORMATS, "e4m3", ("fp8_e4m3", "fp8_e4m3", False))
    p = Paged(fmt, [n], 2, 64, 16)
    cu = np.array([0, rows])
    q = random_query(rows, 8, 64)
    b, off = p.table[0, key // 16], key % 16
    clean = prefill(p, q, cu)
    bad = torch.zeros(64, dtype=torch.bool, device=DEV)
    if p.cache.v_meta is not None:
        code = p.cache.v_cache[b, off, 0]
        if fmt == "int4":
            code = torch.stack((code & 15, code >> 4), -1).flatten()
        scale = 5000.0 if fmt == "int4" else 300.0
        p.cache.v_meta[b, 0, :2, off] = torch.tensor([scale, 0.0], dtype=torch.float16, device=DEV)
        bad = torch.isinf((code.double() * scale).half())
        if fmt == "kvarn":
            p.cache.v_meta[b, 0, 2, off] = 1.0
            bad = torch.full_like(bad, bool(bad.any()))
    elif fmt == "e4m3":
        bad[[5, 63]] = True
        p.cache.v_cache[b, off, 0, 5], p.cache.v_cache[b, off, 0, 63] = 0x7F, 0xFF  # its NaN
    else:
        bad[[5, 9, 40]] = True
        t = {"e5m2": torch.float8_e5m2, "bf16": torch.bfloat16}[fmt]
        values = torch.tensor([float("inf"), float("nan"), -float("inf")]).to(t).view(torch.uint8).to(DEV)
        row = p.cache.v_cache[b, off, 0].view(64, -1)
        row[[5, 9, 40]] = values.view(3, -1)
    assert bad.any()
    out = prefill(p, q, cu)
    assert kvq.kvq_get_device_error() == 0
    first = key - (n - rows)  # the first row that sees the key
    assert torch.equal(bits(out[:first]), bits(clean[:first])) and torch.equal(bits(out[:, 4:]), bits(clean[:, 4:]))
    finite = torch.isfinite(out[first:, :4])
    assert (finite == ~bad).all()
    if not bad.all():  # the other elements against the oracle, where they are finite
        good = (~bad).cpu().numpy()
        with np.errstate(all="ignore"):
            ref, tol = p.expect(q, cu, 0.125)
        # within the derived bound; check_close's mean limit of 2e-3 is for values of size one
        # (of outputs near 10 the rounding to bf16 alone is off by 10 * 2^-10 = 1e-2 on average)
        err = np.abs(out[first:, :4][..., ~bad].double().cpu().numpy() - ref[first:, :4][..., good])
        assert (err <= tol[first:, :4][..., good]).all()
    # a NaN among the row's fields: all of the row
    if p.cache.v_meta is not None:
        for field in range(p.cache.v_meta.shape[2]):
            keep = p.cache.v_meta[b, 0, field, off].clone()
            p.cache.v_meta[b, 0, field, off] = float("nan")
            out = prefill(p, q, cu)
            assert torch.equal(bits(out[:first]), bits(clean[:first])) and torch.equal(bits(out[:, 4:]), bits(clean[:, 4:]))
            assert not torch.isfinite(out[first:, :4]).any()
            p.cache.v_meta[b, 0, field, off] = keep


@pytest.mark.parametrize("way", sorted(NOT_FINITE))
@pytest.mark.parametrize("fmt", ["uint8", "kvarn", "e5m2", "bf16"])
def test_one_key_row_not_finite(fmt, way):
    """Rows that see a key that is NaN are NaN, and no others."""
    n, rows, key = NOT_FINITE[way]
    p = Paged(fmt, [n], 2, 64, 16)
    cu = np.array([0, rows])
    q = random_query(rows, 8, 64)
    b, off = p.table[0, key // 16], key % 16
    clean = prefill(p, q, cu)
    if p.cache.k_meta is not None:
        p.cache.k_meta[b, 0, 1, off] = float("nan")
    else:
        p.cache.k_cache[b, off, 0] = 0x7F if fmt == "e5m2" else 0xFF
    out = prefill(p, q, cu)
    first = key - (n - rows)
    assert torch.equal(bits(out[:first]), bits(clean[:first])) and torch.equal(bits(out[:, 4:]), bits(clean[:, 4:]))
    assert torch.isnan(out[first:, :4]).all()
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("way", sorted(NOT_FINITE))
def test_large_finite_values(way):
    """Rows near the end of fp16's range, whose bound passes it although no value does."""
    n, rows, key = NOT_FINITE[way]
    p = Paged("uint8", [n], 2, 64, 16)
    b, off = p.table[0, key // 16], key % 16
    p.cache.v_meta[b, 0, :2, off] = torch.tensor([200.0, -30000.0], dtype=torch.float16, device=DEV)
    cu = np.array([0, rows])
    q = random_query(rows, 8, 64)
    ref, tol = p.expect(q, cu, 0.125)
    out = prefill(p, q, cu)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all() and kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("seqs", [1, 40])  # keys cut into parts, and a CTA for all of them
@pytest.mark.parametrize("rows", [1, 2, 16, 30])
@pytest.mark.parametrize("n", [129, 256, 700, 1281])
def test_a_new_maximum_in_every_tile_of_few_rows(n, rows, seqs):
    """The accumulators are scaled in every tile, the second and the last among them, when
    the products before are done."""
    p = Paged("bf16", [n] * seqs, 2, 64, 16)
    g = torch.Generator(DEV).manual_seed(n)
    k = torch.ones((n, 2, 64), device=DEV) * torch.linspace(-8, 8, n, device=DEV)[:, None, None]
    v = torch.randn((n, 2, 64), device=DEV, generator=g).to(torch.bfloat16)
    q = torch.ones((rows * seqs, 8, 64), dtype=torch.bfloat16, device=DEV)
    cu = np.arange(seqs + 1) * rows
    for keys, sm in ((k, 1.0), (k.flip(0), -1.0), (k, 0.125)):
        for s in range(seqs):
            slots = ints([p.table[s, t // 16] * 16 + t % 16 for t in range(n)], torch.int64)
            kvq.kvq_write_cache(p.cache, keys.to(torch.bfloat16).contiguous(), v, slots)
        out = prefill(p, q, cu, sm=sm)
        each = bits(out).view(seqs, rows, 8, 64)
        assert (each == each[:1]).all()  # the sequences are alike
        ref, tol = expected_of_the_first(p, q[:rows], sm)
        check_close(out[:rows], ref, tol)
    assert kvq.kvq_get_device_error() == 0


def expected_of_the_first(p, q, sm):
    """The oracle's result for p's first sequence."""
    lens, table = p.lens, p.table
    p.lens, p.table = lens[:1], table[:1]
    try:
        return p.expect(q, [0, q.shape[0]], sm)
    finally:
        p.lens, p.table = lens, table


@pytest.mark.parametrize("fmt", ["int8", "e5m2", "uint8", "bf16"])
@pytest.mark.parametrize("rows,g,seqs", [(2, 1, 1), (40, 2, 1), (300, 1, 1), (600, 4, 1),  # keys cut into parts
                                         (2, 1, 100), (40, 2, 100), (100, 2, 100), (600, 4, 10)])  # not; 64 to 256 rows
def test_many_light_keys_beside_a_heavy_one(fmt, rows, g, seqs):
    """One key that dominates, its value zero, and 131,071 of 2^-25.4 its weight: what
    they weigh together is the output."""
    n, d, weight = 131072, 64, 2.0 ** -25.4
    k, v = torch.zeros((n, 1, d), device=DEV), torch.full((n, 1, d), 100.0, device=DEV)
    k[0], v[0] = 1.0, 0.0
    p = Paged(fmt, [n], 1, d, 128)
    if fmt == "int8":
        p.cache.k_scale, p.cache.v_scale = 1.0, 1.0
    slots = ints(p.table[0, np.arange(n) // 128] * 128 + np.arange(n) % 128, torch.int64)
    kvq.kvq_write_cache(p.cache, k.to(torch.bfloat16), v.to(torch.bfloat16), slots)
    p.lens = p.lens.repeat(seqs)  # sequences of the same pages
    p.block_table, p.context_lens = p.block_table.repeat(seqs, 1), p.context_lens.repeat(seqs)
    q = torch.ones((rows * seqs, g, d), dtype=torch.bfloat16, device=DEV)
    out = prefill(p, q, np.arange(seqs + 1) * rows, sm=float(-np.log(weight) / d)).double().cpu().numpy()
    light = np.tile(np.arange(n - rows, n), seqs)[:, None, None] * weight
    value = 96.0 if fmt == "e5m2" else 100.0  # as the format holds it
    ref = np.broadcast_to(light / (1 + light) * value, out.shape)
    # a probability of 2^(7 - 25.4) in fp16 is off by 2^-25, 2^-6.6 of it, the same in every
    # key (bf16: 2^-8); a logit of 17.6 by 2^-22; the output by 2^-8
    assert np.abs(out / ref - 1).max() <= (2.0 ** -8 if fmt == "bf16" else 2.0 ** -6.6) + 2.0 ** -8 + 1e-4
    assert kvq.kvq_get_device_error() == 0
