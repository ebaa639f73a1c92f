"""Block-scaled pages at the ends of what their scales and codes hold: pages of zeros, codes that are
not finite, and chunk attention over pages of any size."""
import numpy as np
import pytest
import torch

from quantized_paged_kv_kvq_gb300 import kvq

from block_testing import Blocked
from step_testing import DEV, check_close, garbage, ints, random_query

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [8, 128])
@pytest.mark.parametrize("num_ctas", [1, 2, 3])
def test_decode_of_many_pages_of_zeros(bs, num_ctas):
    """655,360 keys of one logit whose values are zero but for the last quarter's: every key weighs the
    same, in ranges of zeros alone, too."""
    n, d = 5 << 17, 64
    nb = n // bs
    cache = kvq.alloc_kv_cache("int8_block", "int8_block", nb, bs, 1, d, device=DEV, fill=0)
    cache.v_cache[3 * nb // 4:] = 127
    cache.v_meta[3 * nb // 4:] = 1.0 / 127
    table, lens = torch.arange(nb, dtype=torch.int32, device=DEV)[None], ints([n])
    q = random_query(1, 4, d)
    out = torch.full_like(q, 7.0)
    ws = garbage(kvq.kvq_decode_workspace_size(cache, 1, 4, n, num_ctas))
    kvq.kvq_paged_decode(cache, q, out, table, lens, n, 0.125, ws, num_ctas)
    assert kvq.kvq_get_device_error() == 0
    # a quarter: equal terms, 40,960 tiles of 16 keys added up in float32 in turn, each sum off by 2^-23
    # of itself at most, numerator and denominator; the probability times 1 / 127 and a range's
    # result rounded to fp16, the output to bf16
    assert (out.double() - 0.25).abs().max() <= 0.25 * (2 * 40960 * 2.0 ** -23 + 2 * 2.0 ** -11 + 2.0 ** -8)


@pytest.mark.parametrize("num_ctas", range(1, 10))
@pytest.mark.parametrize("at", [0, 500, 1439])
def test_decode_of_a_key_that_is_not_a_number(num_ctas, at):
    """Whichever range holds it, and whichever others are merged with it: every element of its
    kv-head's outputs is NaN, the other head's are not."""
    p = Blocked("e4m3", [1440], 2, 64, 16)
    p.fill()
    q = random_query(1, 8, 64)
    ref = p.decode(q, num_ctas=num_ctas)
    p.cache.k_cache[p.table[0, at // 16], at % 16, 1, 7] = 0x7F
    out = p.decode(q, num_ctas=num_ctas)
    assert torch.equal(out[:, :4], ref[:, :4]) and torch.isfinite(ref).all()
    assert torch.isnan(out[:, 4:]).all()


@pytest.mark.parametrize("fmt", ["fp8_e4m3", "fp8_e4m3_block"])
@pytest.mark.parametrize("num_ctas", [2, 5, 9, 33])
def test_decode_of_a_range_of_keys_that_are_not_numbers(fmt, num_ctas):
    """From some key on all of them, wherever that is: the last range may hold nothing else."""
    n, bs, d = 1440, 16, 64
    cache = kvq.alloc_kv_cache(fmt, fmt, n // bs, bs, 1, d, device=DEV, fill=0x30)
    for m in (cache.k_meta, cache.v_meta):
        if m is not None:
            m.fill_(1.0)
    q = random_query(1, 4, d)
    out = torch.full_like(q, 7.0)
    ws = garbage(kvq.kvq_decode_workspace_size(cache, 1, 4, n, num_ctas))
    table, lens = torch.arange(n // bs, dtype=torch.int32, device=DEV)[None], ints([n])
    for page in range(n // bs - 1, n // bs // 2, -1):
        cache.k_cache[page] = 0x7F
        kvq.kvq_paged_decode(cache, q, out, table, lens, n, 0.125, ws, num_ctas)
        assert torch.isnan(out).all(), f"from page {page} on"
    assert kvq.kvq_get_device_error() == 0


# ---- chunk attention: the same pages give the same answer as the decode, whatever their size
def chunks(p, counts, g, sm, window=0, sinks=0):
    cu = np.concatenate([[0], np.cumsum(counts)])
    q = random_query(int(cu[-1]), p.hkv * g, p.d)
    ref, tol = p.expect(q, cu, sm, window, sinks)  # codes are exact operands: keys are not rounded
    most = int(np.max(counts))
    ws = garbage(kvq.kvq_prefill_workspace_size(p.cache, len(p.lens), q.shape[1], q.shape[0], most, p.max_len))
    out = torch.full_like(q, 7.0)
    kvq.kvq_paged_prefill(p.cache, q, out, ints(cu), p.block_table, p.context_lens, most, p.max_len, sm, window, sinks, ws)
    assert kvq.kvq_get_device_error() == 0
    return out.double().cpu().numpy(), ref, tol


# sequences of 700 with few rows, with 128 and 256 a tile, dequantized ahead, and keys in parts
FORMS = {"64_rows": ([700, 700], [5, 16], 2), "128_rows": ([700, 700], [40, 60], 2), "256_rows": ([700, 700], [90, 100], 4),
         "ahead": ([700, 700], [700, 500], 4), "parts": ([3000], [3], 8)}


@pytest.mark.parametrize("f", [1e-30, 1e-20, 1e-6, 1e5, 1e15, 1e30])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("pair,bs", [("int8", 8), ("e4m3", 16), ("e4m3_int8", 128)])
def test_chunks_of_values_of_any_size(form, f, pair, bs):
    """A whole sequence's, and a page's beside others."""
    lens, counts, g = FORMS[form]
    p = Blocked(pair, lens, 2, 64, bs)
    p.fill()
    for s, n in enumerate(lens):
        k, v = p.rows(n)
        v = (v.float() * f).to(torch.bfloat16)
        if s == 0 and len(lens) > 1:
            p.store(k, v, p.slots(s, np.arange(n)))
        else:
            p.store(k[:bs], v[:bs], p.slots(s, np.arange(2 * bs, 3 * bs)))
    got, ref, tol = chunks(p, counts, g, 0.125)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("f", [1e-30, 1e-6, 1e5, 1e30])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_chunks_of_keys_of_any_size(form, f):
    """Logits of ordinary size from keys of any: sm_scale makes up for theirs."""
    lens, counts, g = FORMS[form]
    p = Blocked("e4m3_int8", lens, 2, 128, 16)
    p.fill(f)
    for s, n in enumerate(lens):
        k, v = p.rows(n)
        k = (k.float() * f).to(torch.bfloat16)
        p.store(k, v, p.slots(s, np.arange(n)))
    got, ref, tol = chunks(p, counts, g, 128 ** -0.5 / f)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 5)])
def test_chunks_of_pages_of_zeros(form, window, sinks):
    """Keys of zeros, values of zeros, one after the other and both, beside pages of tiny and large ones."""
    lens, counts, g = FORMS[form]
    p = Blocked("int8", lens, 2, 64, 16)
    for s, n in enumerate(lens):
        size = 10.0 ** p.rng.integers(-3, 3, (2, n // 16 + 1, 2, 1)) * (p.rng.random((2, n // 16 + 1, 2, 1)) < 0.6)
        size[0] = np.minimum(size[0], 1.0)
        p.store(*p.rows(n, np.repeat(size, 16, 1)[:, :n]), p.slots(s, np.arange(n)))
    got, ref, tol = chunks(p, counts, g, 0.125, window, sinks)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("form", ["64_rows", "256_rows", "ahead"])
def test_chunks_where_a_page_out_of_sight_is_anything(form):
    """Scales that are not numbers, of keys and of values, reach the rows that see their page alone."""
    lens, counts, g = FORMS[form]
    counts = [16, 5] if form == "64_rows" else counts
    p = Blocked("int8", lens, 2, 64, 8)
    p.fill()
    clean, _, _ = chunks(p, counts, g, 0.125)
    begin = lens[0] - counts[0]
    first = -(-(begin + counts[0] // 2) // 8) * 8  # of a page that the rows in front of it do not see
    for value in (float("nan"), float("inf")):
        for of_keys in (True, False):
            q = Blocked("int8", lens, 2, 64, 8)
            q.fill()
            (q.cache.k_meta if of_keys else q.cache.v_meta)[q.table[0, first // 8], 0] = value
            got, _, _ = chunks(q, counts, g, 0.125)
            row = first - begin
            assert np.array_equal(got[:row], clean[:row]) and np.array_equal(got[counts[0]:], clean[counts[0]:])
            assert np.array_equal(got[:, g:], clean[:, g:])
            if not of_keys or np.isnan(value):
                assert not np.isfinite(got[row:counts[0], :g]).any()


@pytest.mark.parametrize("form", ["64_rows", "256_rows", "ahead"])
@pytest.mark.parametrize("pair", ["e4m3", "int8_e4m3"])
def test_chunks_with_a_code_that_is_not_a_number(form, pair):
    """Of a value: its element of the rows that see it, and nothing else."""
    lens, counts, g = FORMS[form]
    p = Blocked(pair, lens, 2, 64, 16)
    p.fill()
    clean, _, _ = chunks(p, counts, g, 0.125)
    at = lens[0] - counts[0] // 2
    p.cache.v_cache[p.table[0, at // 16], at % 16, 1, 9] = 0x7F
    got, _, _ = chunks(p, counts, g, 0.125)
    row = at - (lens[0] - counts[0])
    assert np.isnan(got[row:counts[0], g:, 9]).all()
    got[row:counts[0], g:, 9] = clean[row:counts[0], g:, 9]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("tile", [0, 1, 4])
@pytest.mark.parametrize("form", ["64_rows", "128_rows", "256_rows", "ahead"])
def test_a_wait_of_the_chunks_that_runs_out(form, tile):
    """The products of one CTA wait for what nothing signals: the launch ends, the next one is whole.
    (As many sequences, of the same pages, as leave a CTA all of its keys; of one length, so that CTA 0
    has rows.)"""
    lens, counts, g = FORMS[form]
    counts = [max(counts)] * 2
    p = Blocked("e4m3_int8", lens, 2, 64, 16)
    p.fill()
    table, context, n = p.block_table.repeat(40, 1), ints(lens * 40), 80
    cu, most = np.concatenate([[0], np.cumsum(counts * 40)]), max(counts)
    q = random_query(int(cu[-1]), 2 * g, 64)
    ws = garbage(kvq.kvq_prefill_workspace_size(p.cache, n, 2 * g, int(cu[-1]), most, 700))

    def call():
        out = torch.full_like(q, 7.0)
        kvq.kvq_paged_prefill(p.cache, q, out, ints(cu), table, context, most, 700, 0.125, 0, 0, ws)
        return out, kvq.kvq_get_device_error()

    ref, found = call()
    assert found == 0
    kvq.kvq_debug_arm_wait_timeout(1 << 12, 0, tile)
    _, found = call()
    assert found & kvq.DEVERR_TIMEOUT
    out, found = call()
    assert found == 0 and torch.equal(out, ref)


# ---- store
@pytest.mark.parametrize("pair", ["int8", "e4m3"])
def test_an_infinity_among_zeros(pair):
    """A page without a scale has no code for an infinity: 0, or e4m3's NaN, as for a NaN; behind rows
    that gave the page a scale it is the largest code."""
    p = Blocked(pair, [16, 16], 1, 64, 16)
    x = torch.zeros((4, 1, 64), dtype=torch.bfloat16, device=DEV)
    x[1, 0, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    p.store(x, x, p.slots(0, np.arange(4)))
    ones = torch.ones_like(x)
    p.store(ones, ones, p.slots(1, np.arange(4)))
    p.store(x, x, p.slots(1, np.arange(4, 8)))
    p.same()
    nan, most, least = (0, 127, 128) if pair == "int8" else (0x7F, 0x7E, 0xFE)
    for codes, scales in ((p.cache.k_cache, p.cache.k_meta), (p.cache.v_cache, p.cache.v_meta)):
        assert scales[p.table[0, 0], 0] == 0 and (codes[p.table[0, 0], 1, 0, :3].int() & 0x7F).tolist() == [nan] * 3
        assert codes[p.table[1, 0], 5, 0, :2].tolist() == [most, least]


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("sm", [-0.125, 0.0, 1.0])
def test_chunks_of_any_sm_scale(form, sm):
    lens, counts, g = FORMS[form]
    p = Blocked("int8_e4m3", lens, 2, 64, 32)
    p.fill()
    got, ref, tol = chunks(p, counts, g, sm)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()
