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
