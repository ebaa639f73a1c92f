"""Decode over asymmetric value rows whose scales, times the probabilities, leave fp16's
range at either end: many light keys beside one that dominates, and large scales behind a
maximum that lags.  Against the oracle, within its derived bound."""
import numpy as np
import pytest
import torch

from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, Paged, bits, garbage, ints

pytestmark = pytest.mark.gpu


def decodes(p, q, sm, ctas):
    """Outputs of the decode and of the same through a window that holds everything."""
    s, hq = q.shape[:2]
    ws = garbage(kvq.kvq_decode_workspace_size(p.cache, s, hq, p.max_len, ctas))
    a = kvq.kvq_paged_decode(p.cache, q, torch.full_like(q, 7.0), p.block_table, p.context_lens, p.max_len, sm, ws, ctas)
    b = kvq.kvq_decode_window(p.cache, q, torch.full_like(q, 7.0), p.block_table, p.context_lens, p.max_len, sm, p.max_len,
                              0, ws, ctas)
    assert torch.equal(bits(a), bits(b))
    return a


def store(p, k, v):
    n = k.shape[0]
    slots = ints(p.table[0, np.arange(n) // p.bs] * p.bs + np.arange(n) % p.bs, torch.int64)
    kvq.kvq_write_cache(p.cache, k.to(torch.bfloat16), v.to(torch.bfloat16), slots)


def check(out, ref, tol):
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("seqs", [1, 40, 310])  # several CTAs a sequence, and less than one
@pytest.mark.parametrize("fmt", ["int4", "uint8", "kvarn"])
@pytest.mark.parametrize("d,bs,light", [(64, 128, 20.0), (128, 8, 20.0), (64, 16, 24.0)])
def test_many_light_keys_beside_a_heavy_one(fmt, d, bs, light, seqs):
    """32,767 keys of 2^-light the weight of one whose value is zero."""
    n = 32768
    p = Paged(fmt, [n], 1, d, bs)
    g = torch.Generator(DEV).manual_seed(d)
    k, v = torch.zeros((n, 1, d), device=DEV), torch.randn((n, 1, d), device=DEV, generator=g)
    k[0], v[0] = 1.0, 0.0
    store(p, k, v)
    q = torch.ones((1, 2, d), dtype=torch.bfloat16, device=DEV)
    sm = float(light * np.log(2) / d)
    ref, tol = p.expect(q, [0, 1], sm)
    p.block_table, p.context_lens = p.block_table.repeat(seqs, 1), p.context_lens.repeat(seqs)  # of the same pages
    out = decodes(p, q.repeat(seqs, 1, 1), sm, 0)
    check(out, np.repeat(ref, seqs, 0), np.repeat(tol, seqs, 0))


@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("fmt,scale", [("int4", 4000.0), ("uint8", 250.0), ("kvarn", 250.0), ("uint8", 2.0 ** -14)])
@pytest.mark.parametrize("rise", [0.0, 5.0, 7.5, 30.0])
def test_scales_behind_a_maximum_that_lags(fmt, scale, rise, ctas):
    """Rows of ordinary scales, then keys 2^rise as heavy whose values reach 63,750."""
    n, d = 400, 64
    p = Paged(fmt, [n], 2, d, 16, seed=3)
    k = torch.zeros((n, 2, d), device=DEV)
    k[300:330] = 1.0
    store(p, k, torch.randn((n, 2, d), device=DEV, generator=torch.Generator(DEV).manual_seed(1)))
    for t in range(300, 330):
        m = p.cache.v_meta[p.table[0, t // 16], :, :, t % 16]
        m[:, 0], m[:, 1] = scale, -scale
        if fmt == "kvarn":
            m[:, 2] = 0.25 + 0.02 * (t - 300)
    q = torch.ones((1, 8, d), dtype=torch.bfloat16, device=DEV)
    sm = float(rise * np.log(2) / d)
    ref, tol = p.expect(q, [0, 1], sm)
    check(decodes(p, q, sm, ctas), ref, tol)


@pytest.mark.parametrize("ctas", [1, 3])
@pytest.mark.parametrize("step", [0.0, 1.0, 30.0, 100.0, -30.0])
@pytest.mark.parametrize("fmt", ["int4", "uint8", "kvarn"])
def test_rows_without_a_scale(fmt, step, ctas):
    """Scales of zero: the rows are their zero points.  Logits that move by 2^step from
    tile to tile, by more than float32's range in all."""
    n, d = 300, 64
    p = Paged(fmt, [n], 2, d, 16, seed=5)
    k = (torch.arange(n, device=DEV) // 16 / 20.0)[:, None, None].expand(n, 2, d)  # 0 .. 0.9 by 0.05 a tile
    store(p, k, torch.randn((n, 2, d), device=DEV, generator=torch.Generator(DEV).manual_seed(1)))
    p.cache.v_meta[:, :, 0] = 0.0
    q = torch.ones((1, 8, d), dtype=torch.bfloat16, device=DEV)
    sm = float(step * np.log(2) / (0.05 * d))
    # the oracle's bound holds for sm >= 0 (its logits' part is sm * 2u * |q| |k|): a
    # negative one is the other sign of the queries, the same logits exactly
    ref, tol = p.expect(q if sm >= 0 else -q, [0, 1], abs(sm))
    check(decodes(p, q, sm, ctas), ref, tol)
