"""kvq_read_cache against the oracle's dequantization, every format."""
import numpy as np
import pytest
import torch

from oracle import cache as OC
from quantized_paged_kv_kvq_gb300 import kvq

from block_testing import PAIRS, Blocked
from step_testing import DEV, FORMATS, Paged, bits, ints

pytestmark = pytest.mark.gpu


def read(cache, slots, hkv, d, fill=7.0):
    out = [torch.full((len(slots), hkv, d), fill, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kvq.kvq_read_cache(cache, ints(np.asarray(slots), torch.int64), *out)
    return out


def close(got, ref, parts):
    """Float32 operations (at most 24, each 2^-24 of what it adds up), one rounding to bf16."""
    got = got.double().cpu().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + 24 * 2.0 ** -24 * parts + 1e-38).all()


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("hkv,d,bs,heads", [(8, 128, 16, False), (2, 64, 8, False), (1, 128, 128, False), (3, 64, 32, True), (5, 128, 64, True)])
def test_every_format(fmt, hkv, d, bs, heads):
    p = Paged(fmt, [130, 1, 77], hkv, d, bs, head_scales=heads)
    rng = np.random.default_rng(1)
    pos = [(s, t) for s, n in enumerate(p.lens) for t in range(n)]
    pos = [pos[i] for i in rng.integers(0, len(pos), 301)]  # any order, some twice
    pages = np.array([p.table[s, t // bs] for s, t in pos])
    offs = np.array([t % bs for _, t in pos])
    got = read(p.cache, pages * bs + offs, hkv, d)
    kc, km, vc, vm = p.numpy()
    for out, codes, meta, f, scale in ((got[0], kc, km, p.k_fmt, p.k_scale), (got[1], vc, vm, p.v_fmt, p.v_scale)):
        for h in range(hkv):
            m = meta[pages, h][:, :, :].transpose(0, 2, 1)[np.arange(len(pos)), offs] if meta.shape[2] else np.zeros((len(pos), 0), np.uint16)
            ref = OC.decode_rows(codes[pages, offs, h], m, f, scale[h] if np.ndim(scale) else scale, p.kvarn, p.signs, d)
            parts = np.abs(ref)
            if f.endswith("asym"):  # code * scale and the zero point may cancel; a rotation mixes the row
                fields = [np.abs(OC.F.F16.decode(m[:, i]))[:, None] for i in range(m.shape[1])]
                parts = (OC.F.unpack_int4(codes[pages, offs, h]) if f == "int4_asym" else codes[pages, offs, h]) * fields[0] + fields[1]
                if p.kvarn:
                    parts = np.broadcast_to((parts * fields[2]).sum(1, keepdims=True) / np.sqrt(d), parts.shape)
            close(out[:, h], ref, parts)
            if f == "bf16":
                assert np.array_equal(bits(out[:, h]).cpu().numpy().view(np.uint16), codes[pages, offs, h].view(np.uint16))
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("pair", sorted(PAIRS))
@pytest.mark.parametrize("hkv,d,bs", [(8, 128, 16), (2, 64, 8), (5, 128, 64)])
def test_block_formats(pair, hkv, d, bs):
    p = Blocked(pair, [130, 77], hkv, d, bs)
    p.fill()
    for s, n in enumerate(p.lens):
        got = read(p.cache, p.slots(s, np.arange(n)), hkv, d)
        for out, ref in zip(got, p.sequence(s, n)):
            close(out, ref, np.abs(ref))


@pytest.mark.parametrize("fmt", ["int8", "kvarn", "int4", "bf16"])
def test_skipped_and_bad_slots_leave_their_rows(fmt):
    p = Paged(fmt, [50], 2, 64, 16)
    slots = p.table[0, np.arange(50) // 16] * 16 + np.arange(50) % 16
    full = read(p.cache, slots, 2, 64)
    some = slots.copy()
    some[[0, 3, 4, 49]] = [-1, -5, p.cache.num_blocks * 16, 1 << 40]
    got = read(p.cache, some, 2, 64)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_SLOT_RANGE
    for a, b in zip(full, got):
        assert (b[[0, 3, 4, 49]] == 7).all()
        a[[0, 3, 4, 49]] = 7.0
        assert torch.equal(bits(a), bits(b))


def test_strides_graphs_and_an_empty_call():
    p = Paged("uint8", [90], 4, 128, 32)
    slots = ints(p.table[0, np.arange(90) // 32] * 32 + np.arange(90) % 32, torch.int64)
    k, v = read(p.cache, slots.cpu().numpy(), 4, 128)
    wide = torch.full((90, 11, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    kvq.kvq_read_cache(p.cache, slots, wide[:, 1:5], wide[:, 6:10])
    assert torch.equal(bits(wide[:, 1:5]), bits(k)) and torch.equal(bits(wide[:, 6:10]), bits(v))
    assert (wide[:, [0, 5, 10]] == 7).all()
    kvq.kvq_read_cache(p.cache, slots[:0], k[:0], v[:0])
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = [torch.zeros_like(k), torch.zeros_like(v)]
    with torch.cuda.graph(g, stream=s):
        kvq.kvq_read_cache(p.cache, slots, *out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out[0]), bits(k)) and torch.equal(bits(out[1]), bits(v))


@pytest.mark.parametrize("fmt", ["kvarn", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_that_are_16_byte_aligned_only(fmt, d):
    """Rows that begin in the middle of a 32-byte sector, in either way, give the same bits."""
    p = Paged(fmt, [70], 3, d, 16)
    slots = p.table[0, np.arange(70) // 16] * 16 + np.arange(70) % 16
    k, v = read(p.cache, slots, 3, d)
    for off, stride in ((8, 3 * d + 16), (0, 3 * d + 8), (8, 3 * d + 8)):
        flat = torch.full((2, 72 * (3 * d + 16)), 7.0, dtype=torch.bfloat16, device=DEV)
        ko, vo = (torch.as_strided(x[off:], (70, 3, d), (stride, d, 1)) for x in flat)
        kvq.kvq_read_cache(p.cache, ints(slots, torch.int64), ko, vo)
        assert torch.equal(bits(ko), bits(k)) and torch.equal(bits(vo), bits(v))
        rest = flat.clone()
        for x in rest:
            torch.as_strided(x[off:], (70, 3, d), (stride, d, 1)).fill_(7.0)
        assert (rest == 7).all()


def test_reading_and_writing_again_gives_the_same_codes():
    """INT8 rows survive the round trip through bf16 (codes of 8 bits, values of 8)."""
    p = Paged("int8", [200], 2, 128, 16)
    slots = p.table[0, np.arange(200) // 16] * 16 + np.arange(200) % 16
    before = p.cache.k_cache.clone(), p.cache.v_cache.clone()
    k, v = read(p.cache, slots, 2, 128)
    kvq.kvq_write_cache(p.cache, k, v, ints(slots, torch.int64))
    assert torch.equal(before[0], p.cache.k_cache) and torch.equal(before[1], p.cache.v_cache)
