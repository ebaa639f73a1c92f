"""kvq_rope_table, kvq_norm_rope and kvq_norm_rope_write."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from oracle import step as OS
from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, FORMATS, bits, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("positions,rot,base,scaling", [
    (1, 2, 10000.0, None), (3, 64, 10000.0, None), (1000, 128, 10000.0, kvq.RopeScaling("linear", 4.0)),
    (131072, 64, 500000.0, kvq.RopeScaling("bands", 8.0, 8192, 1.0, 4.0)),
    (5001, 96, 10000.0, kvq.RopeScaling("ntk", 2.0)), (777, 256, 1e6, None), (65, 6, 100.0, None),
    (40000, 128, 10000.0, kvq.RopeScaling("yarn", 16.0, 4096, 1.0, 32.0, 1.277))])
def test_table(positions, rot, base, scaling):
    table = torch.full((positions + 1, rot // 2, 2), 7.0, device=DEV)
    kvq.kvq_rope_table(table[:positions], base, scaling)
    s = scaling or kvq.RopeScaling("none")
    theta = OS.rope_theta(rot, base, s.kind, s.factor, s.original_len, s.low, s.high)
    pos = np.arange(positions) if positions < 6000 else np.concatenate([np.arange(300), np.arange(positions - 3000, positions)])
    ref = OS.rope_table(pos, theta, s.amplitude)
    got = table.cpu().numpy()
    # an angle of at most pi/4 rounded to float32 (2^-24 of it), the functions' own 2^-23,
    # the product with the amplitude 2^-24; float64 angles to 2^-52 * 131072 turns
    assert np.abs(got[pos] - ref).max() <= 3e-7 * s.amplitude
    assert (got[positions:] == 7.0).all()


def test_table_at_far_positions():
    """Angles keep their digits at positions where float32 products lose all of them."""
    n = 1 << 24
    table = torch.empty((n, 1, 2), device=DEV)
    kvq.kvq_rope_table(table, 10000.0)
    pos = np.array([n - 1, n - 12345, 8388607])
    ref = OS.rope_table(pos, np.array([1.0]))
    assert np.abs(table[ints(pos, torch.int64)].cpu().numpy() - ref).max() <= 3e-7


def packed(t, hq, hkv, d, seed=0):
    """Queries, keys and values as slices of one projection."""
    g = torch.Generator(DEV).manual_seed(seed)
    x = (torch.randn((t, (hq + 2 * hkv) * d), device=DEV, generator=g) * 1.7).to(torch.bfloat16)
    cut = lambda a, b: x[:, a * d:b * d].unflatten(1, (b - a, d))
    return cut(0, hq), cut(hq, hq + hkv), cut(hq + hkv, hq + 2 * hkv)


def make_rope(d, rot, interleaved, norm, positions=500, offset=0.0):
    g = torch.Generator(DEV).manual_seed(9)
    w = (torch.randn((2, d), device=DEV, generator=g) * 0.2 + (1 - offset)).to(torch.bfloat16)
    table = None
    if rot:
        table = torch.empty((positions, rot // 2, 2), device=DEV)
        kvq.kvq_rope_table(table, 10000.0)
    return kvq.Rope(table, interleaved, w[0] if norm else None, w[1] if norm else None, 1e-6, offset)


def check_rotated(rope, x, weight, positions, out):
    rows = None if rope.table is None else rope.table[positions.long()].cpu().numpy()
    ref = OS.norm_rope(x.double().cpu().numpy(), None if weight is None else weight.double().cpu().numpy(),
                       rope.eps, rope.weight_offset, rows, rope.interleaved)
    # one rounding to bf16 (2^-8 of the value) and some twenty float32 operations on
    # values up to the row's largest: 32 * 2^-24 of it
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * np.sqrt(2) * np.abs(ref).max(-1, keepdims=True)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("t,hq,hkv,d,rot,interleaved,norm", [
    (1, 32, 8, 128, 128, False, True), (5, 8, 2, 64, 64, True, True), (33, 3, 1, 64, 16, False, False),
    (64, 32, 8, 128, 112, False, True), (7, 64, 8, 128, 48, True, False), (9, 5, 5, 256, 256, False, True),
    (12, 16, 16, 256, 96, True, True), (4, 9, 3, 128, 0, False, True), (6, 17, 2, 64, 48, False, False),
    (300, 1, 1, 128, 32, False, True)])
def test_norm_rope(t, hq, hkv, d, rot, interleaved, norm):
    q, k, _ = packed(t, hq, hkv, d)
    rope = make_rope(d, rot, interleaved, norm)
    pos = ints(np.random.default_rng(t).integers(0, 500, t))
    qo, ko = torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV), torch.empty((t, hkv, d), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_norm_rope(rope, q, k, pos, qo, ko)
    check_rotated(rope, q, rope.q_weight, pos, qo)
    check_rotated(rope, k, rope.k_weight, pos, ko)
    kvq.kvq_norm_rope(rope, q, k, pos, q, k)  # in place, inside the packed projection
    assert torch.equal(bits(q), bits(qo)) and torch.equal(bits(k), bits(ko))
    assert kvq.kvq_get_device_error() == 0


def test_weight_offset_one_sided_norm_and_zero_rows():
    q, k, _ = packed(6, 4, 4, 128)
    q[2] = 0
    rope = make_rope(128, 128, False, True, offset=1.0)
    rope.k_weight = None
    pos = ints([0, 1, 2, 3, 499, 5])
    qo, ko = torch.empty((6, 4, 128), dtype=torch.bfloat16, device=DEV), torch.empty((6, 4, 128), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_norm_rope(rope, q, k, pos, qo, ko)
    check_rotated(rope, q, rope.q_weight, pos, qo)
    check_rotated(rope, k, None, pos, ko)
    assert (qo[2] == 0).all()


def test_positions_outside_the_table():
    q, k, v = packed(4, 4, 2, 64)
    rope = make_rope(64, 64, False, True)
    pos = ints([3, 500, -1, 7])
    qo, ko = torch.full((4, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV), torch.full((4, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    kvq.kvq_norm_rope(rope, q, k, pos, qo, ko)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_POSITION
    assert (qo[1:3] == 5).all() and (ko[1:3] == 5).all() and not (qo[3] == 5).all()
    cache = kvq.alloc_kv_cache("int8", "int8", 4, 8, 2, 64, 0.05, 0.05, device=DEV, fill=0x11)
    qo.fill_(5.0)
    kvq.kvq_norm_rope_write(rope, cache, q, k, v, pos, ints([0, 9, 10, 30], torch.int64), qo)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_POSITION
    assert (qo[1:3] == 5).all() and (cache.k_cache[1] == 0x11).all() and (cache.v_cache[1] == 0x11).all()
    assert not (cache.v_cache[3, 6] == 0x11).all()


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("t,hq,hkv,d,rot,interleaved,norm,bs", [
    (1, 32, 8, 128, 128, False, True, 16), (37, 8, 2, 64, 32, True, True, 8), (50, 6, 3, 128, 64, False, False, 64),
    (19, 16, 16, 64, 64, False, True, 128), (21, 10, 10, 128, 0, False, True, 32)])
def test_write_is_the_two_calls(fmt, t, hq, hkv, d, rot, interleaved, norm, bs):
    """Codes, fields and queries bit-equal to kvq_norm_rope then kvq_write_cache."""
    kf, vf, kvarn = FORMATS[fmt]
    rng = np.random.default_rng(t + d)
    q, k, v = packed(t, hq, hkv, d, seed=t)
    rope = make_rope(d, rot, interleaved, norm)
    pos = ints(rng.integers(0, 500, t))
    nb = -(-t // bs) + 2
    slots = rng.permutation(nb * bs)[:t]
    slots[rng.random(t) < 0.1] = -1
    slots = ints(slots, torch.int64)
    signs = ints(rng.integers(0, 2, d) * 2 - 1, torch.int8) if kvarn else None
    a, b = (kvq.alloc_kv_cache(kf, vf, nb, bs, hkv, d, 0.04, 0.05, kvarn, signs, device=DEV, fill=0x5A) for _ in range(2))
    if fmt in ("int8", "e4m3_int8"):
        for c in (a, b):
            c.k_head_scales = torch.linspace(0.02, 0.09, hkv, device=DEV)
    qo, ko = torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV), torch.empty((t, hkv, d), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_norm_rope(rope, q, k, pos, qo, ko)
    kvq.kvq_write_cache(a, ko, v, slots)
    got = kvq.kvq_norm_rope_write(rope, b, q, k, v, pos, slots, torch.empty_like(qo))
    assert torch.equal(bits(got), bits(qo))
    assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)
    if a.k_meta is not None:
        assert torch.equal(bits(a.k_meta), bits(b.k_meta)) and torch.equal(bits(a.v_meta), bits(b.v_meta))
    assert kvq.kvq_get_device_error() == 0


def test_slot_past_the_cache():
    q, k, v = packed(3, 4, 2, 64)
    rope = make_rope(64, 64, True, False)
    cache = kvq.alloc_kv_cache("bf16", "bf16", 2, 16, 2, 64, device=DEV, fill=0x11)
    qo = torch.empty((3, 4, 64), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_norm_rope_write(rope, cache, q, k, v, ints([1, 2, 3]), ints([32, 1 << 40, 31], torch.int64), qo)
    assert kvq.kvq_get_device_error() == kvq.DEVERR_SLOT_RANGE
    check_rotated(rope, q, None, ints([1, 2, 3]), qo)
    assert (cache.k_cache[0] == 0x11).all() and not (cache.k_cache[1, 15] == 0x11).all()


def test_no_tokens_and_no_heads():
    rope = make_rope(64, 64, True, False)
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_norm_rope(rope, e, e, ints([]), e, e)
    q, k, _ = packed(3, 4, 2, 64)
    qo, none = torch.empty((3, 4, 64), dtype=torch.bfloat16, device=DEV), torch.empty((3, 0, 64), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_norm_rope(rope, q, none, ints([1, 2, 3]), qo, none)
    check_rotated(rope, q, None, ints([1, 2, 3]), qo)


def exact_rotation(p, base, i, rot):
    """cos and sin of p * base^(-2i/rot), from decimals of 60 digits."""
    getcontext().prec = 60
    turn = Decimal("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256")
    angle = Decimal(p) * (Decimal(base).ln() * (-2 * i) / rot).exp()
    x = float(angle - turn * int(angle / turn))  # rounded by 4e-16
    return math.cos(x), math.sin(x)


@pytest.mark.parametrize("base", [1.298, 1.175, 10000.0])
def test_table_at_the_last_positions(base):
    """Every pair up to the last position that the call takes."""
    n = (1 << 31) - 1  # 34 GB
    table = torch.empty((n, 2, 2), device=DEV)
    kvq.kvq_rope_table(table, base)
    pos = [n - 1, n - 2, n - 12345, (1 << 30) + 7, 1 << 24] + list(range(n - 300, n - 100))
    got = table[ints(pos, torch.int64)].cpu().numpy()
    ref = np.array([[exact_rotation(p, base, i, 4) for i in range(2)] for p in pos])
    assert np.abs(got - ref).max() <= 3e-7


def test_table_at_far_positions_of_every_pair():
    n = 1 << 24  # 8.6 GB
    table = torch.empty((n, 64, 2), device=DEV)
    kvq.kvq_rope_table(table, 1e6)
    pos = [n - 1, n - 12345, 8388607, 5000001]
    got = table[ints(pos, torch.int64)].cpu().numpy()
    ref = np.array([[exact_rotation(p, 1e6, i, 128) for i in range(64)] for p in pos])
    assert np.abs(got - ref).max() <= 3e-7


@pytest.mark.parametrize("fmt", ["int8", "e4m3_int8", "e5m2"])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
@pytest.mark.parametrize("d,interleaved", [(128, False), (64, True)])
def test_write_with_head_scales(fmt, which, d, interleaved):
    """Each tensor with its own scales per kv-head, or with its one scale: the two calls' codes."""
    kf, vf, _ = FORMATS[fmt]
    t, hq, hkv = 45, 12, 6
    q, k, v = packed(t, hq, hkv, d, seed=d)
    rope = make_rope(d, d, interleaved, True)
    pos, slots = ints(np.arange(t) * 7 % 500), ints(np.random.default_rng(1).permutation(64)[:t], torch.int64)
    a, b = (kvq.alloc_kv_cache(kf, vf, 4, 16, hkv, d, 0.04, 0.05, device=DEV, fill=0x5A) for _ in range(2))
    for c in (a, b):
        if "k" in which:
            c.k_head_scales = torch.linspace(0.02, 0.09, hkv, device=DEV)
        if "v" in which:
            c.v_head_scales = torch.linspace(0.11, 0.03, hkv, device=DEV)
    qo, ko = torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV), torch.empty((t, hkv, d), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_norm_rope(rope, q, k, pos, qo, ko)
    kvq.kvq_write_cache(a, ko, v, slots)
    kvq.kvq_norm_rope_write(rope, b, q, k, v, pos, slots, torch.empty_like(qo))
    assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)
    plain = kvq.alloc_kv_cache(kf, vf, 4, 16, hkv, d, 0.04, 0.05, device=DEV, fill=0x5A)
    kvq.kvq_norm_rope_write(rope, plain, q, k, v, pos, slots, torch.empty_like(qo))
    assert torch.equal(plain.k_cache, b.k_cache) == ("k" not in which)
    assert torch.equal(plain.v_cache, b.v_cache) == ("v" not in which)
    assert kvq.kvq_get_device_error() == 0
