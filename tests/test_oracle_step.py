"""Pins of the serving step's oracle to something other than itself."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle import step as OS
from quantized_paged_kv_kvq_gb300 import workloads as W

from kvq_testing import OracleRun


def test_plan_by_hand():
    # bs 8: request 0 holds 8 tokens (1 page) and adds 1; request 1 adds none;
    # request 2 starts with 17 tokens (3 pages)
    table = np.array([[5, -1, -1], [2, 7, -1], [-1, -1, -1]])
    slots, pos, after, cu, t2, fr = OS.plan_step([8, 12, 0], [1, 0, 17], table, [90, 91, 92, 93, 94, 95],
                                                 [1, 6], 8, 20)
    assert t2.tolist() == [[5, 91, -1], [2, 7, -1], [92, 93, 94]]
    assert cu.tolist() == [0, 1, 1, 18] and after.tolist() == [9, 12, 17] and fr.tolist() == [5, 6]
    assert slots[:3].tolist() == [728, 736, 737] and slots[17] == 94 * 8 and slots[18:].tolist() == [-1, -1]
    assert pos.tolist() == [8] + list(range(17)) + [0, 0]


def test_plan_matches_the_workloads_slots():
    wl = W.workload("tiny_int8", seed=3)
    slots, pos, *_ = OS.plan_step(np.zeros(wl.num_seqs, int), wl.context_lens, np.full_like(wl.block_table, -1),
                                  wl.block_table[wl.block_table >= 0], [0, 10 ** 6], wl.block_size, wl.num_tokens)
    assert np.array_equal(slots, wl.slot_mapping)
    assert np.array_equal(pos, np.concatenate([np.arange(c) for c in wl.context_lens]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_positions(interleaved):
    rng = np.random.default_rng(0)
    theta = OS.rope_theta(64, 10000.0)
    q, k = rng.standard_normal((2, 1, 1, 64))
    at = lambda x, p: OS.norm_rope(x, None, 0, 0, OS.rope_table([p], theta), interleaved)[0, 0]
    assert np.isclose(np.linalg.norm(at(q, 777)), np.linalg.norm(q))
    assert np.isclose(at(q, 900) @ at(k, 893), at(q, 7) @ at(k, 0))
    assert np.allclose(at(q, 0), q[0, 0])


def test_rotation_is_a_complex_product():
    x = np.arange(1.0, 5.0).reshape(1, 1, 4)
    t = OS.rope_table([3], np.array([0.5, 0.25]))
    z = np.array([1 + 2j, 3 + 4j]) * np.exp(1j * np.array([1.5, 0.75]))
    assert np.allclose(OS.norm_rope(x, None, 0, 0, t, True)[0, 0], [z[0].real, z[0].imag, z[1].real, z[1].imag])
    z = np.array([1 + 3j, 2 + 4j]) * np.exp(1j * np.array([1.5, 0.75]))
    assert np.allclose(OS.norm_rope(x, None, 0, 0, t, False)[0, 0], [z[0].real, z[1].real, z[0].imag, z[1].imag])


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(1).standard_normal((3, 2, 64)) * 40
    y = OS.norm_rope(x, np.zeros(64), 0.0, 1.0, None, False)
    assert np.allclose((y * y).mean(-1), 1.0)
    assert np.allclose(OS.norm_rope(x, np.full(64, 2.0), 0.0, 0.0, None, False), 2 * y)


def test_stretched_angles():
    plain = OS.rope_theta(128, 1e4)
    assert np.allclose(OS.rope_theta(128, 1e4, "linear", 4.0), plain / 4)
    ntk = OS.rope_theta(128, 1e4, "ntk", 4.0)
    assert ntk[0] == plain[0] and np.isclose(ntk[-1], plain[-1] / 4)  # the slowest pair slows by the factor
    for kind, low, high in (("yarn", 1.0, 32.0), ("bands", 1.0, 4.0)):
        th = OS.rope_theta(128, 1e4, kind, 8.0, 4096.0, low, high)
        turns = 4096 * plain / (2 * np.pi)
        fast, slow = turns > high * 1.3, turns < low / 1.3
        assert np.allclose(th[fast], plain[fast]) and np.allclose(th[slow], plain[slow] / 8)
        assert (th <= plain * (1 + 1e-12)).all() and (th >= plain / 8 * (1 - 1e-12)).all()


def test_visible_positions():
    assert OS.visible(4, 0, 0).tolist() == [0, 1, 2, 3, 4]
    assert OS.visible(9, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert OS.visible(3, 3, 2).tolist() == [0, 1, 2, 3]
    assert OS.visible(0, 1, 0).tolist() == [0] and OS.visible(-1, 4, 4).size == 0


@pytest.mark.parametrize("name", ["tiny_int8", "kvarn_131k", "llama8b_bf16"])
def test_attention_reduces_to_the_decode(name):
    wl = W.workload(name, num_seqs=2, ctx_lo=5, ctx_hi=40)
    o = OracleRun(wl)
    sm = float(OA.default_sm_scale(wl.head_dim))
    args = ((o.kc, o.km, o.vc, o.vm), wl.block_table, wl.context_lens, wl.block_size, wl.k_fmt, wl.v_fmt,
            o.k_scale, o.v_scale, sm)
    kw = dict(kvarn=wl.kvarn, signs=wl.signs)
    one, tol = OS.paged_attention(wl.query, [0, 1, 2], *args, **kw)
    assert np.allclose(one, o.decode(), atol=1e-6)
    assert (tol > 0).all() and np.median(tol) < 0.3
    # a window as long as the context hides nothing; rows of a chunk are decodes of shorter contexts
    assert np.allclose(OS.paged_attention(wl.query, [0, 1, 2], *args, window=40, **kw)[0], one)
    two, _ = OS.paged_attention(np.concatenate([wl.query[:1], wl.query]), [0, 2, 3], *args, **kw)
    short = wl.context_lens.copy()
    short[0] -= 1
    ref, _ = OS.paged_attention(wl.query, [0, 1, 2], args[0], wl.block_table, short, *args[3:], **kw)
    assert np.allclose(two[0], ref[0]) and np.allclose(two[1], one[0])
    # a window of one token alone: its value
    v = OA.dequant_sequence(o.vc, o.vm, wl.block_table[0], wl.context_lens[0], wl.block_size, 0, wl.v_fmt,
                            o.v_scale, wl.kvarn, wl.signs, wl.head_dim)
    last, _ = OS.paged_attention(wl.query, [0, 1, 2], *args, window=1, **kw)
    assert np.allclose(last[0, 0], v[-1], atol=1e-6)
