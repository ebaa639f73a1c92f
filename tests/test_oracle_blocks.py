"""Pins of the block-scaled oracle: page scales, codes and the dense attention."""
import numpy as np
import pytest

from oracle import blocks as B

FMTS = sorted(B.QMAX)


def bf16(x):
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def empty(nb=4, bs=8, hkv=2, d=64):
    return np.full((nb, bs, hkv, d), 0xFF, np.uint8), np.full((nb, 4), np.nan, np.float32)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_page_written_at_once_has_the_scale_of_its_largest_value(fmt):
    x = bf16(np.random.default_rng(0).standard_normal((8, 2, 64)))
    codes, scales = B.write(*empty(), x, np.arange(8, 16), fmt)
    assert (codes[[0, 2, 3]] == 0xFF).all() and np.isnan(scales[[0, 2, 3]]).all() and np.isnan(scales[1, 2:]).all()
    for h in range(2):
        assert scales[1, h] == np.float32(np.abs(x[:, h]).max()) / np.float32(B.QMAX[fmt])
        err = np.abs(B.rows(codes, scales, fmt, 1, np.arange(8))[:, h] - x[:, h])
        step = scales[1, h] * (1.0 if fmt == "int8_block" else np.maximum(np.abs(x[:, h] / scales[1, h]) * 2.0 ** -3, 2.0 ** -9))
        assert (err <= 0.5 * step * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_growth_is_by_powers_of_two_and_keeps_the_error_below_a_step(fmt):
    rng = np.random.default_rng(1)
    x = bf16(rng.standard_normal((8, 2, 64)) * 1.5 ** np.arange(8)[:, None, None])
    codes, scales = empty()
    last = None
    for t in range(8):
        B.write(codes, scales, x[t:t + 1], [t], fmt)
        s = scales[0, :2].copy()
        if last is not None:
            k = np.log2(s / last)
            assert (k == np.rint(k)).all() and (k >= 0).all()
            need = np.abs(x[t]).max(1) / B.QMAX[fmt]
            assert (s >= need * (1 - 1e-6)).all() and ((k == 0) | (s < 2 * need)).all()
        last = s
    got = B.rows(codes, scales, fmt, 0, np.arange(8))
    if fmt == "int8_block":
        assert (np.abs(got - x) <= scales[0, :2][None, :, None] * (1 + 1e-6)).all()
    else:
        assert (np.abs(got - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scales[0, :2][None, :, None] * 2.0 ** -9) * (1 + 1e-6)).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_zero_rows_and_values_not_finite(fmt):
    codes, scales = empty()
    B.write(codes, scales, np.zeros((2, 2, 64)), [0, 1], fmt)
    assert (scales[0, :2] == 0).all() and (B.rows(codes, scales, fmt, 0, [0, 1]) == 0).all()
    x = np.ones((1, 2, 64), np.float32)
    x[0, 0, :3] = [np.inf, -np.inf, np.nan]
    B.write(codes, scales, x, [2], fmt)  # the first scale of the page that says something
    assert (scales[0, :2] == np.float32(1) / np.float32(B.QMAX[fmt])).all()
    v = B.values(codes[0, 2], fmt)
    top = B.QMAX[fmt]
    assert v[0, 0] == top and v[0, 1] in (-top, -top - 1) and (v[1] == top).all()
    assert v[0, 2] == 0 if fmt == "int8_block" else np.isnan(v[0, 2])


def test_runs():
    assert B.runs([0, 1, 7, 8, -1, 9, 100, 3], 8, 4) == [(0, [0, 1, 2]), (1, [3, 5]), (0, [7])]


def test_dense_attention_is_the_definition():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, tol = B.attention(q, k, v, 0.3, first=2, window=2, sinks=1)
    for j, ids in enumerate(([0, 1, 2], [0, 2, 3], [0, 3, 4])):
        for h in range(4):
            e = np.exp(0.3 * k[ids, h // 2] @ q[j, h])
            np.testing.assert_allclose(out[j, h], e @ v[ids, h // 2] / e.sum(), rtol=1e-12)
    assert (tol > 0).all()
    assert (B.attention(q, k, v, 0.3, first=-5)[0] == 0).all()  # sees nothing
