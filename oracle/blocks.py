"""Oracle: 8-bit codes with a scale per (page, kv-head), and attention of rows that
are at hand as numbers (test infrastructure only).

The store is the definition in include/kvq.h, page by page and head by head, in float32
where it decides a code or a scale (one IEEE operation a step); attention is float64.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from .step import visible

F32 = np.float32
QMAX = {"int8_block": 127, "fp8_e4m3_block": 448}
CODE = {"int8_block": "int8", "fp8_e4m3_block": "fp8_e4m3"}


def values(codes, fmt):
    """The numbers that codes stand for, float64."""
    return F.dequant_sym(codes, CODE[fmt], 1.0)


def encode(x, fmt):
    """Float32 values to codes."""
    x = np.asarray(x, F32)
    if fmt == "int8_block":
        return F.quant_int8(np.where(np.isnan(x), F32(0), x), F32(1))
    return F.quant_fp8(x, F32(1), "fp8_e4m3")


def runs(slots, block_size, num_blocks):
    """(page, tokens) of what consecutive tokens put into one page; skipped ones do not part them."""
    found, last = [], None
    for t, slot in enumerate(int(s) for s in slots):
        if not 0 <= slot < num_blocks * block_size:
            continue
        page = slot // block_size
        if page == last:
            found[-1][1].append(t)
        else:
            found.append((page, [t]))
        last = page
    return found


def page_scale(rows, old, begun, fmt):
    """(scale, k) of one head's rows [n, D]: k doublings of the old scale."""
    finite = np.abs(rows[np.isfinite(rows)])
    most = F32(finite.max()) if finite.size else F32(0)
    need = F32(0) if most == 0 else max(F32(most / F32(QMAX[fmt])), F32(2.0 ** -126))
    if begun or not (2.0 ** -126 <= old < np.inf):
        return need, 0
    k = 0
    while F32(old) * F32(2.0) ** k < need:
        k += 1
    return F32(np.ldexp(F32(old), k)), k


def write(codes, scales, x, slots, fmt):
    """Store x [T, Hkv, D] (float32 of bf16 values) into codes [NB, bs, Hkv, D] and scales
    [NB, P], in place."""
    x = np.asarray(x, F32)
    nb, bs, hkv, _ = codes.shape
    for page, tokens in runs(slots, bs, nb):
        offsets = [int(slots[t]) % bs for t in tokens]
        front = min(offsets)
        for h in range(hkv):
            scale, k = page_scale(x[tokens, h], scales[page, h], front == 0, fmt)
            if k > 0:
                codes[page, :front, h] = encode(values(codes[page, :front, h], fmt) * 2.0 ** -k, fmt)
            scales[page, h] = scale
            with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                inv = F32(1) / F32(scale) if scale > 0 else F32(0)
                codes[page, offsets, h] = encode(x[tokens, h] * inv, fmt)
    return codes, scales


def rows(codes, scales, fmt, pages, offsets):
    """Rows [n, Hkv, D] as numbers."""
    hkv = codes.shape[2]
    return values(codes[pages, offsets], fmt) * scales[pages, :hkv].astype(np.float64)[..., None]


def attention(query, keys, vals, sm_scale, first=0, window=0, sinks=0, operand=0.0, key=0.0, prob=2.0 ** -8, lost=0.0):
    """out [q, Hq, D] of queries at positions first, first + 1, ... over keys, vals
    [n, Hkv, D] at 0, 1, ..., and per element a bound on what rounding may change of it:

      * a query and a key element rounded to within `operand` and `key` of themselves: a
        logit moves by 8 (operand + key) sm_scale sqrt(sum_d (q_d k_d)^2) (roundings of
        different elements count as independent, at eight times their root of summed
        squares); the D products and additions of float32 by 2^-23 D of the same; 2^-18
        for the exponential;
      * logits that move by at most e change out by at most (e^(2e) - 1) sum_t p_t |v_t - out|;
      * a probability (times its value's scale) rounded to within `prob` of itself, and,
        of quantized formats, partial results in fp16: 8 * prob (3 of those where operand > 0)
        sqrt(sum_t (p_t v_t)^2); `lost` for each key of the largest |v_t|, where 16 bits
        drop small ones; the sums over n positions 2^-23 n sum_t p_t |v_t|;
      * the output's own rounding to bf16: 2^-8 of it.
    """
    query, keys, vals = (np.asarray(x, np.float64) for x in (query, keys, vals))
    nq, hq, d = query.shape
    g = hq // keys.shape[1]
    out, tol = np.zeros(query.shape), np.full(query.shape, 1e-30)
    seen = np.zeros((nq, keys.shape[0]), bool)
    for j in range(nq):
        seen[j, visible(first + j, window, sinks)] = True
    some = seen.any(1)
    for h in range(hq if nq else 0):
        k, v, q = keys[:, h // g], vals[:, h // g], query[:, h]
        logit = np.where(seen, sm_scale * (q @ k.T), -np.inf)
        p = np.exp(logit - np.where(some, logit.max(1), 0.0)[:, None])
        p /= np.where(some, p.sum(1), 1.0)[:, None]
        o = p @ v
        e = np.sqrt(np.where(seen, (q * q) @ (k * k).T, 0.0)).max(1)
        e = (abs(sm_scale) * (8 * (operand + key) + d * 2.0 ** -23) * e + 2.0 ** -18)[:, None]
        spread = p @ np.abs(v) + np.abs(o)  # >= sum_t p_t |v_t - out|
        n = seen.sum(1)[:, None]
        out[:, h] = o
        tol[:, h] += np.expm1(2 * e) * spread + (24 if operand else 8) * prob * np.sqrt((p * p) @ (v * v)) \
            + n * lost * np.abs(v).max() + n * 2.0 ** -23 * (p @ np.abs(v)) + 2.0 ** -8 * np.abs(o)
    return out, tol
