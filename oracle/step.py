"""Oracle: the rest of a serving step in float64 (test infrastructure only).

Block tables, slots and positions from request lengths; rotation tables; norm
and rotation of query and key heads; and attention of any number of new tokens
per sequence to the dequantized cache, causal, through a window with kept first
tokens.  Each function is the definition in include/kvq.h written out request by
request, row by row.
"""
from __future__ import annotations

import math

import numpy as np

from . import formats as F
from .attention import dequant_sequence
from .hadamard import rotate_f32


def plan_step(context_lens, new_lens, block_table, free_blocks, free_range, block_size, max_tokens):
    """(slots, positions, context lengths after, cu, block table, free range) of valid inputs;
    a page for which no free block is left gets -1, its tokens slot -1."""
    table = np.array(block_table, np.int32)
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.zeros(max_tokens, np.int32)
    nxt, end = int(free_range[0]), int(free_range[1])
    cu = [0]
    for s, (old, new) in enumerate(zip(context_lens, new_lens)):
        for page in range(-(-int(old) // block_size), -(-int(old + new) // block_size)):
            table[s, page] = free_blocks[nxt] if nxt < end else -1
            nxt = min(nxt + 1, end)
        for j in range(int(new)):
            t, pos = cu[-1] + j, int(old) + j
            if t < max_tokens:
                b = int(table[s, pos // block_size])
                positions[t] = pos
                slots[t] = b * block_size + pos % block_size if b >= 0 else -1
        cu.append(cu[-1] + int(new))
    after = np.asarray(context_lens, np.int32) + np.asarray(new_lens, np.int32)
    return slots, positions, after, np.array(cu, np.int32), table, np.array([nxt, end], np.int32)


def rope_theta(rot_dim, base, kind="none", factor=1.0, original_len=1.0, low=1.0, high=2.0):
    """Angle per position of every pair [rot_dim / 2]."""
    out = []
    for i in range(rot_dim // 2):
        if kind == "ntk":
            theta = (base * factor ** (rot_dim / (rot_dim - 2))) ** (-2 * i / rot_dim)
        else:
            theta = base ** (-2 * i / rot_dim)
        if kind == "linear":
            theta /= factor
        elif kind == "yarn":
            d = lambda x: rot_dim * math.log(original_len / (2 * math.pi * x)) / (2 * math.log(base))
            a, b = max(math.floor(d(high)), 0), min(math.ceil(d(low)), rot_dim - 1)
            g = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            theta = theta * (1 - g) + theta / factor * g
        elif kind == "bands":
            h = min(max((original_len * theta / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            theta = theta * h + theta / factor * (1 - h)
        out.append(theta)
    return np.array(out)


def rope_table(positions, theta, amplitude=1.0):
    """[len(positions), pairs, 2] of (cos, sin)."""
    angle = np.asarray(positions, np.float64)[:, None] * theta
    return amplitude * np.stack((np.cos(angle), np.sin(angle)), -1)


def norm_rope(x, weight, eps, offset, table_rows, interleaved):
    """x [T, H, D] normalised over D (weight None: not) and turned by table_rows
    [T, r/2, 2] (None: not), in float64."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)
    if table_rows is not None:
        pairs = table_rows.shape[1]
        for i in range(pairs):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
            c, s = table_rows[:, None, i, 0].astype(np.float64), table_rows[:, None, i, 1].astype(np.float64)
            ya, yb = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
            y[..., a], y[..., b] = ya, yb
    return y


def visible(p, window, sinks):
    """Positions that the query at position p sees (window 0: every earlier one)."""
    if p < 0:
        return np.zeros(0, np.int64)
    first = max(0, p - window + 1) if window else 0
    return np.concatenate([np.arange(min(sinks, first)), np.arange(first, p + 1)]).astype(np.int64)


def paged_attention(query, cu, cache, block_table, context_lens, block_size, k_fmt, v_fmt, k_scale,
                    v_scale, sm_scale, window=0, sinks=0, kvarn=False, signs=None, gather_lens=None):
    """out [T, Hq, D] and per element a bound on what 16-bit operands and float32
    sums may change of it.

    cache: (k codes, k meta, v codes, v meta).  The bound, with u = 2^-11 for
    quantized formats (fp16 operands) and 2^-8 for the 16-bit cache (bf16, exact
    but for the probabilities); roundings of different elements count as
    independent, at eight times their root of summed squares:
      * the query, and a key row once dequantized, rounded to fp16: a logit moves
        by 8 * 2u * sm_scale * sqrt(sum_d (q_d k_d)^2), where rotated rows (KVarN)
        have sqrt(sum_d (q'_d k'_d)^2) <= max_d |q'_d| |k|; the D products and
        additions of a dot product by 2^-23 D of the same; 2^-18 for the exponential;
      * logits that move by at most e change out by at most (e^(2e) - 1) sum_t p_t |v_t - out|;
      * a probability and a value row rounded, and partial results: 8 * 3u *
        sqrt(sum_t (p_t a_t)^2), a_t = |v_t| or, of an asymmetric row, its parts
        |code * scale| + |zero point|, and for rotated rows the largest element
        4 |v| / sqrt(D) counts; the sums over n positions 2^-23 n sum_t p_t a_t;
      * the output's own rounding to bf16: 2^-8 of it.
    """
    query = np.asarray(query, np.float64)
    hq, d = query.shape[1:]
    kc, km, vc, vm = cache
    hkv = kc.shape[2]
    g = hq // hkv
    out = np.zeros(query.shape)
    tol = np.zeros(query.shape)
    u = 2.0 ** -8 if k_fmt == "bf16" else 2.0 ** -11
    uq = (0.0 if k_fmt == "bf16" else 8 * 2 * u) + d * 2.0 ** -23
    head = lambda sc, h: sc[h] if np.ndim(sc) == 1 else sc

    def parts(ids, row, h, values):
        """a_t of the value rows."""
        if not v_fmt.endswith("asym"):
            return np.abs(values)
        blk, off = row[ids // block_size], ids % block_size
        c, m = vc[blk, off, h], vm[blk, h, :, off]
        f = [F.F16.decode(m[:, i])[:, None] for i in range(m.shape[1])]
        a = np.abs((F.unpack_int4(c) if v_fmt == "int4_asym" else c) * f[0]) + np.abs(f[1])
        if kvarn:
            a = np.broadcast_to(4 * np.linalg.norm(a * np.abs(f[2]), axis=1, keepdims=True) / np.sqrt(d), a.shape)
        return a

    for s in range(len(context_lens)):
        n, q0, q1 = int(context_lens[s]), int(cu[s]), int(cu[s + 1])
        if q1 == q0 or n <= 0:
            continue
        # only positions that some row sees are read: the others' pages may be gone
        seen = np.unique(np.concatenate([visible(n - (q1 - q0) + j, window, sinks) for j in range(q1 - q0)]))
        row = np.zeros(-(-n // block_size) or 1, np.int64)
        pages = np.unique(seen // block_size)
        row[pages] = np.asarray(block_table)[s, pages]
        for h in range(hkv):
            k = np.zeros((n, d))
            v = np.zeros((n, d))
            va = np.zeros((n, d))
            for codes, meta, fmt, scale, to in ((kc, km, k_fmt, k_scale, k), (vc, vm, v_fmt, v_scale, v)):
                full = dequant_sequence(codes, meta, row, n, block_size, h, fmt, head(scale, h), kvarn, signs, d)
                to[seen] = full[seen]
            va[seen] = parts(seen, row, h, v[seen])
            for j in range(q1 - q0):
                t = visible(n - (q1 - q0) + j, window, sinks)
                if not t.size:
                    continue
                x = query[q0 + j, h * g:(h + 1) * g]
                logit = sm_scale * (x @ k[t].T)
                p = np.exp(logit - logit.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                o = p @ v[t]
                if kvarn:
                    e = np.abs(rotate_f32(x, signs)).max(1) * np.linalg.norm(k[t], axis=1).max()
                else:
                    e = np.sqrt((x * x) @ (k[t] * k[t]).T).max(1)
                e = (sm_scale * uq * e + 2.0 ** -18)[:, None]
                spread = np.stack([r @ np.abs(v[t] - m) for r, m in zip(p, o)])
                out[q0 + j, h * g:(h + 1) * g] = o
                tol[q0 + j, h * g:(h + 1) * g] = np.expm1(2 * e) * spread \
                    + 24 * u * np.sqrt((p * p) @ (va[t] * va[t])) + t.size * 2.0 ** -23 * (p @ va[t]) \
                    + 2.0 ** -8 * np.abs(o) + 1e-30
    return out, tol
