"""Shared helpers for the block-scaled cache's tests: a cache on the GPU beside the
oracle's arrays."""
from __future__ import annotations

import numpy as np
import torch

from oracle import blocks as B
from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, garbage, ints

PAIRS = {"int8": ("int8_block", "int8_block"), "e4m3": ("fp8_e4m3_block", "fp8_e4m3_block"),
         "e4m3_int8": ("fp8_e4m3_block", "int8_block"), "int8_e4m3": ("int8_block", "fp8_e4m3_block")}


class Blocked:
    """A cache whose every byte is 0xFF (NaN scales) until it is written, in random pages;
    `store` writes rows to the cache and to the oracle's arrays alike."""

    def __init__(self, pair, lens, hkv, d, bs, seed=0, spare=3):
        self.k_fmt, self.v_fmt = PAIRS[pair]
        self.rng = np.random.default_rng(seed)
        self.lens, self.bs, self.d, self.hkv = np.asarray(lens), bs, d, hkv
        need = [-(-int(n) // bs) for n in lens]
        self.nb = sum(need) + spare
        perm, at = self.rng.permutation(self.nb), 0
        self.table = np.full((len(lens), max(need + [1]) + 1), 999999, np.int64)
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n]
            at += n
        self.cache = kvq.alloc_kv_cache(self.k_fmt, self.v_fmt, self.nb, bs, hkv, d, device=DEV, fill=0xFF)
        self.kc, self.vc = (np.full((self.nb, bs, hkv, d), 0xFF, np.uint8) for _ in range(2))
        self.ks, self.vs = (np.full((self.nb, kvq.scale_pitch(hkv)), 0xFFFFFFFF, np.uint32).view(np.float32) for _ in range(2))
        self.block_table, self.context_lens = ints(self.table), ints(self.lens)
        self.max_len = int(self.lens.max()) if len(lens) else 0

    def slots(self, s, positions):
        positions = np.asarray(positions, np.int64)
        return self.table[s, positions // self.bs] * self.bs + positions % self.bs

    def rows(self, n, scale=1.0):
        """bf16 keys and values [n, Hkv, D], sizes by row."""
        x = self.rng.standard_normal((2, n, self.hkv, self.d)) * np.asarray(scale)
        return tuple(torch.from_numpy(x[i].astype(np.float32)).to(DEV).to(torch.bfloat16) for i in range(2))

    def record(self, k, v, slots):
        for x, codes, scales, fmt in ((k, self.kc, self.ks, self.k_fmt), (v, self.vc, self.vs, self.v_fmt)):
            B.write(codes, scales, x.float().cpu().numpy(), slots, fmt)

    def store(self, k, v, slots):
        kvq.kvq_write_cache(self.cache, k, v, ints(np.asarray(slots), torch.int64))
        self.record(k, v, slots)

    def fill(self, scale=1.0):
        """Every sequence, in chunks of random sizes, rows of random sizes."""
        at = np.zeros(len(self.lens), np.int64)
        while (at < self.lens).any():
            new = np.minimum(self.rng.integers(0, 90, len(at)) + (self.rng.random(len(at)) < 0.5), self.lens - at)
            slots = np.concatenate([self.slots(s, np.arange(a, a + n)) for s, (a, n) in enumerate(zip(at, new))])
            if len(slots):
                size = np.exp(0.7 * self.rng.standard_normal((2, len(slots), self.hkv, 1))) * scale
                self.store(*self.rows(len(slots), size), slots)
            at += new

    def same(self):
        """Codes and scales bit for bit, the unwritten ones and the padding too."""
        c = self.cache
        for got, want in ((c.k_cache, self.kc), (c.v_cache, self.vc)):
            assert np.array_equal(got.cpu().numpy(), want)
        for got, want in ((c.k_meta, self.ks), (c.v_meta, self.vs)):
            assert np.array_equal(got.view(torch.int32).cpu().numpy().view(np.uint32), want.view(np.uint32))

    def sequence(self, s, n):
        """The first n keys and values of sequence s as numbers (pages outside the pool: 0)."""
        t = np.arange(n)
        pages = self.table[s, t // self.bs]
        ok = pages < self.nb
        out = []
        for codes, scales, fmt in ((self.kc, self.ks, self.k_fmt), (self.vc, self.vs, self.v_fmt)):
            x = B.rows(codes, scales, fmt, np.where(ok, pages, 0), t % self.bs)
            x[~ok] = 0.0
            out.append(x)
        return out

    def expect(self, query, cu, sm_scale, window=0, sinks=0, key=0.0):
        """Attention of each sequence's last rows.  Queries and probabilities are rounded to
        fp16 (2^-11), keys where `key` says so; probabilities below 2^-34 of the
        largest times the largest value of a tile are dropped."""
        q = query.double().cpu().numpy()
        out, tol = np.zeros(q.shape), np.full(q.shape, 1e-30)
        for s, n in enumerate(int(x) for x in self.lens):
            a, b = int(cu[s]), int(cu[s + 1])
            if a < b and n > 0:
                out[a:b], tol[a:b] = B.attention(q[a:b], *self.sequence(s, n), sm_scale, n - (b - a), window, sinks,
                                                 operand=2.0 ** -11, key=key, prob=2.0 ** -11, lost=2.0 ** -34)
        return out, tol

    def decode(self, q, out=None, window=0, sinks=0, num_ctas=0, sm=None, new=None):
        out = torch.full_like(q, 7.0) if out is None else out
        ws = garbage(kvq.kvq_decode_workspace_size(self.cache, len(self.lens), q.shape[1], self.max_len, num_ctas))
        args = (self.block_table, self.context_lens, self.max_len, self.d ** -0.5 if sm is None else sm)
        if window:
            k, v = new or (None, None)
            return kvq.kvq_decode_window(self.cache, q, out, *args, window, sinks, ws, num_ctas, k, v)
        if new:
            return kvq.kvq_decode_append(self.cache, *new, q, out, *args, ws, num_ctas)
        return kvq.kvq_paged_decode(self.cache, q, out, *args, ws, num_ctas)
