"""Shared helpers for the serving-step tests: caches of given lengths on the GPU
and as numpy, and the comparison with the oracle's bound."""
from __future__ import annotations

import numpy as np
import torch

from oracle import step as OS
from quantized_paged_kv_kvq_gb300 import kvq

FORMATS = {  # k, v, KVarN
    "int8": ("int8", "int8", False),
    "e4m3_int8": ("fp8_e4m3", "int8", False),
    "e5m2": ("fp8_e5m2", "fp8_e5m2", False),
    "int4": ("int4_asym", "int4_asym", False),
    "uint8": ("uint8_asym", "uint8_asym", False),
    "kvarn": ("int4_asym", "uint8_asym", True),
    "bf16": ("bf16", "bf16", False),
}
DEV = "cuda"


def ints(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), device=DEV).to(dtype)


def bits(t):
    """A bf16 or fp16 tensor's bits, for exact comparison."""
    return t.contiguous().view(torch.int16)


class Paged:
    """A cache holding `lens` tokens per sequence, in random pages; every other byte,
    code or field, is 0xFF (NaN in the floating formats).  Pages of positions that
    `keep(s, t)` rejects are taken out of the block table (entry 999999)."""

    def __init__(self, fmt, lens, hkv, d, bs, seed=0, head_scales=False, keep=None, spare=3, k_std=1.0):
        self.k_fmt, self.v_fmt, self.kvarn = FORMATS[fmt]
        rng = np.random.default_rng(seed)
        self.lens, self.bs, self.d, self.hkv = np.asarray(lens), bs, d, hkv
        need = [-(-int(n) // bs) for n in lens]
        nb = sum(need) + spare
        perm = rng.permutation(nb)
        self.table = np.full((len(lens), max(need + [1]) + 1), 999999, np.int64)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n]
            at += n
        signs = rng.integers(0, 2, d) * 2 - 1
        self.signs = signs.astype(np.int8) if self.kvarn else None
        scale = lambda f: 4.5 / 127 if f == "int8" else 1.0
        self.cache = kvq.alloc_kv_cache(self.k_fmt, self.v_fmt, nb, bs, hkv, d, scale(self.k_fmt),
                                        scale(self.v_fmt), self.kvarn,
                                        None if self.signs is None else ints(self.signs, torch.int8),
                                        device=DEV, fill=0xFF)
        self.k_scale, self.v_scale = np.float32(scale(self.k_fmt)), np.float32(scale(self.v_fmt))
        if head_scales and self.k_fmt in ("int8", "fp8_e4m3", "fp8_e5m2"):
            self.k_scale = (self.k_scale * (0.5 + rng.random(hkv))).astype(np.float32)
            self.v_scale = (self.v_scale * (0.5 + rng.random(hkv))).astype(np.float32)
            self.cache.k_head_scales = torch.from_numpy(self.k_scale).to(DEV)
            self.cache.v_head_scales = torch.from_numpy(self.v_scale).to(DEV)
        slots = [self.table[s, t // bs] * bs + t % bs for s, n in enumerate(lens) for t in range(int(n))]
        t = len(slots)
        if t:
            rows = rng.standard_normal((2, t, hkv, d)).astype(np.float32)
            rows[0] *= k_std
            k, v = (torch.from_numpy(x).to(DEV).to(torch.bfloat16) for x in rows)
            kvq.kvq_write_cache(self.cache, k, v, ints(np.array(slots), torch.int64))
        if keep is not None:
            for s, n in enumerate(lens):
                pages = {t // bs for t in range(int(n)) if keep(s, t)}
                for page in range(need[s]):
                    if page not in pages:
                        self.table[s, page] = 999999
        self.block_table, self.context_lens = ints(self.table), ints(self.lens)
        self.max_len = int(self.lens.max()) if len(lens) else 0

    def numpy(self):
        c = self.cache
        meta = lambda m, codes: (np.zeros((codes.shape[0], c.num_kv_heads, 0, c.block_size), np.uint16) if m is None
                                 else m.view(torch.int16).cpu().numpy().view(np.uint16))
        kc, vc = c.k_cache.cpu().numpy(), c.v_cache.cpu().numpy()
        return kc, meta(c.k_meta, kc), vc, meta(c.v_meta, vc)

    def expect(self, query, cu, sm_scale, window=0, sinks=0):
        return OS.paged_attention(query.double().cpu().numpy(), cu, self.numpy(), self.table, self.lens, self.bs,
                                  self.k_fmt, self.v_fmt, self.k_scale, self.v_scale, sm_scale, window, sinks,
                                  self.kvarn, self.signs)


def random_query(n, hq, d, seed=1):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn((n, hq, d), device=DEV, generator=g).to(torch.bfloat16)


def garbage(nbytes):
    """A workspace whose contents mean nothing."""
    ws = torch.empty(max(nbytes, 16) // 4 + 4, dtype=torch.float32, device=DEV)
    ws.view(torch.int32).random_()
    return ws


def check_close(out, ref, tol, what=""):
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)) if got.size else 0.0
    mean = np.abs(got - ref).mean() if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"
    assert mean <= 2e-3, f"{what}: mean error {mean:.2e}"
