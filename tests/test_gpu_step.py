"""The operators together, as a serving loop runs them: plan a step, normalise, rotate
and store its tokens, attend to the cache; prompts first, then single tokens, then a
request that ends and one that joins.  Every token's key and value are kept on the side
and the whole attention is compared with the definition on them."""
from dataclasses import replace

import numpy as np
import pytest
import torch

from oracle import step as OS
from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, FORMATS, bits, garbage, ints

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, SEQS, WIDTH, POOL = 8, 2, 128, 16, 4, 40, 120


class Loop:
    """One layer of a server: its cache, tables and buffers, all made once."""

    def __init__(self, fmt, window, sinks, seed=0):
        kf, vf, kvarn = FORMATS[fmt]
        rng = np.random.default_rng(seed)
        self.g = torch.Generator(DEV).manual_seed(seed)
        signs = ints(rng.integers(0, 2, D) * 2 - 1, torch.int8) if kvarn else None
        scale = lambda f: 0.05 if f == "int8" else 1.0
        self.cache = kvq.alloc_kv_cache(kf, vf, POOL, BS, HKV, D, scale(kf), scale(vf), kvarn, signs, device=DEV, fill=0xFF)
        table = torch.empty((1024, D // 2, 2), device=DEV)
        kvq.kvq_rope_table(table, 10000.0, kvq.RopeScaling("bands", 4.0, 256, 1.0, 4.0))
        w = (1 + 0.1 * torch.randn((2, D), device=DEV, generator=self.g)).to(torch.bfloat16)
        self.rope = kvq.Rope(table, False, w[0], w[1])
        self.window, self.sinks = window, sinks
        self.block_table = torch.full((SEQS, WIDTH), -1, dtype=torch.int32, device=DEV)
        self.free = ints(rng.permutation(POOL))
        self.free_range, self.next_range = ints([0, POOL]), ints([0, 0])
        self.lens, self.next_lens = ints([0] * SEQS), ints([0] * SEQS)
        self.cu = ints([0] * (SEQS + 1))
        self.keys = [torch.empty((0, HKV, D), dtype=torch.float64) for _ in range(SEQS)]
        self.values = [torch.empty((0, HKV, D), dtype=torch.float64) for _ in range(SEQS)]

    def step(self, new):
        total = int(sum(new))
        pad = 5  # the packed buffers are longer than the tokens
        slots = torch.empty(total + pad, dtype=torch.int64, device=DEV)
        pos = torch.empty(total + pad, dtype=torch.int32, device=DEV)
        kvq.kvq_plan_step(self.lens, ints(new), self.block_table, self.free, self.free_range, BS, POOL, slots, pos,
                          self.next_lens, self.cu, self.next_range)
        self.lens, self.next_lens = self.next_lens, self.lens
        self.free_range, self.next_range = self.next_range, self.free_range
        qkv = torch.randn((total + pad, (HQ + 2 * HKV) * D), device=DEV, generator=self.g).to(torch.bfloat16)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        query = torch.empty((total + pad, HQ, D), dtype=torch.bfloat16, device=DEV)
        kvq.kvq_norm_rope_write(self.rope, self.cache, q, k, v, pos, slots, query)
        lens = self.lens.tolist()
        n, most = max(lens), max(new)
        out = torch.full_like(query, 3.0)
        ws = garbage(kvq.kvq_prefill_workspace_size(self.cache, SEQS, HQ, total + pad, most, n))
        kvq.kvq_paged_prefill(self.cache, query, out, self.cu, self.block_table, self.lens, most, n, D ** -0.5,
                              self.window, self.sinks, ws)
        assert (out[total:] == 3.0).all()
        # the tokens on the side, from the projection alone
        t = pos.long()
        for x, w, kept in ((k, self.rope.k_weight, self.keys), (v, None, self.values)):
            rows = self.rope.table[t].cpu().numpy() if w is not None else None
            y = OS.norm_rope(x.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), 1e-6, 0.0, rows, False)
            at = 0
            for s, c in enumerate(new):
                kept[s] = torch.cat([kept[s], torch.from_numpy(y[at:at + c])])
                at += c
        return query[:total], out[:total], new

    def reference(self, query, new):
        q = query.double().cpu()
        ref = torch.zeros(q.shape, dtype=torch.float64)
        at = 0
        for s, c in enumerate(new):
            n = self.keys[s].shape[0]
            for j in range(c):
                t = torch.from_numpy(OS.visible(n - c + j, self.window, self.sinks))
                k, v = self.keys[s][t].repeat_interleave(HQ // HKV, 1), self.values[s][t].repeat_interleave(HQ // HKV, 1)
                p = torch.softmax(torch.einsum("hd,thd->ht", q[at + j], k) * D ** -0.5, -1)
                ref[at + j] = torch.einsum("ht,thd->hd", p, v)
            at += c
        return ref


# how far a quantized cache may take the output: the mean over everything, in units of the
# values' deviation 1 (a code step is at most 5 / 127 for int8, 2^-3 of a value for e4m3
# keys, an eighth of a row's range for 4 bits; they average over hundreds of tokens)
MEAN = {"bf16": 2e-3, "int8": 1e-2, "e4m3_int8": 3e-2, "kvarn": 6e-2, "uint8": 1e-2}


@pytest.mark.parametrize("fmt", sorted(MEAN))
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_a_serving_loop(fmt, window, sinks):
    loop = Loop(fmt, window, sinks)
    steps = [[200, 37, 0, 129], [1, 1, 64, 1], [1, 1, 1, 1], [3, 1, 200, 1]] + [[1, 1, 1, 1]] * 3
    for i, new in enumerate(steps):
        if i == 3:  # request 1 has ended: its pages stay with it, its row is used anew
            loop.lens[1] = 0
            loop.block_table[1].fill_(-1)
            loop.keys[1], loop.values[1] = loop.keys[1][:0], loop.values[1][:0]
        query, out, _ = loop.step(new)
        err = (out.double().cpu() - loop.reference(query, new)).abs()
        assert torch.isfinite(err).all()
        assert err.mean() <= MEAN[fmt], f"step {i}: {err.mean():.2e}"
    assert loop.free_range.tolist()[0] == sum(-(-n // BS) for n in loop.lens.tolist()) + 3  # and request 1's first three
    assert kvq.kvq_get_device_error() == 0
    # the single tokens of the last step through the decode: the same rows
    one = torch.empty_like(query)
    ws = garbage(kvq.kvq_decode_workspace_size(loop.cache, SEQS, HQ, 600))
    if window:
        kvq.kvq_decode_window(loop.cache, query, one, loop.block_table, loop.lens, 600, D ** -0.5, window, sinks, ws)
    else:
        kvq.kvq_paged_decode(loop.cache, query, one, loop.block_table, loop.lens, 600, D ** -0.5, ws)
    assert (one.double() - out.double()).abs().max() <= 4e-2
    assert (one.double() - out.double()).abs().mean() <= 2e-3


def test_two_captured_steps_share_nothing():
    """Two steps' calls captured into graphs of their own, each with its workspace, replayed in turn."""
    loops = [Loop("int8", 64, 3, seed=i) for i in range(2)]
    runs = []
    for loop in loops:
        loop.step([150, 20, 3, 70])
        q = torch.randn((SEQS, HQ, D), device=DEV, generator=loop.g).to(torch.bfloat16)
        out, one = torch.empty_like(q), torch.empty_like(q)
        cu = ints([0, 1, 2, 3, 4])
        ws = [garbage(kvq.kvq_prefill_workspace_size(loop.cache, SEQS, HQ, SEQS, 1, 150)),
              garbage(kvq.kvq_decode_workspace_size(loop.cache, SEQS, HQ, 150))]

        def run(loop=loop, q=q, out=out, one=one, cu=cu, ws=ws):
            kvq.kvq_paged_prefill(loop.cache, q, out, cu, loop.block_table, loop.lens, 1, 150, 0.1, 64, 3, ws[0])
            kvq.kvq_decode_window(loop.cache, q, one, loop.block_table, loop.lens, 150, 0.1, 64, 3, ws[1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run()
        runs.append((run, g, q, out, one))
    for turn in range(3):
        for run, g, q, out, one in runs:
            q.copy_(torch.randn(q.shape, device=DEV).to(torch.bfloat16))
        for _, g, *_ in runs:
            g.replay()
        torch.cuda.synchronize()
        for run, g, q, out, one in runs:
            a, b = out.clone(), one.clone()
            run()
            torch.cuda.synchronize()
            assert torch.equal(bits(a), bits(out)) and torch.equal(bits(b), bits(one))
            assert (a.double() - b.double()).abs().max() <= 4e-2


def test_blocks_past_32_bits():
    """The same tokens in the first blocks of a pool and in blocks beyond 4 GiB: same bits."""
    bs, hkv, d, nb = 128, 8, 128, 34000  # 131,072 bytes a block and tensor: 4.46 GB each
    cache = kvq.KVCache("int8", "int8", hkv, d, bs, nb, torch.empty((nb, bs, hkv, d), dtype=torch.uint8, device=DEV),
                        torch.empty((nb, bs, hkv, d), dtype=torch.uint8, device=DEV), k_scale=0.04, v_scale=0.04)
    n = 700
    g = torch.Generator(DEV).manual_seed(1)
    q, k, v = (torch.randn((n, h, d), device=DEV, generator=g).to(torch.bfloat16) for h in (32, hkv, hkv))
    rope = kvq.Rope(None)
    pos, query = ints(np.arange(n)), torch.empty_like(q)
    pages = -(-n // bs)
    found = []
    for first in (0, nb - pages):
        free = ints(np.arange(first, first + pages))
        table, slots = torch.full((1, pages), -1, dtype=torch.int32, device=DEV), torch.empty(n, dtype=torch.int64, device=DEV)
        lens, cu, rng = ints([0]), ints([0, 0]), ints([0, 0])
        at = torch.empty(n, dtype=torch.int32, device=DEV)
        kvq.kvq_plan_step(ints([0]), ints([n]), table, free, ints([0, pages]), bs, nb, slots, at, lens, cu, rng)
        assert slots[0] == first * bs and torch.equal(at, pos)
        kvq.kvq_norm_rope_write(rope, cache, q, k, v, pos, slots, query)
        assert torch.equal(bits(query), bits(q))
        outs = []
        for rows in (n, 40, 1):  # dequantized ahead, by each CTA, and one token through the decode
            sub, out = query[n - rows:].contiguous(), torch.empty((rows, 32, d), dtype=torch.bfloat16, device=DEV)
            ws = garbage(kvq.kvq_prefill_workspace_size(cache, 1, 32, rows, rows, n))
            outs.append(kvq.kvq_paged_prefill(cache, sub, out, ints([0, rows]), table, lens, rows, n, d ** -0.5, 300, 7, ws))
        ws = garbage(kvq.kvq_decode_workspace_size(cache, 1, 32, n))
        one = query[n - 1:].contiguous()
        outs.append(kvq.kvq_decode_window(cache, one, torch.empty_like(one), table, lens, n, d ** -0.5, 300, 7, ws))
        found.append([bits(o) for o in outs])
    assert all(torch.equal(a, b) for a, b in zip(*found))
    assert kvq.kvq_get_device_error() == 0


def test_the_binding_refuses_wrong_tensors():
    loop = Loop("int8", 0, 0)
    loop.step([20, 1, 1, 1])
    q = torch.zeros((SEQS, HQ, D), dtype=torch.bfloat16, device=DEV)
    ws = garbage(1 << 22)
    good = dict(query=q, out=torch.empty_like(q), block_table=loop.block_table, context_lens=loop.lens)
    call = lambda **kw: kvq.kvq_decode_window(loop.cache, **{**good, **kw}, max_context_len=20, sm_scale=0.1, window=5,
                                              workspace=ws)
    call()
    for kw in (dict(query=q.float()), dict(query=q.cpu()), dict(out=q[:, ::2]), dict(query=q[:, :, :64]),
               dict(block_table=loop.block_table.long()), dict(block_table=loop.block_table[:, ::2]),
               dict(context_lens=loop.lens[:2]), dict(new_key=q[:, :HKV])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(kvq.KvqError):  # a head ratio above 8
        big = torch.zeros((SEQS, 32, D), dtype=torch.bfloat16, device=DEV)
        call(query=big, out=torch.empty_like(big))
    rope = loop.rope
    k = torch.zeros((3, HKV, D), dtype=torch.bfloat16, device=DEV)
    for args in ((q[:3], k, ints([0, 1])), (q[:3], k[:2], ints([0, 1, 2])), (q[:3].transpose(0, 1), k, ints([0, 1, 2])),
                 (q[:3], k, torch.zeros(3, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            kvq.kvq_norm_rope(rope, *args, torch.empty_like(q[:3]), torch.empty_like(k))
    with pytest.raises(kvq.KvqError):  # an output over another input
        kvq.kvq_norm_rope(rope, q[:3], k, ints([0, 1, 2]), torch.empty_like(q[:3]), q[:3, :HKV])


@pytest.mark.parametrize("fmt", ["int8", "kvarn"])
def test_the_binding_refuses_caches_that_do_not_fit(fmt):
    """A cache with a tensor elsewhere, of another type or too small reaches no kernel."""
    loop = Loop(fmt, 0, 0)
    loop.step([20, 1, 1, 1])
    q = torch.zeros((SEQS, HQ, D), dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros((SEQS, HKV, D), dtype=torch.bfloat16, device=DEV)
    out, ws, pos = torch.empty_like(q), garbage(1 << 22), ints([0, 1, 2, 3])
    calls = (lambda c: kvq.kvq_decode_window(c, q, out, loop.block_table, loop.lens, 20, 0.1, 5, workspace=ws),
             lambda c: kvq.kvq_paged_prefill(c, q, out, ints([0, 1, 2, 3, 4]), loop.block_table, loop.lens, 1, 20, 0.1, workspace=ws),
             lambda c: kvq.kvq_norm_rope_write(loop.rope, c, q, kv, kv, pos, ints([0, 1, 2, 3], torch.int64), out))
    for call in calls:
        call(loop.cache)
    torch.cuda.synchronize()
    bad = [dict(k_cache=loop.cache.k_cache.cpu()), dict(v_cache=loop.cache.v_cache.float()),
           dict(k_cache=loop.cache.k_cache[:1]), dict(num_blocks=loop.cache.num_blocks + 1),
           dict(v_cache=loop.cache.v_cache.transpose(1, 2))]
    if loop.cache.k_meta is not None:
        bad += [dict(k_meta=None), dict(v_meta=loop.cache.v_meta.float()), dict(signs=loop.cache.signs.cpu())]
    for kw in bad:
        for call in calls:
            with pytest.raises(ValueError):
                call(replace(loop.cache, **kw))
    for call in calls:
        call(loop.cache)
    assert kvq.kvq_get_device_error() == 0
