"""Prompts and block-scaled pages, as cases to measure.

A prompt's queries, keys and values are all at hand in 16 bits, so its
attention needs no cache.  A cache of 8-bit codes with one scale for each page
and kv-head is written run by run (a page that is begun takes the scale of its
rows, one that goes on grows its scale by a power of two where a new row asks
for it), attended to by single tokens and by chunks, and read back to 16 bits,
as is a cache of any other format.

`run` computes an operator with elementary torch operations in float32
(`own` false) or calls the library (`own` true); `exact` computes it in
float64.  The float32 and float64 forms share nothing but the inputs.
"""
import math
import random

import numpy as np
import torch

own = False

CUDA = "cuda"
# (query heads, kv-heads, head_dim) of the bench's workloads, multi-head attention, odd groups
SHAPES = ((32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 16, 128), (24, 8, 64), (7, 1, 128), (20, 4, 64))
CACHES = (("int8", "int8", False), ("fp8_e4m3", "int8", False), ("fp8_e5m2", "fp8_e5m2", False),
          ("int4_asym", "int4_asym", False), ("uint8_asym", "uint8_asym", False),
          ("int4_asym", "uint8_asym", True), ("bf16", "bf16", False))
BLOCKED = (("int8_block", "int8_block"), ("fp8_e4m3_block", "fp8_e4m3_block"),
           ("fp8_e4m3_block", "int8_block"))
SMALLEST = 2.0 ** -126  # of a page's scale
MOST = 64 * 16384 ** 2  # scores of the largest listed prompt


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    c8b = dict(hq=32, hkv=8, d=128)
    return [
        # one short question: latency
        dict(name="prompt_short", op="prompt", seqs=1, lo=333, hi=333, window=0, sinks=0, layout=1, **c8b),
        # a batch of prompts of very different lengths, packed
        dict(name="prompt_packed", op="prompt", seqs=16, lo=1, hi=4096, window=0, sinks=0, layout=2, **c8b),
        # one long document, 64 query heads: the compute-bound end
        dict(name="prompt_long", op="prompt", seqs=1, lo=16384, hi=16384, hq=64, hkv=8, d=128, window=0,
             sinks=0, layout=3),
        # narrow heads in groups of three through a window behind kept first tokens
        dict(name="prompt_window", op="prompt", seqs=6, lo=1, hi=7001, hq=24, hkv=8, d=64, window=1024, sinks=4,
             layout=4),
        # a decode step's new rows: one token of each request, somewhere in its page
        dict(name="write_step", op="write", seqs=64, lo=256, hi=4096, new_lo=1, new_hi=1, bs=16,
             k="int8_block", v="int8_block", layout=5, hkv=8, d=128),
        # a step of prompt chunks behind what is cached already
        dict(name="write_chunks", op="write", seqs=24, lo=0, hi=2048, new_lo=1, new_hi=1365, bs=16,
             k="fp8_e4m3_block", v="fp8_e4m3_block", layout=6, hkv=8, d=128),
        # large pages of narrow heads
        dict(name="write_large_pages", op="write", seqs=3, lo=0, hi=999, new_lo=8191, new_hi=8191, bs=128,
             k="fp8_e4m3_block", v="int8_block", layout=7, hkv=2, d=64),
        # decode of a full batch, one scale for each page and head
        dict(name="block_decode", op="attend", seqs=64, bs=16, k="int8_block", v="int8_block", lo=256, hi=4096,
             q_lo=1, q_hi=1, window=0, sinks=0, chunk=False, layout=8, **c8b),
        # few long requests, large pages, a window over most of them
        dict(name="block_decode_long", op="attend", seqs=12, bs=64, k="fp8_e4m3_block", v="fp8_e4m3_block",
             lo=4096, hi=32768, q_lo=1, q_hi=1, window=20000, sinks=4, chunk=False, layout=9, hq=64, hkv=8, d=128),
        # chunks of prompts on what their requests have cached
        dict(name="block_chunks", op="attend", seqs=8, bs=32, k="fp8_e4m3_block", v="int8_block", lo=0, hi=4096,
             q_lo=1, q_hi=777, window=0, sinks=0, chunk=True, layout=10, **c8b),
        # one request's context brought back to 16 bits, to be moved or attended to densely
        dict(name="read_request", op="read", tokens=2049, bs=16, k="int8_block", v="int8_block", kvarn=False,
             layout=11, hkv=8, d=128),
        # a very long request out of the rotated 4-bit cache
        dict(name="read_kvarn_131k", op="read", tokens=131072, bs=32, k="int4_asym", v="uint8_asym", kvarn=True,
             layout=12, hkv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "prompt", "write", "write", "attend", "attend", "attend", "read"))
    layout = rng.randrange(1 << 30)
    bs = rng.choice((8, 16, 32, 64, 128))
    hq, hkv, d = rng.choice(SHAPES)
    window = rng.choice((0, 0, 0, 1, 100, 1024, 4097))
    sinks = rng.choice((0, 1, 4, 130)) if window else 0
    k, v = rng.choice(BLOCKED)
    if op == "prompt":
        seqs, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 16384)
        while 4 * seqs * hq * hi * hi > MOST:
            seqs, hi = (3 * seqs + 3) // 4, 4 * hi // 5
        return dict(op=op, seqs=seqs, lo=rng.choice((0, 1, (hi + 1) // 2, hi)), hi=hi, hq=hq, hkv=hkv, d=d,
                    window=window, sinks=sinks, layout=layout)
    if op == "write":
        seqs = _log_int(rng, 1, 512)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, 16384 // seqs))
        return dict(op=op, seqs=seqs, lo=0, hi=min(4096, (1 << 17) // seqs), new_lo=rng.choice((0, 1, new)),
                    new_hi=new, bs=bs, k=k, v=v, layout=layout, hkv=hkv, d=d)
    if op == "read":
        if rng.random() < 0.6:
            k, v, kvarn = rng.choice(CACHES)
        else:
            kvarn = False
        return dict(op=op, tokens=_log_int(rng, 1, 131072 * 8 // max(hkv, 8)), bs=bs, k=k, v=v, kvarn=kvarn, layout=layout,
                    hkv=hkv, d=d)
    if rng.random() < 0.6:
        seqs = _log_int(rng, 1, 128)
        hi = _log_int(rng, 16, min(65536, 262144 // seqs))
        return dict(op=op, seqs=seqs, bs=bs, k=k, v=v, lo=rng.choice((0, 1, hi // 2)), hi=hi, q_lo=1, q_hi=1,
                    window=window, sinks=sinks, chunk=False, layout=layout, hq=hq, hkv=hkv, d=d)
    seqs, q, hi = _log_int(rng, 1, 32), _log_int(rng, 1, 2048), _log_int(rng, 16, 8192)
    while seqs * hq * q * (q + hi) > 1 << 31:
        seqs, q, hi = (seqs + 1) // 2, (q + 1) // 2, (hi + 1) // 2
    return dict(op=op, seqs=seqs, bs=bs, k=k, v=v, lo=0, hi=hi, q_lo=rng.choice((0, 1, (q + 1) // 2)), q_hi=q,
                window=window, sinks=sinks, chunk=True, layout=layout, hq=hq, hkv=hkv, d=d)


def _lengths(case):
    """(tokens already there, new tokens) of every request: fixed by the case."""
    r = np.random.default_rng(case["layout"])
    n = case["seqs"]
    old = r.integers(case["lo"], case["hi"], n, endpoint=True)
    if case["op"] == "prompt":
        old[-1] = max(old[-1], 1)
        return np.zeros(n, np.int64), old
    if case["op"] == "attend" and not case["chunk"]:  # the context includes the query's own token
        old[0] = max(old[0], 1)
        return old - 1, np.ones(n, np.int64)
    lo, hi = ("new_lo", "new_hi") if case["op"] == "write" else ("q_lo", "q_hi")
    new = r.integers(case[lo], case[hi], n, endpoint=True)
    new[0] = max(new[0], 1)
    return old, new


def _row_bytes(fmt, d):
    return d // 2 if fmt == "int4_asym" else 2 * d if fmt == "bf16" else d


def _fields(fmt, kvarn):
    return (3 if kvarn else 2) if fmt.endswith("asym") else 0


def _pages_of(old, new, bs):
    return np.where(new > 0, (old + new + bs - 1) // bs - old // bs, 0)


def work(case):
    """Bytes each input and output once; operations of the products."""
    op, hkv, d = case["op"], case["hkv"], case["d"]
    if op == "read":
        t = case["tokens"]
        per = 8 + hkv * sum(_row_bytes(case[x], d) + 2 * _fields(case[x], case["kvarn"]) + 2 * d for x in ("k", "v"))
        scales = sum(4 * hkv * -(-t // case["bs"]) for x in ("k", "v") if case[x].endswith("block"))
        return {"bytes": t * per + scales, "flops": 0}
    old, new = _lengths(case)
    if op == "write":
        pages = int(_pages_of(old, new, case["bs"]).sum())
        return {"bytes": int(new.sum()) * (8 + 6 * hkv * d) + pages * hkv * 16, "flops": 0}
    hq, w = case["hq"], case["window"] or 1 << 40
    pairs = seen = pages = 0
    for first, n in zip(old.tolist(), new.tolist()):
        if first + n <= 0 or first < 0:
            continue
        p = np.arange(first, first + n, dtype=np.int64)
        pairs += int((np.minimum(p + 1, w) + np.minimum(case["sinks"], np.maximum(p + 1 - w, 0))).sum())
        if n and op == "attend":
            a = max(0, first - w + 1)
            seen += first + n - a + min(case["sinks"], a)
            pages += -(-(first + n) // case["bs"]) - a // case["bs"]
    total = int(new[old + new > 0].sum())
    rows = total * hq * d * 4
    if op == "prompt":
        return {"bytes": rows + total * hkv * d * 4, "flops": int(4 * d * hq * pairs)}
    return {"bytes": rows + seen * hkv * d * 2 + pages * hkv * 8, "flops": int(4 * d * hq * pairs)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _ints(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), device=CUDA).to(dtype)


def _pages(lens, bs, rng, spare):
    """A random page for every bs tokens: (table with -1 behind them, pool size)."""
    need = -(-lens // bs)
    pool = int(need.sum()) + spare
    width = max(1, int(need.max(initial=1)))
    table = np.full((len(lens), width), -1, np.int32)
    table[np.arange(width)[None] < need[:, None]] = rng.permutation(pool).astype(np.int32)[:int(need.sum())]
    return table, pool


def _fp8(fmt):
    return torch.float8_e5m2 if fmt == "fp8_e5m2" else torch.float8_e4m3fn


def _codes(fmt, kvarn, shape, g, x_scale):
    """A cache's bytes and metadata as quantising random rows leaves them, and its tensor scale."""
    nb, bs, hkv, d = shape
    x = torch.randn(shape, device=CUDA, generator=g) * x_scale
    if fmt.endswith("block"):  # rows of a page differ in size, pages too
        x *= torch.exp(0.3 * torch.randn((nb, bs, hkv, 1), device=CUDA, generator=g) +
                       torch.randn((nb, 1, hkv, 1), device=CUDA, generator=g))
        scale = x.abs().amax((1, 3)) / (127 if fmt == "int8_block" else 448)
        x /= scale[:, None, :, None]
        x = x.round().to(torch.int8) if fmt == "int8_block" else x.clamp(-448, 448).to(torch.float8_e4m3fn)
        meta = torch.zeros((nb, (hkv + 3) // 4 * 4), device=CUDA)
        meta[:, :hkv] = scale
        return x.view(torch.uint8), meta, 1.0
    if fmt == "bf16":
        return x.to(torch.bfloat16).view(torch.uint8).reshape(nb, bs, hkv, 2 * d), None, 1.0
    if fmt == "int8":
        scale = 4.5 * x_scale / 127
        return (x / scale).round().clamp(-128, 127).to(torch.int8).view(torch.uint8), None, scale
    if fmt.startswith("fp8"):
        return x.to(_fp8(fmt)).view(torch.uint8), None, 1.0
    top = 15 if fmt == "int4_asym" else 255
    x = x / x_scale
    lo, hi = x.amin(-1), x.amax(-1)
    s, z = ((hi - lo) / top).half(), lo.half()
    c = ((x - z[..., None].float()) / s[..., None].float()).round().clamp(0, top).to(torch.uint8)
    if fmt == "int4_asym":
        c = c[..., 0::2] | (c[..., 1::2] << 4)
    sigma = torch.exp(0.5 * torch.randn((nb, bs, hkv), device=CUDA, generator=g)).half()
    fields = [s, z, sigma] if kvarn else [s, z]
    return c, torch.stack([f.permute(0, 2, 1) for f in fields], 2).contiguous(), 1.0


def prepare(case, seed):
    g = torch.Generator(CUDA).manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, hkv, d = case["op"], case["hkv"], case["d"]
    st = dict(case)
    if op == "prompt":
        _, n = _lengths(case)
        total, hq = int(n.sum()), case["hq"]
        # the projection's output: queries, keys and values of a token side by side
        qkv = torch.randn((total, (hq + 2 * hkv) * d), device=CUDA, generator=g)
        qkv[:, :(hq + hkv) * d] *= 1.3  # logits spread over some units
        qkv = qkv.to(torch.bfloat16)
        st["query"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        st["key"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        st["value"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        st["cu"], st["max_len"], st["sm_scale"] = _ints(np.concatenate([[0], np.cumsum(n)])), int(n.max()), d ** -0.5
        st["out"] = torch.empty((total, hq, d), dtype=torch.bfloat16, device=CUDA)
        return st
    bs = case["bs"]
    if op == "read":
        n = case["tokens"]
        table, nb = _pages(np.array([n]), bs, rng, 3)
        t = np.arange(n)
        st["slots"] = _ints(table[0].astype(np.int64)[t // bs] * bs + t % bs, torch.int64)
        st["key_out"], st["value_out"] = torch.empty((2, n, hkv, d), dtype=torch.bfloat16, device=CUDA)
    else:
        old, new = _lengths(case)
        lens = old + new
        table, nb = _pages(lens, bs, rng, 3)
    kvarn = case.get("kvarn", False)
    st["k_cache"], st["k_meta"], st["k_scale"] = _codes(case["k"], kvarn, (nb, bs, hkv, d), g, 1.5)
    st["v_cache"], st["v_meta"], st["v_scale"] = _codes(case["v"], kvarn, (nb, bs, hkv, d), g, 1.0)
    st["pool"], st["signs"] = nb, None
    if kvarn:
        st["signs"] = _ints(rng.integers(0, 2, d) * 2 - 1, torch.int8)
    if op == "write":
        seq = np.repeat(np.arange(len(old)), new)
        pos = np.concatenate([np.arange(a, a + b) for a, b in zip(old, new)])
        st["slots"] = _ints(table[seq, pos // bs].astype(np.int64) * bs + pos % bs, torch.int64)
        rows = torch.randn((2, len(pos), hkv, d), device=CUDA, generator=g)
        # tokens differ in size, so that a page's largest value is not always among its first rows
        rows *= torch.exp(0.5 * torch.randn((2, len(pos), hkv, 1), device=CUDA, generator=g))
        st["key"], st["value"] = rows.to(torch.bfloat16)
    if op == "attend":
        st["block_table"], st["lens"] = _ints(table), _ints(lens)
        st["max_len"], st["max_q"], st["sm_scale"] = int(lens.max()), int(new.max()), d ** -0.5
        cu = np.concatenate([[0], np.cumsum(new)])
        st["cu"] = _ints(cu)
        st["query"] = torch.randn((int(cu[-1]), case["hq"], d), device=CUDA, generator=g).to(torch.bfloat16)
        st["out"] = torch.zeros_like(st["query"])
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    if own:
        return _OWN[st["op"]](st)
    return _PLAIN[st["op"]](st)


def _cache(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    return kvq.KVCache(st["k"], st["v"], st["hkv"], st["d"], st["bs"], st["pool"], st["k_cache"], st["v_cache"],
                       st["k_meta"], st["v_meta"], st["k_scale"], st["v_scale"], st.get("kvarn", False), st["signs"])


def _workspace(nbytes):
    return torch.empty(nbytes // 4 + 4, dtype=torch.float32, device=CUDA)


def _own_prompt(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    return kvq.kvq_prompt_attention(st["query"], st["key"], st["value"], st["out"], st["cu"], st["max_len"],
                                    st["sm_scale"], st["window"], st["sinks"])


def _own_write(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    if "cache" not in st:
        st["cache"] = _cache(st)
    kvq.kvq_write_cache(st["cache"], st["key"], st["value"], st["slots"])
    return _written(st)


def _own_attend(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    if "cache" not in st:
        c = st["cache"] = _cache(st)
        st["workspace"] = _workspace(
            kvq.kvq_prefill_workspace_size(c, st["seqs"], st["hq"], st["query"].shape[0], st["max_q"], st["max_len"])
            if st["chunk"] else kvq.kvq_decode_workspace_size(c, st["seqs"], st["hq"], st["max_len"]))
    if st["chunk"]:
        return kvq.kvq_paged_prefill(st["cache"], st["query"], st["out"], st["cu"], st["block_table"], st["lens"],
                                     st["max_q"], st["max_len"], st["sm_scale"], st["window"], st["sinks"],
                                     st["workspace"])
    if st["window"]:
        return kvq.kvq_decode_window(st["cache"], st["query"], st["out"], st["block_table"], st["lens"],
                                     st["max_len"], st["sm_scale"], st["window"], st["sinks"], st["workspace"])
    return kvq.kvq_paged_decode(st["cache"], st["query"], st["out"], st["block_table"], st["lens"], st["max_len"],
                                st["sm_scale"], st["workspace"])


def _own_read(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    if "cache" not in st:
        st["cache"] = _cache(st)
    kvq.kvq_read_cache(st["cache"], st["slots"], st["key_out"], st["value_out"])
    return {"key": st["key_out"], "value": st["value_out"]}


def _plain_softmax_product(p, v, seen, g):
    """Logits p [n, hkv, g * lq, lk] and what each query sees [n, 1, 1, lq, lk] -> [n, lq, hq, d]."""
    n, hkv, rows, lk = p.shape
    p = p.view(n, hkv, g, rows // g, lk)
    p.masked_fill_(~seen, -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(n, hkv, rows, lk) @ v).view(n, hkv, g, rows // g, -1)
    out = torch.where(total > 0, out / total, 0.0)
    return out.permute(0, 3, 1, 2, 4).reshape(n, rows // g, hkv * g, -1)


def _plain_prompt(st):
    hq, hkv, d, n, length = st["hq"], st["hkv"], st["d"], st["seqs"], st["max_len"]
    g, cu = hq // hkv, st["cu"].long()
    count = cu[1:] - cu[:-1]
    j = torch.arange(length, device=CUDA)
    rows = (cu[:-1, None] + j).clamp(max=st["query"].shape[0] - 1)  # padded to the longest
    seen = (j <= j[:, None]) & (j < count[:, None, None])
    if st["window"]:
        seen &= (j > j[:, None] - st["window"]) | (j < st["sinks"])
    q = st["query"][rows].float() * st["sm_scale"]
    q = q.view(n, length, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * length, d)
    k, v = st["key"][rows].float(), st["value"][rows].float()
    out = _plain_softmax_product(q @ k.permute(0, 2, 3, 1), v.permute(0, 2, 1, 3), seen[:, None, None], g)
    t = torch.arange(st["query"].shape[0], device=CUDA)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return out[seq, t - cu[seq]].to(torch.bfloat16)


def _written(st):
    types = {"int8_block": torch.int8, "fp8_e4m3_block": torch.float8_e4m3fn}
    return {"k": st["k_cache"].view(types[st["k"]]), "v": st["v_cache"].view(types[st["v"]]),
            "k_scales": st["k_meta"], "v_scales": st["v_meta"]}


def _power(k):
    """2 ** k as float32, exactly."""
    return ((k + 127).clamp(1, 254).int() << 23).view(torch.float32)


def _plain_store(st, fmt, cache, meta, x):
    hkv, bs, slots = st["hkv"], st["bs"], st["slots"]
    x = x.float()
    page, offset = slots // bs, slots % bs
    first = torch.ones_like(page, dtype=torch.bool)
    first[1:] = page[1:] != page[:-1]  # of the run that fills a page
    run_of = first.long().cumsum(0) - 1
    run_page, run_offset = page[first], offset[first]
    most = torch.zeros((run_page.numel(), hkv), device=CUDA)
    most.scatter_reduce_(0, run_of[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    top = torch.full_like(most, 127 if fmt == "int8_block" else 448)  # a tensor: divided by, not multiplied by 1 / top
    need = torch.where(most > 0, (most / top).clamp(min=SMALLEST), 0.0)
    had = torch.where((run_offset > 0)[:, None], meta[run_page, :hkv], 0.0)
    (nm, ne), (hm, he) = torch.frexp(need), torch.frexp(had)
    grow = torch.where((need > had) & (had > 0), (ne - he + (nm > hm)).clamp(min=0), 0)
    scale = torch.where(had > 0, had * _power(grow), need)
    meta[run_page, :hkv] = scale
    # rows in front of a run whose scale has grown
    old = cache.view(torch.int8 if fmt == "int8_block" else torch.float8_e4m3fn)
    j = torch.arange(bs, device=CUDA)
    again = (j < run_offset[:, None])[..., None] & (grow > 0)[:, None]
    shrunk = old[run_page].float() * _power(-grow)[:, None, :, None]
    shrunk = (shrunk.round().to(torch.int8) if fmt == "int8_block" else shrunk.to(torch.float8_e4m3fn)).view(torch.uint8)
    cache[run_page] = torch.where(again[..., None], shrunk, cache[run_page])
    y = x * torch.where(scale > 0, torch.ones_like(scale) / scale, 0.0)[run_of][..., None]
    y = y.round().clamp(-128, 127).to(torch.int8) if fmt == "int8_block" else y.clamp(-448, 448).to(torch.float8_e4m3fn)
    cache[page, offset] = y.view(torch.uint8)


def _plain_write(st):
    _plain_store(st, st["k"], st["k_cache"], st["k_meta"], st["key"])
    _plain_store(st, st["v"], st["v_cache"], st["v_meta"], st["value"])
    return _written(st)


def _hadamard(d, dtype):
    i = torch.arange(d, device=CUDA)
    bits = (i & i[:, None])[..., None] >> torch.arange(8, device=CUDA) & 1
    return (1 - 2 * (bits.sum(-1) & 1)).to(dtype) * d ** -0.5


def _dequantised(st, which, page, offset, dtype):
    """Rows (page, offset) of one of the caches as numbers, [..., kv-heads, head_dim]."""
    fmt, meta = st[which], st[which + "_meta"]
    raw = st[which + "_cache"][page, offset]
    if fmt == "bf16":
        return raw.view(torch.bfloat16).to(dtype)
    if fmt.endswith("block"):
        raw = raw.view(torch.int8 if fmt == "int8_block" else torch.float8_e4m3fn).to(dtype)
        return raw * meta[page, :st["hkv"]].to(dtype)[..., None]
    if fmt == "int8":
        return raw.view(torch.int8).to(dtype) * st[which + "_scale"]
    if fmt.startswith("fp8"):
        return raw.view(_fp8(fmt)).to(dtype) * st[which + "_scale"]
    if fmt == "int4_asym":
        raw = torch.stack((raw & 15, raw >> 4), -1).flatten(-2)
    x = raw.to(dtype) * meta[page, :, 0, offset].to(dtype)[..., None] + meta[page, :, 1, offset].to(dtype)[..., None]
    if st["kvarn"]:  # times the row's deviation, then the inverse rotation
        x = x * meta[page, :, 2, offset].to(dtype)[..., None]
        x = (x @ _hadamard(st["d"], dtype)) * st["signs"].to(dtype)
    return x


def _plain_attend(st):
    hq, hkv, d, n, lq, lk = st["hq"], st["hkv"], st["d"], st["seqs"], st["max_q"], st["max_len"]
    g = hq // hkv
    key_pos = torch.arange(lk, device=CUDA)
    page = st["block_table"].long()[:, key_pos // st["bs"]].clamp(min=0)
    offset = (key_pos % st["bs"]).expand(n, -1)
    k = _dequantised(st, "k", page, offset, torch.float32)
    v = _dequantised(st, "v", page, offset, torch.float32)
    cu, lens = st["cu"].long(), st["lens"].long()
    count = cu[1:] - cu[:-1]
    j = torch.arange(lq, device=CUDA)
    rows = (cu[:-1, None] + j).clamp(max=st["query"].shape[0] - 1)  # padded to the longest
    q_pos = (lens - count)[:, None] + j
    seen = (key_pos <= q_pos[..., None]) & (j < count[:, None])[..., None] & (key_pos < lens[:, None])[:, None]
    if st["window"]:
        seen &= (key_pos > q_pos[..., None] - st["window"]) | (key_pos < st["sinks"])
    q = st["query"][rows].float() * st["sm_scale"]
    q = q.view(n, lq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * lq, d)
    out = _plain_softmax_product(q @ k.permute(0, 2, 3, 1), v.permute(0, 2, 1, 3), seen[:, None, None], g)
    t = torch.arange(st["query"].shape[0], device=CUDA)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return out[seq, t - cu[seq]].to(torch.bfloat16)


def _plain_read(st):
    page, offset = st["slots"] // st["bs"], st["slots"] % st["bs"]
    return {"key": _dequantised(st, "k", page, offset, torch.float32).to(torch.bfloat16),
            "value": _dequantised(st, "v", page, offset, torch.float32).to(torch.bfloat16)}


_OWN = {"prompt": _own_prompt, "write": _own_write, "attend": _own_attend, "read": _own_read}
_PLAIN = {"prompt": _plain_prompt, "write": _plain_write, "attend": _plain_attend, "read": _plain_read}


# --------------------------------------------------------------------------
# the definitions in float64
# --------------------------------------------------------------------------
def _exact_heads(q, k, v, pos, key_pos, st):
    """Queries [n, hq, d] at positions pos over keys [t, hkv, d] at key_pos."""
    w = st["window"] or 1 << 40
    hidden = (key_pos[None] > pos[:, None]) | ((pos[:, None] - key_pos[None] >= w) & (key_pos[None] >= st["sinks"]))
    out = torch.empty(q.shape, dtype=torch.float64, device=CUDA)
    g = st["hq"] // st["hkv"]
    for h in range(st["hq"]):
        logit = q[:, h].double() @ k[:, h // g].double().T * st["sm_scale"]
        out[:, h] = torch.softmax(logit.masked_fill_(hidden, -math.inf), -1) @ v[:, h // g].double()
    return out


def _exact_prompt(st):
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device=CUDA)
    cu = st["cu"].tolist()
    for a, b in zip(cu, cu[1:]):
        for c in range(a, b, 2048):  # rows see what lies in front of them
            e = min(c + 2048, b)
            first = 0 if not st["window"] or st["sinks"] else max(0, c - a - st["window"] + 1)
            at = torch.arange(first, e - a, device=CUDA)
            out[c:e] = _exact_heads(st["query"][c:e], st["key"][a + first:e], st["value"][a + first:e],
                                    torch.arange(c - a, e - a, device=CUDA), at, st)
    return out


def _rounded(x):
    """float64 to the nearest float32, as float64."""
    return x.float().double()


def _exact_store(st, which, x):
    """Codes and scales after the write, run by run: each float32 step of the definition rounded from float64."""
    fmt, bs, hkv = st[which], st["bs"], st["hkv"]
    eight = torch.int8 if fmt == "int8_block" else torch.float8_e4m3fn
    codes = st[which + "_cache"].view(eight).double()
    scales = st[which + "_meta"].double()
    top = 127.0 if fmt == "int8_block" else 448.0

    def coded(y):
        if fmt == "int8_block":
            return torch.round(y).clamp(-128, 127)
        return y.float().clamp(-448, 448).to(eight).double()  # y is a float32 value

    slots = st["slots"].tolist()
    t = 0
    while t < len(slots):
        page, off = divmod(slots[t], bs)
        e = t
        while e < len(slots) and slots[e] // bs == page:
            e += 1
        rows = x[t:e].double()
        most = rows.abs().amax((0, 2))
        need = torch.where(most > 0, _rounded(most / top).clamp(min=SMALLEST), 0.0)
        had = scales[page, :hkv] if off else torch.zeros_like(need)
        new = torch.where(had > 0, had, need)
        short = (had > 0) & (new < need)
        while bool(short.any()):
            new = torch.where(short, new * 2, new)
            short = (had > 0) & (new < need)
        if off:
            ratio = torch.where(had > 0, had / new, 1.0)[None, :, None]
            front = codes[page, :off]
            codes[page, :off] = torch.where(ratio < 1, coded(front * ratio), front)
        scales[page, :hkv] = new
        inv = torch.where(new > 0, _rounded(1 / new), 0.0)
        at = torch.as_tensor([s % bs for s in slots[t:e]], device=CUDA)
        codes[page, at] = coded(_rounded(rows * inv[None, :, None]))
        t = e
    return (codes.to(torch.int8) if fmt == "int8_block" else codes), scales


def _exact_attend(st):
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device=CUDA)
    cu, lens, w = st["cu"].tolist(), st["lens"].tolist(), st["window"] or 1 << 40
    for s in range(st["seqs"]):
        n, length = cu[s + 1] - cu[s], lens[s]
        if not n or not length:
            continue
        pos = torch.arange(length - n, length, device=CUDA)
        first = max(0, length - n - w + 1)  # before it: kept tokens alone
        t = torch.cat((torch.arange(min(st["sinks"], first), device=CUDA), torch.arange(first, length, device=CUDA)))
        page, offset = st["block_table"][s].long()[t // st["bs"]], t % st["bs"]
        k = _dequantised(st, "k", page, offset, torch.float64)
        v = _dequantised(st, "v", page, offset, torch.float64)
        out[cu[s]:cu[s + 1]] = _exact_heads(st["query"][cu[s]:cu[s + 1]], k, v, pos, t, st)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(st)
    if case["op"] == "write":
        (k, ks), (v, vs) = _exact_store(st, "k", st["key"]), _exact_store(st, "v", st["value"])
        return {"k": k, "v": v, "k_scales": ks, "v_scales": vs}
    if case["op"] == "attend":
        return _exact_attend(st)
    page, offset = torch.div(st["slots"], st["bs"], rounding_mode="floor"), st["slots"] % st["bs"]
    found = {"key": [], "value": []}
    for a in range(0, case["tokens"], 16384):
        for name, which in (("key", "k"), ("value", "v")):
            found[name].append(_dequantised(st, which, page[a:a + 16384], offset[a:a + 16384], torch.float64))
    return {name: torch.cat(x) for name, x in found.items()}


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(40)]:
        w = work(c)
        print("%-18s %10.3f MB %12.3f GFLOP  %s" % (c.get("name", "-"), w["bytes"] / 1e6, w["flops"] / 1e9, c))
