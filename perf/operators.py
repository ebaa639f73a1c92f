"""The operators of a paged serving step, as cases to measure.

One step of a serving loop plans where each request's new tokens go (block
tables, slots, positions), normalises and rotates the queries and keys of
every head, stores keys and values in the paged cache, and attends: each
request's new tokens to its own cached context, all of it or a sliding window
with the first few tokens kept visible.

`run` computes an operator with elementary torch operations in float32
(`own` false) or calls the library (`own` true); `exact` computes it in
float64.  The float32 and float64 forms share nothing but the inputs.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
CUDA = "cuda"
# (query heads, kv-heads, head_dim) of the bench's workloads, and multi-head attention
SHAPES = ((32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 16, 128), (24, 8, 64))
CACHES = (("int8", "int8", False), ("fp8_e4m3", "int8", False), ("fp8_e5m2", "fp8_e5m2", False),
          ("int4_asym", "int4_asym", False), ("uint8_asym", "uint8_asym", False),
          ("int4_asym", "uint8_asym", True), ("bf16", "bf16", False))


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    c8b = dict(hq=32, hkv=8, d=128)
    return [
        # a decode step of a full batch: one new token each, now and then a new page
        dict(name="plan_decode", op="plan", seqs=64, lo=256, hi=4096, new_lo=1, new_hi=1, bs=16,
             pad=0, layout=1),
        # a step that admits many prompts at once, with a padded token buffer
        dict(name="plan_chunks", op="plan", seqs=256, lo=0, hi=4096, new_lo=1, new_hi=4096, bs=16,
             pad=777, layout=2),
        # the rotation table of a short-context model, half of each head rotated
        dict(name="table_4k", op="table", positions=4096, rot=64, base=10000.0, kind="none",
             factor=1.0),
        # the table of a model stretched to 131,072 positions, frequency bands scaled apart
        dict(name="table_131k", op="table", positions=131072, rot=128, base=500000.0,
             kind="bands", factor=8.0),
        # the queries and keys of one decode step of 64 requests, normalised and rotated
        dict(name="rope_decode", op="rope", tokens=64, rot=128, interleaved=False, norm=True,
             write="", bs=16, table=4096, layout=3, **c8b),
        # a prefill chunk's queries and keys, the keys and values going to an FP8 cache
        dict(name="rope_write_chunk", op="rope", tokens=16384, rot=128, interleaved=False,
             norm=True, write="fp8_e4m3", bs=16, table=131072, layout=4, **c8b),
        # neighbouring pairs rotated in half of a narrow head, no norm, into the 16-bit cache
        dict(name="rope_write_odd", op="rope", tokens=1001, hq=8, hkv=2, d=64, rot=32,
             interleaved=True, norm=False, write="bf16", bs=32, table=8192, layout=5),
        # decode of the batch above with a 1,024-token window behind 4 kept tokens
        dict(name="window_int8", op="window", seqs=64, bs=16, k="int8", v="int8", kvarn=False,
             lo=256, hi=4096, window=1024, sinks=4, layout=6, **c8b),
        # four very long requests in the rotated 4-bit cache, a quarter of them in view
        dict(name="window_kvarn_131k", op="window", seqs=4, bs=32, k="int4_asym", v="uint8_asym",
             kvarn=True, lo=131072, hi=131072, window=32768, sinks=128, layout=7, **c8b),
        # checking a few drafted tokens of each request against its whole context
        dict(name="prefill_verify", op="prefill", seqs=32, q_lo=1, q_hi=8, bs=16, k="int8",
             v="int8", kvarn=False, lo=256, hi=4096, window=0, sinks=0, layout=8, **c8b),
        # two long chunks behind long cached contexts: the compute-bound end
        dict(name="prefill_long", op="prefill", seqs=2, q_lo=4096, q_hi=4096, bs=16, k="int8",
             v="int8", kvarn=False, lo=4096, hi=8192, window=0, sinks=0, layout=9, **c8b),
        # ragged chunks through a window with kept tokens, on the rotated 4-bit cache
        dict(name="prefill_window", op="prefill", seqs=8, q_lo=1, q_hi=2048, bs=32,
             k="int4_asym", v="uint8_asym", kvarn=True, lo=0, hi=6144, window=2048, sinks=64,
             layout=10, **c8b),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "table", "rope", "rope", "window", "window", "prefill", "prefill",
                     "prefill"))
    layout = rng.randrange(1 << 30)
    bs = rng.choice((8, 16, 32, 64, 128))
    if op == "plan":
        seqs = _log_int(rng, 1, 1024)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 1, min(4096, (1 << 19) // seqs))
        return dict(op=op, seqs=seqs, lo=0, hi=min(8192, (1 << 20) // seqs), new_lo=rng.choice((0, 1)),
                    new_hi=new, bs=bs, pad=rng.choice((0, 1, 333)), layout=layout)
    if op == "table":
        rot = rng.choice((32, 64, 96, 128))
        return dict(op=op, positions=_log_int(rng, 1, 131072), rot=rot,
                    base=rng.choice((10000.0, 500000.0, 1000000.0)),
                    kind=rng.choice(("none", "linear", "ntk", "yarn", "bands")),
                    factor=rng.choice((2.0, 4.0, 8.0, 32.0)))
    hq, hkv, d = rng.choice(SHAPES)
    if op == "rope":
        return dict(op=op, tokens=_log_int(rng, 1, 16384 * 32 // max(hq, 32)), hq=hq, hkv=hkv, d=d,
                    rot=rng.choice((d, d // 2, d // 4, d - 16)), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.6, write=rng.choice(("", "fp8_e4m3", "fp8_e5m2", "bf16")),
                    bs=bs, table=32768, layout=layout)
    k, v, kvarn = rng.choice(CACHES)
    window = rng.choice((0, 1, 100, 512, 1024, 4097))
    sinks = rng.choice((0, 1, 4, 20, 130)) if window else 0
    if op == "window":
        seqs = _log_int(rng, 1, 128)
        hi = _log_int(rng, 16, min(131072, 400000 // seqs))
        return dict(op=op, seqs=seqs, hq=hq, hkv=hkv, d=d, bs=bs, k=k, v=v, kvarn=kvarn,
                    lo=rng.choice((0, 1, hi // 2)), hi=hi, window=max(window, 1), sinks=sinks,
                    layout=layout)
    seqs = _log_int(rng, 1, 32)
    q = 1 if rng.random() < 0.1 else _log_int(rng, 1, 4096)
    hi = _log_int(rng, 16, 8192)
    while seqs * hq * q * (q + hi) > 1 << 31:
        seqs, q, hi = (seqs + 1) // 2, (q + 1) // 2, (hi + 1) // 2
    return dict(op=op, seqs=seqs, hq=hq, hkv=hkv, d=d, bs=bs, k=k, v=v, kvarn=kvarn,
                q_lo=rng.choice((0, 1, (q + 1) // 2)), q_hi=q, lo=0, hi=hi, window=window,
                sinks=sinks, layout=layout)


def _lengths(case):
    """(tokens already cached, new tokens) of every request: fixed by the case."""
    r = np.random.default_rng(case["layout"])
    n = case["seqs"]
    old = r.integers(case["lo"], case["hi"], n, endpoint=True)
    if case["op"] == "window":  # the cached context includes the query's own token
        old[0] = max(old[0], 1)
        return old, np.ones(n, np.int64)
    lo, hi = ("new_lo", "new_hi") if case["op"] == "plan" else ("q_lo", "q_hi")
    new = r.integers(case[lo], case[hi], n, endpoint=True)
    new[0] = max(new[0], 1)
    return old, new


def _row_bytes(fmt, d):
    return d // 2 if fmt == "int4_asym" else 2 * d if fmt == "bf16" else d


def _fields(fmt, kvarn):
    return (3 if kvarn else 2) if fmt.endswith("asym") else 0


def work(case):
    """Bytes each input and output once; operations of the products."""
    op = case["op"]
    if op == "table":
        return {"bytes": case["positions"] * case["rot"] * 4, "flops": 0}
    if op == "plan":
        old, new = _lengths(case)
        total, bs = int(new.sum()), case["bs"]
        pages = np.ceil((old + new) / bs).astype(np.int64)
        fresh = pages - np.ceil(old / bs).astype(np.int64)
        touched = np.where(new > 0, pages - old // bs, 0)  # pages that new tokens land in
        return {"bytes": int((total + case["pad"]) * 12 + 4 * touched.sum() + 8 * fresh.sum() + 16 * len(old)),
                "flops": 0}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "rope":
        n = case["tokens"]
        out = (hq + hkv) * d * 2
        if case["write"]:
            out = hq * d * 2 + 2 * hkv * _row_bytes(case["write"], d) + 8
        read = (hq + (2 if case["write"] else 1) * hkv) * d * 2 + 4
        return {"bytes": n * (read + out + case["rot"] * 4), "flops": 0}
    old, new = _lengths(case)
    last = old + new if op == "prefill" else old  # tokens of the context
    first = np.where(new > 0, last - new, 0)  # position of the first query
    new = np.where(last > 0, new, 0)
    w = case["window"] or 1 << 40
    pairs, seen = 0, 0
    for f, n, l in zip(first.tolist(), new.tolist(), last.tolist()):
        p = np.arange(f, f + n, dtype=np.int64) if op == "prefill" else np.arange(l - 1, l)[:n]
        pairs += int((np.minimum(p + 1, w) + np.minimum(case["sinks"], np.maximum(p + 1 - w, 0))).sum())
        if n:
            a = max(0, int(p[0]) - w + 1)
            seen += l - a + min(case["sinks"], a)
    per = sum(_row_bytes(case[x], d) + 2 * _fields(case[x], case["kvarn"]) for x in ("k", "v"))
    return {"bytes": int(seen * hkv * per + new.sum() * hq * d * 4), "flops": int(4 * d * hq * pairs)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _table(positions, rot, base, kind, factor):
    """cos and sin of every position and pair, in float64."""
    angle = torch.arange(positions, device=CUDA, dtype=torch.float64)[:, None] * _theta(rot, base, kind, factor)
    return torch.stack((angle.cos(), angle.sin()), -1) * _amplitude(kind, factor)


ORIGINAL = 8192  # positions before stretching
LOW, HIGH = {"yarn": 1.0, "bands": 1.0}, {"yarn": 32.0, "bands": 4.0}


def _amplitude(kind, factor):
    return 0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0


def _theta(rot, base, kind, factor):
    i = torch.arange(rot // 2, device=CUDA, dtype=torch.float64)
    if kind == "ntk":  # a larger base, so that the slowest pair slows by the factor
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2 * i / rot)
    if kind == "linear":
        return theta / factor
    if kind == "yarn":  # a ramp over pairs between two numbers of turns
        def at(turns):
            return rot * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(at(HIGH[kind])), 0)
        hi = min(math.ceil(at(LOW[kind])), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return theta / factor * ramp + theta * (1 - ramp)
    if kind == "bands":  # fast pairs kept, slow ones divided, a blend between
        turns = ORIGINAL * theta / (2 * math.pi)
        blend = ((turns - LOW[kind]) / (HIGH[kind] - LOW[kind])).clamp(0, 1)
        return theta / factor * (1 - blend) + theta * blend
    return theta


def _ints(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), device=CUDA).to(dtype)


def _pages(lens, bs, rng, spare):
    """A random page for every bs tokens: (table with -1 behind them, unused pages, pool size)."""
    need = -(-lens // bs)
    pool = int(need.sum()) + spare
    perm = rng.permutation(pool).astype(np.int32)
    width = max(1, int(need.max(initial=1)))
    table = np.full((len(lens), width), -1, np.int32)
    inside = np.arange(width)[None] < need[:, None]
    table[inside] = perm[:int(need.sum())]
    return table, perm[int(need.sum()):], pool


def _codes(fmt, kvarn, shape, g, x_scale):
    """A cache's bytes (and its fp16 fields) as quantising random rows leaves them."""
    nb, bs, hkv, d = shape
    x = torch.randn(shape, device=CUDA, generator=g) * x_scale
    if fmt == "bf16":
        return x.to(torch.bfloat16).view(torch.uint8).reshape(nb, bs, hkv, 2 * d), None, 1.0
    if fmt == "int8":
        scale = 4.5 * x_scale / 127
        return (x / scale).round().clamp(-128, 127).to(torch.int8).view(torch.uint8), None, scale
    if fmt.startswith("fp8"):
        t = torch.float8_e4m3fn if fmt == "fp8_e4m3" else torch.float8_e5m2
        return x.to(t).view(torch.uint8), None, 1.0
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
    op = case["op"]
    st = dict(case)
    if op == "table":
        # the inputs are numbers: another seed stretches a little differently
        st["base"] = case["base"] * (1 + seed % 97 / 1000)
        st["table"] = torch.empty((case["positions"], case["rot"] // 2, 2), device=CUDA)
        return st
    if op == "plan":
        old, new = _lengths(case)
        bs = case["bs"]
        table, unused, pool = _pages(old, bs, rng, 100 + int((-(-new // bs) + 1).sum()))
        full = np.full((len(old), int((-(-(old + new) // bs)).max(initial=0)) + 3), -1, np.int32)
        full[:, :min(full.shape[1], table.shape[1])] = table[:, :full.shape[1]]
        total = int(new.sum()) + case["pad"]
        st.update(pool=pool, old=_ints(old), new=_ints(new), block_table=_ints(full),
                  free=_ints(unused), free_range=_ints([7, len(unused)]),
                  slots=torch.empty(total, dtype=torch.int64, device=CUDA),
                  positions=torch.empty(total, dtype=torch.int32, device=CUDA),
                  lens=torch.empty(len(old), dtype=torch.int32, device=CUDA),
                  cu=torch.empty(len(old) + 1, dtype=torch.int32, device=CUDA),
                  free_out=torch.empty(2, dtype=torch.int32, device=CUDA))
        return st
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    if op == "rope":
        n, rot = case["tokens"], case["rot"]
        # the projection's output: queries, keys and values of a token side by side
        qkv = torch.randn((n, (hq + 2 * hkv) * d), device=CUDA, generator=g).to(torch.bfloat16)
        st["query"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        st["key"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        st["value"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        start = int(rng.integers(0, max(1, case["table"] - n)))
        pos = np.arange(start, start + n) if n > 256 else rng.integers(0, case["table"], n)
        st["positions"] = _ints(pos)
        st["table"] = _table(case["table"], rot, 500000.0, "none", 1.0).float()
        st["q_weight"] = st["k_weight"] = None
        if case["norm"]:
            st["q_weight"], st["k_weight"] = (1 + 0.1 * torch.randn((2, d), device=CUDA, generator=g)).to(torch.bfloat16)
        st["query_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device=CUDA)
        st["key_out"] = torch.empty((n, hkv, d), dtype=torch.bfloat16, device=CUDA)
        if case["write"]:
            nb = -(-n // bs) + 3
            st["slots"] = _ints(rng.permutation(nb)[np.arange(n) // bs] * bs + np.arange(n) % bs, torch.int64)
            shape = (nb, bs, hkv, _row_bytes(case["write"], d))
            st["k_cache"] = torch.zeros(shape, dtype=torch.uint8, device=CUDA)
            st["v_cache"] = torch.zeros(shape, dtype=torch.uint8, device=CUDA)
        return st
    old, new = _lengths(case)
    lens = old + new if op == "prefill" else old
    table, _, nb = _pages(lens, bs, rng, 3)
    st["k_cache"], st["k_meta"], st["k_scale"] = _codes(case["k"], case["kvarn"], (nb, bs, hkv, d), g, 1.5)
    st["v_cache"], st["v_meta"], st["v_scale"] = _codes(case["v"], case["kvarn"], (nb, bs, hkv, d), g, 1.0)
    st["signs"] = None
    if case["kvarn"]:
        st["signs"] = _ints(rng.integers(0, 2, d) * 2 - 1, torch.int8)
    st["pool"], st["sm_scale"] = nb, d ** -0.5
    st["block_table"], st["lens"] = _ints(table), _ints(lens)
    st["max_len"], st["max_q"] = int(lens.max(initial=0)), int(new.max(initial=0))
    cu = np.concatenate([[0], np.cumsum(new)])
    st["cu"] = _ints(cu)
    st["query"] = torch.randn((int(cu[-1]), hq, d), device=CUDA, generator=g).to(torch.bfloat16)
    st["out"] = torch.zeros_like(st["query"])
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    op = st["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _plan_outputs(st):
    return {"slots": st["slots"], "positions": st["positions"], "lens": st["lens"], "cu": st["cu"],
            "table": st["block_table"], "free": st["free_out"]}


def _own_plan(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    kvq.kvq_plan_step(st["old"], st["new"], st["block_table"], st["free"], st["free_range"], st["bs"],
                      st["pool"], st["slots"], st["positions"], st["lens"], st["cu"], st["free_out"])
    return _plan_outputs(st)


def _plain_plan(st):
    bs = st["bs"]
    old, new = st["old"].long(), st["new"].long()
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    have, need = (old + bs - 1) // bs, (old + new + bs - 1) // bs
    before = (need - have).cumsum(0) - (need - have)  # fresh pages of the requests before
    table = st["block_table"].long()
    page = torch.arange(table.shape[1], device=CUDA)[None]
    fresh = (page >= have[:, None]) & (page < need[:, None])
    source = st["free_range"][0] + before[:, None] + page - have[:, None]
    table = torch.where(fresh, st["free"].long()[source.clamp(0, st["free"].numel() - 1)], table)
    t = torch.arange(st["slots"].numel(), device=CUDA)
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=old.numel() - 1)
    valid = t < cu[-1]
    pos = torch.where(valid, old[seq] + t - cu[seq], 0)
    slots = torch.where(valid, table[seq, pos // bs] * bs + pos % bs, -1)
    free = torch.stack((st["free_range"][0] + (need - have).sum(), st["free_range"][1].long()))
    return {"slots": slots, "positions": pos.int(), "lens": (old + new).int(), "cu": cu.int(),
            "table": table.int(), "free": free.int()}


def _own_table(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    kind, scaling = st["kind"], None
    if kind != "none":
        scaling = kvq.RopeScaling(kind, st["factor"], ORIGINAL, LOW.get(kind, 0.0), HIGH.get(kind, 0.0),
                                  _amplitude(kind, st["factor"]))
    return kvq.kvq_rope_table(st["table"], st["base"], scaling)


def _plain_table(st):
    return _table(st["positions"], st["rot"], st["base"], st["kind"], st["factor"]).float()


def _fp8(fmt):
    return {"fp8_e4m3": torch.float8_e4m3fn, "fp8_e5m2": torch.float8_e5m2, "bf16": torch.bfloat16}[fmt]


def _rope_outputs(st):
    if not st["write"]:
        return {"query": st["query_out"], "key": st["key_out"]}
    t = _fp8(st["write"])
    return {"query": st["query_out"], "k_cache": st["k_cache"].view(t), "v_cache": st["v_cache"].view(t)}


def _own_rope(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    if "rope" not in st:  # the layer's handles
        st["rope"] = kvq.Rope(st["table"], st["interleaved"], st["q_weight"], st["k_weight"], EPS)
        if st["write"]:
            st["cache"] = kvq.KVCache(st["write"], st["write"], st["hkv"], st["d"], st["bs"],
                                      st["k_cache"].shape[0], st["k_cache"], st["v_cache"])
    if st["write"]:
        kvq.kvq_norm_rope_write(st["rope"], st["cache"], st["query"], st["key"], st["value"],
                                st["positions"], st["slots"], st["query_out"])
    else:
        kvq.kvq_norm_rope(st["rope"], st["query"], st["key"], st["positions"], st["query_out"],
                          st["key_out"])
    return _rope_outputs(st)


def _plain_norm_rope(st, x, weight):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    rot = st["rot"]
    cos, sin = st["table"][st["positions"].long()][:, None].unbind(-1)
    if st["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1).to(torch.bfloat16)


def _plain_store(st, cache, x):
    t = _fp8(st["write"])
    if t is not torch.bfloat16:
        top = torch.finfo(t).max
        x = x.float().clamp(-top, top)
    cache.flatten(0, 1)[st["slots"]] = x.to(t).view(torch.uint8)


def _plain_rope(st):
    q = _plain_norm_rope(st, st["query"], st["q_weight"])
    k = _plain_norm_rope(st, st["key"], st["k_weight"])
    if not st["write"]:
        return {"query": q, "key": k}
    _plain_store(st, st["k_cache"], k)
    _plain_store(st, st["v_cache"], st["value"])
    return {**_rope_outputs(st), "query": q}


def _cache(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    return kvq.KVCache(st["k"], st["v"], st["hkv"], st["d"], st["bs"], st["pool"], st["k_cache"],
                       st["v_cache"], st["k_meta"], st["v_meta"], st["k_scale"], st["v_scale"],
                       st["kvarn"], st["signs"])


def _workspace(nbytes):
    return torch.empty(nbytes // 4 + 4, dtype=torch.float32, device=CUDA)


def _own_window(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    if "cache" not in st:
        st["cache"] = _cache(st)
        st["workspace"] = _workspace(kvq.kvq_decode_workspace_size(st["cache"], st["seqs"], st["hq"],
                                                                   st["max_len"]))
    return kvq.kvq_decode_window(st["cache"], st["query"], st["out"], st["block_table"], st["lens"],
                                 st["max_len"], st["sm_scale"], st["window"], st["sinks"],
                                 st["workspace"])


def _own_prefill(st):
    from quantized_paged_kv_kvq_gb300 import kvq
    if "cache" not in st:
        st["cache"] = _cache(st)
        st["workspace"] = _workspace(kvq.kvq_prefill_workspace_size(
            st["cache"], st["seqs"], st["hq"], st["query"].shape[0], st["max_q"], st["max_len"]))
    return kvq.kvq_paged_prefill(st["cache"], st["query"], st["out"], st["cu"], st["block_table"],
                                 st["lens"], st["max_q"], st["max_len"], st["sm_scale"],
                                 st["window"], st["sinks"], st["workspace"])


def _hadamard(d, dtype):
    h = torch.ones((1, 1), dtype=dtype, device=CUDA)
    while h.shape[0] < d:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h * d ** -0.5


def _dequantised(st, which, page, offset, dtype):
    """Rows (page, offset) of one of the caches as numbers, [..., kv-heads, head_dim]."""
    fmt = st[which]
    raw = st[which + "_cache"][page, offset]
    if fmt == "bf16":
        return raw.view(torch.bfloat16).to(dtype)
    if fmt == "int8":
        return raw.view(torch.int8).to(dtype) * st[which + "_scale"]
    if fmt.startswith("fp8"):
        return raw.view(_fp8(fmt)).to(dtype) * st[which + "_scale"]
    if fmt == "int4_asym":
        raw = torch.stack((raw & 15, raw >> 4), -1).flatten(-2)
    meta = st[which + "_meta"]
    x = raw.to(dtype) * meta[page, :, 0, offset].to(dtype)[..., None] + meta[page, :, 1, offset].to(dtype)[..., None]
    if st["kvarn"]:  # times the row's deviation, then the inverse rotation
        x = x * meta[page, :, 2, offset].to(dtype)[..., None]
        x = (x @ _hadamard(st["d"], dtype)) * st["signs"].to(dtype)
    return x


def _plain_attention(st):
    hq, hkv, d, n, lq, lk = st["hq"], st["hkv"], st["d"], st["seqs"], st["max_q"], st["max_len"]
    key_pos = torch.arange(lk, device=CUDA)
    page = st["block_table"].long()[:, key_pos // st["bs"]].clamp(min=0)
    offset = (key_pos % st["bs"]).expand(n, -1)
    k = _dequantised(st, "k", page, offset, torch.float32)
    v = _dequantised(st, "v", page, offset, torch.float32)
    # queries of every request side by side, padded to the longest
    cu, lens = st["cu"].long(), st["lens"].long()
    count = cu[1:] - cu[:-1]
    j = torch.arange(lq, device=CUDA)
    rows = (cu[:-1, None] + j).clamp(max=max(st["query"].shape[0] - 1, 0))
    q_pos = (lens - count)[:, None] + j
    seen = (key_pos <= q_pos[..., None]) & (j < count[:, None])[..., None] & (key_pos < lens[:, None])[:, None]
    if st["window"]:
        seen &= (key_pos > q_pos[..., None] - st["window"]) | (key_pos < st["sinks"])
    seen = seen[:, None, None]
    q = st["query"][rows].float() * st["sm_scale"]
    q = q.view(n, lq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    p = (q @ k.permute(0, 2, 3, 1)).view(n, hkv, hq // hkv, lq, lk)
    p.masked_fill_(~seen, -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(n, hkv, -1, lk) @ v.permute(0, 2, 1, 3)).view(n, hkv, hq // hkv, lq, d)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, lq, hq, d)
    t = torch.arange(st["query"].shape[0], device=CUDA)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return out[seq, t - cu[seq]].to(torch.bfloat16)


_OWN = {"plan": _own_plan, "table": _own_table, "rope": _own_rope, "window": _own_window,
        "prefill": _own_prefill}
_PLAIN = {"plan": _plain_plan, "table": _plain_table, "rope": _plain_rope,
          "window": _plain_attention, "prefill": _plain_attention}


# --------------------------------------------------------------------------
# the definitions in float64
# --------------------------------------------------------------------------
def _exact_rotated(st, x, weight):
    x = x.double()
    d, rot = x.shape[-1], st["rot"]
    if weight is not None:
        x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * weight.double()
    c, s = st["table"].double()[st["positions"].long()].unbind(-1)
    turn = torch.complex(c, s)[:, None]
    i = torch.arange(rot // 2, device=CUDA)
    re, im = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + rot // 2)
    z = torch.complex(x[..., re], x[..., im]) * turn
    y = x.clone()
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_attention(st):
    hq, hkv, d, bs = st["hq"], st["hkv"], st["d"], st["bs"]
    gq = hq // hkv
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device=CUDA)
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    w = st["window"] or 1 << 40
    for s in range(st["seqs"]):
        n, length = cu[s + 1] - cu[s], lens[s]
        if not n or not length:
            continue
        pos = torch.arange(length - n, length, device=CUDA)
        first = max(0, length - n - w + 1)  # before it: kept tokens alone
        t = torch.cat((torch.arange(min(st["sinks"], first), device=CUDA), torch.arange(first, length, device=CUDA)))
        page, offset = st["block_table"][s].long()[t // bs], t % bs
        k = _dequantised(st, "k", page, offset, torch.float64)
        v = _dequantised(st, "v", page, offset, torch.float64)
        hidden = (t[None] > pos[:, None]) | ((pos[:, None] - t[None] >= w) & (t[None] >= st["sinks"]))
        for h in range(hkv):
            q = st["query"][cu[s]:cu[s + 1], h * gq:(h + 1) * gq].double()
            logit = torch.einsum("qgd,td->gqt", q, k[:, h]) * st["sm_scale"]
            p = torch.softmax(logit.masked_fill_(hidden, -math.inf), -1)
            out[cu[s]:cu[s + 1], h * gq:(h + 1) * gq] = torch.einsum("gqt,td->qgd", p, v[:, h])
    return out


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    st = prepare(case, seed)
    if op == "table":
        turn = torch.arange(case["positions"], device=CUDA, dtype=torch.float64)
        z = torch.polar(torch.full((1,), _amplitude(case["kind"], case["factor"]), dtype=torch.float64, device=CUDA),
                        torch.outer(turn, _theta(case["rot"], st["base"], case["kind"], case["factor"])))
        return torch.view_as_real(z)
    if op == "rope":
        q = _exact_rotated(st, st["query"], st["q_weight"])
        k = _exact_rotated(st, st["key"], st["k_weight"])
        if not case["write"]:
            return {"query": q, "key": k}
        t = _fp8(case["write"])
        found = {"query": q}
        for name, x in (("k_cache", k.to(torch.bfloat16)), ("v_cache", st["value"])):
            shape = st[name].shape[:3] + (case["d"],)
            y = torch.zeros(shape, dtype=torch.float64, device=CUDA)
            if t is not torch.bfloat16:
                x = x.float().clamp(-torch.finfo(t).max, torch.finfo(t).max).to(t)
            y.flatten(0, 1)[st["slots"]] = x.double()
            found[name] = y
        return found
    return _exact_attention(st)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(40)]:
        w = work(c)
        print("%-18s %10.3f MB %12.3f GFLOP  %s" % (c.get("name", "-"), w["bytes"] / 1e6, w["flops"] / 1e9, c))
