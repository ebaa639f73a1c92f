"""The prompt attention, the cache read-back and the block formats refuse bad arguments on
the host, without a GPU."""
import ctypes

import pytest
import torch

from quantized_paged_kv_kvq_gb300 import kvq

from test_abi import FAKE, _decode, _desc, _write, lib  # noqa: F401  (fixture)

MB = 1 << 20


def at(n):  # disjoint 16-byte aligned addresses, never dereferenced
    return 0x100000000 + n * MB


def prompt(lib, **kw):
    a = dict(out=at(0), os=1024, q=at(1), qs=1024, k=at(2), ks=256, v=at(3), vs=256, cu=at(4), s=2, t=64, n=64, hq=8,
             hkv=2, d=128, sm=0.1, w=0, sinks=0)
    a.update(kw)
    return lib.kvq_prompt_attention(*[a[x] for x in ("out", "os", "q", "qs", "k", "ks", "v", "vs", "cu", "s", "t", "n", "hq",
                                                     "hkv", "d", "sm", "w", "sinks")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(s=-1), 1), (dict(t=-1), 1), (dict(n=-1), 1), (dict(hq=0), 1), (dict(hkv=0), 1), (dict(d=0), 1),
    (dict(hq=9), 1), (dict(hq=18), 2), (dict(d=96), 2), (dict(d=256), 2), (dict(t=(1 << 30) + 1), 2),
    (dict(sm=float("nan")), 1), (dict(sm=float("inf")), 1), (dict(w=-1), 1), (dict(sinks=-1), 1),
    (dict(out=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(cu=None), 1),
    (dict(q=at(1) + 8), 1), (dict(cu=at(4) + 2), 1), (dict(qs=1016), 1), (dict(ks=252), 1), (dict(vs=260), 1),
    (dict(os=(1 << 31) + 8), 1),
    (dict(out=at(1)), 1), (dict(out=at(2)), 1), (dict(out=at(3) + 512), 1),  # not in place
    (dict(s=0), 0), (dict(t=0, q=None), 0), (dict(n=0), 0)])
def test_prompt(lib, kw, status):
    assert prompt(lib, **kw) == status


def block(**kw):
    return _desc(**{**dict(k_fmt=7, v_fmt=8, k_meta=at(20), v_meta=at(21)), **kw})


def read(lib, desc=None, **kw):
    a = dict(k=at(0), v=at(1), ko=at(2), vo=at(3), ks=1024, vs=1024, slots=at(4), n=4)
    a.update(kw)
    d = block() if desc is None else desc
    return lib.kvq_read_cache(ctypes.byref(d), a["k"], a["v"], a["ko"], a["vo"], a["ks"], a["vs"], a["slots"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(ko=None), 1), (dict(vo=None), 1), (dict(slots=None), 1),
    (dict(k=at(0) + 8), 1), (dict(ko=at(2) + 8), 1), (dict(slots=at(4) + 4), 1), (dict(ks=1016), 1), (dict(vs=1028), 1),
    (dict(vo=at(2)), 1), (dict(vo=at(2) + 64), 1), (dict(n=0, k=None), 0), (dict(n=(1 << 34) + 1), 2)])
def test_read(lib, kw, status):
    assert read(lib, **kw) == status
    assert lib.kvq_read_cache(None, at(0), at(1), at(2), at(3), 1024, 1024, at(4), 4, None) == 1


def test_block_formats(lib):
    for kf, vf in ((7, 1), (1, 8), (7, 6), (4, 8), (7, 5)):  # with a block format both have one
        assert _write(lib, block(k_fmt=kf, v_fmt=vf)) == 2
    assert _write(lib, block(k_meta=None)) == 1 and _write(lib, block(v_meta=None)) == 1
    assert _write(lib, block(k_meta=at(20) + 8)) == 1
    assert _write(lib, block(flags=1)) == 2  # rotation needs asymmetric formats
    assert _write(lib, block(k_head_scales=at(22))) == 1 and _write(lib, block(v_head_scales=at(22))) == 1
    assert _write(lib, block(k_fmt=9)) == 1
    assert _write(lib, block(k_scale=0.0, v_scale=0.0), n=0) == 0  # the tensor scales are unused
    assert _decode(lib, block(), hq=30) == 1 and _decode(lib, block(), hq=128) == 2
    assert _decode(lib, block(), ws=None, wsb=0) == 3


def test_calls_without_block_formats(lib):
    d = block()
    rope = kvq._RopeDesc(128, 128, 0, 1e-6, 0.0, None, None, at(9), 100)
    assert lib.kvq_norm_rope_write(ctypes.byref(rope), ctypes.byref(d), at(0), at(1), at(2), 1024, at(3), 1024, at(4), 1024,
                                   at(5), 1024, at(6), at(7), 4, 8, None) == 2
    one = (kvq._CacheDesc * 1)(d)
    pools = (ctypes.c_void_p * 1)(at(0))
    assert lib.kvq_decode_mixed(one, 1, pools, pools, at(1), None, None, 0, 0, at(2), at(3), 4, 32, at(4), 64, at(5), 1024,
                                0.1, 1, None, 0, None) == 2


def test_binding():
    x = torch.zeros((4, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.kvq_prompt_attention(x, x, x, x, torch.zeros(2, dtype=torch.int32), 4, 0.1)
    with pytest.raises(ValueError, match="32 bits"):
        kvq.kvq_prompt_attention(x, x, x, x, torch.zeros(2, dtype=torch.int32), 1 << 40, 0.1)
    with pytest.raises(ValueError, match="entry more"):
        kvq.kvq_prompt_attention(x, x, x, x, torch.zeros(0, dtype=torch.int32), 4, 0.1)
    c = kvq.alloc_kv_cache("int8_block", "fp8_e4m3_block", 4, 16, 6, 64, device="cpu", fill=0)
    assert c.k_meta.shape == c.v_meta.shape == (4, 8) and c.k_meta.dtype == torch.float32
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.kvq_read_cache(c, torch.zeros(4, dtype=torch.int64), x, x)


def test_the_binding_checks_a_block_cache(monkeypatch):
    """Scales of another shape, type or device are refused before an address leaves."""
    c = kvq.alloc_kv_cache("int8_block", "int8_block", 4, 16, 6, 64, device="cpu", fill=0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    kvq._cache_desc(0, c)
    for bad in (None, c.k_meta[:3], c.k_meta[:, :6], c.k_meta.double(), c.k_meta.t(), c.k_meta[0], torch.zeros((4, 16))[:, ::2]):
        for name in ("k_meta", "v_meta"):
            good = getattr(c, name)
            setattr(c, name, bad)
            with pytest.raises(ValueError, match=name):
                kvq._cache_desc(0, c)
            setattr(c, name, good)
