"""The serving-step entry points refuse bad arguments on the host, without a GPU."""
import ctypes
import importlib.util
import sys

import pytest
import torch

from quantized_paged_kv_kvq_gb300 import kvq

from test_abi import FAKE, _desc, lib  # noqa: F401  (fixture)

MB = 1 << 20


def at(n):  # disjoint 16-byte aligned addresses, never dereferenced
    return 0x100000000 + n * MB


def plan(lib, **kw):
    a = dict(cl=at(0), nl=at(1), s=4, bt=at(2), w=64, bs=16, nb=100, fb=at(3), cap=50, fr=at(4), slots=at(5),
             pos=at(6), t=64, clo=at(7), cu=at(8), fro=at(9))
    a.update(kw)
    return lib.kvq_plan_step(a["cl"], a["nl"], a["s"], a["bt"], a["w"], a["bs"], a["nb"], a["fb"], a["cap"], a["fr"],
                             a["slots"], a["pos"], a["t"], a["clo"], a["cu"], a["fro"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(s=-1), 1), (dict(w=-1), 1), (dict(bs=0), 1), (dict(nb=0), 1), (dict(cap=-1), 1), (dict(t=-1), 1),
    (dict(bs=24), 2), (dict(bs=4), 2), (dict(w=(1 << 30) // 16 + 1), 2), (dict(t=1 << 31), 2),
    (dict(cl=None), 1), (dict(nl=None), 1), (dict(bt=None), 1), (dict(fb=None), 1), (dict(fr=None), 1),
    (dict(slots=None), 1), (dict(pos=None), 1), (dict(clo=None), 1), (dict(cu=None), 1), (dict(fro=None), 1),
    (dict(cl=at(0) + 2), 1), (dict(slots=at(5) + 8), 1), (dict(pos=at(6) + 4), 1),
    # nothing written may overlap what is read or written
    (dict(clo=at(0)), 1), (dict(clo=at(0) + 12), 1), (dict(cu=at(1)), 1), (dict(fro=at(4)), 1),
    (dict(bt=at(3) + 100), 1), (dict(slots=at(6)), 1), (dict(cu=at(7) + 8), 1), (dict(pos=at(5) + 256), 1)])
def test_plan(lib, kw, status):
    assert plan(lib, **kw) == status


def table(lib, n=100, rot=64, base=10000.0, scaling=None, p=FAKE):
    sc = None if scaling is None else ctypes.byref(kvq._RopeScaling(*scaling))
    return lib.kvq_rope_table(p, n, rot, base, sc, None)


def test_rope_table(lib):
    inf, nan = float("inf"), float("nan")
    assert table(lib, n=-1) == 1 and table(lib, rot=63) == 1 and table(lib, rot=0) == 1
    assert table(lib, rot=258) == 2 and table(lib, n=1 << 31) == 2
    assert table(lib, base=1.0) == 1 and table(lib, base=nan) == 1 and table(lib, base=inf) == 1
    assert table(lib, p=None) == 1 and table(lib, p=FAKE + 8) == 1
    assert table(lib, n=0, p=None) == 0
    assert table(lib, scaling=(5, 2.0, 1.0, 1.0, 2.0, 1.0)) == 1  # no such kind
    assert table(lib, scaling=(1, 0.0, 1.0, 1.0, 2.0, 1.0)) == 1 and table(lib, scaling=(1, nan, 1.0, 1.0, 2.0, 1.0)) == 1
    assert table(lib, rot=2, scaling=(2, 2.0, 1.0, 1.0, 2.0, 1.0)) == 1  # the stretched base needs r > 2
    assert table(lib, scaling=(3, 2.0, 0.0, 1.0, 2.0, 1.0)) == 1 and table(lib, scaling=(4, 2.0, 64.0, 4.0, 4.0, 1.0)) == 1
    assert table(lib, scaling=(4, 2.0, 64.0, 0.0, 4.0, 1.0)) == 1 and table(lib, scaling=(0, 1.0, 1.0, 1.0, 2.0, inf)) == 1


def rope_desc(**kw):
    a = dict(head_dim=128, rot_dim=128, interleaved=0, eps=1e-6, weight_offset=0.0, q_weight=at(20), k_weight=at(21),
             table=at(22), num_positions=100)
    a.update(kw)
    return kvq._RopeDesc(**a)


def norm_rope(lib, d=None, **kw):
    a = dict(qo=at(0), qos=4096, ko=at(8), kos=1024, q=at(16), qs=4096, k=at(24), ks=1024, pos=at(32), t=10, hq=32, hkv=8)
    a.update(kw)
    d = rope_desc() if d is None else d
    return lib.kvq_norm_rope(ctypes.byref(d), a["qo"], a["qos"], a["ko"], a["kos"], a["q"], a["qs"], a["k"], a["ks"],
                             a["pos"], a["t"], a["hq"], a["hkv"], None)


BAD_ROPE = [(dict(rot_dim=-16), 1), (dict(rot_dim=144), 1), (dict(interleaved=2), 1), (dict(eps=-1.0), 1),
            (dict(eps=float("nan")), 1), (dict(weight_offset=float("inf")), 1), (dict(rot_dim=40), 2),
            (dict(head_dim=96, rot_dim=96), 2), (dict(q_weight=at(20) + 8), 1), (dict(table=None), 1),
            (dict(table=at(22) + 4), 1), (dict(num_positions=-1), 1)]


@pytest.mark.parametrize("kw,status", BAD_ROPE)
def test_rope_descriptions(lib, kw, status):
    assert norm_rope(lib, rope_desc(**kw)) == status
    assert write(lib, rope_desc(**kw)) == status


@pytest.mark.parametrize("kw", [
    dict(t=-1), dict(hq=-1), dict(hkv=-1), dict(q=None), dict(ko=None), dict(pos=None), dict(pos=at(32) + 2),
    dict(q=at(16) + 8), dict(qos=4088), dict(qs=4100), dict(ks=1016),
    dict(qo=at(16) + 16), dict(qo=at(24)), dict(ko=at(16)), dict(ko=at(0)), dict(qo=at(16), qos=6144),
    # one projection's queries over its keys: rows 4,096 + 1,024 wide, 5,120 apart
    dict(q=at(16), qs=5120, k=at(16) + 2 * 4096, ks=5120, qo=at(16) + 2 * 1024, qos=5120)])
def test_norm_rope(lib, kw):
    assert norm_rope(lib, **kw) == 1


def test_norm_rope_nothing_to_do(lib):
    assert lib.kvq_norm_rope(None, at(0), 4096, at(8), 1024, at(16), 4096, at(24), 1024, at(32), 4, 32, 8, None) == 1
    assert norm_rope(lib, t=0, q=None) == 0
    assert norm_rope(lib, hq=0, hkv=0, q=None, k=None, qo=None, ko=None) == 0


def write(lib, d=None, c=None, **kw):
    a = dict(kc=at(40), vc=at(48), qo=at(0), qos=4096, q=at(16), qs=4096, k=at(24), ks=1024, v=at(28), vs=1024,
             pos=at(32), slots=at(33), t=10, hq=32)
    a.update(kw)
    d = rope_desc() if d is None else d
    c = _desc() if c is None else c
    return lib.kvq_norm_rope_write(ctypes.byref(d), ctypes.byref(c), a["kc"], a["vc"], a["qo"], a["qos"], a["q"], a["qs"],
                                   a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["slots"], a["t"], a["hq"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(kc=None), 1), (dict(vc=at(48) + 8), 1), (dict(slots=None), 1), (dict(v=None), 1), (dict(vs=1000), 1),
    (dict(qo=at(24)), 1), (dict(qo=at(28)), 1), (dict(t=0, kc=None, slots=None), 0)])
def test_norm_rope_write(lib, kw, status):
    assert write(lib, **kw) == status


def test_norm_rope_write_descriptions(lib):
    assert write(lib, rope_desc(head_dim=64, rot_dim=64)) == 1  # not the cache's
    assert write(lib, c=_desc(head_dim=256)) == 2
    assert write(lib, c=_desc(k_scale=0.0)) == 1
    assert write(lib, c=_desc(k_fmt=4, v_fmt=4)) == 1  # asymmetric needs metadata


def window(lib, c=None, **kw):
    a = dict(nk=None, nv=None, s=4, hq=32, mb=64, mc=1024, sm=0.088, w=16, sinks=4, p=256, ws=None, wsb=0)
    a.update(kw)
    c = _desc() if c is None else c
    return lib.kvq_decode_window(ctypes.byref(c), FAKE, FAKE, a["nk"], a["nv"], 1024, 1024, FAKE, FAKE, a["s"], a["hq"],
                                 FAKE, a["mb"], FAKE, a["mc"], a["sm"], a["w"], a["sinks"], a["p"], a["ws"], a["wsb"], None)


def test_decode_window(lib):
    assert window(lib, w=0) == 1 and window(lib, w=-5) == 1 and window(lib, sinks=-1) == 1
    assert window(lib) == 3  # needs a workspace
    assert window(lib, nk=FAKE) == 1 and window(lib, nv=FAKE) == 1  # one without the other
    assert window(lib, hq=30) == 1 and window(lib, mb=10) == 1 and window(lib, sm=float("nan")) == 1
    assert window(lib, _desc(head_dim=96)) == 2
    assert window(lib, s=0) == 0


def prefill(lib, c=None, **kw):
    a = dict(kc=at(0), vc=at(8), out=at(16), q=at(24), cu=at(32), s=4, total=20, mq=8, hq=32, bt=at(33), mb=64,
             cl=at(34), mc=1024, sm=0.088, w=0, sinks=0, ws=None, wsb=0)
    a.update(kw)
    c = _desc() if c is None else c
    return lib.kvq_paged_prefill(ctypes.byref(c), a["kc"], a["vc"], a["out"], a["q"], a["cu"], a["s"], a["total"],
                                 a["mq"], a["hq"], a["bt"], a["mb"], a["cl"], a["mc"], a["sm"], a["w"], a["sinks"],
                                 a["ws"], a["wsb"], None)


def test_prefill_shapes(lib):
    n = ctypes.c_size_t(7)
    size = lambda c, *a: lib.kvq_prefill_workspace_size(ctypes.byref(c), *a, ctypes.byref(n))
    assert size(_desc(), -1, 32, 10, 4, 100) == 1 and size(_desc(), 4, 0, 10, 4, 100) == 1
    assert size(_desc(), 4, 32, -1, 4, 100) == 1 and size(_desc(), 4, 32, 10, -1, 100) == 1
    assert size(_desc(), 4, 32, 10, 4, -1) == 1 and size(_desc(), 4, 30, 10, 4, 100) == 1
    assert size(_desc(), 4, 128, 10, 4, 100) == 2  # 16 query heads a kv-head
    assert size(_desc(), 4, 32, 1 << 31, 4, 100) == 2 and size(_desc(), 4, 32, 10, 4, (1 << 30) + 1) == 2
    assert size(_desc(head_dim=256), 4, 32, 10, 4, 100) == 2
    assert lib.kvq_prefill_workspace_size(ctypes.byref(_desc()), 4, 32, 10, 4, 100, None) == 1
    assert size(_desc(), 0, 32, 0, 0, 0) == 0 and n.value == 0
    assert prefill(lib, w=-1) == 1 and prefill(lib, sinks=-1) == 1 and prefill(lib, sm=float("inf")) == 1 \
        if torch.cuda.is_available() else True
    # nothing to do, whatever the pointers
    assert prefill(lib, s=0, kc=None) == 0 and prefill(lib, total=0, q=None) == 0 and prefill(lib, mq=0, cu=None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(w=-1), 1), (dict(sinks=-1), 1), (dict(sm=float("inf")), 1), (dict(sm=float("nan")), 1),
    (dict(kc=None), 1), (dict(vc=None), 1), (dict(out=None), 1), (dict(q=None), 1), (dict(cu=None), 1),
    (dict(bt=None), 1), (dict(cl=None), 1),
    (dict(kc=at(0) + 8), 1), (dict(vc=at(8) + 4), 1), (dict(out=at(16) + 8), 1), (dict(q=at(24) + 2), 1),
    (dict(cu=at(32) + 2), 1), (dict(bt=at(33) + 1), 1), (dict(cl=at(34) + 2), 1),
    # 20 rows of 32 heads of 128: the output over the queries, whole or by 16 bytes at either end
    (dict(out=at(24)), 1), (dict(out=at(24) + 20 * 32 * 128 * 2 - 16), 1), (dict(out=at(24) - 20 * 32 * 128 * 2 + 16), 1),
    (dict(mb=63), 1), (dict(mb=-1), 1), (dict(s=-1), 1), (dict(total=-1), 1), (dict(mq=-1), 1), (dict(mc=-1), 1),
    (dict(hq=30), 1), (dict(hq=128), 2), (dict(total=1 << 31), 2), (dict(mc=(1 << 30) + 1), 2)])
def test_prefill(lib, kw, status):
    """Refused on the host, before the device is asked for anything."""
    assert prefill(lib, **kw) == status


def test_binding_checks_before_the_call():
    """Tensors that are not on the GPU are refused by the binding itself."""
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        kvq.kvq_rope_table(torch.empty(4, 8, 2), 10000.0)


def test_rope_table_factors_without_a_fraction_to_keep(lib):
    assert table(lib, scaling=(1, 1e-9, 1.0, 1.0, 2.0, 1.0)) == 1  # 1.6e8 turns a position
    assert table(lib, n=0, scaling=(1, 1e-6, 1.0, 1.0, 2.0, 1.0)) == 0


CACHE_FORMATS = [("int8", "fp8_e4m3", False), ("int4_asym", "uint8_asym", True), ("uint8_asym", "uint8_asym", False), ("bf16", "bf16", False)]


def host_cache(kf, vf, kvarn):
    signs = torch.ones(64, dtype=torch.int8) if kvarn else None
    c = kvq.alloc_kv_cache(kf, vf, 3, 16, 2, 64, 0.1, 0.1, kvarn, signs, device="cpu")
    if not kf.endswith("asym") and kf != "bf16":
        c.k_head_scales, c.v_head_scales = torch.ones(2), torch.ones(2)
    return c


@pytest.mark.parametrize("kf,vf,kvarn", CACHE_FORMATS)
def test_caches_whose_tensors_do_not_fit_are_refused(kf, vf, kvarn):
    """The check that the binding makes before a cache's addresses leave it (here of CPU
    tensors, which are those of device -1)."""
    kvq._cache_desc(-1, host_cache(kf, vf, kvarn))
    more = host_cache(kf, vf, kvarn)
    more.num_blocks = 2  # tensors with a block more than it is told of
    kvq._cache_desc(-1, more)
    wrong = {}
    for name in ("k_cache", "v_cache", "k_meta", "v_meta", "signs", "k_head_scales", "v_head_scales"):
        t = getattr(host_cache(kf, vf, kvarn), name)
        if t is None:
            continue
        wrong[name] = [t.double(), t[..., :-1], t[:1], torch.stack((t, t), -1)[..., 0], t.unsqueeze(0)]
        if name.endswith("meta"):
            wrong[name] += [None, t[:, :, :1].contiguous(), t[:, :1].contiguous()]
    for name, values in wrong.items():
        for x in values:
            c = host_cache(kf, vf, kvarn)
            setattr(c, name, x)
            with pytest.raises(ValueError, match=name):
                kvq._cache_desc(-1, c)
        with pytest.raises(ValueError, match="k_cache"):  # on another device than the call's
            kvq._cache_desc(0, host_cache(kf, vf, kvarn))
    c = host_cache(kf, vf, kvarn)
    c.num_blocks = 4  # more blocks than its tensors hold
    with pytest.raises(ValueError, match="k_cache"):
        kvq._cache_desc(-1, c)


def test_the_binding_does_without_torchs_shortcuts(monkeypatch):
    """A torch without its private device and stream queries: the public ones serve."""
    class Stream:
        def __init__(self, dev):
            self.cuda_stream = 100 + dev
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 5)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("kvq_without_shortcuts", kvq.__file__)
    other = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, other)
    spec.loader.exec_module(other)

    class OnDevice:
        def __init__(self, dev):
            self.dev = self.device = dev

        def get_device(self):
            return self.dev
    assert other._device_of("x", OnDevice(5)) == 5 and other._raw_stream(5, None) == 105
    assert other._raw_stream(5, Stream(7)) == 107
    for dev in (4, -1):
        with pytest.raises(ValueError, match="current CUDA device"):
            other._device_of("x", OnDevice(dev))


@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 5, 1 << 40, -(1 << 31) - 1, -(1 << 32) + 7])
def test_numbers_beyond_32_bits_are_refused(value):
    """ctypes cuts them: a window of 2^32 + 5 would be one of 5."""
    c, i32 = host_cache("int8", "int8", False), torch.int32
    q, table, lens = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 3), dtype=i32), torch.zeros(2, dtype=i32)
    cu, slots, two = torch.zeros(3, dtype=i32), torch.zeros(4, dtype=torch.int64), torch.zeros(2, dtype=i32)
    decode = dict(max_context_len=9, window=4, num_sinks=0, num_ctas=0)
    prefill = dict(max_query_len=1, max_context_len=9, window=4, num_sinks=0)
    size = dict(num_seqs=2, num_q_heads=4, max_query_len=1, max_context_len=9)
    plan = dict(block_size=16, num_blocks=3)
    for good, call in (
            (decode, lambda **kw: kvq.kvq_decode_window(c, q, q, table, lens, sm_scale=0.1, **kw)),
            (prefill, lambda **kw: kvq.kvq_paged_prefill(c, q, q, cu, table, lens, sm_scale=0.1, **kw)),
            (size, lambda **kw: kvq.kvq_prefill_workspace_size(c, total_q=2, **kw)),
            (plan, lambda **kw: kvq.kvq_plan_step(lens, lens, table, lens, two, slot_mapping=slots, positions=slots.int(),
                                                  context_lens_out=lens, cu_new=cu, free_range_out=two, **kw))):
        for name in good:
            with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
                call(**{**good, name: value})
