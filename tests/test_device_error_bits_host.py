"""The device error word: the header's bits and the binding's are the same, each its own."""
import os
import re

from quantized_paged_kv_kvq_gb300 import kvq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def read(*path):
    with open(os.path.join(ROOT, *path), encoding="utf-8") as f:
        return f.read()


def test_header_and_binding_agree():
    header = {n: int(v) for n, v in re.findall(r"#define KVQ_(DEVERR_\w+) (\d+)u", read("include", "kvq.h"))}
    binding = {n: v for n, v in vars(kvq).items() if n.startswith("DEVERR_")}
    assert header == binding
    assert sorted(header.values()) == [1 << i for i in range(len(header))]


def test_a_window_out_of_place_is_not_reported_as_a_wait():
    """It cannot be brought about here, so the source: the check raises a bit of its own."""
    source = read("quantized_paged_kv_kvq_gb300", "csrc", "decode.cuh")
    check = source[source.index("if (C::BLOCK && base_s != raw_s)"):]
    assert f"raise_error({kvq.DEVERR_SHARED_WINDOW}u)" in check[:check.index("return;")]
