"""kvq_plan_step against the oracle, all outputs equal."""
import numpy as np
import pytest
import torch

from oracle import step as OS
from quantized_paged_kv_kvq_gb300 import kvq

from step_testing import DEV, ints

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, old, new, bs, max_tokens, free=None, width=None, seed=0, num_blocks=None, first=2):
        rng = np.random.default_rng(seed)
        self.old, self.new, self.bs, self.max_tokens = np.asarray(old), np.asarray(new), bs, max_tokens
        have, need = -(-self.old // bs), -(-(self.old + self.new) // bs)
        fresh = int((need - have).sum())
        nb = int(have.sum()) + fresh + 5 if num_blocks is None else num_blocks
        perm = rng.permutation(nb)
        width = int(need.max(initial=0)) + 1 if width is None else width
        self.table = np.full((len(old), width), -7)
        at = 0
        for s, n in enumerate(have):
            self.table[s, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:] if free is None else np.asarray(free)
        self.free = np.concatenate([np.full(first, -1, int), self.free])
        self.range = [first, len(self.free)]
        self.num_blocks = nb
        self.lens, self.add = ints(self.old), ints(self.new)
        self.block_table, self.free_blocks, self.free_range = ints(self.table), ints(self.free), ints(self.range)
        s = len(old)
        # one element more than the call is told of, to see that it stays as it was
        self.out = {"slots": torch.full((max_tokens + 4,), -99, dtype=torch.int64, device=DEV),
                    "positions": torch.full((max_tokens + 4,), -99, dtype=torch.int32, device=DEV),
                    "lens": torch.full((s,), -99, dtype=torch.int32, device=DEV),
                    "cu": torch.full((s + 1,), -99, dtype=torch.int32, device=DEV),
                    "range": torch.full((2,), -99, dtype=torch.int32, device=DEV)}

    def call(self, stream=None):
        o = self.out
        kvq.kvq_plan_step(self.lens, self.add, self.block_table, self.free_blocks, self.free_range, self.bs,
                          self.num_blocks, o["slots"][:self.max_tokens], o["positions"][:self.max_tokens],
                          o["lens"], o["cu"], o["range"], stream=stream)

    def check(self):
        slots, pos, after, cu, table, rng = OS.plan_step(self.old, self.new, self.table, self.free, self.range,
                                                         self.bs, self.max_tokens)
        torch.cuda.synchronize()
        for name, ref in (("slots", slots), ("positions", pos), ("lens", after), ("cu", cu), ("range", rng)):
            got = self.out[name].cpu().numpy()
            assert np.array_equal(got[:len(ref)], ref), name
            assert (got[len(ref):] == -99).all(), name
        assert np.array_equal(self.block_table.cpu().numpy(), table)


@pytest.mark.parametrize("seqs,old_hi,new_hi,bs,pad", [
    (1, 0, 1, 16, 0), (1, 5000, 1, 16, 3), (64, 4096, 1, 16, 0), (3, 9, 40, 8, 0), (300, 200, 20, 32, 11),
    (512, 64, 9, 64, 1), (513, 64, 9, 128, 2), (1500, 30, 12, 8, 0), (7, 1000, 6001, 16, 5), (5, 10, 0, 16, 9)])
def test_against_the_oracle(seqs, old_hi, new_hi, bs, pad):
    rng = np.random.default_rng(seqs + bs)
    old, new = rng.integers(0, old_hi + 1, seqs), rng.integers(0, new_hi + 1, seqs)
    st = Step(old, new, bs, int(new.sum()) + pad)
    st.call()
    st.check()
    st.call()  # nothing was consumed: the same again
    st.check()
    assert kvq.kvq_get_device_error() == 0


def test_lengths_at_page_edges():
    old = [0, 0, 1, 15, 16, 17, 31, 32, 0, 16]
    new = [0, 16, 15, 1, 1, 15, 2, 32, 17, 0]
    st = Step(old, new, 16, sum(new) + 1)
    st.call()
    st.check()
    assert kvq.kvq_get_device_error() == 0


def test_no_requests_and_no_tokens():
    for st in (Step([], [], 16, 5, width=2), Step([], [], 16, 0, width=0), Step([4, 0], [0, 0], 16, 0)):
        st.call()
        st.check()
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("free", [0, 1, 5])
def test_free_blocks_run_out(free):
    st = Step([20, 0, 3], [30, 40, 50], 16, 130, free=np.arange(free), num_blocks=40)
    st.call()
    st.check()  # the oracle gives -1 to the pages left over
    assert kvq.kvq_get_device_error() == kvq.DEVERR_FREE_BLOCKS


def test_more_tokens_than_room():
    st = Step([4, 9], [30, 40], 16, 33)
    st.call()
    st.check()
    assert kvq.kvq_get_device_error() == kvq.DEVERR_TOKENS


def test_bad_ids_and_lengths_are_flagged():
    st = Step([20, 8], [1, 30], 16, 31)
    st.block_table[0, 1] = st.num_blocks  # the page that request 0's token lands in
    st.free_blocks[2] = -3                # the first free block
    st.call()
    slots = st.out["slots"].cpu().numpy()
    table = st.block_table.cpu().numpy()
    assert kvq.kvq_get_device_error() == kvq.DEVERR_BLOCK_RANGE
    assert slots[0] == -1 and table[0, 1] == st.num_blocks
    assert table[1, 1] == -1 and (slots[9:25] == -1).all() and (slots[1:9] >= 0).all() and (slots[25:31] >= 0).all()

    st = Step([20, 8], [1, 3], 16, 8, width=2)
    st.lens[0], st.add[1] = -5, 1000  # below zero; wider than the table
    st.call()
    assert kvq.kvq_get_device_error() & kvq.DEVERR_CONTEXT_RANGE
    assert st.out["lens"].tolist() == [1, 32] and st.out["cu"].tolist() == [0, 1, 25]

    st = Step([20], [1], 16, 1)
    st.free_range[1] = 10 ** 6
    st.call()
    assert kvq.kvq_get_device_error() == kvq.DEVERR_FREE_BLOCKS
    assert st.out["range"].tolist() == [2, len(st.free)]


def test_replayed_from_a_graph_and_on_another_stream():
    st = Step([100, 3, 0], [1, 1, 1], 16, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    st.call(stream=s)
    s.synchronize()
    st.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        st.call()
    for step in range(1, 20):  # the lengths grow from step to step on the device
        st.old = st.old + 1
        st.lens.copy_(ints(st.old))
        st.table = st.block_table.cpu().numpy()
        st.range = st.out["range"].tolist() if step > 1 else st.range
        st.free_range.copy_(ints(st.range))
        g.replay()
        st.check()
    assert kvq.kvq_get_device_error() == 0


@pytest.mark.parametrize("rng", [(2, -2 ** 31), (2, -2 ** 31 + 1), (7, -2 ** 31 + 6), (2, 1), (2, -1), (-5, -3),
                                 (-2 ** 31, -2 ** 31), (2 ** 31 - 1, -2 ** 31), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_ranges_that_end_before_they_begin_hold_nothing(rng):
    """However far the end lies before the beginning: no entry of the list is taken."""
    st = Step([20, 0], [30, 20], 16, 50)
    st.free_range.copy_(ints(rng))
    st.call()
    first = min(max(rng[0], 0), len(st.free))
    assert kvq.kvq_get_device_error() == kvq.DEVERR_FREE_BLOCKS
    assert st.out["range"].tolist() == [first, first]
    table, slots = st.block_table.tolist(), st.out["slots"].tolist()
    assert table[0][2:4] == [-1, -1] and table[1][:2] == [-1, -1]
    assert table[0][:2] == st.table[0, :2].tolist()
    assert all(x >= 0 for x in slots[:12]) and slots[12:50] == [-1] * 38  # the held page's 12 free places
    assert st.out["cu"].tolist() == [0, 30, 50] and st.out["lens"].tolist() == [50, 20]
