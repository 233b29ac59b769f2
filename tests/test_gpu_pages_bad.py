"""GPU tests of page operators on rows that list pages they should not: pages that nobody counts, and
page ids outside the pool."""
import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import _lib
from tests.test_gpu_pages import _i32, _same, _state

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def test_compact_leaves_entries_of_uncounted_pages():
    """A row lists pages whose count is 0, below the live ones' number and beyond it: the entries stay and
    the flag tells of them, whatever an earlier call has left in the workspace."""
    for beside in (False, True):
        pool, ref, dev = _state("kv8", 20, [0, 0, 0], 6, 3)
        ref.table[0, :3], ref.lens[0] = [9, 3, 12], 300
        ref.table[1, :2], ref.lens[1] = [15, 8], 256
        ref.refs[[9, 3, 12, 15, 8]] = 1
        for t, a in ((pool.block_table, ref.table), (pool.seq_lens, ref.lens), (pool.ref_counts, ref.refs)):
            t.copy_(torch.from_numpy(a))
        assert ref.compact() == 5
        pool.compact()                                       # leaves a map of these pages behind
        assert pool.errors() == 0
        _same(pool, ref, dev)
        # row 1 ends twice in the counts: its pages are free although row 2 still lists them and others
        ref.table[2, :5], ref.lens[2] = [2, 17, ref.table[1, 0], ref.table[1, 1], 19], 600
        ref.refs[ref.table[1, :2]] = 0
        ref.lens[1] = 0
        ref.refs[[2, 17]] = 1
        for t, a in ((pool.block_table, ref.table), (pool.seq_lens, ref.lens), (pool.ref_counts, ref.refs)):
            t.copy_(torch.from_numpy(a))
        counted = ref.refs > 0
        live = int(counted.sum())
        holes = [p for p in range(live) if not counted[p]]
        movers = [p for p in range(live, 20) if counted[p]]
        to = {m: h for m, h in zip(movers, holes)}
        want = ref.table.copy()
        uncounted = 0
        for s in range(3):
            for c in range((ref.lens[s] + 127) // 128):
                uncounted += not counted[ref.table[s, c]]
                want[s, c] = to.get(ref.table[s, c], ref.table[s, c])
        assert uncounted == 3
        t, r = pool.block_table, pool.ref_counts
        if beside:
            t, r = torch.full_like(t, 77), torch.full_like(r, 77)
            pool.compact(t, r)
        else:
            pool.compact()
        assert pool.errors() == _lib.FLAG_BAD_PAGE
        assert np.array_equal(t.cpu().numpy(), want)
        refs = np.zeros_like(ref.refs)
        for p in np.flatnonzero(counted):
            refs[to.get(p, p)] = ref.refs[p]
        assert np.array_equal(r.cpu().numpy(), refs)


def test_fork_of_a_row_with_a_bad_full_page():
    """The child is made with the entry as it stands; the page is counted nowhere and flagged."""
    for bad in (30, -3):
        pool, ref, dev = _state("kv8", 30, [400, 0, 0], 5, 3)
        before = ref.refs.copy()
        pool.block_table[0, 1] = bad
        pool.fork(_i32(0), _i32(1))
        assert pool.errors() == _lib.FLAG_BAD_PAGE
        t = pool.block_table.cpu().numpy()
        assert pool.seq_lens.tolist() == [400, 400, 0] and np.array_equal(t[1, :3], t[0, :3])
        free = int(np.flatnonzero(before == 0)[0])
        before[[t[0, 0], t[0, 2]]] += 1
        before[free] = 1
        assert t[1, 3] == free and np.array_equal(pool.ref_counts.cpu().numpy(), before)
        pool.free(_i32(1))                                   # and freed but for that entry
        assert pool.errors() == _lib.FLAG_BAD_PAGE
        before[[t[0, 0], t[0, 2]]] -= 1
        before[free] = 0
        assert np.array_equal(pool.ref_counts.cpu().numpy(), before) and pool.seq_lens.tolist() == [400, 0, 0]


def test_fork_of_a_row_with_a_bad_last_page():
    """Its partly filled last page cannot be copied: the entry does nothing, the others are served."""
    pool, ref, dev = _state("kv8", 30, [400, 300, 0, 0], 5, 3)
    pool.block_table[0, 3] = 30
    pool.fork(_i32(0, 1), _i32(2, 3))
    assert pool.errors() == _lib.FLAG_BAD_PAGE
    ref.fork([1], [3])
    ref.table[0, 3] = 30
    _same(pool, ref, dev)


def test_compact_beside_then_the_next_operator():
    """Tables of their own are copied over the pool's before it goes on."""
    pool, ref, dev = _state("kv8", 30, [0, 900, 0, 300], 9, 3, shared=False)
    t, r = torch.empty_like(pool.block_table), torch.empty_like(pool.ref_counts)
    pool.compact(t, r)
    assert ref.compact() == 11
    pool.block_table.copy_(t)
    pool.ref_counts.copy_(r)
    pool.reserve(_i32(0, 3), _i32(1000, 700))
    ref.reserve([0, 3], [1000, 700])
    pool.fork(_i32(1), _i32(2))
    ref.fork([1], [2])
    assert pool.errors() == 0
    _same(pool, ref, dev)
