"""GPU tests of the page operators against plain Python over the same state: every length, table
entry, count and plane byte equal."""
import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache, KVCache, PagePool, _lib
from tests import _kv8

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.asarray(a).dtype)).cuda()


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _state(kind, pages, lens, width, seed, heads=3, shared=True):
    """A pool with sequences of the given lengths on shuffled pages, and the same in plain Python."""
    rng = np.random.default_rng(seed)
    u8 = lambda *s: rng.integers(0, 256, s, dtype=np.uint8)  # noqa: E731
    planes = {}
    if kind in ("nvfp4", "both"):
        planes.update(k_data=u8(pages, 4, 128, 64), k_scale=u8(pages, 4, 128, 8), v_data=u8(pages, 4, 128, 64),
                      v_scale=u8(pages, 4, 128, 8), ki_data=u8(pages, 128, 64), ki_scale=u8(pages, 128, 8))
    if kind in ("kv8", "both"):
        f = lambda: rng.random((pages, heads), dtype=np.float32)  # noqa: E731
        planes.update(k8_data=u8(pages, heads, 128, 128), k8_scale=f(), v8_data=u8(pages, heads, 128, 128), v8_scale=f())
    table = np.full((len(lens), width), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    free = list(rng.permutation(pages))
    for s, n in enumerate(lens):
        full = n // 128
        prev = s - 1
        for c in range((n + 127) // 128):
            if shared and prev >= 0 and c < full and c < lens[prev] // 128 and c < 2 and s % 2:
                table[s, c] = table[prev, c]          # a shared prefix of full pages
            else:
                table[s, c] = free.pop()
            refs[table[s, c]] += 1
    ref = _kv8.Pool(np.asarray(lens, np.int32), table, refs, planes)
    dev = {n: _cuda(a) for n, a in planes.items()}
    caches = []
    if kind in ("nvfp4", "both"):
        caches.append(KVCache(*(dev[n] for n in ("k_data", "k_scale", "v_data", "v_scale", "ki_data", "ki_scale"))))
    if kind in ("kv8", "both"):
        caches.append(KV8Cache(*(dev[n] for n in ("k8_data", "k8_scale", "v8_data", "v8_scale"))))
    pool = PagePool(caches, _cuda(np.asarray(lens, np.int32)), _cuda(table), _cuda(refs))
    return pool, ref, dev


def _same(pool, ref, dev):
    assert np.array_equal(pool.seq_lens.cpu().numpy(), ref.lens)
    assert np.array_equal(pool.block_table.cpu().numpy(), ref.table)
    assert np.array_equal(pool.ref_counts.cpu().numpy(), ref.refs)
    for n, a in ref.planes.items():
        assert np.array_equal(dev[n].cpu().numpy().view(np.uint8), a.view(np.uint8)), n


KINDS = ["nvfp4", "kv8", "both"]


@pytest.mark.parametrize("kind", KINDS)
def test_copy(kind):
    pool, ref, dev = _state(kind, 40, [300], 4, 1)
    rng = np.random.default_rng(2)
    perm = rng.permutation(40).astype(np.int32)
    dst, src = perm[:15].copy(), rng.choice(perm[15:], 15).astype(np.int32)
    src[3], dst[4] = -1, -9                                   # skipped
    dst[5] = src[5]                                           # onto itself
    tokens = rng.integers(0, 129, 15).astype(np.int32)
    tokens[:3] = [0, 128, 1]
    pool.copy(_cuda(src), _cuda(dst), _cuda(tokens))
    ref.copy(src, dst, tokens)
    assert pool.errors() == 0
    _same(pool, ref, dev)
    src[5], dst[5] = perm[20], perm[5]
    pool.copy(_cuda(src), _cuda(dst))
    ref.copy(src, dst)
    assert pool.errors() == 0
    _same(pool, ref, dev)


def test_copy_bad_entries_are_flagged_and_skipped():
    pool, ref, dev = _state("kv8", 20, [300], 4, 1)
    pool.copy(_i32(1, 20, 3), _i32(2, 4, 1 << 30), _i32(5, 6, 7))
    ref.copy([1], [2], [5])
    assert pool.errors() == _lib.FLAG_BAD_PAGE
    pool.copy(_i32(1, 2), _i32(8, 9), _i32(129, -1))
    assert pool.errors() == _lib.FLAG_BAD_LENGTH
    _same(pool, ref, dev)


@pytest.mark.parametrize("kind", KINDS)
def test_fork_then_grow_then_free(kind):
    lens = [300, 512, 129, 0, 1, 128] + [0] * 12
    pool, ref, dev = _state(kind, 64, lens, 9, 3)
    parents = [0, 0, 1, 2, 4, 5, 3, 0]
    children = [6, 7, 8, 9, 10, 11, 12, 13]
    pool.fork(_i32(*parents), _i32(*children))
    ref.fork(parents, children)
    assert pool.errors() == 0
    _same(pool, ref, dev)
    rows, to = [6, 8, 12, 9, 0, 15], [301, 900, 130, 100, 384, 9 * 128]
    pool.reserve(_i32(*rows), _i32(*to))
    ref.reserve(rows, to)
    assert pool.errors() == 0
    _same(pool, ref, dev)
    gone = [0, 6, 9, 13, 3]
    pool.free(_i32(*gone))
    ref.free(gone)
    assert pool.errors() == 0
    _same(pool, ref, dev)
    pool.fork(_i32(1, 8), _i32(0, 6))                        # freed pages and rows are used again
    ref.fork([1, 8], [0, 6])
    assert pool.errors() == 0
    _same(pool, ref, dev)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool.compact(num_live=live)
    assert int(live) == ref.compact()
    assert pool.errors() == 0
    _same(pool, ref, dev)


def test_fork_reads_every_parent_as_it_was():
    """A parent may be another entry's child: it is still empty then."""
    pool, ref, dev = _state("kv8", 30, [300, 0, 0, 0], 4, 3)
    pool.fork(_i32(0, 1, 0), _i32(1, 2, 3))
    ref.fork([0, 1, 0], [1, 2, 3])
    assert pool.errors() == 0
    _same(pool, ref, dev)
    assert pool.seq_lens.tolist() == [300, 300, 0, 300]


def test_fork_bad_entries():
    pool, ref, dev = _state("kv8", 30, [300, 200, 0, 0, 0], 4, 3)
    parents, children = [0, 5, 0, -1, 0, 1, 2, 0], [2, 3, 1, 3, 2, 9, 2, 4]
    with pytest.raises(_lib.MSAError):
        pool.fork(_i32(*parents), _i32(*children))           # more entries than sequences
    pool.fork(_i32(*parents[:5]), _i32(*children[:5]))
    ref.fork(parents[:1], children[:1])                      # the others: bad parent, child in use, bad parent, twice
    assert pool.errors() == _lib.FLAG_BAD_SEQ
    _same(pool, ref, dev)
    pool.fork(_i32(*parents[5:]), _i32(*children[5:]))
    ref.fork(parents[7:], children[7:])
    assert pool.errors() == _lib.FLAG_BAD_SEQ
    _same(pool, ref, dev)


def test_fork_and_reserve_out_of_pages():
    pool, ref, dev = _state("kv8", 8, [300, 256, 0, 0, 0, 0, 0], 6, 3, shared=False)    # 3 free pages
    pool.fork(_i32(0, 0, 1, 0, 0), _i32(2, 3, 4, 5, 6))      # the fourth tail finds none; row 4 needs none
    ref.fork([0, 0, 1, 0], [2, 3, 4, 5])
    assert pool.errors() == _lib.FLAG_NO_PAGE
    _same(pool, ref, dev)
    pool.free(_i32(2, 3))
    ref.free([2, 3])
    pool.reserve(_i32(0, 1, 4, 5), _i32(384, 600, 257, 380))  # 0, then 3 of 2 free pages, then nothing more
    ref.reserve([0, 1, 4, 5], [384, 600, 257, 380])
    assert pool.errors() == _lib.FLAG_NO_PAGE
    _same(pool, ref, dev)
    pool.reserve(_i32(0, 1, 4, 1, 7, -1), _i32(384, 6 * 128 + 1, 100, 300, 5, 5))
    assert pool.errors() == _lib.FLAG_BAD_LENGTH | _lib.FLAG_BAD_SEQ   # 1 beyond its row, 1 again, no such rows
    ref.reserve([0, 1, 4], [384, 6 * 128 + 1, 100])
    _same(pool, ref, dev)


def test_free_bad_entries():
    pool, ref, dev = _state("kv8", 20, [300, 200, 500], 4, 3)
    pool.free(_i32(1, 1, -1, 1, 3))
    ref.free([1])
    assert pool.errors() == _lib.FLAG_BAD_SEQ
    _same(pool, ref, dev)
    page = int(pool.block_table[0, 0])
    pool.ref_counts[page] = 0                                # a page that nobody counted
    pool.free(_i32(0))
    assert pool.errors() == _lib.FLAG_BAD_PAGE
    assert int(pool.ref_counts[page]) == 0 and int(pool.ref_counts.min()) == 0


@pytest.mark.parametrize("pages,seqs,live", [(1, 1, 1), (5, 2, 0), (64, 7, 40), (300, 20, 299), (3000, 40, 1500), (3000, 3, 10)])
def test_compact_beside_the_old_tables(pages, seqs, live):
    rng = np.random.default_rng(pages + live)
    cuts = np.sort(rng.integers(0, live + 1, seqs - 1))
    counts = np.diff(np.concatenate([[0], cuts, [live]]))
    lens = [int(c) * 128 - (int(rng.integers(0, 128)) if c else 0) for c in counts]
    pool, ref, dev = _state("kv8" if pages > 1000 else "both", pages, lens, max(1, int(counts.max())), pages, heads=1, shared=False)
    t, r = torch.full_like(pool.block_table, 77), torch.full_like(pool.ref_counts, 77)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):                                       # the inputs are as they were: the same again
        pool.compact(t, r, n)
        assert pool.errors() == 0
    assert np.array_equal(pool.block_table.cpu().numpy(), ref.table)
    assert np.array_equal(pool.ref_counts.cpu().numpy(), ref.refs)
    assert int(n) == ref.compact() == live
    assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(r.cpu().numpy(), ref.refs)
    for name, a in ref.planes.items():
        assert np.array_equal(dev[name].cpu().numpy().view(np.uint8), a.view(np.uint8)), name


def test_many_forks_in_a_graph():
    """Sums over more entries than a block has threads, and a replayed capture."""
    S = 2600
    lens = [int(x) for x in np.random.default_rng(0).integers(1, 700, 40)] + [0] * (S - 40)
    pool, ref, dev = _state("kv8", 4000, lens, 8, 3, heads=1)
    parents = [i % 40 for i in range(S - 40)]
    children = list(range(40, S))
    p, c = _i32(*parents), _i32(*children)
    grown = [min(lens[x] + 130, 8 * 128) for x in parents]
    to = _i32(*grown)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.fork(p, c)
        pool.free(c)
        pool.fork(p, c)
        pool.reserve(c[:700], to[:700])
    g.replay()
    torch.cuda.synchronize()
    assert pool.errors() == 0
    ref.fork(parents, children)
    ref.free(children)
    ref.fork(parents, children)
    ref.reserve(children[:700], grown[:700])
    _same(pool, ref, dev)


def test_refusals():
    pool, ref, dev = _state("kv8", 20, [300, 200], 4, 3)
    for bad in (torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32),
                torch.zeros((2, 1), dtype=torch.int32, device="cuda"), _i32(1, 2, 3, 4)[::2]):
        with pytest.raises(ValueError):
            pool.free(bad)
    with pytest.raises(ValueError):
        pool.copy(_i32(1, 2), _i32(3))
    with pytest.raises(ValueError):
        pool.compact(pool.block_table, None)
    with pytest.raises(ValueError):
        PagePool(pool.caches, pool.seq_lens, pool.block_table, pool.ref_counts[:10].clone())
    with pytest.raises(ValueError):
        PagePool(pool.caches, pool.seq_lens.long(), pool.block_table, pool.ref_counts)
    with pytest.raises(ValueError):
        PagePool(pool.caches * 5, pool.seq_lens, pool.block_table, pool.ref_counts)
    pool.free(_i32(0)[:0])
    pool.copy(_i32(0)[:0], _i32(0)[:0])
    assert pool.errors() == 0
    _same(pool, ref, dev)


def test_a_serving_run_over_the_8_bit_cache():
    """Prompts reserved and appended, attended, forked into samples, each continued on its own,
    some ended, the pool compacted: every step's attention against the same history kept apart."""
    rng = np.random.default_rng(7)
    H, G, P, S, M = 2, 8, 40, 6, 8
    cache = KV8Cache.empty(P, H)
    pool = PagePool.empty([cache], S, M)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    history = {}                                             # the pages of a sequence as they should be
    val = torch.from_numpy(_kv8.e4m3_values()).cuda()

    def step(rows):                                          # rows: {sequence: new tokens}
        seqs = sorted(rows)
        for s in seqs:
            history.setdefault(s, 0)
            history[s] += rows[s]
        lens = torch.tensor([history[s] for s in seqs], dtype=torch.int32, device="cuda")
        pool.reserve(_i32(*seqs), lens)
        indptr = np.concatenate([[0], np.cumsum([rows[s] for s in seqs])]).astype(np.int32)
        total = int(indptr[-1])
        k, v, q = (torch.from_numpy(rng.standard_normal((total, n, 128))).to(torch.bfloat16).cuda()
                   for n in (H, H, H * G))
        at = torch.tensor(seqs, device="cuda")
        batch = KV8Batch(pool.seq_lens[at].contiguous(), _cuda(indptr), pool.block_table[at].contiguous(), q,
                         total_rows=total, max_rows_per_req=max(rows.values()))
        cache.append(batch, k, v, ws)
        att = KV8Attention(cache, batch)
        out = att.attend()
        table = batch.block_table.cpu().numpy()
        want = _kv8.attend(q.double().view(total, H, G, 128), cache, [history[s] for s in seqs], indptr, table)
        o, _, tol, _ = want
        assert bool(((out.double() - o).abs() <= tol).all())
        for i, s in enumerate(seqs):                         # what was appended is what the cache holds
            for j in range(rows[s]):
                pos = history[s] - rows[s] + j
                page = int(table[i, pos // 128])
                x = k[indptr[i] + j].double()
                sc = cache.k_scale[page].double()[:, None]
                got = val[cache.k_data[page, :, pos % 128].long()] * sc
                # half a step: 2^-4 of the value, 2^-10 scales for subnormals; a second rounding to
                # subnormals when the page's scale grew later in this call is not possible
                assert bool(((got - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * sc).all())
        assert pool.errors() == 0 and att.errors() == 0 and _lib.msa_get_error(ws) == 0

    step({0: 300, 1: 77})
    step({0: 1, 1: 1})
    pool.fork(_i32(0, 0, 1), _i32(2, 3, 4))
    history.update({2: history[0], 3: history[0], 4: history[1]})
    step({0: 1, 2: 1, 3: 3, 4: 8})
    before = cache.k_data[pool.block_table[2, :3].long()].clone(), cache.k_scale[pool.block_table[2, :3].long()].clone()
    step({0: 90})                                            # the parent goes on: the samples keep theirs
    after = cache.k_data[pool.block_table[2, :3].long()], cache.k_scale[pool.block_table[2, :3].long()]
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    pool.free(_i32(1, 3))
    history.pop(1), history.pop(3)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool.compact(num_live=live)
    assert int(live) == int((pool.ref_counts > 0).sum()) and torch.all(pool.ref_counts[int(live):] == 0)
    step({0: 1, 2: 2, 4: 1, 5: 130})
    pool.free(_i32(0, 2, 4, 5))
    assert pool.errors() == 0 and torch.all(pool.ref_counts == 0)


@pytest.mark.parametrize("S,pages", [(9000, 30000), (50, 5003)])
def test_plans_over_large_pools(S, pages):
    """More sequences and pages than one pass of the planning code takes; no cache bytes."""
    rng = np.random.default_rng(S)
    lens = [int(x) for x in rng.integers(0, 700 if S > 1000 else 9000, S)]
    empty = [int(x) for x in rng.permutation(S)[:S // 3]]
    for s in empty:
        lens[s] = 0
    pool, ref, dev = _state(None, pages, lens, 80, 5, shared=False)
    others = np.array([s for s in range(S) if lens[s] > 0])
    parents = [int(x) for x in rng.choice(others, len(empty))]
    pool.fork(_i32(*parents), _i32(*empty))
    ref.fork(parents, empty)
    assert pool.errors() == 0
    _same(pool, ref, dev)
    rows = [int(x) for x in rng.permutation(S)[:S // 2]]
    to = [min(int(ref.lens[s]) + int(rng.choice([0, 1, 130, 700])), 80 * 128) for s in rows]
    pool.reserve(_i32(*rows), _i32(*to))
    ref.reserve(rows, to)
    assert pool.errors() == 0
    _same(pool, ref, dev)
    gone = [int(x) for x in rng.permutation(S)[:S // 2]]
    pool.free(_i32(*gone))
    ref.free(gone)
    assert pool.errors() == 0
    _same(pool, ref, dev)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool.compact(num_live=live)
    assert int(live) == ref.compact()
    assert pool.errors() == 0
    _same(pool, ref, dev)


def test_replaced_tensors_are_refused():
    pool, ref, dev = _state("kv8", 20, [300, 0], 4, 3)
    pool.fork(_i32(0), _i32(1))
    pool.caches[0].k_data = pool.caches[0].k_data.clone()
    with pytest.raises(ValueError):
        pool.free(_i32(1))
    pool, ref, dev = _state("kv8", 20, [300, 0], 4, 3)
    pool.block_table = pool.block_table.clone()
    with pytest.raises(ValueError):
        pool.fork(_i32(0), _i32(1))


def test_a_pool_of_counts_alone():
    """No sequences and no caches: compact moves the counts, the other operators have nothing to do."""
    z = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    pool = PagePool([], none, torch.zeros((0, 3), dtype=torch.int32, device="cuda"), z(0, 2, 0, 1, 5))
    live = z(-1)
    pool.compact(num_live=live)
    pool.fork(none, none)
    pool.reserve(none, none)
    pool.free(none)
    pool.copy(none, none)
    assert int(live) == 3 and pool.ref_counts.tolist() == [1, 2, 5, 0, 0] and pool.errors() == 0
