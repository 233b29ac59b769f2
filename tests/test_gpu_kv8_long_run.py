"""The operators for long sequences over the 8-bit cache in one serving run, on the pool's own tables, and calls that the
other tests do not make."""
import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import DecodeBatch, KV8Attention, KV8Batch, KV8Cache, PagePool
from tests import _kv8, _kv8_long

pytestmark = pytest.mark.gpu

ALL = lambda t, p: t >= 0  # noqa: E731


def ints(x):
    return torch.tensor(np.asarray(x, np.int64).tolist(), dtype=torch.int32, device="cuda")


def test_prompt_beams_weights_eviction_window():
    """A prompt in two chunks with its weights; beams forked, decoded on shared pages; one of them cut to its heaviest tokens
    where it stands; it goes on with full attention and weights, then with a window."""
    H, G, n, beams = 2, 8, 1400, 4
    cache = KV8Cache.empty(80, H)
    pool = PagePool.empty([cache], 1 + beams, 16)
    w = torch.zeros((1 + beams, H, 16 * 128), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def step(first, count, rows, how="attend", **kw):
        total = count * rows
        k, v, q = (torch.randn((total, h, 128), device="cuda", generator=g).to(torch.bfloat16) for h in (H, H, H * G))
        batch = KV8Batch(pool.seq_lens[first:first + count], ints(range(0, total + 1, rows)), pool.block_table[first:first + count], q,
                         total_rows=total, max_rows_per_req=rows)
        cache.append(batch, k, v, ws)
        att = KV8Attention(cache, batch, max_groups=1, with_weights=True)
        out = getattr(att, how)(**kw)
        lens, table = batch.context_lens.cpu().numpy(), batch.block_table.cpu().numpy()
        indptr, q64 = np.arange(0, total + 1, rows), q.double().view(total, H, G, 128)
        window = kw.get("window")
        sees = ALL if window is None else (lambda t, p: (t > p - window) | (t < kw["sinks"]))
        want, lse, tol, tol_lse = _kv8_long.attend(q64, cache, lens, indptr, table, sees, False)
        _kv8_long.close(out, want, tol, f"{how} out")
        _kv8_long.close(att.lse, lse, tol_lse, f"{how} lse")
        if window is None:
            mine = w[first:first + count]
            before = mine.clone()
            att.add_weights(mine, mine, keep=0.75)
            got = _kv8_long.weights(q64, att.lse, cache, lens, indptr, table, before, 0.75, False)
            for (b, h), (x, bound) in got.items():
                _kv8_long.close(mine[b, h, :int(lens[b])], x, bound, f"weights {b} {h}")
        assert att.errors() == 0 and pool.errors() == 0

    pool.reserve(ints([0]), ints([900]))
    step(0, 1, 900)
    pool.reserve(ints([0]), ints([n]))
    step(0, 1, 500)
    pool.fork(ints([0] * beams), ints(range(1, beams + 1)))
    w[1:] = w[0]
    for i in range(1, 4):
        pool.reserve(ints(range(1, beams + 1)), ints([n + i] * beams))
        step(1, beams, 1, "attend_shared", group_indptr=ints([0, beams]), min_saved=1)
    pool.evict(ints([2]), ints([2]), w, keep=400, sinks=4, recent=100)
    assert pool.errors() == 0 and int(pool.seq_lens[2]) == 400
    for i in range(1, 3):
        pool.reserve(ints([2]), ints([400 + i]))
        step(2, 1, 1)
    pool.reserve(ints([2]), ints([405]))
    step(2, 1, 3, window=130, sinks=4)
    # the other beams still decode on what they share
    for b in (1, 3, 4):
        pool.reserve(ints([b]), ints([n + 4]))
    step(3, 2, 1, "attend_shared", group_indptr=ints([0, 2]), min_saved=1)
    pool.free(ints(range(1 + beams)))
    assert int(pool.ref_counts.sum()) == 0 and pool.errors() == 0


def _setup(lens, rows, H, G, seed):
    lens_, indptr, table, pages = _kv8.batch_of(lens, rows, seed)
    k, ks = _kv8.fill(pages, H, seed + 1)
    v, vs = _kv8.fill(pages, H, seed + 2)
    q = torch.randn((int(indptr[-1]), H * G, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    batch = KV8Batch(ints(lens_), ints(indptr), torch.from_numpy(table).cuda(), q.to(torch.bfloat16), total_rows=int(indptr[-1]),
                     max_rows_per_req=max(1, max(rows)))
    return KV8Cache(k, ks, v, vs), batch


def test_batches_without_rows_and_without_requests():
    cache, batch = _setup([300, 0, 77], [0, 0, 0], 2, 4, 3)
    att = KV8Attention(cache, batch, max_groups=1, with_weights=True)
    att.attend(window=5, sinks=1)
    att.attend_shared(ints([0, 3]), min_saved=1)
    old = torch.rand((3, 2, 3 * 128), device="cuda")
    new = torch.full_like(old, -1.0)
    att.add_weights(old, new, keep=0.5)
    assert att.errors() == 0
    for b, n in enumerate((300, 0, 77)):
        assert torch.equal(new[b, :, :n], 0.5 * old[b, :, :n]) and (new[b, :, n:] == -1.0).all()
    none = KV8Batch(ints([]), ints([0]), torch.zeros((0, 3), dtype=torch.int32, device="cuda"), batch.q, total_rows=0, max_rows_per_req=1)
    att = KV8Attention(cache, none, max_groups=1, with_weights=True)
    att.attend(window=5)
    att.attend_shared(ints([0, 0]), min_saved=1)
    att.add_weights(old[:0], new[:0])
    assert att.errors() == 0


def test_calls_on_a_given_stream_see_what_it_wrote():
    """Every operator with stream=: inputs written there just before, results read there."""
    cache, batch = _setup([3000, 900], [2, 1], 4, 8, 5)
    att = KV8Attention(cache, batch, max_groups=1, with_weights=True)
    other = KV8Attention(cache, batch, max_groups=1, with_weights=True)
    old = torch.rand((2, 4, batch.block_table.shape[1] * 128), device="cuda")
    want = [att.attend(window=300, sinks=4).clone(), att.attend_shared(ints([0, 2]), min_saved=1).clone()]
    att.attend()
    want_w = att.add_weights(old, torch.zeros_like(old)).clone()
    q, o = batch.q.clone(), old.clone()
    batch.q.zero_()
    old.zero_()
    groups, lse = ints([0, 2]), att.lse.clone()
    new = torch.zeros_like(old)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        batch.q.copy_(q)
        old.copy_(o)
    got = [other.attend(window=300, sinks=4, stream=s)]
    with torch.cuda.stream(s):
        got[0] = got[0].clone()
    got.append(other.attend_shared(groups, stream=s, min_saved=1))
    with torch.cuda.stream(s):
        got[1] = got[1].clone()
    other.add_weights(old, new, lse=lse, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(new, want_w)


def test_decode_batches_and_replaced_tensors():
    """A DecodeBatch serves as a batch; tensors replaced in it are seen by the next call of every form."""
    cache, batch = _setup([2000, 300], [1, 1], 4, 8, 7)
    q8 = batch.q.to(torch.float8_e4m3fn).view(torch.uint8)
    db = DecodeBatch(batch.context_lens, batch.q_indptr, batch.block_table, q8, torch.zeros((2, 4, 128), dtype=torch.uint8, device="cuda"),
                     total_rows=2, max_rows_per_req=1)
    att = KV8Attention(cache, db, max_groups=1, with_weights=True)
    old = torch.rand((2, 4, batch.block_table.shape[1] * 128), device="cuda")

    def check(lens):
        q64 = db.q.view(torch.float8_e4m3fn).double().view(2, 4, 8, 128)
        table = db.block_table.cpu().numpy()
        out = att.attend(window=100, sinks=3)
        want, _, tol, _ = _kv8_long.attend(q64, cache, lens, [0, 1, 2], table, lambda t, p: (t > p - 100) | (t < 3))
        _kv8_long.close(out, want, tol, "window")
        want, _, tol, _ = _kv8_long.attend(q64, cache, lens, [0, 1, 2], table, ALL)
        _kv8_long.close(att.attend_shared(ints([0, 2]), min_saved=1), want, tol, "shared")
        att.attend()
        new = att.add_weights(old, torch.zeros_like(old))
        for (b, h), (x, bound) in _kv8_long.weights(q64, att.lse, cache, lens, [0, 1, 2], table, old, 1.0).items():
            _kv8_long.close(new[b, h, :lens[b]], x, bound, "weights")

    check([2000, 300])
    db.context_lens = ints([1500, 299])
    check([1500, 299])
    db.q = db.q.flip(0).contiguous()
    check([1500, 299])
    assert att.errors() == 0


def test_weights_at_the_end_of_a_wide_table():
    """Tables and weight rows far wider than the contexts; rows of weights that start on 4 bytes only."""
    cache, batch = _setup([300, 1000], [1, 4], 2, 8, 9)
    wide = torch.full((2, 2000), -1, dtype=torch.int32, device="cuda")
    wide[:, :batch.block_table.shape[1]] = batch.block_table
    batch.block_table = wide
    att = KV8Attention(cache, batch, max_groups=1, with_weights=True)
    att.attend()
    L = 2000 * 128 + 3
    old, new = torch.rand((2, 2, L), device="cuda"), torch.full((2, 2, L), -2.0, device="cuda")
    att.add_weights(old, new)
    q64 = batch.q.double().view(5, 2, 8, 128)
    for (b, h), (x, bound) in _kv8_long.weights(q64, att.lse, cache, [300, 1000], [0, 1, 5], wide.cpu().numpy(), old, 1.0, False).items():
        _kv8_long.close(new[b, h, :len(x)], x, bound, "weights")
        assert (new[b, h, len(x):] == -2.0).all()
    # a table so wide that the sizes alone let attend_shared look for common pages
    out, plain = att.attend_shared(ints([0, 2])).clone(), att.attend()
    want, _, tol, _ = _kv8_long.attend(q64, cache, [300, 1000], [0, 1, 5], wide.cpu().numpy(), ALL, False)
    _kv8_long.close(out, want, tol, "shared")
    _kv8_long.close(plain, want, tol, "plain")
    assert att.errors() == 0
