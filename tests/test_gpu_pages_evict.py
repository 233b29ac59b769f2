"""msa_pages_evict: sequences cut to their heaviest tokens, against a plain form, bit for bit."""
import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache, KVCache, PagePool, _lib
from tests import _kv8, _kv8_long

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x, np.int64).tolist(), dtype=torch.int32, device="cuda")


def setup(lens, empty, heads, seed, spare=0, pow2=True, share=0, width=None, extra=0):
    """A pool of len(lens) sequences and `empty` empty ones over len(heads) caches; `share`: pages that the second and later
    sequences have in common with the first."""
    rng = np.random.default_rng(seed)
    need = [(n + 127) // 128 for n in lens]
    total = sum(need) + spare
    perm = rng.permutation(total).astype(np.int32)
    M = width or max(need + [1])
    table = np.full((len(lens) + empty, M), -1, np.int32)
    refs = np.zeros(total, np.int32)
    at = 0
    for b, m in enumerate(need):
        row = perm[at:at + m].copy()
        at += m
        if b and share:
            k = min(share, m, need[0])
            row[:k] = table[0, :k]
        table[b, :m] = row
        for x in row:
            refs[x] += 1
    caches, weights = [], []
    for c, h in enumerate(heads):
        k, ks = _kv8.fill(total, h, seed + 10 * c + 1)
        v, vs = _kv8.fill(total, h, seed + 10 * c + 2)
        if pow2:
            ks, vs = (torch.exp2(torch.ceil(torch.log2(s))) for s in (ks, vs))
        caches.append(KV8Cache(k, ks, v, vs))
        w = rng.standard_normal((len(lens) + empty, h, M * 128 + extra)).astype(np.float32)
        weights.append(torch.from_numpy(np.exp(2 * w) * (rng.random(w.shape) > 0.2)).float().cuda())
    pool = PagePool(caches, ints(list(lens) + [0] * empty), torch.from_numpy(table).cuda(), torch.from_numpy(refs).cuda())
    return pool, weights


def host(pool, weights):
    state = tuple(t.cpu().numpy().copy() for t in (pool.seq_lens, pool.block_table, pool.ref_counts))
    planes = [{n: getattr(c, n).cpu().numpy().copy() for n in ("k_data", "k_scale", "v_data", "v_scale")} for c in pool.caches]
    return state, planes, [w.cpu().numpy().copy() for w in weights]


def same_codes(a, b):
    """Equal codes; NaN codes of either sign count alike."""
    return np.array_equal(np.where((a & 127) == 127, 127, a), np.where((b & 127) == 127, 127, b))


def check(pool, weights, parents, children, keep, sinks, recent, flags=0):
    state, planes, w = host(pool, weights)
    _kv8_long.evict(state, planes, w, parents, children, keep, sinks, recent)
    pool.evict(ints(parents), ints(children), weights, keep, sinks, recent)
    assert pool.errors() == flags
    got_state, got_planes, got_w = host(pool, weights)
    for name, a, b in zip(("lens", "table", "refs"), got_state, state):
        assert np.array_equal(a, b), name
    for a, b in zip(got_w, w):
        assert np.array_equal(a.view(np.uint32), b.view(np.uint32))
    for a, b in zip(got_planes, planes):
        for n in a:
            if n.endswith("scale"):
                assert np.array_equal(a[n].view(np.uint32), b[n].view(np.uint32)), n
            else:
                assert same_codes(a[n], b[n]), n


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (100, 4, 30), (127, 0, 0), (128, 0, 128), (129, 129, 0),
                                               (300, 4, 296), (500, 130, 0), (1000, 1, 333), (4000, 4, 64)])
@pytest.mark.parametrize("heads", [[4], [1, 3]])
def test_into_children(heads, keep, sinks, recent):
    lens = [1, 2, 127, 128, 129, 300, 1001, 2500]
    pool, weights = setup(lens, 8, heads, 3, spare=8 * 32 + 2)
    check(pool, weights, list(range(8)), list(range(15, 7, -1)), keep, sinks, recent)


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (130, 4, 60), (640, 1, 639), (2048, 4, 256)])
def test_where_they_stand(keep, sinks, recent):
    lens = [1, 200, 2048, 3001, 2049, 0]
    pool, weights = setup(lens, 0, [2, 2], 5, spare=70, share=9)
    check(pool, weights, [0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], keep, sinks, recent)


def test_children_of_one_parent_beside_cuts_in_place():
    pool, weights = setup([1500, 900, 700], 4, [3], 7, spare=60, share=4)
    check(pool, weights, [0, 1, 0, 2, 0], [3, 1, 4, 5, 6], 300, 4, 100)


@pytest.mark.parametrize("kind", ["equal", "zeros", "negative", "nan", "inf", "tiny", "neighbours", "few"])
def test_weights_that_tie_or_are_none(kind):
    """Ties go to the lowest positions, whatever passes of the selection they need."""
    pool, (w,) = setup([9000, 20000, 700], 3, [2], 11, spare=3 * 40)
    rng = np.random.default_rng(2)
    x = {"equal": np.full(w.shape, 0.5), "zeros": np.zeros(w.shape), "negative": -rng.random(w.shape),
         "nan": np.where(rng.random(w.shape) < 0.5, np.nan, rng.random(w.shape)),
         "inf": np.where(rng.random(w.shape) < 0.1, np.inf, rng.random(w.shape)),
         "tiny": rng.integers(0, 9, w.shape) * 2.0 ** -149,
         "neighbours": (rng.integers(0, 5, w.shape) + 0x3F800000).astype(np.int32).view(np.float32).reshape(w.shape),
         "few": rng.integers(0, 3, w.shape)}[kind]
    w.copy_(torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)))
    check(pool, [w], [0, 1, 2], [3, 4, 5], 1999, 3, 50)


@pytest.mark.parametrize("count", [1, 1023, 1024, 1025, 3000])
def test_tokens_that_share_all_but_the_last_digits(count):
    """`count` weights between 1 and 1 + 1024 steps, equal ones among them, and the last token kept is one of them."""
    N, heavy = 10_000, 500
    pool, (w,) = setup([N], 1, [2], 12, spare=20)
    rng = np.random.default_rng(count)
    x = rng.random((2, N)).astype(np.float32) * 0.5
    for h in range(2):
        at = rng.permutation(np.arange(10, N - 100))
        x[h, at[:heavy]] = 2 + rng.random(heavy)
        x[h, at[heavy:heavy + count]] = (rng.integers(0, 1024, count) + 0x3F800000).astype(np.int32).view(np.float32)
    w[0, :, :N] = torch.from_numpy(x).cuda()
    check(pool, [w], [0], [1], heavy + (count + 1) // 2 + 7 + 90, 7, 90)


@pytest.mark.parametrize("N", [4095, 4097, 8191, 8192, 8193, 8321, 12_289, 16_384, 20_481])
def test_lengths_around_what_warps_take(N):
    pool, weights = setup([N], 2, [1], 14, spare=60)
    check(pool, weights, [0], [1], 1000, 5, 77)
    check(pool, weights, [0], [2], 1000, 400, 600)   # none by its weight


def test_scales_that_are_no_powers_of_two_and_none():
    pool, weights = setup([1200, 600], 2, [2], 13, spare=20, pow2=False)
    c = pool.caches[0]
    for i, s in enumerate((0.0, -1.0, float("nan"), float("inf"), 2.0 ** -60, 2.0 ** 60, 1e-40)):
        c.k_scale[pool.block_table[0, i].long()] = s
    c.v_scale[pool.block_table[1].clamp(min=0).long()] = 0.0
    c.v_data[pool.block_table[0, 3].long(), 0, :, 5] = 0x7F
    check(pool, weights, [0, 1], [2, 3], 500, 4, 100)


def test_long_sequence_odd_table():
    pool, weights = setup([70_001], 1, [1], 17, spare=140, width=600, extra=3)
    check(pool, weights, [0], [1], 17_003, 5, 1000)


def test_entries_that_do_nothing():
    pool, weights = setup([900, 500, 300, 400], 4, [2], 19, spare=12)
    # out of range, child not empty, child twice, parent that is cut where it stands (as many entries as sequences)
    check(pool, weights, [-1, 0, 9, 0, 0, 1, 1, 3], [4, 8, 4, 1, 5, 5, 1, 6], 200, 4, 10, flags=_lib.FLAG_BAD_SEQ)


def test_parent_cut_in_place_is_nobody_elses():
    pool, weights = setup([900, 500], 3, [2], 23, spare=12)
    check(pool, weights, [0, 0, 1, 1], [2, 0, 3, 4], 200, 4, 10, flags=_lib.FLAG_BAD_SEQ)


def test_pages_run_out():
    pool, weights = setup([900, 500, 700], 3, [2], 29, spare=5)
    check(pool, weights, [0, 1, 2], [3, 4, 5], 300, 4, 10, flags=_lib.FLAG_NO_PAGE)


def test_bad_lengths_and_pages():
    pool, weights = setup([900, 500], 2, [2], 31, spare=12)
    pool.block_table[0, 2], pool.block_table[0, 4] = 10 ** 6, -3
    check(pool, weights, [0], [2], 300, 4, 10, flags=_lib.FLAG_BAD_PAGE)
    check(pool, weights, [0], [0], 300, 4, 10, flags=_lib.FLAG_BAD_PAGE)
    pool.seq_lens[1] = 10 ** 6
    pool.evict(ints([1]), ints([3]), weights, 300, 4, 10)
    assert pool.errors() == _lib.FLAG_BAD_LENGTH and pool.seq_lens[3] == 0


def test_more_sequences_than_a_plan_takes_at_once():
    n = 1500
    rng = np.random.default_rng(3)
    pool, weights = setup([int(x) for x in rng.integers(1, 200, n)], n, [1], 37, spare=n + 5)
    check(pool, weights, list(range(n)), list(range(n, 2 * n)), 50, 1, 10)


def test_equal_runs_and_growing_scratch():
    pool, weights = setup([3000, 2000], 2, [4], 41, spare=60)
    want = None
    for keep in (10, 2000, 300, 2000, 10, 2000):
        pool.evict(ints([0, 1]), ints([2, 3]), weights, keep, 4, 5)
        got = host(pool, weights)
        if keep == 2000:
            want = want or got
            for a, b in zip(got[0], want[0]):
                assert np.array_equal(a, b)
            for n in got[1][0]:
                assert np.array_equal(got[1][0][n][pool.block_table[2].clamp(min=0).cpu()], want[1][0][n][pool.block_table[2].clamp(min=0).cpu()])
        pool.free(ints([2, 3]))
    assert pool.errors() == 0


def test_captured_and_replayed():
    pool, weights = setup([3000, 2000, 900], 3, [2], 43, spare=60)
    par, ch = ints([0, 1, 2]), ints([3, 4, 5])
    pool.evict(par, ch, weights, 700, 4, 50)
    pool.free(ch)
    want = host(pool, weights)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.evict(par, ch, weights, 700, 4, 50)
        pool.free(ch)
    pool.evict(par, ch, weights, 900, 4, 50)      # (a larger scratch, while the graph keeps its own)
    pool.free(ch)
    weights[0][3:] = -1.0
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert pool.errors() == 0
    got = host(pool, weights)
    for b, n in ((3, 700), (4, 700), (5, 700)):
        assert np.array_equal(got[2][0][b, :, :n], want[2][0][b, :, :n])
        p = want[0][1][b, :6]
        assert np.array_equal(got[0][1][b, :6], p)
        for name in got[1][0]:
            x, y = got[1][0][name][p], want[1][0][name][p]
            if name.endswith("data"):
                x, y = x[:-1], y[:-1]              # (behind the last token the larger call's tokens stay)
            assert np.array_equal(x, y), name


def test_a_serving_run():
    """Prompt, weights, eviction, further tokens with weights, eviction where it stands: attention and weights over what
    is kept, against 64 bits on the pool's own tables."""
    H, G, n, keep = 2, 4, 1000, 300
    cache = KV8Cache.empty(40, H)
    pool = PagePool.empty([cache], 2, 12)
    w = torch.zeros((2, H, 12 * 128), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def step(s, rows):
        k, v, q = (torch.randn((rows, h, 128), device="cuda", generator=g).to(torch.bfloat16) for h in (H, H, H * G))
        batch = KV8Batch(pool.seq_lens[s:s + 1], ints([0, rows]), pool.block_table[s:s + 1], q, total_rows=rows, max_rows_per_req=rows)
        cache.append(batch, k, v, ws)
        att = KV8Attention(cache, batch, with_weights=True)
        out = att.attend()
        before = w[s:s + 1].clone()
        att.add_weights(w[s:s + 1], w[s:s + 1])
        assert att.errors() == 0 and pool.errors() == 0
        lens, table = pool.seq_lens[s:s + 1].cpu().numpy(), pool.block_table[s:s + 1].cpu().numpy()
        q64 = q.double().view(rows, H, G, 128)
        want, lse, tol, tol_lse = _kv8_long.attend(q64, cache, lens, [0, rows], table, lambda t, p: t >= 0, False)
        _kv8_long.close(out, want, tol, "out")
        got = _kv8_long.weights(q64, att.lse, cache, lens, [0, rows], table, before, 1.0, False)
        for (_, h), (x, bound) in got.items():
            _kv8_long.close(w[s, h, :int(lens[0])], x, bound, "weights")

    pool.reserve(ints([0]), ints([n]))
    step(0, n)
    check(pool, [w], [0], [1], keep, 4, 64)
    for i in range(1, 6):
        pool.reserve(ints([1]), ints([keep + i]))
        step(1, 1)
    check(pool, [w], [1], [1], 200, 4, 64)
    pool.reserve(ints([1]), ints([203]))
    step(1, 3)
    pool.free(ints([0, 1]))
    assert int(pool.ref_counts.sum()) == 0


def test_refusals():
    pool, weights = setup([300], 1, [2], 47, spare=5)
    a, b, (w,) = ints([0]), ints([1]), weights
    for args in ((a, b, w, 0), (a, b, w, 10, 5, 6), (a, b, w, 10, -1), (a, b, w, 10, 0, -1), (a, b, [w, w], 10), (a, b, w[..., :128], 10),
                 (a, b, w.double(), 10), (a, b, w[:1], 10), (a.long(), b, w, 10), (a, ints([1, 1]), w, 10), (a.cpu(), b, w, 10)):
        with pytest.raises(ValueError):
            pool.evict(*args)
    with pytest.raises(_lib.MSAError):
        pool.evict(ints([0, 0, 0]), ints([1, 1, 1]), w, 10)      # more entries than sequences
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    nvfp4 = KVCache(z(8, 4, 128, 64), z(8, 4, 128, 8), z(8, 4, 128, 64), z(8, 4, 128, 8), z(8, 128, 64), z(8, 128, 8))
    with pytest.raises(ValueError):
        PagePool.empty([nvfp4], 2, 4).evict(a, b, w, 10)
    assert pool.errors() == 0 and int(pool.seq_lens[1]) == 0
