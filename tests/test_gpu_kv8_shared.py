"""msa_kv8_attn_shared: requests whose block tables begin with the same pages, against 64 bits."""
import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache, PagePool, _lib
from tests import _kv8, _kv8_long

pytestmark = pytest.mark.gpu

ALL = lambda t, p: t >= 0  # noqa: E731


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def setup(groups, H, G, qtype, seed):
    """groups: [(shared pages, [(tokens of its own, rows), ..]), ..]; returns what the tests need of the batch."""
    rng = np.random.default_rng(seed)
    lens = [p * 128 + n for p, members in groups for n, _ in members]
    rows = [r for _, members in groups for _, r in members]
    need = sum(p + sum((n + 127) // 128 for n, _ in members) for p, members in groups)
    perm = rng.permutation(need + 3).astype(np.int32)
    table = np.full((len(lens), max((n + 127) // 128 for n in lens) + 1), -1, np.int32)
    at, b, indptr_g = 0, 0, [0]
    for p, members in groups:
        front, at = perm[at:at + p], at + p
        for n, _ in members:
            m = (n + 127) // 128
            table[b, :p], table[b, p:p + m] = front, perm[at:at + m]
            at, b = at + m, b + 1
        indptr_g.append(b)
    pages = len(perm)
    k, ks = _kv8.fill(pages, H, seed + 1)
    v, vs = _kv8.fill(pages, H, seed + 2)
    cache = KV8Cache(k, ks, v, vs)
    g = torch.Generator(device="cuda").manual_seed(seed + 3)
    indptr = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    n = int(indptr[-1])
    q = torch.randn((n, H * G, 128), device="cuda", generator=g)
    q = q.to(torch.bfloat16) if qtype == "bf16" else q.to(torch.float8_e4m3fn)
    batch = KV8Batch(ints(lens), ints(indptr), torch.from_numpy(table).cuda(), q, total_rows=n, max_rows_per_req=max(1, max(rows)))
    return cache, batch, np.array(lens), indptr, table, indptr_g


def check(cache, batch, lens, indptr, table, indptr_g, flags=0, most=None, what=""):
    att = KV8Attention(cache, batch, max_groups=most or len(indptr_g) - 1)
    att.out.fill_(7.0)
    att.lse.fill_(7.0)
    out = att.attend_shared(ints(indptr_g), min_saved=1)
    assert att.errors() == flags
    n, heads = batch.q.shape[:2]
    q64 = batch.q.double().view(n, cache.num_kv_heads, heads // cache.num_kv_heads, 128)
    want, lse, tol, tol_lse = _kv8_long.attend(q64, cache, lens, indptr, table, ALL, batch.q.dtype != torch.bfloat16)
    _kv8_long.close(out, want, tol, f"{what} out")
    _kv8_long.close(att.lse, lse, tol_lse, f"{what} lse")
    return att


@pytest.mark.parametrize("H,G,qtype", [(4, 8, "e4m3"), (4, 8, "bf16"), (1, 1, "bf16"), (3, 5, "e4m3"), (2, 64, "bf16")])
@pytest.mark.parametrize("groups", [
    [(32, [(1, 1)] * 4)],                                            # samples of one prompt
    [(9, [(n, 1) for n in range(1, 40)])],                           # beams, own lengths around nothing
    [(20, [(128, 1), (129, 2), (300, 8), (8, 8)]), (40, [(5, 1), (1000, 3)]), (3, [(64, 1)])],
    [(17, [(1, 1), (4, 0), (9, 2), (700, 0)]), (0, [(50, 1), (60, 1)]), (11, [(3, 3)] * 3)],   # members without rows
], ids=["samples", "beams", "ragged", "rowless"])
def test_groups(groups, H, G, qtype):
    check(*setup(groups, H, G, qtype, 7), what="groups")


def test_prompts_that_share_a_prefix():
    check(*setup([(12, [(200, 150), (333, 333), (140, 129)]), (6, [(90, 70), (300, 1)])], 2, 4, "bf16", 17))


def test_prompts_of_many_chunks():
    """64 queries a KV head: a chunk has two rows, and a prompt more chunks than a warp has lanes."""
    check(*setup([(12, [(400, 300), (3, 1), (90, 70)]), (6, [(500, 480), (2, 2), (131, 129)])], 1, 64, "bf16", 19))
    check(*setup([(5, [(4300, 4200), (1, 1), (4000, 1)])], 1, 64, "e4m3", 20))


def test_more_members_than_a_plan_takes_at_once():
    check(*setup([(10, [(1 + i % 130, 1) for i in range(700)]), (12, [(3, 1)] * 40)], 1, 4, "e4m3", 27))


def test_deep_prefix():
    check(*setup([(700, [(n, 1) for n in (1, 50, 128, 200, 1000, 129)])], 2, 8, "bf16", 37))


def test_requests_outside_groups_and_empty_groups():
    cache, batch, lens, indptr, table, _ = setup([(16, [(5, 1), (7, 2)]), (16, [(40, 1)] * 3), (9, [(80, 1)] * 2)], 2, 8, "e4m3", 47)
    for indptr_g in ([2, 5], [0, 2, 2, 2], [7, 7], [1, 1, 7], [0], [3, 4, 4, 6]):
        check(cache, batch, lens, indptr, table, indptr_g, most=4, what=str(indptr_g))


def test_groups_that_share_less_than_they_say():
    """Tables that differ on some page, rows that begin inside a shared page, groups over unrelated requests."""
    cache, batch, lens, indptr, table, g = setup([(30, [(5, 1), (7, 1), (300, 2)]), (30, [(40, 8), (3, 1)])], 2, 8, "e4m3", 57)
    table[1, 17] = cache.num_pages - 1
    table[3, 0] = cache.num_pages - 2
    batch.block_table = torch.from_numpy(table).cuda()
    check(cache, batch, lens, indptr, table, g)
    check(cache, batch, lens, indptr, table, [0, 5])
    lens2 = lens.copy()
    lens2[0] = 16 * 128 + 3          # a member that ends inside the shared pages
    batch.context_lens = ints(lens2)
    check(cache, batch, lens2, indptr, table, g)


@pytest.mark.parametrize("indptr_g", [[0, 3, 2, 5], [-1, 5], [0, 6], [4, 1]])
def test_bad_groups_are_flagged_and_taken_alone(indptr_g):
    args = setup([(20, [(5, 1), (7, 1), (300, 2)]), (20, [(40, 8), (3, 1)])], 2, 8, "e4m3", 67)
    check(*args[:5], indptr_g, flags=_lib.FLAG_BAD_LENGTH)


def test_a_request_with_a_bad_length_leaves_its_group_alone():
    cache, batch, lens, indptr, table, g = setup([(20, [(5, 1), (7, 1), (300, 2)]), (20, [(40, 8), (3, 1)])], 2, 8, "e4m3", 77)
    bad = lens.copy()
    bad[1] = -4
    batch.context_lens = ints(bad)
    att = KV8Attention(cache, batch, max_groups=2)
    att.out.fill_(7.0)
    out = att.attend_shared(ints(g), min_saved=1)
    assert att.errors() == _lib.FLAG_BAD_LENGTH
    q64 = batch.q.double().view(-1, 2, 8, 128)
    want, _, tol, _ = _kv8_long.attend(q64, cache, lens, indptr, table, ALL)
    others = [0, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12]
    _kv8_long.close(out[others], want[others], tol[others], "others")
    assert (out[1] == 7.0).all()


def test_bad_pages_in_the_shared_part_and_behind():
    cache, batch, lens, indptr, table, g = setup([(24, [(5, 1), (200, 1), (300, 2)])], 2, 8, "e4m3", 87)
    table[:, 5] = cache.num_pages
    table[1, 24] = -1
    batch.block_table = torch.from_numpy(table).cuda()
    check(cache, batch, lens, indptr, table, g, flags=_lib.FLAG_BAD_PAGE)


def test_nan_and_scales():
    cache, batch, lens, indptr, table, g = setup([(24, [(5, 3), (200, 1), (300, 2)]), (10, [(9, 1)] * 3)], 2, 8, "e4m3", 97)
    cache.v_data[table[0, 3], 0, 17, 5] = 0x7F                 # every row of the first group sees it
    cache.v_data[table[1, 24], 1, 100, 9] = 0xFF               # one member
    cache.v_data[table[0, 24], 1, 4, 3] = 0x7F                 # the last of three rows
    cache.k_data[table[4, 10], 0, 8, 77] = 0x7F
    for i, e in enumerate((-60, 60, 0, 30)):
        cache.v_scale[table[2, 20 + i], :] = 2.0 ** e
    cache.v_scale[table[0, 4], :] = 0.0
    check(cache, batch, lens, indptr, table, g, what="NaN")


def test_one_half_far_below_the_other():
    """Keys of one half weigh nothing beside the other's."""
    cache, batch, lens, indptr, table, g = setup([(16, [(5, 1), (90, 1)])], 1, 8, "e4m3", 107)
    cache.k_scale[table[0, 16]] *= 60.0
    cache.k_scale[table[0, :16]] *= 1e-3
    check(cache, batch, lens, indptr, table, g)
    cache.k_scale[table[0, :16]] *= 6e4
    cache.k_scale[table[1, 16]] *= 1e-3
    check(cache, batch, lens, indptr, table, g)


def test_rows_behind_stay_and_runs_are_equal():
    cache, batch, lens, indptr, table, g = setup([(24, [(5, 1), (200, 1), (300, 2)])], 4, 8, "bf16", 117)
    q = torch.cat([batch.q, batch.q[:2]])
    batch = KV8Batch(batch.context_lens, batch.q_indptr, batch.block_table, q, total_rows=6, max_rows_per_req=2)
    att = KV8Attention(cache, batch, max_groups=1)
    att.out.fill_(3.0)
    first = att.attend_shared(ints(g), min_saved=1).clone()
    assert (first[4:] == 3.0).all()
    for _ in range(30):
        assert torch.equal(att.attend_shared(ints(g), min_saved=1), first)
    # calls with and without groups take turns on one workspace
    plain = att.attend().clone()
    assert torch.equal(att.attend_shared(ints(g), min_saved=1), first) and torch.equal(att.attend(), plain)


def test_captured_and_replayed_on_two_streams():
    cache, batch, *_, g = setup([(40, [(5 + i, 1) for i in range(20)])], 4, 8, "bf16", 127)
    gi = ints(g)
    a, b = (KV8Attention(cache, batch, max_groups=1) for _ in range(2))
    want = a.attend_shared(gi, min_saved=1).clone(), a.lse.clone()
    graphs = []
    for att in (a, b):
        att.attend_shared(gi, min_saved=1)
        torch.cuda.synchronize()
        att.out.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            att.attend_shared(gi, min_saved=1)
        graphs.append((graph, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for att in (a, b):
        assert torch.equal(att.out, want[0]) and torch.equal(att.lse, want[1])


def test_beams_forked_on_the_pool():
    """A prompt forked to beams that append tokens: the pool's own tables, their groups' pages found in them."""
    H, G = 4, 8
    cache = KV8Cache.empty(96, H)
    pool = PagePool.empty([cache], 9, 24)
    g = torch.Generator(device="cuda").manual_seed(3)
    n = 1500
    pool.reserve(ints([0]), ints([n]))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def append(first, count, rows):
        total = count * rows
        kv = [torch.randn((total, H, 128), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
        q = torch.randn((total, H * G, 128), device="cuda", generator=g).to(torch.bfloat16)
        batch = KV8Batch(pool.seq_lens[first:first + count], ints(range(0, total + 1, rows)), pool.block_table[first:first + count],
                         q, total_rows=total, max_rows_per_req=rows)
        cache.append(batch, *kv, ws)
        return batch

    append(0, 1, n)
    pool.fork(ints([0] * 8), ints(range(1, 9)))
    for step in range(1, 4):
        pool.reserve(ints(range(1, 9)), ints([n + step] * 8))
        batch = append(1, 8, 1)
        att = KV8Attention(cache, batch, max_groups=1)
        out = att.attend_shared(ints([0, 8]), min_saved=1).clone()
        assert pool.errors() == 0 and att.errors() == 0
        want, _, tol, _ = _kv8_long.attend(batch.q.double().view(8, H, G, 128), cache, [n + step] * 8, np.arange(9),
                                           pool.block_table[1:].cpu().numpy(), ALL, False)
        _kv8_long.close(out, want, tol, f"step {step}")


def test_what_sharing_has_to_save():
    """A group that saves too little is taken alone, by the same kernel or by the plain call; the bits tell them apart from
    the shared form only within its bounds."""
    cache, batch, lens, indptr, table, g = setup([(40, [(5 + i, 1) for i in range(20)]), (12, [(9, 2)] * 3)], 4, 8, "bf16", 147)
    att = KV8Attention(cache, batch, max_groups=2)
    plain = att.attend().clone(), att.lse.clone()
    want, lse, tol, tol_lse = _kv8_long.attend(batch.q.double().view(-1, 4, 8, 128), cache, lens, indptr, table, ALL, False)
    for least in (None, 0, 1, 2 * 12 * 2 * 4, 2 * 12 * 2 * 4 + 1, 2 * 40 * 19 * 4, 2 * 40 * 19 * 4 + 1, 2 ** 31 - 1):
        out = att.attend_shared(ints(g), min_saved=least)
        _kv8_long.close(out, want, tol, f"out at {least}")
        _kv8_long.close(att.lse, lse, tol_lse, f"lse at {least}")
    assert att.errors() == 0
    narrow = setup([(3, [(5, 1), (7, 1)])], 2, 8, "bf16", 157)
    att = KV8Attention(*narrow[:2], max_groups=1)
    plain = att.attend().clone(), att.lse.clone()
    out = att.attend_shared(ints([5, -1]))          # too little to save by the sizes: the groups are not looked at
    assert torch.equal(out, plain[0]) and torch.equal(att.lse, plain[1]) and att.errors() == 0


def test_refusals():
    cache, batch, *_ = setup([(3, [(5, 1), (7, 1)])], 2, 8, "e4m3", 137)
    att = KV8Attention(cache, batch, max_groups=2)
    for g in (ints([0, 1, 2, 2]), ints([]), torch.tensor([0, 2], device="cuda"), torch.tensor([0, 2], dtype=torch.int32),
              ints([[0, 2]]), ints([0, 9, 2, 9])[::2]):
        with pytest.raises(ValueError):
            att.attend_shared(g)
    for least in (-1, 2 ** 31):
        with pytest.raises(ValueError):
            att.attend_shared(ints([0, 2]), min_saved=least)
    with pytest.raises(ValueError):
        KV8Attention(cache, batch).attend_shared(ints([0, 2]))
    with pytest.raises(_lib.MSAError):
        KV8Attention(cache, batch, max_groups=-1)
