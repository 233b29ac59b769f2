"""msa_kv8_attn_shared: what one member of a group has stays with it, and what the groups' kernel decides."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, _lib
from tests import _kv8_long
from tests.test_gpu_kv8_shared import ALL, ints, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("plane", ["v_scale", "k_scale"])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -1.0, 1e-40, 2.0 ** 100])
@pytest.mark.parametrize("members,H,G,qtype", [(16, 2, 8, "bf16"), (16, 2, 8, "e4m3"), (8, 2, 8, "bf16"), (4, 2, 8, "e4m3"),
                                               (32, 1, 1, "bf16")])
def test_a_bad_scale_stays_with_its_member(members, H, G, qtype, scale, plane):
    """A scale outside what the cache allows on one member's own page: the other members' rows as if it were
    another, bit for bit. (With 16, 8 and 4 members of 8 queries the tile has 1, 2 and 4 copies of the rows.)"""
    cache, batch, lens, indptr, table, g = setup([(16, [(100 + 7 * i, 1) for i in range(members)])], H, G, qtype, 167)
    att = KV8Attention(cache, batch, max_groups=1)
    bad = 1
    page = int(table[bad, 16])
    want, want_lse = att.attend_shared(ints(g), min_saved=1).clone(), att.lse.clone()
    getattr(cache, plane)[page] = scale
    out, lse = att.attend_shared(ints(g), min_saved=1), att.lse
    others = [r for r in range(members) if r != bad]
    assert torch.isfinite(want).all()
    assert torch.equal(out[others], want[others]) and torch.equal(lse[others], want_lse[others])
    assert att.errors() == 0
    # and those bits are right
    q64 = batch.q.double().view(members, H, G, 128)
    ref, _, tol, _ = _kv8_long.attend(q64, cache, lens, indptr, table, ALL, qtype != "bf16")
    _kv8_long.close(out[others], ref[others], tol[others], "others")


def decided(att, num_reqs, groups):
    """What the groups' kernel left in the workspace behind the plain call's: [shared pages, first row, rows, first member]
    of each group, and each request's shared pages."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    n = ctypes.c_size_t(0)
    assert _lib.load().msa_kv8_attn_workspace_size(att._ref, ctypes.byref(n)) == 0
    at = up(n.value)
    g = att.ws[at:at + 16 * groups].view(torch.int32).view(groups, 4).tolist()
    at += up(16 * groups)
    return g, att.ws[at:at + 4 * num_reqs].view(torch.int32).tolist()


def expected(lens, indptr, table, indptr_g, H, G, min_saved):
    """The same from the rule: a group's pages are the leading ones that all members with rows list and that all their rows
    see whole; they are shared when that saves its part of min_saved reads of a page by a row chunk and head."""
    rows = np.diff(indptr)
    n = len(indptr_g) - 1
    most = max(min(-(-int(indptr[-1]) // n), 32), max(1, int(rows.max())))
    m = (1 << (min(most, 128) - 1).bit_length()) * G
    room = 128 // (4 if m <= 32 else 2 if m <= 64 else 1) // G
    alone = 1 << (room.bit_length() - 1)
    chunk = min(alone, 32)
    least = -(-min_saved // n)
    groups, skip = [], [0] * len(rows)
    for b0, b1 in zip(indptr_g[:-1], indptr_g[1:]):
        who = [b for b in range(b0, b1) if rows[b] > 0]
        pages = min((int(lens[b] - rows[b]) // 128 for b in who), default=0) if len(who) > 1 else 0
        for b in who:
            differs = np.nonzero(table[b, :pages] != table[b0, :pages])[0]
            pages = min([pages, *differs[:1]])
        tiles = lambda b, a, z: (int(lens[b]) - int(rows[b]) + z - 1) // 128 + 1  # noqa: E731  (its rows a .. z - 1)
        apart = sum(tiles(b, a, min(a + alone, int(rows[b]))) for b in who for a in range(0, int(rows[b]), alone))
        r0, r1 = int(indptr[b0]), int(indptr[b1])
        together = 0
        for a in range(r0, r1, chunk):
            together += pages
            for b in who:
                x, z = max(a, int(indptr[b])), min(a + chunk, int(indptr[b + 1]))
                together += tiles(b, x - int(indptr[b]), z - int(indptr[b])) - pages if x < z else 0
        # (what the kernel asks first, too: the others' pages at most)
        if pages and (min((len(who) - 1) * pages, apart - together) * H < least):
            pages = 0
        groups.append([int(pages), r0 if b0 < b1 else 0, r1 - r0, b0])
        for b in range(b0, b1):
            skip[b] = int(pages)
    return groups, skip


def check_decision(cache, batch, lens, indptr, table, g, min_saved, H, G):
    att = KV8Attention(cache, batch, max_groups=len(g) - 1)
    att.attend_shared(ints(g), min_saved=min_saved)
    assert att.errors() == 0
    got, want = decided(att, len(lens), len(g) - 1), expected(lens, indptr, table, g, H, G, min_saved)
    assert [x for x in got[0] if x[0]] == [x for x in want[0] if x[0]] and [x[0] for x in got[0]] == [x[0] for x in want[0]]
    assert got[1] == want[1]
    return want[1]


BEAMS = [(128, [(1 + 4 * i, 1) for i in range(64)])]


@pytest.mark.parametrize("H,G", [(32, 1), (16, 2), (4, 8)])
@pytest.mark.parametrize("groups,shares", [
    (BEAMS, True),                                                    # single rows: nearly all reads are saved
    ([(20, [(500 + 40 * i, 8) for i in range(16)])], None),           # speculative rows: see below
    ([(100, [(500 + 40 * i, 8) for i in range(16)])], True),
    ([(40, [(1 + 4 * i, 1) for i in range(63)] + [(300, 257)])], True),  # a prompt among them
    ([(64, [(549, 512), (613, 512)])], False),                        # prompts read the pages for each chunk of theirs
    ([(64, [(2085, 2048), (2149, 2048)])], False),
], ids=["beams", "speculative", "speculative_deep", "mixed", "prompts_512", "prompts_2048"])
def test_what_is_shared_goes_by_row_chunks(groups, shares, H, G):
    skip = check_decision(*setup(groups, H, G, "bf16", 177), 768, H, G)
    if shares is None:      # 8 queries a head: a chunk has two members' rows, so 16 - 8 of 16 reads of 20 pages by 4 heads are
        shares = G < 8      # saved, 640; with fewer there are 4 chunks of 32 rows and more heads: 16 x 12 x 20 and more
    assert (skip[0] > 0) == shares


@pytest.mark.parametrize("H,G", [(2, 8), (3, 1), (1, 64), (2, 5)])
def test_the_least_that_is_saved(H, G):
    """Both sides of the threshold: what the group saves, and one more."""
    for groups in ([(12, [(9, 2)] * 3)], [(40, [(5 + i, 1) for i in range(20)])], [(30, [(40 + 9 * i, 1 + i) for i in range(9)])]):
        args = setup(groups, H, G, "e4m3", 187)
        below, least = 0, 2 * 40 * 20 * H       # the group shares at the one (saving nothing is no loss), not at the other
        while least - below > 1:
            mid = (below + least) // 2
            below, least = (mid, least) if expected(*args[2:], H, G, mid)[0][0][0] else (below, mid)
        assert check_decision(*args, least - 1, H, G)[0] == groups[0][0]
        assert check_decision(*args, least, H, G)[0] == 0


def test_the_common_pages_of_a_group():
    """Tables that differ on some page, members that end inside the common pages, members without rows, empty groups."""
    H, G = 2, 8     # (chunks of 8 rows: the second group's 9 lie in as many as its members' do, so only nothing is saved)
    cache, batch, lens, indptr, table, g = setup([(30, [(5, 1), (7, 1), (300, 2)]), (30, [(40, 8), (3, 1), (9, 0)])], H, G, "e4m3", 197)
    assert check_decision(cache, batch, lens, indptr, table, g, 0, H, G) == [30] * 6
    for b, page in ((1, 17), (2, 29), (4, 0), (5, 3)):               # (the last has no rows: its entry does not count)
        t = table.copy()
        t[b, page] = cache.num_pages - 1
        batch.block_table = torch.from_numpy(t).cuda()
        skip = check_decision(cache, batch, lens, indptr, t, g, 0, H, G)
        assert skip == [page if b < 3 else 30] * 3 + [30 if b != 4 else page] * 3
    batch.block_table = torch.from_numpy(table).cuda()
    for b, n, pages in ((0, 16 * 128 + 1, 16), (0, 16 * 128, 15), (3, 20 * 128 + 8, 20), (3, 20 * 128 + 7, 19)):
        short = lens.copy()
        short[b] = n
        batch.context_lens = ints(short)
        skip = check_decision(cache, batch, short, indptr, table, g, 0, H, G)
        assert skip[3 * (b // 3)] == pages
    batch.context_lens = ints(lens)
    for indptr_g in ([0, 0, 3, 6], [1, 5], [2, 3, 5], [6, 6], [0, 6]):
        check_decision(cache, batch, lens, indptr, table, indptr_g, 0, H, G)


@pytest.mark.parametrize("H,G,qtype", [(4, 1, "bf16"), (2, 2, "bf16"), (4, 1, "e4m3"), (2, 2, "e4m3"), (1, 3, "bf16")])
@pytest.mark.parametrize("groups", [
    [(12, [(500, 300), (333, 333), (140, 129)]), (6, [(90, 70), (300, 1)])],          # prompts, as a rule alone
    [(40, [(1 + 4 * i, 1) for i in range(50)] + [(700, 300), (40, 33)]), (3, [(260, 256)])],   # one among beams: shared
    [(12, [(90, 50), (64, 64), (70, 33)]), (20, [(1 + i, 1) for i in range(10)] + [(60, 40)])],    # two copies of 64 rows
], ids=["alone", "mixed", "short"])
@pytest.mark.parametrize("least", [0, 1, 2 ** 31 - 1])
def test_prompts_of_few_queries_a_head(groups, H, G, qtype, least):
    """1 to 3 queries a KV head: a chunk of a request alone has up to 128 rows, one of a group 32. NaN values that some rows
    of a chunk see and others do not, in the first, the middle and the last chunks."""
    cache, batch, lens, indptr, table, g = setup(groups, H, G, qtype, 207)
    for b, n in enumerate(lens):
        r = int(indptr[b + 1] - indptr[b])
        for i, back in enumerate((r - 1, r - 2, r // 2, r // 2 - 40, 33, 32, 1, 0)):     # tokens of its own
            if 0 <= back < r:
                t = int(n) - 1 - back
                cache.v_data[int(table[b, t // 128]), i % H, t % 128, (37 * i + b) % 128] = 0x7F if i % 2 else 0xFF
    att = KV8Attention(cache, batch, max_groups=len(g) - 1)
    out = att.attend_shared(ints(g), min_saved=least)
    assert att.errors() == 0
    q64 = batch.q.double().view(len(batch.q), H, G, 128)
    want, lse, tol, tol_lse = _kv8_long.attend(q64, cache, lens, indptr, table, ALL, qtype != "bf16")
    assert torch.isnan(want).any() and not torch.isnan(want).all()
    _kv8_long.close(out, want, tol, "out")
    _kv8_long.close(att.lse, lse, tol_lse, "lse")


def test_tables_of_more_than_44_million_tokens_take_the_plain_call():
    """The groups' kernel adds up the own tiles of 2,048 row chunks in 32 bits: as many as 2,048 + 4,096 pieces of members,
    times the table's pages, have to fit."""
    cache, batch, lens, indptr, table, g = setup([(16, [(100 + 7 * i, 1) for i in range(3)])], 2, 8, "bf16", 217)
    for pages, shared in ((349_525, True), (349_526, False)):
        assert ((2048 + 4096) * pages < 2 ** 31) == shared
        wide = torch.full((3, pages), -1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = torch.from_numpy(table).cuda()
        batch.block_table = wide
        att = KV8Attention(cache, batch, max_groups=1)
        att.ws[256:].fill_(0x77)
        plain = att.attend().clone(), att.lse.clone()
        out = att.attend_shared(ints(g), min_saved=1)
        assert att.errors() == 0
        assert (decided(att, 3, 1)[0][0][0] == 16) == shared
        assert shared or (torch.equal(out, plain[0]) and torch.equal(att.lse, plain[1]))


@pytest.mark.parametrize("H,G", [(32, 1), (16, 2), (4, 8)])
@pytest.mark.parametrize("groups,at,looks", [
    (BEAMS, [0, 64], True),
    ([(256, [(1 + 4 * i, 1) for i in range(8)]), (0, [(2048, 2048)])], [0, 8], True),    # a long prompt beside them: 129 of its chunks
    ([(256, [(1 + 4 * i, 1) for i in range(8)] + [(2100, 2048)])], [0, 9], True),        # or with them
    ([(600, [(549, 512), (613, 512)])], [0, 2], False),                                   # nothing but prompts
    ([(600, [(549, 512), (613, 300), (700, 250)])], [0, 3], False),
    ([(600, [(549, 512), (613, 300), (700, 200)])], [0, 3], True),                        # 512 rows in all may be one request's
    ([(600, [(549, 512), (613, 1)])], [0, 2], False),                                     # 1 of 5 chunks and more
], ids=["beams", "beside", "among", "prompts", "uneven", "short", "one"])
def test_the_librarys_own_choice(groups, at, looks, H, G):
    """Whether the groups are looked at, by the sizes alone: where they are not, the call is attend() and their place in the
    workspace stays as it was."""
    cache, batch, lens, indptr, table, _ = setup(groups, H, G, "bf16", 227)
    att = KV8Attention(cache, batch, max_groups=1)
    att.ws[256:].fill_(0x77)
    plain = att.attend().clone(), att.lse.clone()
    out = att.attend_shared(ints(at))
    assert att.errors() == 0
    got, skip = decided(att, len(lens), 1)
    assert (got[0][0] != 0x77777777) == looks
    if looks:
        want = expected(lens, indptr, table, at, H, G, 768)
        assert got[0][0] == want[0][0][0] and skip[:at[1]] == want[1][:at[1]]
    else:
        assert torch.equal(out, plain[0]) and torch.equal(att.lse, plain[1])
