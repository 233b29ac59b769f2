"""GPU tests of the 8-bit cache: the append bit for bit against its rule in 64 bits, the attention
against softmax attention in 64 bits within bounds derived from its roundings (tests/_kv8.py)."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache, _lib
from tests import _kv8

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------------- append
APPENDS = [
    # lens, rows, heads
    ([1], [1], 4),
    ([128, 129, 127, 1, 256], [1, 1, 1, 1, 1], 4),
    ([700, 130, 2000, 1, 450, 300], [3, 8, 0, 1, 5, 2], 4),
    ([131, 260, 8], [8, 8, 8], 1),
    ([133, 5], [7, 5], 3),
    ([300], [300], 4),                       # a whole prompt
    ([1000, 129, 640, 77], [873, 9, 0, 77], 8),
    ([128 * 9 + 1], [128 * 7], 2),
]


def _append_case(lens, rows, heads, dtype, seed, spread=6.0):
    lens, indptr, table, pages = _kv8.batch_of(lens, rows, seed)
    rng = np.random.default_rng(seed)
    total = int(indptr[-1])
    x = {}
    for n in ("k", "v"):
        a = rng.standard_normal((total, heads, 128)) * np.exp2(rng.uniform(-spread, spread, (total, heads, 1)))
        a[rng.random(a.shape) < 0.02] = 0.0
        x[n] = torch.from_numpy(a).to(dtype)
    planes = {}
    for n in ("k", "v"):
        planes[n + "_data"] = rng.integers(0, 256, (pages, heads, 128, 128), dtype=np.uint8)
        s = np.exp2(rng.uniform(-8, 4, (pages, heads))).astype(np.float32)
        s[rng.random(s.shape) < 0.5] = 2.0 ** -5
        planes[n + "_scale"] = s
    return lens, indptr, table, pages, x, planes


def _check_append(lens, rows, heads, dtype, seed, change=None):
    lens, indptr, table, pages, x, planes = _append_case(lens, rows, heads, dtype, seed)
    if change is not None:
        change(x, planes, table)
    cache = KV8Cache(**{n: _cuda(a) for n, a in planes.items()})
    batch = KV8Batch(_cuda(lens), _cuda(indptr), _cuda(table), total_rows=int(indptr[-1]),
                     max_rows_per_req=max(1, max(rows)))
    ws = _ws()
    cache.append(batch, x["k"].cuda(), x["v"].cuda(), ws)
    assert _lib.msa_get_error(ws) == 0
    for n in ("k", "v"):
        _kv8.append_plane(x[n].double().numpy(), lens, indptr, table, planes[n + "_data"], planes[n + "_scale"])
        got = getattr(cache, n + "_data").cpu().numpy()
        assert np.array_equal(getattr(cache, n + "_scale").cpu().numpy(), planes[n + "_scale"]), n
        bad = np.argwhere(got != planes[n + "_data"])
        # a NaN of either sign is the same NaN
        bad = [i for i in map(tuple, bad) if not (got[i] & 127 == 127 and planes[n + "_data"][i] & 127 == 127)]
        assert not bad, (n, len(bad), bad[0], got[bad[0]], planes[n + "_data"][bad[0]])


@pytest.mark.parametrize("lens,rows,heads", APPENDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_append_matches_the_rule_bit_for_bit(lens, rows, heads, dtype):
    _check_append(lens, rows, heads, dtype, seed=len(lens) * 100 + heads)


def test_append_scale_borders_and_special_values():
    def change(x, planes, table):
        for n in ("k", "v"):
            t = x[n]
            t[0] = 0.0                                   # nothing but zeros in a page
            t[1].fill_(448.0 * 2.0 ** -3)                 # exactly on a border
            t[2].fill_(448.0 * 2.0 ** -3 * (1 + 2.0 ** -7))
            t[3].fill_(1e-30)                            # below the smallest scale
            t[4, :, 5] = math.inf
            t[4, :, 6] = -math.inf
            t[5, :, 7] = math.nan
            t[6].fill_(-0.0)
            planes[n + "_scale"][table[7, 0]] = 0.0      # old slots that hold nothing
            planes[n + "_scale"][table[8, 0]] = math.nan
            planes[n + "_scale"][table[9, 0]] = 3.0 * 2.0 ** 20
    for dtype in (torch.bfloat16, torch.float32):
        _check_append([1, 2, 1, 1, 1, 1, 129, 9, 9, 9], [1] * 10, 2, dtype, seed=5, change=change)


def test_append_takes_strided_rows_one_source_and_leaves_the_rest():
    lens, indptr, table, pages, x, planes = _append_case([200, 77], [100, 77], 4, torch.bfloat16, 3)
    fused = torch.randn(177, 48 * 128).to(torch.bfloat16).cuda()
    k = fused.view(177, 48, 128)[:, 32:36]                # a slice of a fused projection's rows
    cache = KV8Cache(**{n: _cuda(a) for n, a in planes.items()})
    batch = KV8Batch(_cuda(lens), _cuda(indptr), _cuda(table), total_rows=177, max_rows_per_req=100)
    ws = _ws()
    cache.append(batch, k, None, ws)
    _kv8.append_plane(k.double().cpu().numpy(), lens, indptr, table, planes["k_data"], planes["k_scale"])
    for n, a in planes.items():                           # v untouched, slots past the end untouched
        assert np.array_equal(getattr(cache, n).cpu().numpy(), a), n
    assert _lib.msa_get_error(ws) == 0


def test_append_bad_pages_and_lengths_are_flagged_and_skipped():
    lens, indptr, table, pages, x, planes = _append_case([200, 77, 300], [2, 3, 1], 4, torch.float32, 9)
    table[1, 0] = pages + 5
    bad = lens.copy()
    bad[2] = 128 * table.shape[1] + 1                     # longer than its row
    cache = KV8Cache(**{n: _cuda(a) for n, a in planes.items()})
    batch = KV8Batch(_cuda(bad), _cuda(indptr), _cuda(table), total_rows=6, max_rows_per_req=3)
    ws = _ws()
    cache.append(batch, x["k"].cuda(), x["v"].cuda(), ws)
    assert _lib.msa_get_error(ws) == _lib.FLAG_BAD_PAGE | _lib.FLAG_BAD_LENGTH
    for n in ("k", "v"):
        _kv8.append_plane(x[n].double().numpy()[:2], lens[:1], indptr[:2], table[:1], planes[n + "_data"], planes[n + "_scale"])
        assert np.array_equal(getattr(cache, n + "_data").cpu().numpy(), planes[n + "_data"])
        assert np.array_equal(getattr(cache, n + "_scale").cpu().numpy(), planes[n + "_scale"])


def test_append_many_requests_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(1)
    lens = rng.integers(1, 500, 700).tolist()
    rows = [int(rng.integers(0, min(n, 8) + 1)) for n in lens]
    lens, indptr, table, pages, x, planes = _append_case(lens, rows, 2, torch.bfloat16, 21)
    cache = KV8Cache(**{n: _cuda(a) for n, a in planes.items()})
    batch = KV8Batch(_cuda(lens), _cuda(indptr), _cuda(table), total_rows=int(indptr[-1]), max_rows_per_req=8)
    ws, k, v = _ws(), x["k"].cuda(), x["v"].cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.append(batch, k, v, ws)
    g.replay()
    torch.cuda.synchronize()
    assert _lib.msa_get_error(ws) == 0
    for n in ("k", "v"):
        _kv8.append_plane(x[n].double().numpy(), lens, indptr, table, planes[n + "_data"], planes[n + "_scale"])
        assert np.array_equal(getattr(cache, n + "_data").cpu().numpy(), planes[n + "_data"])
        assert np.array_equal(getattr(cache, n + "_scale").cpu().numpy(), planes[n + "_scale"])


# ---------------------------------------------------------------------------------- attention
def _attn_case(lens, rows, H, G, q_type, seed, n_ids=0, q_level=1.5, pad_rows=0):
    lens, indptr, table, pages = _kv8.batch_of(lens, rows, seed)
    kd, ks = _kv8.fill(pages, H, seed + 1)
    vd, vs = _kv8.fill(pages, H, seed + 2)
    cache = KV8Cache(kd, ks, vd, vs)
    for b, n in enumerate(lens):              # slots past a context hold NaN codes
        if n % 128 and n > 0:
            page = int(table[b, n // 128])
            kd[page, :, n % 128:] = 0x7F
            vd[page, :, n % 128:] = 0xFF
    total = int(indptr[-1])
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((total, H * G, 128), device="cuda", generator=g) * q_level
    if q_type == "e4m3":
        q = x.to(torch.float8_e4m3fn).view(torch.uint8)
        qv = q.view(torch.float8_e4m3fn).double()
    else:
        q = x.to(torch.bfloat16)
        qv = q.double()
    ids = None
    if n_ids:
        rng = np.random.default_rng(seed)
        ids = np.full((len(lens), H, n_ids), -1, np.int32)
        for b, n in enumerate(lens):
            nb = (int(n) + 127) // 128
            for h in range(H):
                m = min(nb, n_ids)
                some = np.concatenate([rng.permutation(nb - 1)[:m - 1], [nb - 1]]) if nb else np.zeros(0, int)
                ids[b, h, rng.permutation(n_ids)[:len(some)]] = rng.permutation(some)
    batch = KV8Batch(_cuda(lens), _cuda(indptr), _cuda(table), q, total_rows=total, max_rows_per_req=max(1, max(rows)))
    return cache, batch, lens, indptr, table, qv.view(total, H, G, 128), ids


def _assert_attends(got, lse, ref):
    out, want_lse, tol, tol_lse = ref
    g, l = got.double(), lse.double()
    assert torch.equal(torch.isnan(g), torch.isnan(out))
    assert torch.equal(torch.isnan(l), torch.isnan(want_lse))
    over = torch.nan_to_num((g - out).abs() - tol, nan=-1.0)
    i = int(over.argmax())
    assert over.max() <= 0, (np.unravel_index(i, over.shape), float(g.view(-1)[i]), float(out.view(-1)[i]), float(tol.view(-1)[i]))
    inf = torch.isinf(want_lse)
    assert torch.equal(l[inf], want_lse[inf])
    fin = torch.isfinite(want_lse)
    assert bool(((l - want_lse)[fin].abs() <= tol_lse[fin]).all()), float(((l - want_lse)[fin].abs() - tol_lse[fin]).max())


def _check_attend(lens, rows, H, G, q_type, seed, n_ids=0, **kw):
    cache, batch, lens, indptr, table, qv, ids = _attn_case(lens, rows, H, G, q_type, seed, n_ids, **kw)
    att = KV8Attention(cache, batch)
    out = att.attend(None if ids is None else _cuda(ids))
    assert att.errors() == 0
    ref = _kv8.attend(qv, cache, lens, indptr, table, ids)
    _assert_attends(out, att.lse, ref)
    return att


ATTENDS = [
    # lens, rows, KV heads, query heads per KV head
    ([1], [1], 4, 8),
    ([127, 128, 129], [1, 1, 1], 4, 8),
    ([4096], [1], 4, 8),
    ([700, 130, 2000, 1, 4500, 3000], [3, 8, 1, 1, 5, 2], 4, 8),
    ([700, 0, 2000, 9], [3, 0, 0, 9], 4, 8),
    ([5000, 129], [8, 2], 1, 1),
    ([3000, 260], [4, 1], 3, 5),
    ([3000, 260], [2, 4], 2, 7),
    ([1025, 64], [1, 1], 8, 16),
    ([900, 200], [3, 2], 1, 64),
    ([20000], [8], 1, 8),
    ([300], [300], 4, 8),                      # whole prompts
    ([1000, 129, 77], [873, 9, 77], 2, 4),
    ([1500], [700], 1, 3),
    ([2100], [130], 1, 64),
    ([640] * 40, [1] * 40, 4, 8),
]


@pytest.mark.parametrize("lens,rows,H,G", ATTENDS)
@pytest.mark.parametrize("q_type", ["e4m3", "bf16"])
def test_attend_all_blocks(lens, rows, H, G, q_type):
    _check_attend(lens, rows, H, G, q_type, seed=sum(lens) % 1000)


@pytest.mark.parametrize("lens,rows,H,G,n_ids", [
    ([4096], [1], 4, 8, 16),
    ([9000, 130, 5000, 1, 4500], [3, 8, 1, 1, 5], 4, 8, 16),
    ([9000, 700], [8, 8], 2, 7, 4),
    ([6000] * 20, [2] * 20, 4, 8, 32),
    ([3000], [200], 2, 8, 5),
    ([500], [4], 1, 8, 1),
])
@pytest.mark.parametrize("q_type", ["e4m3", "bf16"])
def test_attend_listed_blocks(lens, rows, H, G, n_ids, q_type):
    _check_attend(lens, rows, H, G, q_type, seed=sum(lens) % 1000 + 1, n_ids=n_ids)


def test_attend_sharp_and_flat_scores():
    for level in (0.0, 0.05, 12.0):
        _check_attend([3000, 50], [4, 1], 2, 8, "bf16", seed=8, q_level=level)


def test_rows_that_see_nothing_are_zero():
    cache, batch, lens, indptr, table, qv, ids = _attn_case([3000, 700], [4, 2], 2, 8, "e4m3", 4, n_ids=8)
    ids[0] = -1                                          # no block at all
    ids[1, 0] = -1
    ids[1, 0, 3] = 5                                     # only the block that holds the rows themselves
    att = KV8Attention(cache, batch)
    out = att.attend(_cuda(ids))
    assert att.errors() == 0
    assert torch.all(out[:4] == 0) and torch.all(att.lse[:4] == -math.inf)
    _assert_attends(out, att.lse, _kv8.attend(qv, cache, lens, indptr, table, ids))
    # a prompt whose rows come before the only listed block see nothing either
    cache, batch, lens, indptr, table, qv, ids = _attn_case([300], [300], 1, 8, "bf16", 6, n_ids=2)
    ids[0, 0] = [-1, 2]
    att = KV8Attention(cache, batch)
    out = att.attend(_cuda(ids))
    assert torch.all(out[:256] == 0) and torch.all(att.lse[:256] == -math.inf)
    _assert_attends(out, att.lse, _kv8.attend(qv, cache, lens, indptr, table, ids))


def test_bad_ids_are_flagged_and_left_out():
    cache, batch, lens, indptr, table, qv, ids = _attn_case([3000, 700], [4, 2], 2, 8, "e4m3", 4, n_ids=8)
    ids[0, 0] = [3, 1, 3, 3, -1, 0, 1, -1]               # listed again: counted once
    ids[1, 1] = [0, 1, 99, 2, -5, 1 << 30, -1, -1]       # outside the context
    att = KV8Attention(cache, batch)
    out = att.attend(_cuda(ids))
    assert att.errors() == _lib.FLAG_BAD_IDS
    assert att.errors() == 0
    _assert_attends(out, att.lse, _kv8.attend(qv, cache, lens, indptr, table, ids))


def test_bad_pages_and_lengths():
    cache, batch, lens, indptr, table, qv, _ = _attn_case([3000, 700, 900], [4, 2, 1], 2, 8, "bf16", 4)
    table[0, 3], table[1, 5] = cache.num_pages, -7
    batch.block_table.copy_(_cuda(table))
    att = KV8Attention(cache, batch)
    out = att.attend()
    assert att.errors() == _lib.FLAG_BAD_PAGE
    _assert_attends(out, att.lse, _kv8.attend(qv, cache, lens, indptr, table))
    for bad in (-1, 24 * 128 + 1, 1):                    # negative, beyond its row, fewer than its rows
        l2 = lens.copy()
        l2[1] = bad
        batch.context_lens.copy_(_cuda(l2))
        att.out.fill_(7.0)
        att.lse.fill_(7.0)
        att.attend()
        assert att.errors() == _lib.FLAG_BAD_LENGTH | _lib.FLAG_BAD_PAGE
        assert torch.all(att.out[4:6] == 7.0) and torch.all(att.lse[4:6] == 7.0)
    batch.context_lens.copy_(_cuda(lens))


def test_values_that_a_row_does_not_see_never_reach_it():
    """NaN keys and values of later rows of the same step, and a NaN that is seen."""
    for rows, G in ((6, 8), (40, 8)):
        cache, batch, lens, indptr, table, qv, _ = _attn_case([261 + rows], [rows], 1, G, "bf16", 11)
        n = 261 + rows
        t = n - 3                                         # seen by the last three rows alone
        cache.v_data[int(table[0, t // 128]), 0, t % 128, 17] = 0x7F
        cache.v_data[int(table[0, t // 128]), 0, t % 128, 90] = 0xFF
        t = n - 2                                         # a key: its rows become NaN everywhere
        cache.k_data[int(table[0, t // 128]), 0, t % 128, 3] = 0x7F
        att = KV8Attention(cache, batch)
        out = att.attend()
        assert att.errors() == 0
        assert not torch.isnan(out[:rows - 3]).any()
        nan = torch.isnan(out[rows - 3])
        assert nan[:, [17, 90]].all() and int(nan.sum()) == 2 * G
        assert torch.isnan(out[rows - 2:]).all()
        ref = _kv8.attend(qv[:rows - 3], cache, [n - 3], np.array([0, rows - 3]), table)
        _assert_attends(out[:rows - 3], att.lse[:rows - 3], ref)


def test_scales_over_their_whole_range():
    for seed in (1, 2):
        cache, batch, lens, indptr, table, qv, _ = _attn_case([1500, 900], [4, 1], 2, 8, "e4m3", seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = cache.v_scale.shape
        cache.v_scale.copy_(torch.exp2(torch.randint(-60, 61, shape, device="cuda", generator=g).float()))
        cache.v_scale[torch.rand(shape, device="cuda", generator=g) < 0.2] = 0.0
        cache.k_scale.mul_(torch.exp2(torch.randint(-60, 1, shape, device="cuda", generator=g).float()))
        cache.k_scale[torch.rand(shape, device="cuda", generator=g) < 0.2] = 0.0
        att = KV8Attention(cache, batch)
        out = att.attend()
        assert att.errors() == 0
        _assert_attends(out, att.lse, _kv8.attend(qv, cache, lens, indptr, table))
        cache.v_scale.zero_()                             # nothing but zeros
        out = att.attend()
        assert torch.all(out == 0)
        _assert_attends(out, att.lse, _kv8.attend(qv, cache, lens, indptr, table))


def test_queries_of_wide_range():
    """Rows of very large and very small queries, zero rows, elements far below a row's largest."""
    cache, batch, lens, indptr, table, qv, _ = _attn_case([900], [8], 2, 8, "bf16", 3)
    q = batch.q
    q[0] = 0.0
    q[1] *= 2.0 ** -90
    q[2, :, ::2] *= 2.0 ** -12
    q[3, :, 1:] *= 2.0 ** -20
    q[4] *= 2.0 ** -130
    att = KV8Attention(cache, batch)
    out = att.attend()
    assert att.errors() == 0
    _assert_attends(out, att.lse, _kv8.attend(q.double().view(8, 2, 8, 128), cache, lens, indptr, table))
    q[5, 3, 7] = math.nan                                 # a NaN or an infinity stays in its row and head
    q[6, 1, 2] = math.inf
    again = att.attend()
    keep = torch.ones(8, 16, dtype=torch.bool)
    keep[5, 3] = keep[6, 1] = False
    assert torch.equal(again[keep], out[keep])
    assert torch.isnan(again[5, 3]).all() and torch.isnan(again[6, 1]).all()


def test_strided_queries_and_rows_behind_the_last_sequence():
    cache, batch, lens, indptr, table, qv, _ = _attn_case([300, 500], [5, 3], 2, 8, "bf16", 3)
    ref = KV8Attention(cache, batch).attend().clone()
    wide = torch.randn((11, 40, 128), device="cuda").to(torch.bfloat16)
    wide[:8, 4:20] = batch.q
    more = KV8Batch(batch.context_lens, batch.q_indptr, batch.block_table, wide[:, 4:20], total_rows=11, max_rows_per_req=6)
    att = KV8Attention(cache, more)
    att.out.fill_(3.0)
    att.lse.fill_(3.0)
    out = att.attend()
    assert att.errors() == 0
    assert torch.equal(out[:8], ref)
    assert torch.all(out[8:] == 3.0) and torch.all(att.lse[8:] == 3.0)


def test_same_bits_again_on_another_stream_and_in_a_graph():
    cache, batch, lens, indptr, table, qv, ids = _attn_case([20000, 3000, 700], [4, 8, 1], 4, 8, "bf16", 3, n_ids=16)
    ids = _cuda(ids)
    for sel in (None, ids):
        att = KV8Attention(cache, batch)
        first = att.attend(sel).clone()
        lse = att.lse.clone()
        for _ in range(3):
            assert torch.equal(att.attend(sel), first) and torch.equal(att.lse, lse)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        att.out.zero_()
        torch.cuda.synchronize()
        att.attend(sel, stream=s)
        s.synchronize()
        assert torch.equal(att.out, first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            att.attend(sel)
        att.out.zero_()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(att.out, first) and torch.equal(att.lse, lse) and att.errors() == 0
        # other lengths in the same captured call
        batch.context_lens.copy_(_cuda(np.array([129, 8, 1], np.int32)))
        batch.q_indptr.copy_(_cuda(indptr))
        if sel is None:
            l2 = np.array([129, 8, 1], np.int32)
            g.replay()
            torch.cuda.synchronize()
            assert att.errors() == 0
            _assert_attends(att.out, att.lse, _kv8.attend(qv, cache, l2, indptr, table))
        batch.context_lens.copy_(_cuda(lens))


def test_no_requests_no_rows():
    cache = KV8Cache.empty(2)
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    batch = KV8Batch(z, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((0, 1), dtype=torch.int32, device="cuda"),
                     torch.zeros((0, 32, 128), dtype=torch.bfloat16, device="cuda"), total_rows=0)
    att = KV8Attention(cache, batch)
    assert att.attend().shape == (0, 32, 128)
    cache.append(batch, torch.zeros((0, 4, 128), device="cuda"), None, _ws())


def test_refusals():
    cache, batch, lens, indptr, table, qv, ids = _attn_case([300, 500], [5, 3], 2, 8, "bf16", 3, n_ids=4)
    q = batch.q
    make = lambda **kw: KV8Batch(**{**dict(context_lens=batch.context_lens, q_indptr=batch.q_indptr,  # noqa: E731
                                           block_table=batch.block_table, q=q, total_rows=8, max_rows_per_req=5), **kw})
    for kw in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :15]), dict(q=q[:7]), dict(q=q[..., :64]),
               dict(context_lens=batch.context_lens.long()), dict(q_indptr=batch.q_indptr[:2]), dict(q=None),
               dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            KV8Attention(cache, make(**kw))
    with pytest.raises(_lib.MSAError):
        KV8Attention(cache, make(max_rows_per_req=2))                 # 8 rows cannot be two requests of 2
    with pytest.raises(_lib.MSAError):
        KV8Attention(cache, make(), sm_scale=0.0)
    odd = torch.zeros(8 * 16 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 16, 128)
    with pytest.raises(_lib.MSAError):
        KV8Attention(cache, make(q=odd)).attend()                     # not 16-byte aligned
    att = KV8Attention(cache, make())
    for bad in (_cuda(ids).long(), _cuda(ids)[:1], _cuda(ids)[:, :1]):
        with pytest.raises(ValueError):
            att.attend(bad)
    with pytest.raises(_lib.MSAError):
        att.attend(torch.zeros((2, 2, 33), dtype=torch.int32, device="cuda"))
    k = torch.zeros((8, 2, 128), device="cuda")
    for kk, vv in ((k.double(), None), (k, k.half()), (k[:7], None), (k[:, :1], None), (k.cpu(), None),
                   (k.transpose(0, 1).contiguous().transpose(0, 1), None)):
        with pytest.raises(ValueError):
            cache.append(make(), kk, vv, _ws())
    with pytest.raises(_lib.MSAError):
        cache.append(make(), k, None, torch.zeros(16, dtype=torch.uint8, device="cuda"))
    bad = torch.zeros(8 * 2 * 128 + 1, device="cuda")[1:].view(8, 2, 128)
    with pytest.raises(_lib.MSAError):
        cache.append(make(), bad, None, _ws())


def test_chosen_blocks_then_attention():
    """The indexer's selection on the NVFP4 index keys feeds the attention over the 8-bit cache."""
    from block_sparse_attention_nvfp4_gb300 import DecodeBatch, KVCache, MSADecoder
    from tests import _wl
    wl = _wl.small([4500, 3000, 700], [3, 8, 1], needles=3, seed=21)
    nv, batch = KVCache.from_host(wl), DecodeBatch.from_host(wl)
    dec = MSADecoder(nv, batch)
    ids = dec.select_blocks()
    kd, ks = _kv8.fill(nv.num_pages, 4, 1)
    vd, vs = _kv8.fill(nv.num_pages, 4, 2)
    cache = KV8Cache(kd, ks, vd, vs)
    att = KV8Attention(cache, batch)                       # a DecodeBatch serves as it is
    out = att.attend(ids)
    assert att.errors() == 0 and dec.errors() == 0
    qv = batch.q.view(torch.float8_e4m3fn).double().view(-1, 4, 8, 128)
    ref = _kv8.attend(qv, cache, wl.context_lens, wl.q_indptr, wl.block_table, ids.cpu().numpy())
    _assert_attends(out, att.lse, ref)


def test_attend_more_requests_than_threads():
    """A thread of the planning code sums several requests; some have no row, some one token."""
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 300, 1500)]
    rows = [min(n, int(r)) for n, r in zip(lens, rng.integers(0, 3, 1500))]
    _check_attend(lens, rows, 1, 4, "e4m3", seed=17)


@pytest.mark.parametrize("lens,rows,H,G", [
    ([4096, 4096, 900], [1, 1, 1], 4, 8),                # few rows: four copies of them in a tile
    ([9000, 260, 3000], [8, 1, 5], 2, 8),                # two
    ([5000, 300], [300, 300], 2, 8),                     # one: rows by chunks
])
@pytest.mark.parametrize("q_type", ["e4m3", "bf16"])
def test_many_runs_give_the_same_bits(lens, rows, H, G, q_type):
    cache, batch, *_ = _attn_case(lens, rows, H, G, q_type, 23)
    att = KV8Attention(cache, batch)
    first, lse = att.attend().clone(), att.lse.clone()
    for _ in range(40):
        att.out.fill_(7.0)
        assert torch.equal(att.attend(), first) and torch.equal(att.lse, lse)
    assert att.errors() == 0


def test_two_calls_at_once():
    """Two attentions, and an append to a third cache, in flight together on their own streams."""
    a = _attn_case([6000, 900], [2, 8], 4, 8, "bf16", 31)
    b = _attn_case([300, 2000], [300, 40], 4, 8, "e4m3", 32)
    atts = [KV8Attention(x[0], x[1]) for x in (a, b)]
    want = [(att.attend().clone(), att.lse.clone()) for att in atts]
    lens, indptr, table, pages, x, planes = _append_case([700, 130, 2000], [3, 8, 1], 4, torch.bfloat16, 33)
    caches = [KV8Cache(**{n: _cuda(p) for n, p in planes.items()}) for _ in range(2)]
    kb = KV8Batch(_cuda(lens), _cuda(indptr), _cuda(table), total_rows=int(indptr[-1]), max_rows_per_req=8)
    k, v, ws = x["k"].cuda(), x["v"].cuda(), _ws()
    caches[0].append(kb, k, v, ws)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for att in atts:
        att.out.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for att, s in zip(atts, streams):
            att.attend(stream=s)
    caches[1].append(kb, k, v, ws, stream=streams[2])
    torch.cuda.synchronize()
    for att, (out, lse) in zip(atts, want):
        assert torch.equal(att.out, out) and torch.equal(att.lse, lse) and att.errors() == 0
    for n in planes:
        assert torch.equal(getattr(caches[0], n), getattr(caches[1], n))
    assert _lib.msa_get_error(ws) == 0


def test_replaced_tensors_are_seen():
    cache, batch, lens, indptr, table, qv, _ = _attn_case([900, 300], [2, 1], 2, 8, "bf16", 41)
    att = KV8Attention(cache, batch)
    att.attend()
    batch.q = (batch.q.float() * -1.5).to(torch.bfloat16)
    _assert_attends(att.attend(), att.lse, _kv8.attend(batch.q.double().view(qv.shape), cache, lens, indptr, table))
    cache.k_data, cache.k_scale = cache.v_data.clone(), cache.v_scale.clone()
    qv = batch.q.double().view(qv.shape)
    _assert_attends(att.attend(), att.lse, _kv8.attend(qv, cache, lens, indptr, table))
    batch.context_lens.data = _cuda(np.array([500, 300], np.int32))       # the same object, another storage
    _assert_attends(att.attend(), att.lse, _kv8.attend(qv, cache, np.array([500, 300], np.int32), indptr, table))
    with pytest.raises(ValueError):
        att.attend(torch.zeros((2, 2, 0), dtype=torch.int32, device="cuda"))
    batch.q = batch.q[:2]
    with pytest.raises(ValueError):
        att.attend()


def test_offsets_past_32_bits():
    """A cache of 4.6 GB a plane: the same tokens on its last pages give the same bits as on a small one."""
    from block_sparse_attention_nvfp4_gb300 import PagePool
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    lens, rows = [900, 300], [900, 300]
    lens, indptr, table, pages, x, planes = _append_case(lens, rows, 4, torch.bfloat16, 51)
    k, v = x["k"].cuda(), x["v"].cuda()
    q = torch.randn((3, 32, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    total = 70000
    got = []
    for size, first in ((pages, 0), (total, total - pages)):
        cache = KV8Cache.empty(size, 4)
        t = _cuda(np.where(table >= 0, table + first, table).astype(np.int32))
        ws = _ws()
        cache.append(KV8Batch(_cuda(lens), _cuda(indptr), t, total_rows=1200, max_rows_per_req=900), k, v, ws)
        att = KV8Attention(cache, KV8Batch(_cuda(lens), _cuda(np.array([0, 2, 3], np.int32)), t, q, total_rows=3,
                                           max_rows_per_req=2))
        att.attend()
        assert _lib.msa_get_error(ws) == 0 and att.errors() == 0
        got.append([att.out, att.lse] + [getattr(cache, n)[first:].clone() for n in planes])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    pool = PagePool([cache], torch.zeros(1, dtype=torch.int32, device="cuda"),
                    torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros(total, dtype=torch.int32, device="cuda"))
    pool.copy(_cuda(np.array([total - 1, total - pages], np.int32)), _cuda(np.array([total // 2, total - pages - 1], np.int32)))
    for n in planes:
        p = getattr(cache, n)
        assert torch.equal(p[total // 2], p[total - 1]) and torch.equal(p[total - pages - 1], p[total - pages])
    assert pool.errors() == 0
