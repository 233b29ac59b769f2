"""msa_kv8_attn_weights: the attention that each cached token got, against 64 bits."""
import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache, _lib
from tests import _kv8, _kv8_long

pytestmark = pytest.mark.gpu


def setup(lens, rows, H, G, qtype, seed, strided=False, extra=0):
    lens_, indptr, table, pages = _kv8.batch_of(lens, rows, seed)
    k, ks = _kv8.fill(pages, H, seed + 1)
    v, vs = _kv8.fill(pages, H, seed + 2)
    cache = KV8Cache(k, ks, v, vs)
    g = torch.Generator(device="cuda").manual_seed(seed + 3)
    n = int(indptr[-1])
    q = torch.randn((n, H * G, 128), device="cuda", generator=g)
    q = q.to(torch.bfloat16) if qtype == "bf16" else q.to(torch.float8_e4m3fn)
    if strided:
        wide = torch.zeros((n, H * G + 2, 128), dtype=q.dtype, device="cuda")
        wide[:, :H * G] = q
        q = wide[:, :H * G]
    batch = KV8Batch(torch.from_numpy(lens_).cuda(), torch.from_numpy(indptr).cuda(), torch.from_numpy(table).cuda(), q,
                     total_rows=n, max_rows_per_req=max(1, max(rows)))
    shape = (len(lens), H, table.shape[1] * 128 + extra)
    old = torch.rand(shape, device="cuda", generator=g) * 3
    return cache, batch, lens_, indptr, table, old


def q64(batch, cache):
    n, heads = batch.q.shape[:2]
    return batch.q.double().view(n, cache.num_kv_heads, heads // cache.num_kv_heads, 128)


def check(cache, batch, lens, indptr, table, old, keep=1.0, restart=False, flags=0, in_place=False, lse=None):
    att = KV8Attention(cache, batch, with_weights=True)
    if lse is None:
        att.attend()
        att.errors()
        lse = att.lse
    new = old.clone() if in_place else torch.full_like(old, -5.0)
    att.add_weights(None if restart else (new if in_place else old), new, keep=keep, lse=lse)
    assert att.errors() == flags
    want = _kv8_long.weights(q64(batch, cache), lse, cache, lens, indptr, table, None if restart else old, keep,
                             batch.q.dtype != torch.bfloat16)
    for (b, h), (w, tol) in want.items():
        n = int(lens[b])
        _kv8_long.close(new[b, h, :n], w, tol, f"request {b} head {h}")
        rest = new[b, h, n:]
        assert torch.equal(rest, old[b, h, n:] if in_place else torch.full_like(rest, -5.0))
    return att, new, want


@pytest.mark.parametrize("H,G,qtype", [(4, 8, "e4m3"), (4, 8, "bf16"), (1, 1, "bf16"), (3, 5, "e4m3"), (2, 64, "bf16")])
@pytest.mark.parametrize("rows", [1, 2, 8])
def test_decode_steps(H, G, qtype, rows):
    lens = [rows, 9, 127, 128, 129, 255, 256, 257, 640, 1500, 3001]
    rs = [min(rows, n) for n in lens]
    check(*setup(lens, rs, H, G, qtype, 11))


@pytest.mark.parametrize("H,G,qtype", [(1, 1, "bf16"), (3, 16, "e4m3"), (2, 64, "bf16"), (4, 8, "bf16"), (5, 7, "e4m3")])
def test_prompts_and_mixed_rows(H, G, qtype):
    check(*setup([700, 5, 1031, 130, 260, 1], [300, 5, 9, 0, 131, 1], H, G, qtype, 21, strided=True))


def test_whole_prompts():
    check(*setup([1300, 513], [1300, 513], 2, 8, "bf16", 31))


@pytest.mark.parametrize("keep,restart,in_place", [(0.5, False, False), (0.0, False, False), (1.0, True, False), (0.9, False, True),
                                                   (2.0, True, True)])
def test_kept_weights(keep, restart, in_place):
    check(*setup([700, 5, 1031], [30, 5, 0], 2, 8, "bf16", 41, extra=36), keep=keep, restart=restart, in_place=in_place)


def test_weights_of_a_row_sum_to_one():
    cache, batch, lens, indptr, table, old = setup([5000, 333], [1, 1], 4, 8, "bf16", 51)
    _, new, _ = check(cache, batch, lens, indptr, table, old, restart=True)
    for b, n in enumerate(lens):
        assert (new[b, :, :n].double().sum(1) - 8).abs().max() < 8 * 2.0 ** -14


def test_rows_without_a_finite_lse_are_left_out():
    cache, batch, lens, indptr, table, old = setup([700, 300], [9, 2], 2, 4, "bf16", 61)
    att = KV8Attention(cache, batch)
    att.attend()
    lse = att.lse.clone()
    lse[3, 2], lse[4, 7], lse[5, 0] = -float("inf"), float("nan"), float("inf")
    batch.q = batch.q.clone()
    batch.q[6, 1, 5], batch.q[7, 4, 9] = float("nan"), float("inf")
    check(cache, batch, lens, indptr, table, old, lse=lse)
    cache2, batch2, *rest = setup([700, 300], [9, 2], 2, 4, "e4m3", 61)
    codes = batch2.q.view(torch.uint8).clone()
    codes[2, 3, 77] = 0xFF
    batch2.q = codes.view(torch.float8_e4m3fn)
    att = KV8Attention(cache2, batch2)
    att.attend()
    lse = att.lse.nan_to_num(nan=1.0)
    check(cache2, batch2, *rest, lse=lse)


def test_nan_keys_get_nothing_and_spoil_nothing():
    """NaN codes behind the context, and in a key that only rows with a NaN lse see."""
    cache, batch, lens, indptr, table, old = setup([400, 300], [60, 1], 2, 4, "e4m3", 71)
    for b, n in enumerate(lens):
        cache.k_data[table[b, (n - 1) // 128], :, (n - 1) % 128 + 1:] = 0x7F
    cache.k_data[table[0, 2], 0, 380 - 256, 5] = 0xFF
    check(cache, batch, lens, indptr, table, old)


def test_far_scales():
    cache, batch, lens, indptr, table, old = setup([600, 300], [3, 1], 2, 4, "bf16", 81)
    cache.k_scale[table[0, 1]] = 0.0
    cache.k_scale[table[0, 2]] *= 2.0 ** -40
    cache.k_scale[table[1, 0]] *= 16.0
    check(cache, batch, lens, indptr, table, old)


def test_bad_pages_and_lengths():
    cache, batch, lens, indptr, table, old = setup([1000, 900, 300], [3, 1, 2], 2, 4, "e4m3", 91)
    table[0, 6], table[1, 0] = -1, cache.num_pages
    batch.block_table = torch.from_numpy(table).cuda()
    check(cache, batch, lens, indptr, table, old, flags=_lib.FLAG_BAD_PAGE)
    bad = lens.copy()
    bad[1] = 10 ** 6
    batch.context_lens = torch.from_numpy(bad).cuda()
    att = KV8Attention(cache, batch, with_weights=True)
    att.attend()
    att.errors()
    new = torch.full_like(old, -5.0)
    att.add_weights(old, new)
    assert att.errors() == _lib.FLAG_BAD_LENGTH | _lib.FLAG_BAD_PAGE
    assert (new[1] == -5.0).all() and not (new[2, :, :300] == -5.0).any()


def test_many_requests_and_far_positions():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 40, 1500)]
    check(*setup(lens, [1] * len(lens), 1, 2, "e4m3", 101))
    n, r = 200_003, 40
    cache, batch, _, indptr, _, _ = setup([1500], [r], 2, 8, "e4m3", 111)
    table = rng.integers(0, cache.num_pages, (1, (n + 127) // 128)).astype(np.int32)
    batch = KV8Batch(torch.tensor([n], dtype=torch.int32, device="cuda"), batch.q_indptr, torch.from_numpy(table).cuda(), batch.q,
                     total_rows=r, max_rows_per_req=r)
    old = torch.rand((1, 2, table.shape[1] * 128), device="cuda")
    check(cache, batch, np.array([n]), indptr, table, old)


def test_equal_bits_captured_and_replayed():
    cache, batch, *_, old = setup([2000, 900, 4100], [300, 1, 80], 4, 8, "bf16", 121)
    a, b = (KV8Attention(cache, batch, with_weights=True) for _ in range(2))
    outs = [torch.zeros_like(old) for _ in range(2)]
    a.attend(), b.attend()
    want = a.add_weights(old, outs[0]).clone()
    for _ in range(20):
        assert torch.equal(a.add_weights(old, outs[0]), want)
    graphs = []
    for att, new in zip((a, b), outs):
        att.add_weights(old, new)
        torch.cuda.synchronize()
        new.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            att.attend()
            att.add_weights(old, new)
        graphs.append((g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for att, new in zip((a, b), outs):
        assert torch.equal(new, want) and att.errors() == 0


def test_steps_add_up():
    """Three decode steps in place: a token's weight is what all rows since its own gave it."""
    H, G, n = 2, 4, 700
    cache, _, _, _, table, _ = setup([n + 3], [1], H, G, "bf16", 131)
    total = torch.zeros((1, H, table.shape[1] * 128), device="cuda")
    want = torch.zeros((H, n + 3), dtype=torch.float64, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    bound = torch.zeros_like(want)
    for step in range(1, 4):
        q = torch.randn((1, H * G, 128), device="cuda", generator=g).to(torch.bfloat16)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        batch = KV8Batch(ints([n + step]), ints([0, 1]), torch.from_numpy(table).cuda(), q, total_rows=1, max_rows_per_req=1)
        att = KV8Attention(cache, batch, with_weights=True)
        att.attend()
        att.add_weights(total, total)
        got = _kv8_long.weights(q64(batch, cache), att.lse, cache, [n + step], [0, 1], table, None, 1.0, False)
        for h in range(H):
            want[h, :n + step] += got[0, h][0]
            bound[h, :n + step] += got[0, h][1]
    for h in range(H):
        _kv8_long.close(total[0, h, :n + 3], want[h], bound[h] + 3 * 2.0 ** -24 * want[h], f"head {h}")


def test_refusals():
    cache, batch, *_, old = setup([300], [1], 2, 4, "e4m3", 141)
    att = KV8Attention(cache, batch, with_weights=True)
    att.attend()
    new = torch.zeros_like(old)
    for o, x, kw in ((old, new[..., :128], {}), (old[:, :1], new, {}), (old, new.double(), {}), (old.cpu(), new, {}),
                     (old, new.transpose(0, 1), {}), (old, new, dict(lse=att.lse[:, :3])), (old, new, dict(lse=att.lse.double()))):
        with pytest.raises(ValueError):
            att.add_weights(o, x, **kw)
    for keep in (-0.5, float("nan"), float("inf")):
        with pytest.raises(_lib.MSAError):
            att.add_weights(old, new, keep=keep)
    with pytest.raises(ValueError):
        KV8Attention(cache, batch).add_weights(old, new)
    with pytest.raises(ValueError):
        KV8Attention(cache, batch, with_lse=False, with_weights=True).add_weights(old, new)
