"""msa_kv8_attn_window: attention to the last tokens and the first ones, against 64 bits."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache, _lib
from tests import _kv8, _kv8_long

pytestmark = pytest.mark.gpu


def setup(lens, rows, H, G, qtype, seed, level=1.0, strided=False):
    lens_, indptr, table, pages = _kv8.batch_of(lens, rows, seed)
    k, ks = _kv8.fill(pages, H, seed + 1, level)
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
    return cache, batch, lens_, indptr, table, q.double().view(n, H, G, 128)


def sees(window, sinks):
    return lambda t, p: (t > p - window) | (t < sinks)


def check(cache, batch, lens, indptr, table, q64, window, sinks, exact_q, what):
    att = KV8Attention(cache, batch)
    att.out.fill_(7.0)
    out = att.attend(window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert att.errors() == 0
    want, lse, tol, tol_lse = _kv8_long.attend(q64, cache, lens, indptr, table, sees(window, sinks), exact_q)
    _kv8_long.close(out, want, tol, f"{what} out")
    _kv8_long.close(att.lse, lse, tol_lse, f"{what} lse")
    return att


# windows below, at and above page and chunk borders; contexts shorter than the window; sinks in a page's middle, at
# its end, past a page and past the context
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (3, 4), (127, 0), (128, 128), (129, 130), (300, 4), (1000, 64),
                                          (100000, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 700)])
@pytest.mark.parametrize("H,G,qtype", [(4, 8, "e4m3"), (2, 5, "bf16")])
def test_single_tokens(H, G, qtype, window, sinks):
    lens = [1, 2, 127, 128, 129, 257, 640, 1500, 3001]
    args = setup(lens, [1] * len(lens), H, G, qtype, 11)
    check(*args, window, sinks, qtype == "e4m3", "tokens")


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (7, 130), (64, 4), (200, 0), (513, 129)])
@pytest.mark.parametrize("H,G,qtype", [(1, 1, "bf16"), (3, 16, "e4m3"), (2, 64, "bf16")])
def test_rows_and_prompts(H, G, qtype, window, sinks):
    lens, rows = [700, 5, 1031, 130, 260], [300, 5, 9, 0, 131]
    args = setup(lens, rows, H, G, qtype, 21)
    check(*args, window, sinks, qtype == "e4m3", "rows")


@pytest.mark.parametrize("qtype", ["bf16", "e4m3"])
def test_speculative_rows_strided(qtype):
    lens, rows = [40, 5000, 9000, 300, 2049], [8, 3, 8, 1, 5]
    args = setup(lens, rows, 4, 8, qtype, 31, strided=True)
    check(*args, 1024, 4, qtype == "e4m3", "speculative")


def test_window_of_everything_equals_the_plain_call():
    lens, rows = [513, 2000, 77], [8, 2, 1]
    cache, batch, *_ = setup(lens, rows, 4, 8, "bf16", 41)
    att = KV8Attention(cache, batch)
    a = att.attend().clone(), att.lse.clone()
    b = att.attend(window=4096).clone(), att.lse.clone()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pages_that_nobody_sees_are_not_looked_up():
    lens, rows = [4000, 2600], [2, 5]
    cache, batch, lens_, indptr, table, q64 = setup(lens, rows, 4, 8, "e4m3", 51)
    window, sinks = 500, 4
    for b, (n, r) in enumerate(zip(lens, rows)):
        first = (n - r - window + 1) // 128
        table[b, 1:first] = [-5, 10 ** 9, 2 ** 31 - 1, -2 ** 31][b % 4]
    batch.block_table = torch.from_numpy(table).cuda()
    check(cache, batch, lens_, indptr, table, q64, window, sinks, True, "stale entries")


def test_bad_pages_are_left_out_and_flagged():
    lens, rows = [1000, 900], [3, 1]
    cache, batch, lens_, indptr, table, q64 = setup(lens, rows, 2, 4, "e4m3", 61)
    table[0, 6] = -1
    table[1, 0] = cache.num_pages
    batch.block_table = torch.from_numpy(table).cuda()
    att = KV8Attention(cache, batch)
    out = att.attend(window=400, sinks=8)
    assert att.errors() == _lib.FLAG_BAD_PAGE
    want, lse, tol, tol_lse = _kv8_long.attend(q64, cache, lens_, indptr, table, sees(400, 8))
    _kv8_long.close(out, want, tol, "out")
    _kv8_long.close(att.lse, lse, tol_lse, "lse")


@pytest.mark.parametrize("window,sinks", [(1, 0), (6, 2), (40, 0), (150, 129)])
def test_nan_reaches_the_rows_that_see_it(window, sinks):
    """NaN codes in K and V at tokens inside and outside of windows; slots past the contexts hold NaN too."""
    lens, rows = [400, 37, 300], [60, 37, 1]
    cache, batch, lens_, indptr, table, q64 = setup(lens, rows, 2, 4, "e4m3", 71)
    rng = np.random.default_rng(5)
    for b, n in enumerate(lens):
        last = table[b, (n - 1) // 128]
        cache.k_data[last, :, (n - 1) % 128 + 1:] = 0x7F
        cache.v_data[last, :, (n - 1) % 128 + 1:] = 0xFF
        for t in rng.integers(0, n, 6):
            cache.v_data[table[b, t // 128], rng.integers(2), t % 128, rng.integers(128)] = 0x7F
    for t in (1, 130, 345, 399):
        cache.v_data[table[0, t // 128], 0, t % 128, t % 128] = 0xFF
    check(cache, batch, lens_, indptr, table, q64, window, sinks, True, "NaN")


def test_value_scales_apart_and_zero():
    lens, rows = [1200, 700], [4, 1]
    cache, batch, lens_, indptr, table, q64 = setup(lens, rows, 2, 8, "e4m3", 81)
    for i, e in enumerate((-60, 60, 0, 30)):
        cache.v_scale[table[0, 5 + i], :] = 2.0 ** e
    cache.v_scale[table[1, 0], :] = 0.0
    check(cache, batch, lens_, indptr, table, q64, 500, 3, True, "scales")


def test_rows_behind_the_last_sequence_stay():
    lens, rows = [300, 200], [2, 1]
    cache, batch, *_ = setup(lens, rows, 2, 4, "e4m3", 91)
    q = torch.cat([batch.q, batch.q[:1]])
    batch = KV8Batch(batch.context_lens, batch.q_indptr, batch.block_table, q, total_rows=4, max_rows_per_req=2)
    att = KV8Attention(cache, batch)
    att.out.fill_(3.0)
    att.lse.fill_(3.0)
    att.attend(window=64, sinks=1)
    assert (att.out[3] == 3.0).all() and (att.lse[3] == 3.0).all() and not (att.out[:3] == 3.0).all()


def test_long_contexts_and_far_positions():
    """260,000 tokens on few pages: positions and tile counts of long requests, the window at the end."""
    n, r = 260_003, 5
    lens_, indptr, table, _ = _kv8.batch_of([1], [r], 1)
    cache, batch, *_ = setup([1500], [r], 4, 8, "e4m3", 101)
    pages = cache.num_pages
    table = np.full((1, (n + 127) // 128), -7, np.int32)
    rng = np.random.default_rng(3)
    table[0, -20:] = rng.integers(0, pages, 20)
    table[0, :2] = rng.integers(0, pages, 2)
    batch = KV8Batch(torch.tensor([n], dtype=torch.int32, device="cuda"), batch.q_indptr, torch.from_numpy(table).cuda(), batch.q,
                     total_rows=r, max_rows_per_req=r)
    check(cache, batch, np.array([n]), indptr, table, batch.q.double().view(r, 4, 8, 128), 2000, 200, True, "far")


def test_captured_and_replayed_on_two_streams():
    lens, rows = [2000, 900, 4100], [3, 1, 8]
    cache, batch, *_ = setup(lens, rows, 4, 8, "bf16", 111)
    a, b = KV8Attention(cache, batch), KV8Attention(cache, batch)
    want = a.attend(window=600, sinks=4).clone(), a.lse.clone()
    torch.cuda.synchronize()
    graphs = []
    for att in (a, b):
        att.out.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            att.attend(window=600, sinks=4)
        graphs.append((g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for att in (a, b):
        assert torch.equal(att.out, want[0]) and torch.equal(att.lse, want[1])
    assert a.errors() == 0 and b.errors() == 0


def test_refusals():
    cache, batch, *_ = setup([300], [1], 2, 4, "e4m3", 121)
    att = KV8Attention(cache, batch)
    for kw in (dict(window=0), dict(window=-1), dict(window=2 ** 31), dict(window=4, sinks=-1), dict(sinks=3)):
        with pytest.raises(ValueError):
            att.attend(**kw)
    with pytest.raises(ValueError):
        att.attend(torch.zeros((1, 2, 4), dtype=torch.int32, device="cuda"), window=4)
    assert math.isfinite(att.attend(window=4).float().sum().item())
