"""GPU tests of calls that the interface allows beside the usual ones: no lse, 8-bit tensor types, the widest
heads, a long context, a DecodeBatch for the append, a serving step captured as one graph, and the decode
path on forked and compacted pages."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import DecodeBatch, KV8Attention, KV8Batch, KV8Cache, KVCache, MSADecoder, PagePool, _lib
from tests import _kv8, _wl
from tests.test_gpu_kv8 import _append_case, _assert_attends, _attn_case, _cuda

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("rows", [[2, 1], [300, 40]])
def test_without_lse_and_with_8_bit_tensor_types(rows):
    cache, batch, lens, indptr, table, qv, _ = _attn_case([900, 300], rows, 2, 8, "e4m3", 41)
    att = KV8Attention(cache, batch)
    want, lse = att.attend().clone(), att.lse.clone()
    bare = KV8Attention(cache, batch, with_lse=False)
    assert torch.equal(bare.attend(), want) and bare.lse is None and bare.errors() == 0
    fp8 = torch.float8_e4m3fn
    typed = KV8Cache(cache.k_data.view(fp8), cache.k_scale, cache.v_data.view(fp8), cache.v_scale)
    batch.q = batch.q.view(fp8)
    att = KV8Attention(typed, batch)
    assert torch.equal(att.attend(), want) and torch.equal(att.lse, lse)


@pytest.mark.parametrize("q_type", ["e4m3", "bf16"])
@pytest.mark.parametrize("lens,rows,H,G", [([130, 1], [1, 1], 64, 64), ([300], [5], 64, 1), ([260000], [1], 1, 8)])
def test_widest_heads_and_a_long_context(lens, rows, H, G, q_type):
    cache, batch, lens, indptr, table, qv, _ = _attn_case(lens, rows, H, G, q_type, 5)
    att = KV8Attention(cache, batch)
    out = att.attend()
    assert att.errors() == 0
    _assert_attends(out, att.lse, _kv8.attend(qv, cache, lens, indptr, table))


def test_append_with_a_decode_batch():
    lens, indptr, table, pages, x, planes = _append_case([700, 130, 2000], [3, 8, 1], 4, torch.bfloat16, 33)
    cache = KV8Cache(**{n: _cuda(p) for n, p in planes.items()})
    none = torch.zeros(0, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cache.append(DecodeBatch(_cuda(lens), _cuda(indptr), _cuda(table), none, none, int(indptr[-1]), 8),
                 x["k"].cuda(), x["v"].cuda(), ws)
    assert _lib.msa_get_error(ws) == 0
    for n in ("k", "v"):
        _kv8.append_plane(x[n].double().numpy(), lens, indptr, table, planes[n + "_data"], planes[n + "_scale"])
        assert np.array_equal(getattr(cache, n + "_data").cpu().numpy(), planes[n + "_data"])
        assert np.array_equal(getattr(cache, n + "_scale").cpu().numpy(), planes[n + "_scale"])


def test_a_serving_step_as_one_graph():
    """Growth, append and attention on the pool's own tensors, captured once and replayed: every step's
    attention against the cache as it is then, the appended tokens against the rule."""
    H, G, S, P, M = 2, 8, 3, 20, 5
    cache = KV8Cache.empty(P, H)
    pool = PagePool.empty([cache], S, M)
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.zeros((S, H, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((S, H * G, 128), dtype=torch.bfloat16, device="cuda")
    seqs, lens = torch.arange(S, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    batch = KV8Batch(pool.seq_lens, torch.arange(S + 1, dtype=torch.int32, device="cuda"), pool.block_table, q,
                     total_rows=S, max_rows_per_req=1)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    att = KV8Attention(cache, batch)

    def step():
        lens.add_(1)
        pool.reserve(seqs, lens)
        cache.append(batch, k, v, ws)
        att.attend()

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens.copy_(torch.tensor([0, 120, 250], dtype=torch.int32))      # (captured, not run)
    pool.reserve(seqs, lens)
    planes = {n: getattr(cache, n).cpu().numpy() for n in ("k_data", "k_scale", "v_data", "v_scale")}
    for _ in range(140):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g) * 2)
        graph.replay()
        table, now = pool.block_table.cpu().numpy(), lens.cpu().numpy()
        assert np.array_equal(pool.seq_lens.cpu().numpy(), now)
        for n, x in (("k", k), ("v", v)):
            _kv8.append_plane(x.double().cpu().numpy(), now, np.arange(S + 1), table, planes[n + "_data"], planes[n + "_scale"])
        if now[0] % 35 == 1:
            assert pool.errors() == 0 and att.errors() == 0 and _lib.msa_get_error(ws) == 0
            for n, a in planes.items():
                assert np.array_equal(getattr(cache, n).cpu().numpy(), a), n
            _assert_attends(att.out, att.lse, _kv8.attend(q.double().view(S, H, G, 128), cache, now, np.arange(S + 1), table))
    assert int((pool.ref_counts > 0).sum()) == sum((int(n) + 127) // 128 for n in lens)


def test_the_decode_path_on_forked_and_compacted_pages():
    """Children of a fork and a compacted pool give the decode path the bits of the parents."""
    wl = _wl.small([4500, 3000, 700], [3, 2, 1], needles=3, seed=21)
    first = KVCache.from_host(wl)
    rows = DecodeBatch.from_host(wl)
    B, M = rows.block_table.shape
    want = [t.clone() for t in MSADecoder(first, rows).decode()]
    cache = KVCache.empty(first.num_pages + 10)                   # with free pages behind
    for n in ("k_data", "k_scale", "v_data", "v_scale", "ki_data", "ki_scale"):
        getattr(cache, n)[:first.num_pages].copy_(getattr(first, n))
    lens = torch.zeros(2 * B, dtype=torch.int32, device="cuda")
    table = torch.full((2 * B, M), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(cache.num_pages, dtype=torch.int32, device="cuda")
    lens[:B], table[:B] = rows.context_lens, rows.block_table
    for b in range(B):
        refs[rows.block_table[b, :(int(rows.context_lens[b]) + 127) // 128].long()] += 1
    pool = PagePool([cache], lens, table, refs)
    parents, children = (torch.arange(a, a + B, dtype=torch.int32, device="cuda") for a in (0, B))
    for act in (lambda: pool.fork(parents, children), lambda: pool.free(parents), lambda: pool.compact()):
        act()
        batch = DecodeBatch(lens[B:].contiguous(), rows.q_indptr, table[B:].contiguous(), rows.q, rows.q_idx,
                            rows.total_rows, rows.max_rows_per_req)
        dec = MSADecoder(cache, batch)
        got = dec.decode()
        assert pool.errors() == 0 and dec.errors() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
