"""Host checks of what KV8Attention and PagePool do when the tensors they are bound to are replaced: the
library is a stand-in that records what a launch would have got."""
import contextlib

import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import DecodeBatch, KV8Attention, KV8Batch, KV8Cache, PagePool, _lib, kv8, pages


class _Lib:
    def msa_kv8_attn_workspace_size(self, args, n):
        n._obj.value = 256
        return 0

    def msa_pages_workspace_size(self, pool, n):
        n._obj.value = 256
        return 0

    def __getattr__(self, name):
        return name


@pytest.fixture
def launches(monkeypatch):
    """Host tensors pass as device ones; a launch appends a copy of its arguments."""
    got = []

    def plain(t, dtype, shape, dev, name):
        dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
        if not (t.dtype in dtypes and t.shape == tuple(shape) and t.is_contiguous()):
            raise ValueError(name)
        return t.data_ptr()

    def call(dev, stream, fn, what, *args):
        a = args[0]._obj
        got.append(type(a).from_buffer_copy(a))

    monkeypatch.setattr(kv8, "_plain", plain)
    monkeypatch.setattr(pages, "_plain", plain)
    monkeypatch.setattr(kv8, "_call", call)
    monkeypatch.setattr(pages, "_call", call)
    monkeypatch.setattr(_lib, "load", lambda: _Lib())
    monkeypatch.setattr(_lib, "msa_workspace_init", lambda ws, stream=None: None)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    return got


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _attention(heads=2):
    cache = KV8Cache.empty(6, heads, device="cpu")
    batch = KV8Batch(_i32(2), _i32(3), _i32(2, 4), torch.zeros((3, 8, 128), dtype=torch.bfloat16), total_rows=3,
                     max_rows_per_req=2)
    return cache, batch, KV8Attention(cache, batch)


def _bound(a):
    return a.block_table, a.max_pages_per_req, a.total_rows, a.q, a.k_data, a.v_scale, a.num_kv_heads


def _raises_until_put_back(att, launches, put_back):
    """A refused replacement is refused again, and nothing is launched in between."""
    before = len(launches)
    for _ in range(3):
        with pytest.raises(ValueError):
            att.attend()
    assert len(launches) == before
    put_back()
    att.attend()
    assert len(launches) == before + 1


def test_a_wider_table_is_refused_every_time(launches):
    cache, batch, att = _attention()
    att.attend()
    old = batch.block_table
    batch.block_table = _i32(2, 9)
    _raises_until_put_back(att, launches, lambda: setattr(batch, "block_table", old))
    assert _bound(launches[-1]) == _bound(launches[0])


def test_another_number_of_rows_is_refused_every_time(launches):
    cache, batch, att = _attention()
    att.attend()
    batch.total_rows = 2
    _raises_until_put_back(att, launches, lambda: setattr(batch, "total_rows", 3))
    batch.max_rows_per_req = 3
    _raises_until_put_back(att, launches, lambda: setattr(batch, "max_rows_per_req", 2))
    assert _bound(launches[-1]) == _bound(launches[0])


def test_planes_of_another_cache_are_refused_every_time(launches):
    cache, batch, att = _attention()
    att.attend()
    old = (cache.k_data, cache.k_scale, cache.v_data, cache.v_scale)
    names = ("k_data", "k_scale", "v_data", "v_scale")

    def put(planes):
        for n, t in zip(names, planes):
            setattr(cache, n, t)

    new = KV8Cache.empty(6, 3, device="cpu")              # 8 query heads do not divide among 3
    put([getattr(new, n) for n in names])
    _raises_until_put_back(att, launches, lambda: put(old))
    # a pool that grew: more pages and a wider table together
    new, table = KV8Cache.empty(12, 2, device="cpu"), batch.block_table
    put([getattr(new, n) for n in names])
    batch.block_table = _i32(2, 8)

    def back():
        put(old)
        batch.block_table = table

    _raises_until_put_back(att, launches, back)
    assert _bound(launches[-1]) == _bound(launches[0])
    # planes that fit are taken, and kept alive while they are bound
    put([getattr(new, n) for n in names])
    addresses = [t.data_ptr() for t in (cache.k_data, cache.v_scale)]
    att.attend()
    assert [launches[-1].k_data, launches[-1].v_scale] == addresses and launches[-1].num_pages == 12
    assert any(t is new.k_data for t in att._held) and any(t is new.v_scale for t in att._held)


def test_a_refused_rebind_leaves_the_old_batch_bound(launches):
    cache, batch, att = _attention()
    att.attend()
    with pytest.raises(ValueError):
        att.rebind(KV8Batch(_i32(2), _i32(3), _i32(2, 9), batch.q, total_rows=3, max_rows_per_req=2))
    att.attend()
    assert att.batch is batch and _bound(launches[-1]) == _bound(launches[0])


@pytest.mark.parametrize("name", ["seq_lens", "block_table", "ref_counts", "k_data", "v_scale"])
def test_a_pool_refuses_tensors_whose_storage_moved(launches, monkeypatch, name):
    cache = KV8Cache.empty(6, 2, device="cpu")
    monkeypatch.setattr(pages, "_planes", lambda c, n, dev: [
        (x, getattr(c, x).data_ptr(), 0, 0, 8) for x in ("k_data", "k_scale", "v_data", "v_scale")])
    monkeypatch.setattr(PagePool, "_list", lambda self, t, n, name: t.data_ptr())
    pool = PagePool([cache], _i32(3), _i32(3, 4), _i32(6))
    seqs = _i32(2)
    pool.free(seqs)
    assert len(launches) == 1
    t = getattr(pool, name) if hasattr(pool, name) else getattr(cache, name)
    keep = t.data                                         # (the old storage stays allocated)
    t.data = keep.clone()
    for call in (lambda: pool.free(seqs), lambda: pool.copy(seqs, seqs), lambda: pool.fork(seqs, seqs),
                 lambda: pool.reserve(seqs, seqs), pool.compact):
        with pytest.raises(ValueError, match=name):
            call()
    assert len(launches) == 1
    t.data = keep
    pool.free(seqs)
    assert len(launches) == 2


def test_replaced_tensors_of_a_decode_batch_are_seen(launches):
    cache = KV8Cache.empty(6, 2, device="cpu")
    q = torch.zeros((3, 8, 128), dtype=torch.uint8)
    batch = DecodeBatch(_i32(2), _i32(3), _i32(2, 4), q, torch.zeros((3, 4, 128), dtype=torch.uint8), 3, 2)
    att = KV8Attention(cache, batch)
    att.attend()
    batch.q = torch.ones_like(q)
    att.attend()
    assert launches[-1].q == batch.q.data_ptr() != launches[0].q
    batch.context_lens = _i32(2)
    att.attend()
    assert launches[-1].context_lens == batch.context_lens.data_ptr()
    batch.context_lens.data = _i32(2)                     # the same object, another storage
    att.attend()
    assert launches[-1].context_lens == batch.context_lens.data_ptr()
    batch.total_rows = 2
    _raises_until_put_back(att, launches, lambda: setattr(batch, "total_rows", 3))
