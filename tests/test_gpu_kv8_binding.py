"""GPU test of KV8Attention when the tensors it is bound to are replaced by ones that do not fit."""
import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache
from tests import _kv8

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def test_a_refused_replacement_is_refused_again_and_can_be_put_back():
    lens, indptr, table, pages = _kv8.batch_of([900, 300], [2, 1], 41)
    kd, ks = _kv8.fill(pages, 2, 42)
    vd, vs = _kv8.fill(pages, 2, 43)
    cache = KV8Cache(kd, ks, vd, vs)
    q = torch.randn((3, 16, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    batch = KV8Batch(_cuda(lens), _cuda(indptr), _cuda(table), q, total_rows=3, max_rows_per_req=2)
    att = KV8Attention(cache, batch)
    want, lse = att.attend().clone(), att.lse.clone()
    names = ("k_data", "k_scale", "v_data", "v_scale")
    wider = torch.full((2, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wider[:, :table.shape[1]] = batch.block_table
    grown = KV8Cache.empty(pages + 8, 2)

    def put(planes, tab, rows=3):
        for n, t in zip(names, planes):
            setattr(cache, n, t)
        batch.block_table, batch.total_rows = tab, rows

    old, tab = [getattr(cache, n) for n in names], batch.block_table
    big = [getattr(grown, n) for n in names]
    for planes, t, rows in ((old, wider, 3), (big, wider, 3), (old, tab, 2)):
        put(planes, t, rows)
        att.out.fill_(7.0)
        for _ in range(2):
            with pytest.raises(ValueError):
                att.attend()
        torch.cuda.synchronize()
        assert torch.all(att.out == 7.0)
        put(old, tab)
        assert torch.equal(att.attend(), want) and torch.equal(att.lse, lse) and att.errors() == 0


@pytest.mark.parametrize("rows", [1, 300])
def test_a_workspace_needs_its_flags_cleared_alone(rows):
    """Whatever the workspace holds behind its flags, and with the clearing held up on the stream that made
    it, a call gives the same."""
    lens, indptr, table, pages = _kv8.batch_of([6000, 300, 700], [rows, 300, 1], 41)
    kd, ks = _kv8.fill(pages, 2, 42)
    vd, vs = _kv8.fill(pages, 2, 43)
    cache = KV8Cache(kd, ks, vd, vs)
    total = int(indptr[-1])
    q = torch.randn((total, 16, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    batch = KV8Batch(_cuda(lens), _cuda(indptr), _cuda(table), q, total_rows=total, max_rows_per_req=300)
    att = KV8Attention(cache, batch)
    want, lse = att.attend().clone(), att.lse.clone()
    for fill in (0xFF, 0x7F, 0x01):
        att.ws[256:].fill_(fill)
        att.out.fill_(7.0)
        assert torch.equal(att.attend(), want) and torch.equal(att.lse, lse) and att.errors() == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        other = KV8Attention(cache, batch)                   # cleared on the current stream
        out = other.attend(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other.lse, lse)


def test_a_pool_needs_its_flags_cleared_alone():
    from tests.test_gpu_pages import _i32, _same, _state
    pool, ref, dev = _state("kv8", 64, [300, 512, 129, 0, 0, 0, 0], 9, 3)
    for fill in (0xFF, 0x01, 0x7F):
        pool.ws[256:].fill_(fill)
        pool.fork(_i32(0, 2), _i32(3, 4))
        ref.fork([0, 2], [3, 4])
        pool.ws[256:].fill_(fill)
        pool.reserve(_i32(3, 5), _i32(700, 200))
        ref.reserve([3, 5], [700, 200])
        pool.ws[256:].fill_(fill)
        pool.compact()
        ref.compact()
        assert pool.errors() == 0
        _same(pool, ref, dev)
        pool.ws[256:].fill_(fill)
        pool.free(_i32(3, 4, 5))
        ref.free([3, 4, 5])
        assert pool.errors() == 0
        _same(pool, ref, dev)
