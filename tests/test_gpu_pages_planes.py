"""A pool over planes that are no 8-bit cache's: copy, fork, reserve, free and compact take them, evict does not."""
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Cache, PagePool

pytestmark = pytest.mark.gpu


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_sixteen_bit_planes():
    g = torch.Generator(device="cuda").manual_seed(3)
    data = lambda: torch.randn((9, 2, 128, 64), device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    scale = lambda: torch.rand((9, 4), device="cuda", generator=g).half()  # noqa: E731
    cache = KV8Cache(data(), scale(), data(), scale())
    pool = PagePool.empty([cache], 3, 4)
    pool.reserve(ints(0), ints(300))
    pool.fork(ints(0), ints(1))
    a, b = pool.block_table[0, :3].tolist(), pool.block_table[1, :3].tolist()
    assert a[:2] == b[:2] and a[2] != b[2] and pool.seq_lens.tolist() == [300, 300, 0]
    for t in (cache.k_data, cache.v_data):
        assert torch.equal(t[a[2], :, :300 - 256], t[b[2], :, :300 - 256])
    for t in (cache.k_scale, cache.v_scale):
        assert torch.equal(t[a[2]], t[b[2]])
    pool.copy(ints(a[0]), ints(7))
    assert torch.equal(cache.k_data[7], cache.k_data[a[0]]) and torch.equal(cache.v_scale[7], cache.v_scale[a[0]])
    with pytest.raises(ValueError, match="k_data"):
        pool.evict(ints(0), ints(2), torch.zeros((3, 2, 512), device="cuda"), 10)
    pool.free(ints(0))
    pool.compact()
    assert pool.errors() == 0 and pool.seq_lens.tolist() == [0, 300, 0]
