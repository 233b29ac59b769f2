"""Host checks of what PagePool.evict binds: its demands on the caches' planes are its own, not the other operators'. The
library is a stand-in that records what a launch would have got."""
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Cache, PagePool, pages
from tests.test_kv8_binding_cpu import _i32, launches  # noqa: F401  (the fixture)


@pytest.fixture
def host(launches, monkeypatch):  # noqa: F811
    """A pool on host tensors."""
    monkeypatch.setattr(pages, "_planes", lambda c, n, dev: [
        (x, getattr(c, x).data_ptr(), 0, 0, 8) for x in ("k_data", "k_scale", "v_data", "v_scale")])
    monkeypatch.setattr(PagePool, "_list", lambda self, t, n, name: t.data_ptr())
    return launches


def _cache(data=torch.uint8, scale=torch.float32, dim=128):
    d = lambda: torch.zeros((6, 2, 128, dim), dtype=data)  # noqa: E731
    s = lambda: torch.zeros((6, 2), dtype=scale)  # noqa: E731
    return KV8Cache(d(), s(), d(), s())


@pytest.mark.parametrize("kw", [dict(data=torch.bfloat16), dict(scale=torch.float16), dict(dim=64)])
def test_planes_that_only_evict_refuses(host, kw):
    """Planes of other types or row lengths: the pool and its other operators take them."""
    cache = _cache(**kw)
    pool = PagePool([cache], _i32(3), _i32(3, 4), _i32(6))
    seqs = _i32(2)
    for call in (lambda: pool.free(seqs), lambda: pool.copy(seqs, seqs), lambda: pool.fork(seqs, seqs),
                 lambda: pool.reserve(seqs, seqs), pool.compact):
        call()
    assert len(host) == 5
    for _ in range(2):
        with pytest.raises(ValueError, match="data|scale"):
            pool.evict(seqs, seqs, torch.zeros((3, 2, 512)), 10)
    assert len(host) == 5
