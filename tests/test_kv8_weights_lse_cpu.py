"""Host checks of which lse KV8Attention.add_weights takes by itself: the one that the last attention to all keys of the
bound batch left, and no other. The library is a stand-in that records what a launch would have got."""
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache, _lib
from tests.test_kv8_binding_cpu import _i32, _Lib, launches  # noqa: F401  (the fixture)


class _WithWeights(_Lib):
    def msa_kv8_attn_weights_workspace_size(self, args, n):
        n._obj.value = 256
        return 0

    def msa_kv8_attn_shared_workspace_size(self, args, groups, n):
        n._obj.value = 256
        return 0


@pytest.fixture
def bound(launches, monkeypatch):  # noqa: F811
    monkeypatch.setattr(_lib, "load", lambda: _WithWeights())
    cache = KV8Cache.empty(6, 2, device="cpu")
    batch = KV8Batch(_i32(2), _i32(3), _i32(2, 4), torch.zeros((3, 8, 128), dtype=torch.bfloat16), total_rows=3, max_rows_per_req=2)
    att = KV8Attention(cache, batch, max_groups=1, with_weights=True)
    new = torch.zeros((2, 2, 512))

    def adds(ok, **kw):
        before = len(launches)
        if ok:
            att.add_weights(None, new, **kw)
        else:
            with pytest.raises(ValueError, match="lse"):
                att.add_weights(None, new, **kw)
        assert len(launches) == before + ok

    return cache, batch, att, adds


def test_only_attention_to_all_keys_leaves_one(bound):
    cache, batch, att, adds = bound
    adds(False)                                   # no attention yet: uninitialised memory
    att.attend()
    adds(True)
    adds(True)
    att.attend(window=5, sinks=1)
    adds(False)
    att.attend_shared(_i32(2))
    adds(True)
    att.attend(_i32(2, 2, 1))
    adds(False)
    adds(True, lse=att.lse)                       # what is given is taken as it is
    adds(False)
    att.attend(window=512)                        # a window as wide as the block table sees all keys
    adds(True)
    att.attend(window=511)
    adds(False)


def test_a_refused_call_leaves_it_as_it_was(bound):
    cache, batch, att, adds = bound
    att.attend()
    for call in (lambda: att.attend(window=0), lambda: att.attend(sinks=1), lambda: att.attend(_i32(2, 2, 0)),
                 lambda: att.attend_shared(_i32(3))):
        with pytest.raises(ValueError):
            call()
        adds(True)


def test_another_batch_has_none(bound):
    cache, batch, att, adds = bound
    att.attend()
    att.rebind(KV8Batch(_i32(2), _i32(3), _i32(2, 4), batch.q, total_rows=3, max_rows_per_req=2))
    adds(False)
    att.attend()
    adds(True)
    att.batch.context_lens = _i32(2)              # replaced in place: the next step of the same requests
    adds(False)
    adds(False)
    att.attend()
    adds(True)
    att.batch.q = torch.ones_like(batch.q)
    adds(False)


def test_a_cache_that_grew_has_the_same_keys(bound):
    cache, batch, att, adds = bound
    att.attend()
    more = KV8Cache.empty(12, 2, device="cpu")
    for n in ("k_data", "k_scale", "v_data", "v_scale"):
        setattr(cache, n, getattr(more, n))
    adds(True)


def test_a_batch_without_rows(bound, launches):  # noqa: F811
    """Queries of no rows have no address; the batch is still the same one from call to call."""
    cache, *_ = bound
    none = KV8Batch(_i32(2), _i32(3), _i32(2, 4), torch.zeros((0, 8, 128), dtype=torch.bfloat16), total_rows=0, max_rows_per_req=2)
    att = KV8Attention(cache, none, max_groups=1, with_weights=True)
    args = att.args
    att.attend_shared(_i32(2))
    att.add_weights(None, torch.zeros((2, 2, 512)))
    assert att.args is args
