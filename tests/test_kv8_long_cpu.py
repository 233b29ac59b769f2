"""Host checks of the operators for long sequences over the 8-bit cache: what the host can see is refused before any
CUDA call; and the plain form of the eviction against a second one."""
import ctypes

import numpy as np
import pytest

from block_sparse_attention_nvfp4_gb300 import _lib
from block_sparse_attention_nvfp4_gb300 import build as msa_build
from tests import _kv8_long


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return _lib.load()


WS = ctypes.c_void_p(1 << 20)       # never dereferenced: checks fail first
X = 1 << 21
BIG = 1 << 40


def _attn(**kw):
    a = _lib.Kv8AttnArgs(num_reqs=2, total_rows=4, max_rows_per_req=2, num_pages=8, max_pages_per_req=4, num_kv_heads=4,
                         q_per_kv=8, n_block_ids=0, q_type=_lib.TYPE_BF16, sm_scale=0.1, q_row_stride=4096, context_lens=X,
                         q_indptr=X, block_table=X, q=X, k_data=X, k_scale=X, v_data=X, v_scale=X, out=X)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


COMMON = [("num_reqs", -1, -1), ("num_reqs", 4097, -1), ("total_rows", 5, -1), ("max_rows_per_req", 0, -1), ("num_kv_heads", 65, -2),
          ("q_per_kv", 65, -2), ("q_type", _lib.TYPE_F16, -2), ("sm_scale", 0.0, -1), ("q_row_stride", 4095, -1), ("q", 0, -1),
          ("k_data", 0, -1), ("k_scale", X + 1, -1), ("context_lens", 0, -1), ("block_table", 0, -1), ("num_pages", 1 << 22, -2),
          ("block_ids", X, -1), ("n_block_ids", 4, -1)]


@pytest.mark.parametrize("field,value,code", COMMON + [("out", 0, -1), ("v_scale", 0, -1), ("lse", X + 2, -1)])
def test_window_and_shared_refuse_what_the_plain_call_refuses(lib, field, value, code):
    a = _attn(**{field: value})
    assert lib.msa_kv8_attn_window(a, 16, 0, WS, BIG, None) == code
    assert lib.msa_kv8_attn_shared(a, 1, X, 0, WS, BIG, None) == code


@pytest.mark.parametrize("field,value,code", COMMON)
def test_weights_refusals(lib, field, value, code):
    assert lib.msa_kv8_attn_weights(_attn(**{field: value}), X, 1.0, X, X, 512, WS, BIG, None) == code


def test_window_arguments(lib):
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        assert lib.msa_kv8_attn_window(_attn(), window, sinks, WS, BIG, None) == -1
    assert lib.msa_kv8_attn_window(None, 4, 0, WS, BIG, None) == -1
    for ws in (None, ctypes.c_void_p((1 << 20) + 64)):
        assert lib.msa_kv8_attn_window(_attn(), 4, 0, ws, BIG, None) == -4


def test_shared_arguments(lib):
    n = ctypes.c_size_t(0)
    for groups, indptr in ((-1, X), (4097, X), (1, None)):
        assert lib.msa_kv8_attn_shared(_attn(), groups, indptr, 0, WS, BIG, None) == -1
    assert lib.msa_kv8_attn_shared(None, 1, X, 0, WS, BIG, None) == -1
    assert lib.msa_kv8_attn_shared_workspace_size(None, 1, ctypes.byref(n)) == -1
    assert lib.msa_kv8_attn_shared_workspace_size(_attn(), 1, None) == -1
    assert lib.msa_kv8_attn_shared_workspace_size(_attn(), -1, ctypes.byref(n)) == -1


def test_weights_arguments(lib):
    n = ctypes.c_size_t(0)
    for lse, keep, old, new, stride in ((None, 1.0, X, X, 512), (X, -1.0, X, X, 512), (X, float("nan"), X, X, 512),
                                        (X, float("inf"), X, X, 512), (X, 1.0, X, None, 512), (X, 1.0, X, X, 511),
                                        (X + 2, 1.0, X, X, 512), (X, 1.0, X + 1, X, 512), (X, 1.0, X, X + 2, 512)):
        assert lib.msa_kv8_attn_weights(_attn(), lse, keep, old, new, stride, WS, BIG, None) == -1
    assert lib.msa_kv8_attn_weights(None, X, 1.0, X, X, 512, WS, BIG, None) == -1
    assert lib.msa_kv8_attn_weights(_attn(), X, 1.0, X, X, 512, None, BIG, None) == -4
    many = dict(num_reqs=4096, max_rows_per_req=1 << 20, total_rows=1 << 26, num_kv_heads=1, q_per_kv=16, q_row_stride=2048)
    assert lib.msa_kv8_attn_weights(_attn(**many), X, 1.0, X, X, 512, WS, BIG, None) == -2
    assert lib.msa_kv8_attn_weights_workspace_size(_attn(**many), ctypes.byref(n)) == -2
    assert lib.msa_kv8_attn_weights_workspace_size(_attn(), None) == -1
    # values that the call does not use may be missing
    assert lib.msa_kv8_attn_weights(_attn(out=0, v_data=0, v_scale=0), X, 1.0, None, X, 511, WS, BIG, None) == -1


def _pool(**kw):
    a = _lib.PagePoolArgs(num_seqs=4, num_pages=16, max_pages_per_seq=4, num_planes=0, seq_lens=X, block_table=X, ref_counts=X)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def _caches(**kw):
    c = (_lib.Kv8EvictCache * 1)(_lib.Kv8EvictCache(X, X, X, X, X, 512, 4))
    for k, v in kw.items():
        setattr(c[0], k, v)
    return c


def _evict(lib, pool=None, n=1, parents=X, children=X, count=1, caches=None, keep=8, sinks=2, recent=2, scratch=X, size=BIG,
           ws=WS):
    return lib.msa_pages_evict(pool or _pool(), n, parents, children, count, caches if caches is not None else _caches(), keep, sinks,
                               recent, scratch, size, ws, 1 << 20, None)


def test_evict_refusals(lib):
    for kw in (dict(n=-1), dict(n=5), dict(parents=None), dict(children=None), dict(count=0), dict(count=5), dict(keep=0),
               dict(sinks=-1), dict(recent=-1), dict(sinks=5, recent=4), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1),
               dict(pool=_pool(num_seqs=-1)), dict(pool=_pool(num_pages=0)), dict(pool=_pool(ref_counts=0)),
               dict(caches=_caches(k_data=0)), dict(caches=_caches(v_data=X + 8)), dict(caches=_caches(k_scale=X + 2)),
               dict(caches=_caches(weights=0)), dict(caches=_caches(weights=X + 1)), dict(caches=_caches(head_stride=511))):
        assert _evict(lib, **kw) == -1, kw
    assert lib.msa_pages_evict(_pool(), 1, X, X, 1, None, 8, 2, 2, X, BIG, WS, 1 << 20, None) == -1
    for kw in (dict(caches=_caches(num_kv_heads=0)), dict(caches=_caches(num_kv_heads=65)), dict(pool=_pool(num_pages=(1 << 20) + 1))):
        assert _evict(lib, **kw) == -2, kw
    for kw in (dict(scratch=None), dict(scratch=X + 8), dict(size=8 * 4 * 8 - 1), dict(ws=None)):
        assert _evict(lib, **kw) == -4, kw


def test_positions_behind_the_longest_sequence_are_ints(lib):
    for pages, code in (((1 << 24) - 255, -2), ((1 << 24) - 1, -2)):
        tokens = pages * 128
        assert _evict(lib, pool=_pool(max_pages_per_seq=pages), caches=_caches(head_stride=tokens)) == code
        assert lib.msa_kv8_attn_weights(_attn(max_pages_per_req=pages), X, 1.0, X, X, tokens, WS, BIG, None) == code


def test_evict_scratch_size(lib):
    n = ctypes.c_size_t(0)
    for count, keep, want in ((3, 100, 8 * 3 * 4 * 100), (0, 5, 0), (4, 10 ** 9, 8 * 4 * 4 * 512)):
        assert lib.msa_pages_evict_scratch_size(_pool(), 1, _caches(), count, keep, ctypes.byref(n)) == 0
        assert n.value == want
    assert lib.msa_pages_evict_scratch_size(_pool(), 1, _caches(), 1, 8, None) == -1
    assert lib.msa_pages_evict_scratch_size(None, 1, _caches(), 1, 8, ctypes.byref(n)) == -1


@pytest.mark.parametrize("seed", range(6))
def test_plain_form_keeps_the_heaviest(seed):
    """The tests' own plain form against one that takes the tokens one by one."""
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 60))
    w = rng.integers(-1, 4, n).astype(np.float32)
    w[rng.random(n) < 0.1] = np.nan
    keep = int(rng.integers(1, n + 4))
    sinks = int(rng.integers(0, keep + 1))
    recent = int(rng.integers(0, keep - sinks + 1))
    got = _kv8_long.kept(w, n, keep, sinks, recent)
    if n <= keep:
        assert list(got) == list(range(n))
        return
    want = set(range(sinks)) | set(range(n - recent, n))
    while len(want) < keep:
        rest = [t for t in range(n) if t not in want]
        want.add(max(rest, key=lambda t: (w[t] if w[t] > 0 else 0.0, -t)))
    assert list(got) == sorted(want)
