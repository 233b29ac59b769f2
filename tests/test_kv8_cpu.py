"""Host checks of the 8-bit cache and page entry points: what the host can see is refused before any
CUDA call, in the library and in the binding."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Attention, KV8Batch, KV8Cache, PagePool, _lib
from block_sparse_attention_nvfp4_gb300 import build as msa_build
from tests import _kv8


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return _lib.load()


WS = ctypes.c_void_p(1 << 20)       # never dereferenced: checks fail first
X = 1 << 21


def _append():
    return _lib.Kv8AppendArgs(num_reqs=2, total_rows=4, max_rows_per_req=2, num_pages=8, max_pages_per_req=4,
                              num_kv_heads=4, src_type=_lib.TYPE_BF16, k_token_stride=512, v_token_stride=512,
                              context_lens=X, q_indptr=X, block_table=X, k=X, v=X, k_data=X, k_scale=X, v_data=X,
                              v_scale=X)


@pytest.mark.parametrize("field,value,code", [
    ("num_reqs", -1, -1), ("num_reqs", 4097, -1), ("total_rows", 5, -1), ("total_rows", -1, -1),
    ("max_rows_per_req", 0, -1), ("num_pages", 0, -1), ("max_pages_per_req", 0, -1), ("num_kv_heads", 0, -2),
    ("num_kv_heads", 65, -2), ("src_type", 0, -2), ("src_type", 9, -2), ("k_token_stride", 511, -1),
    ("k_token_stride", 516, -1), ("v_token_stride", 256, -1), ("context_lens", 0, -1), ("q_indptr", 0, -1),
    ("block_table", 0, -1), ("k", X + 8, -1), ("k_data", 0, -1), ("v_data", X + 4, -1), ("k_scale", 0, -1),
    ("v_scale", X + 2, -1), ("num_pages", 1 << 22, -2), ("max_pages_per_req", 1 << 24, -2),
])
def test_append_refusals(lib, field, value, code):
    a = _append()
    setattr(a, field, value)
    assert lib.msa_kv8_append(ctypes.byref(a), WS, 256, None) == code


def test_append_workspace(lib):
    a = _append()
    assert lib.msa_kv8_append(None, WS, 256, None) == -1
    for ws, n in ((None, 256), (ctypes.c_void_p((1 << 20) + 64), 256), (WS, 255)):
        assert lib.msa_kv8_append(ctypes.byref(a), ws, n, None) == -4


def _attn():
    return _lib.Kv8AttnArgs(num_reqs=2, total_rows=4, max_rows_per_req=2, num_pages=8, max_pages_per_req=4,
                            num_kv_heads=4, q_per_kv=8, n_block_ids=0, q_type=_lib.TYPE_BF16, sm_scale=0.1,
                            q_row_stride=4096, context_lens=X, q_indptr=X, block_table=X, q=X, k_data=X, k_scale=X,
                            v_data=X, v_scale=X, out=X)


@pytest.mark.parametrize("field,value,code", [
    ("num_reqs", -1, -1), ("num_reqs", 4097, -1), ("total_rows", 5, -1), ("max_rows_per_req", 0, -1),
    ("num_kv_heads", 0, -2), ("num_kv_heads", 65, -2), ("q_per_kv", 0, -2), ("q_per_kv", 65, -2),
    ("q_type", _lib.TYPE_F16, -2), ("q_type", -1, -2), ("n_block_ids", 33, -1), ("n_block_ids", 4, -1),
    ("sm_scale", 0.0, -1), ("sm_scale", float("nan"), -1), ("sm_scale", float("inf"), -1), ("q_row_stride", 4095, -1),
    ("q_row_stride", 4100, -1), ("q", 0, -1), ("q", X + 8, -1), ("out", 0, -1), ("out", X + 2, -1),
    ("k_data", 0, -1), ("v_scale", 0, -1), ("k_scale", X + 1, -1), ("lse", X + 2, -1), ("context_lens", 0, -1),
    ("block_table", 0, -1), ("num_pages", 1 << 22, -2), ("block_ids", X, -1),
])
def test_attention_refusals(lib, field, value, code):
    a = _attn()
    setattr(a, field, value)
    assert lib.msa_kv8_attn(ctypes.byref(a), WS, 1 << 30, None) == code


def test_attention_workspace(lib):
    a = _attn()
    n = ctypes.c_size_t(0)
    assert lib.msa_kv8_attn(None, WS, 1 << 30, None) == -1
    assert lib.msa_kv8_attn_workspace_size(None, ctypes.byref(n)) == -1
    assert lib.msa_kv8_attn_workspace_size(ctypes.byref(a), None) == -1
    assert lib.msa_kv8_attn(ctypes.byref(a), None, 1 << 30, None) == -4
    assert lib.msa_kv8_attn(ctypes.byref(a), ctypes.c_void_p((1 << 20) + 16), 1 << 30, None) == -4


def _pool():
    a = _lib.PagePoolArgs(num_seqs=4, num_pages=16, max_pages_per_seq=4, num_planes=2, seq_lens=X, block_table=X,
                          ref_counts=X)
    a.planes[0] = _lib.PagePlane(X, 4, 64, 0)
    a.planes[1] = _lib.PagePlane(X, 0, 0, 16)
    return a


def _calls(lib, a, n=1, ws=WS, size=1 << 20, lst=X):
    p = ctypes.c_void_p(lst) if lst else None
    return [lib.msa_pages_fork(ctypes.byref(a), n, p, p, ws, size, None),
            lib.msa_pages_reserve(ctypes.byref(a), n, p, p, ws, size, None),
            lib.msa_pages_free(ctypes.byref(a), n, p, ws, size, None),
            lib.msa_pages_compact(ctypes.byref(a), p, p, None, ws, size, None),
            lib.msa_pages_copy(ctypes.byref(a), n, p, p, None, ws, size, None)]


@pytest.mark.parametrize("field,value,code", [
    ("num_seqs", -1, -1), ("num_pages", 0, -1), ("max_pages_per_seq", 0, -1), ("num_planes", -1, -1),
    ("num_planes", 17, -1), ("num_pages", (1 << 20) + 1, -2), ("num_seqs", (1 << 20) + 1, -2),
    ("max_pages_per_seq", 1 << 24, -2),
])
def test_pool_refusals(lib, field, value, code):
    a = _pool()
    setattr(a, field, value)
    assert _calls(lib, a) == [code] * 5


def test_plane_refusals(lib):
    for plane in ((0, 4, 64, 0), (X + 8, 4, 64, 0), (X, 0, 64, 0), (X, 4, 4, 0), (X, 4, -8, 0), (X, 0, 0, 6), (X, 0, 0, 0)):
        a = _pool()
        a.planes[0] = _lib.PagePlane(*plane)
        assert _calls(lib, a) == [-1] * 5, plane


def test_pool_lists_and_workspace(lib):
    a = _pool()
    assert _calls(lib, a, n=-1)[:3] == [-1] * 3 and _calls(lib, a, n=5)[:2] == [-1] * 2
    assert _calls(lib, a, lst=0) == [-1] * 5
    assert _calls(lib, a, ws=None) == [-4] * 5
    n = ctypes.c_size_t(0)
    assert lib.msa_pages_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    assert _calls(lib, a, size=n.value - 1) == [-4] * 5
    assert lib.msa_pages_workspace_size(None, ctypes.byref(n)) == -1
    for name in ("seq_lens", "block_table", "ref_counts"):
        a = _pool()
        setattr(a, name, None)
        assert _calls(lib, a)[:4] == [-1] * 4, name


def test_binding_refuses_host_tensors():
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
    cache = KV8Cache.empty(2, 4, device="cpu")
    batch = KV8Batch(z(1), z(2), z(1, 2), z(1, 32, 128, dtype=torch.bfloat16), total_rows=1)
    with pytest.raises(ValueError):
        KV8Attention(cache, batch)
    with pytest.raises(ValueError):
        cache.append(batch, z(1, 4, 128, dtype=torch.float32), None, z(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        PagePool([cache], z(1), z(1, 2), z(2))


def test_plain_forms_agree_with_torch_on_e4m3():
    """The tests' own encoder and decoder against torch's."""
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(_kv8.e4m3_values(), want, equal_nan=True)
    rng = np.random.default_rng(0)
    v = want[np.isfinite(want)]
    s = np.sort(np.unique(v))
    x = np.concatenate([s, (s[1:] + s[:-1]) / 2, rng.standard_normal(4096) * np.exp2(rng.uniform(-14, 9, 4096))])
    got = _kv8.e4m3_codes(x)
    t = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    zero = (got & 127) == 0
    assert np.array_equal(got[~zero], t[~zero]) and np.all(t[zero] & 127 == 0)
