"""Host checks of what PagePool.evict binds: its demands on the caches' planes are its own, not the other operators'. The
library is a stand-in that records what a launch would have got."""
import contextlib
import ctypes
import threading
import time

import pytest
import torch

from block_sparse_attention_nvfp4_gb300 import KV8Cache, PagePool, _lib, pages
from block_sparse_attention_nvfp4_gb300 import build as msa_build
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


def _in_threads(*calls):
    """Runs the calls at once; raises what they raise."""
    start, raised = threading.Barrier(len(calls)), []

    def run(call):
        start.wait()
        try:
            call()
        except BaseException as e:      # noqa: BLE001  (told below)
            raised.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if raised:
        raise raised[0]


@pytest.fixture
def slow(host, monkeypatch):
    """Launches that take a while, with the interpreter free for other threads meanwhile, as a library call leaves it.
    seen: (thread, operator, addresses of the weights at the launch's end, launches under way)."""
    seen, inside = [], []

    def call(dev, stream, fn, what, ref, *args):
        inside.append(what)
        together = len(inside)
        time.sleep(0.05)
        caches = next((a for a in args if isinstance(a, _lib.Kv8EvictCache * 1)), ())
        seen.append((threading.get_ident(), what, [c.weights for c in caches], max(together, len(inside))))
        inside.remove(what)

    monkeypatch.setattr(pages, "_call", call)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return seen


def test_threads_evict_with_their_own_weights(slow):
    pool = PagePool([_cache()], _i32(3), _i32(3, 4), _i32(6))
    seqs, ws = _i32(2), [torch.zeros((3, 2, 512)) for _ in range(4)]
    mine = {}

    def evict(w):
        mine[threading.get_ident()] = w.data_ptr()
        pool.evict(seqs, seqs, w, 10)

    _in_threads(*[lambda w=w: evict(w) for w in ws])
    assert len(slow) == len(ws)
    for thread, what, weights, together in slow:
        assert what == "msa_pages_evict" and weights == [mine[thread]] and together == 1


def test_operators_of_several_threads_are_launched_one_by_one(slow):
    """Their launches share the workspace's lists."""
    pool = PagePool([_cache()], _i32(3), _i32(3, 4), _i32(6))
    seqs, w = _i32(2), torch.zeros((3, 2, 512))
    _in_threads(lambda: pool.fork(seqs, seqs), lambda: pool.evict(seqs, seqs, w, 10), lambda: pool.free(seqs), pool.compact)
    assert sorted(x[1] for x in slow) == ["msa_pages_compact", "msa_pages_evict", "msa_pages_fork", "msa_pages_free"]
    assert [x[3] for x in slow] == [1] * 4


def test_no_scratch_where_no_sequence_can_be_longer_than_keep(slow):
    pool = PagePool([_cache()], _i32(3), _i32(3, 4), _i32(6))
    seqs, w = _i32(2), torch.zeros((3, 2, 512))
    for keep in (512, 10 ** 9):
        pool.evict(seqs, seqs, w, keep)
        assert pool._scratch[1] == 256
    pool.evict(seqs, seqs, w, 511)
    assert pool._scratch[1] == 8 * 2 * 2 * 511


def test_the_library_wants_none_either():
    """Seen by which refusal comes first: so many new pages that no grid holds them, or the scratch that is not there."""
    msa_build.build()
    lib, x = _lib.load(), 1 << 21       # (addresses that are never dereferenced)
    pool = _lib.PagePoolArgs(num_seqs=1 << 20, num_pages=16, max_pages_per_seq=8, num_planes=0, seq_lens=x, block_table=x, ref_counts=x)
    caches = (_lib.Kv8EvictCache * 4)(*[_lib.Kv8EvictCache(x, x, x, x, x, 1024, 64) for _ in range(4)])
    for keep, code in ((1024, -2), (1 << 30, -2), (1023, -4)):
        assert lib.msa_pages_evict(ctypes.byref(pool), 1 << 20, x, x, 4, caches, keep, 0, 0, None, 0, ctypes.c_void_p(1 << 20),
                                   1 << 40, None) == code
