"""A pool of cache pages shared by sequences, on the device: copy, fork, reserve, free and compact
without a synchronisation, and sequences cut to their heaviest tokens (msa_pages_* in include/msa.h)."""
from __future__ import annotations

import ctypes
import operator
import threading
from typing import Optional, Sequence, Union

import torch

from . import _lib
from .api import KVCache
from .kv8 import _INT_MAX, BLOCK, KV8Cache, _call, _need, _plain

_address = torch.Tensor.data_ptr


def _planes(cache, num_pages: int, dev):
    """(name, data, strips, slot_bytes, page_bytes) of every plane of a cache."""
    names = ("k_data", "k_scale", "v_data", "v_scale") + (("ki_data", "ki_scale") if isinstance(cache, KVCache) else ())
    for name in names:
        t = getattr(cache, name)
        _need(t.is_cuda and t.device == dev and t.is_contiguous(), f"{name}: expected a contiguous tensor on {dev}")
        _need(t.shape[0] == num_pages, f"{name}: expected {num_pages} pages, got {t.shape[0]}")
        size = t.element_size()
        if t.dim() == 2:     # scales kept once for a page
            yield name, t.data_ptr(), 0, 0, t.shape[1] * size
        else:
            _need(t.shape[-2] == BLOCK, f"{name}: expected {BLOCK} slots in a page, got shape {tuple(t.shape)}")
            yield name, t.data_ptr(), (t.shape[1] if t.dim() == 4 else 1), t.shape[-1] * size, 0


class PagePool:
    """Sequences over the pages of one or more caches (KVCache, KV8Cache).

    seq_lens int32 [S], block_table int32 [S, M] and ref_counts int32 [P] are the caller's
    tensors (slices of them are the context_lens and block_table of a decode batch); the
    operators change them in place, in stream order. ref_counts[p] is the number of rows that
    hold page p, 0 = free. Sequence and page lists are int32 CUDA tensors. The tensors are bound when
    the pool is made: after one is replaced, or its storage has moved, every operator raises. Calls from several
    threads are launched one after the other; on the device they have to be in stream order, as any two calls."""

    def __init__(self, caches: Sequence[Union[KVCache, KV8Cache]], seq_lens: torch.Tensor, block_table: torch.Tensor,
                 ref_counts: torch.Tensor):
        self.caches, self.seq_lens, self.block_table, self.ref_counts = list(caches), seq_lens, block_table, ref_counts
        _need(block_table.dim() == 2 and ref_counts.dim() == 1, "expected block_table [S, M] and ref_counts [P]")
        self.device = dev = ref_counts.device
        S, M, P = int(block_table.shape[0]), int(block_table.shape[1]), int(ref_counts.shape[0])
        a = self.args = _lib.PagePoolArgs()
        a.num_seqs, a.num_pages, a.max_pages_per_seq = S, P, M
        a.seq_lens = _plain(seq_lens, torch.int32, (S,), dev, "seq_lens")
        a.block_table = _plain(block_table, torch.int32, (S, M), dev, "block_table")
        a.ref_counts = _plain(ref_counts, torch.int32, (P,), dev, "ref_counts")
        planes = [(c, *x) for c in self.caches for x in _planes(c, P, dev)]
        _need(len(planes) <= _lib.MAX_PLANES, f"at most {_lib.MAX_PLANES} planes, got {len(planes)}")
        a.num_planes = len(planes)
        for i, (_, _, data, strips, slot, page) in enumerate(planes):
            a.planes[i].data, a.planes[i].strips, a.planes[i].slot_bytes, a.planes[i].page_bytes = data, strips, slot, page
        # (owner, its tensors' names, how to get them, the ones that are bound), and the addresses of all
        names = [(self, ("seq_lens", "block_table", "ref_counts"))]
        names += [(c, tuple(dict.fromkeys(x[1] for x in planes if x[0] is c))) for c in self.caches]
        self._bound = [(o, n, operator.attrgetter(*n)) for o, n in names]
        self._bound = [(o, n, get, get(o)) for o, n, get in self._bound]
        self._tensors = [t for x in self._bound for t in x[3]]
        self._at = list(map(_address, self._tensors))
        n = ctypes.c_size_t(0)
        _lib._check(_lib.load().msa_pages_workspace_size(ctypes.byref(a), ctypes.byref(n)), "msa_pages_workspace_size")
        with torch.cuda.device(dev):
            self.ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
            _lib.msa_workspace_init(self.ws[:256])   # the flags: a call on another stream may follow at once
        lib = _lib.load()
        self._fns = {n: getattr(lib, n) for n in ("msa_pages_copy", "msa_pages_fork", "msa_pages_reserve",
                                                  "msa_pages_free", "msa_pages_compact", "msa_pages_evict")}
        # evict's; outgrown ones live on, as captured graphs may hold them (together less than the one in use, each being at
        # most half of the next)
        self._scratch, self._scratches = None, []
        self._evict_caches, self._evict_shapes, self._most = None, (), M * BLOCK   # and the shapes of each one's weights
        # An operator is several launches that share the workspace: no other thread's come between them.
        self._lock = threading.RLock()
        self._ref, self._ws, self._index = ctypes.byref(a), (self.ws.data_ptr(), self.ws.numel()), dev.index

    @staticmethod
    def empty(caches: Sequence[Union[KVCache, KV8Cache]], num_seqs: int, max_pages: int) -> "PagePool":
        """A pool of empty sequences over caches whose pages are all free."""
        ref = caches[0].k_data
        z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=ref.device)  # noqa: E731
        return PagePool(caches, z(num_seqs), z(num_seqs, max_pages).fill_(-1), z(ref.shape[0]))

    def _list(self, t: torch.Tensor, n: int, name: str) -> int:
        if t.dtype is not torch.int32 or t.get_device() != self._index or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous int32 list of {n} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _unchanged(self):
        for owner, names, get, bound in self._bound:
            if not all(map(operator.is_, get(owner), bound)):
                changed = [n for n, x, y in zip(names, get(owner), bound) if x is not y]
                raise ValueError(f"{', '.join(changed)}: replaced after the pool was made")
        if list(map(_address, self._tensors)) != self._at:   # the same objects with other storages (set_, resize_, .data)
            names = [n for x in self._bound for n in x[1]]
            changed = [n for n, t, a in zip(names, self._tensors, self._at) if _address(t) != a]
            raise ValueError(f"{', '.join(changed)}: moved after the pool was made")

    def _run(self, name: str, stream, *args):
        self._unchanged()
        with self._lock:
            _call(self.device, stream, self._fns[name], name, self._ref, *args, *self._ws)

    def copy(self, src: torch.Tensor, dst: torch.Tensor, tokens: Optional[torch.Tensor] = None, stream=None):
        """Copy page src[i] to dst[i] in every plane: the first tokens[i] slots, or all."""
        n = src.numel()
        self._run("msa_pages_copy", stream, n, self._list(src, n, "src"), self._list(dst, n, "dst"),
                  None if tokens is None else self._list(tokens, n, "tokens"))

    def fork(self, parents: torch.Tensor, children: torch.Tensor, stream=None):
        """Make the empty sequences children[i] copies of parents[i]: full pages shared, a partly
        filled last page copied to a free page."""
        n = children.numel()
        self._run("msa_pages_fork", stream, n, self._list(parents, n, "parents"), self._list(children, n, "children"))

    def reserve(self, seqs: torch.Tensor, new_lens: torch.Tensor, stream=None):
        """Grow sequences to new_lens tokens, with free pages behind theirs as needed."""
        n = seqs.numel()
        self._run("msa_pages_reserve", stream, n, self._list(seqs, n, "seqs"), self._list(new_lens, n, "new_lens"))

    def free(self, seqs: torch.Tensor, stream=None):
        """End sequences: their pages' counts fall by one, their lengths become 0."""
        n = seqs.numel()
        self._run("msa_pages_free", stream, n, self._list(seqs, n, "seqs"))

    def compact(self, block_table: Optional[torch.Tensor] = None, ref_counts: Optional[torch.Tensor] = None,
                num_live: Optional[torch.Tensor] = None, stream=None):
        """Move the live pages to the ids 0 .. L - 1, in place or with the new tables written to the
        given tensors (both or neither); num_live (int32 [1]) gets L. The pages move either way: with
        tensors of their own, copy them over the pool's before its next operator, whose free pages
        would otherwise be ones in use."""
        if (block_table is None) != (ref_counts is None):
            raise ValueError("compact: give both tables or neither")
        a = self.args
        if block_table is None:
            t, r = a.block_table, a.ref_counts
        else:
            t = _plain(block_table, torch.int32, (a.num_seqs, a.max_pages_per_seq), self.device, "block_table")
            r = self._list(ref_counts, a.num_pages, "ref_counts")
        self._run("msa_pages_compact", stream, t, r, None if num_live is None else self._list(num_live, 1, "num_live"))

    def _evictable(self):
        """The caches as the eviction takes them: what it alone wants of their planes is checked at its first call."""
        if not self.caches or not all(isinstance(c, KV8Cache) for c in self.caches):
            raise ValueError("evict: every cache of the pool has to be a KV8Cache, and at least one")
        caches = (_lib.Kv8EvictCache * len(self.caches))()
        for x, c in zip(caches, self.caches):
            _, _, x.num_kv_heads, x.k_data, x.k_scale, x.v_data, x.v_scale = c._pointers()
        self._evict_shapes = [(self.args.num_seqs, x.num_kv_heads) for x in caches]
        self._evict_bytes = 8 * sum(x.num_kv_heads for x in caches)   # scratch of a kept token
        self._evict_caches = caches
        return caches

    def evict(self, parents: torch.Tensor, children: torch.Tensor, weights: Union[torch.Tensor, Sequence[torch.Tensor]],
              keep: int, sinks: int = 0, recent: int = 0, stream=None):
        """Make children[i] the parents[i] cut to `keep` tokens, on pages of its own: of a longer sequence every KV head
        keeps the first `sinks`, the last `recent` and the heaviest others (equal weights: the lowest
        positions), in the order of their positions. weights (one for each cache) are FP32 [S, H, L], L at least the
        block table's tokens, a row for each sequence as KV8Attention.add_weights fills them; the children's
        rows get the kept tokens' weights. A child is an empty sequence, or its own parent: the
        sequence is cut where it stands, and its old pages are given back. All caches have to be KV8Caches."""
        caches, most, index = self._evict_caches, self._most, self._index
        if caches is None:
            caches = self._evictable()
        weights = (weights,) if isinstance(weights, torch.Tensor) else tuple(weights)
        if len(weights) != len(caches):
            raise ValueError(f"weights: expected {len(caches)} (one for each cache), got {len(weights)}")
        n = children.numel()
        at = self._list(parents, n, "parents"), self._list(children, n, "children")
        if not (0 < keep <= _INT_MAX and 0 <= sinks and 0 <= recent and sinks + recent <= keep):
            raise ValueError(f"evict: expected keep >= 1 and sinks + recent <= keep, got {keep}, {sinks}, {recent}")
        # (what msa_pages_evict_scratch_size says; none where no sequence can be longer than keep)
        need = n * self._evict_bytes * keep if keep < most else 0
        self._unchanged()
        with self._lock:      # (the weights' addresses stand in `caches` until the launch)
            for x, heads, w in zip(caches, self._evict_shapes, weights):
                shape = w.shape
                tokens = shape[-1] if shape else 0
                if tokens < most:
                    raise ValueError(f"weights: expected at least {most} tokens a head, got {tokens}")
                if w.dtype is torch.float32 and w.get_device() == index and shape == (*heads, tokens) and w.is_contiguous():
                    x.weights = w.data_ptr()
                else:
                    x.weights = _plain(w, torch.float32, (*heads, tokens), self.device, "weights")   # (says what is wrong)
                x.head_stride = tokens
            scratch = self._scratch
            if scratch is None or scratch[1] < need:
                if scratch is not None:
                    self._scratches.append(scratch)
                size = max(need, 2 * (scratch[1] if scratch is not None else 0), 256)
                with torch.cuda.device(self.device), torch.cuda.stream(stream):
                    t = torch.empty(size, dtype=torch.uint8, device=self.device)
                scratch = self._scratch = (t.data_ptr(), size, t)
            _call(self.device, stream, self._fns["msa_pages_evict"], "msa_pages_evict", self._ref, n, *at, len(caches), caches,
                  keep, sinks, recent, scratch[0], scratch[1], *self._ws)

    def errors(self, stream=None) -> int:
        """Device error flags since the last read (synchronises the stream)."""
        with torch.cuda.device(self.device):
            return _lib.msa_get_error(self.ws, stream)
