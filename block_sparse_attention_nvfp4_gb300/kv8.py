"""The 8-bit paged cache (E4M3 codes, one FP32 scale for each 128-token page and KV head), the
append that fills it and the attention that reads it. All compute runs in libmsa's kernels
(msa_kv8_append, msa_kv8_attn in include/msa.h)."""
from __future__ import annotations

import ctypes
import dataclasses
import math
import struct
from typing import Optional

import torch

from . import _lib

DIM, BLOCK = 128, 128
_INT_MAX = 2 ** 31 - 1
_SRC_TYPES = {torch.bfloat16: _lib.TYPE_BF16, torch.float16: _lib.TYPE_F16, torch.float32: _lib.TYPE_F32}
_Q_TYPES = {torch.uint8: _lib.TYPE_E4M3, torch.float8_e4m3fn: _lib.TYPE_E4M3, torch.bfloat16: _lib.TYPE_BF16}


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _plain(t: torch.Tensor, dtype, shape, dev, name: str) -> int:
    """The address of a contiguous tensor of the given type and shape on `dev`."""
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    if not (t.dtype in dtypes and t.device == dev and t.is_cuda and t.shape == tuple(shape) and t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {' or '.join(map(str, dtypes))} tensor {tuple(shape)} on {dev} "
                         f"(a GPU), got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _rows(t: torch.Tensor, heads: int, name: str) -> int:
    """The stride between the rows of [rows, heads, 128] whose heads are contiguous."""
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != DIM):
        raise ValueError(f"{name}: the heads of a row must be contiguous, got strides {t.stride()}")
    return row if t.shape[0] > 1 else heads * DIM


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream
_append_args = struct.Struct("@7i2q9P")      # msa_kv8_append_args
assert _append_args.size == ctypes.sizeof(_lib.Kv8AppendArgs)


def _call(dev, stream, fn, what, *args):
    """fn(*args, stream) on the tensors' device; the stream is that device's current one unless given."""
    index = dev.index
    if _current_device() != index:
        with torch.cuda.device(dev):
            return _call(dev, stream, fn, what, *args)
    code = fn(*args, _current_stream(index) if stream is None else stream.cuda_stream)
    if code != _lib.MSA_OK:
        raise _lib.MSAError(code, what)


class _Handle:
    """Tensors that are checked and marshalled once: setting an attribute, or a tensor whose storage
    has moved, marshals again."""

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__.pop("_marshalled", None)


@dataclasses.dataclass
class KV8Batch(_Handle):
    """One step's per-request metadata on the GPU, and its queries: request b owns rows
    q_indptr[b] .. q_indptr[b+1] - 1, at positions context_lens[b] - R .. context_lens[b] - 1."""
    context_lens: torch.Tensor          # int32 [B], this step's rows included
    q_indptr: torch.Tensor              # int32 [B+1]
    block_table: torch.Tensor           # int32 [B, max_pages]
    q: Optional[torch.Tensor] = None    # [rows, heads, 128] bfloat16, or E4M3 (uint8 or float8_e4m3fn); rows may be strided
    total_rows: int = 0
    max_rows_per_req: int = 1

    @property
    def num_reqs(self) -> int:
        return int(self.context_lens.shape[0])


def _geometry(batch, dev):
    """(B, rows, most rows per request, row length of the table, the three tensors' addresses)."""
    got = batch.__dict__.get("_marshalled")
    if got is None or got[0] != dev or got[1][4] != batch.context_lens.data_ptr() or \
            got[1][5] != batch.q_indptr.data_ptr() or got[1][6] != batch.block_table.data_ptr():
        B, M = batch.num_reqs, int(batch.block_table.shape[1])
        got = (dev, (B, int(batch.total_rows), int(batch.max_rows_per_req), M,
                     _plain(batch.context_lens, torch.int32, (B,), dev, "context_lens"),
                     _plain(batch.q_indptr, torch.int32, (B + 1,), dev, "q_indptr"),
                     _plain(batch.block_table, torch.int32, (B, M), dev, "block_table")))
        if isinstance(batch, KV8Batch):
            batch.__dict__["_marshalled"] = got
    return got[1]


@dataclasses.dataclass
class KV8Cache(_Handle):
    """Paged 8-bit K and V: data [P, H, 128, 128] uint8 (E4M3 codes), scale [P, H] float32; the
    value of a slot is E4M3(code) * scale."""
    k_data: torch.Tensor
    k_scale: torch.Tensor
    v_data: torch.Tensor
    v_scale: torch.Tensor

    @property
    def num_pages(self) -> int:
        return int(self.k_data.shape[0])

    @property
    def num_kv_heads(self) -> int:
        return int(self.k_data.shape[1])

    @staticmethod
    def empty(num_pages: int, num_kv_heads: int = 4, device="cuda") -> "KV8Cache":
        data = lambda: torch.zeros((num_pages, num_kv_heads, BLOCK, DIM), dtype=torch.uint8, device=device)  # noqa: E731
        scale = lambda: torch.zeros((num_pages, num_kv_heads), dtype=torch.float32, device=device)  # noqa: E731
        return KV8Cache(data(), scale(), data(), scale())

    def _pointers(self):
        """(device, pages, KV heads, addresses of k_data, k_scale, v_data, v_scale)."""
        got = self.__dict__.get("_marshalled")
        if got is None or got[3] != self.k_data.data_ptr() or got[4] != self.k_scale.data_ptr() or \
                got[5] != self.v_data.data_ptr() or got[6] != self.v_scale.data_ptr():
            P, H, dev = self.num_pages, self.num_kv_heads, self.k_data.device
            codes = (torch.uint8, torch.float8_e4m3fn)
            got = (dev, P, H, _plain(self.k_data, codes, (P, H, BLOCK, DIM), dev, "k_data"),
                   _plain(self.k_scale, torch.float32, (P, H), dev, "k_scale"),
                   _plain(self.v_data, codes, (P, H, BLOCK, DIM), dev, "v_data"),
                   _plain(self.v_scale, torch.float32, (P, H), dev, "v_scale"))
            self.__dict__["_marshalled"] = got
        return got

    def append(self, batch, k: Optional[torch.Tensor], v: Optional[torch.Tensor], ws: torch.Tensor, stream=None):
        """Quantise the batch's new tokens into their pages (msa_kv8_append): k and v
        [rows, H, 128] in bfloat16, float16 or float32 (one type for both; rows may be strided, as
        the parts of a fused projection are), either of them None; ws a zero-filled workspace
        of >= 256 bytes (error flags). `batch` is a KV8Batch or a DecodeBatch; its q is not read."""
        dev, P, H, kd, ks, vd, vs = self._pointers()
        B, total, most, M, lens, indptr, table = _geometry(batch, dev)
        if k is not None:
            kp, kst, kt = self._source(k, total, H, dev, "k")
        if v is not None:
            vp, vst, vt = self._source(v, total, H, dev, "v")
            if k is None:
                kp, kst, kt = 0, 0, vt
            elif vt != kt:
                raise ValueError(f"k and v: expected one type for both, got {k.dtype} and {v.dtype}")
        else:
            vp = vst = 0
            if k is None:
                return
        if ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws: expected a contiguous tensor on {dev}")
        a = _append_args.pack(B, total, most, P, M, H, kt, kst, vst, lens, indptr, table, kp, vp, kd, ks, vd, vs)
        _call(dev, stream, _lib.load().msa_kv8_append, "msa_kv8_append", a, ws.data_ptr(), ws.nbytes)

    @staticmethod
    def _source(t: torch.Tensor, rows: int, heads: int, dev, name: str):
        """Address, row stride and type of new tokens' rows."""
        kind = _SRC_TYPES.get(t.dtype)
        if kind is None or t.shape != (rows, heads, DIM) or t.device != dev:
            raise ValueError(f"{name}: expected [{rows}, {heads}, {DIM}] on {dev} in one of {list(_SRC_TYPES)}, got "
                             f"{tuple(t.shape)} {t.dtype} on {t.device}")
        row, head, one = t.stride()
        if one != 1 or (heads > 1 and head != DIM):
            raise ValueError(f"{name}: the heads of a row must be contiguous, got strides {t.stride()}")
        return t.data_ptr(), row if rows > 1 else heads * DIM, kind


class KV8Attention:
    """Attention over a KV8Cache for a batch; owns its workspace and outputs (`out` BF16
    [rows, heads, 128], `lse` FP32 [rows, heads]). Single tokens, speculative rows and prompts
    (causal) take the same call, to all tokens, to listed blocks, to a window and sinks, or with the pages
    that requests have in common read for their rows together (`attend_shared`, for up to `max_groups` groups);
    `add_weights` (with_weights) says how much attention each cached token got. The workspace is laid out
    for what is asked for here; a batch of the same sizes can be bound with `rebind`, and tensors
    that were replaced in the cache or in the batch (a KV8Batch or a DecodeBatch) are seen by the
    next call, which raises when they do not fit."""

    def __init__(self, cache: KV8Cache, batch: KV8Batch, sm_scale: Optional[float] = None, with_lse: bool = True,
                 max_groups: int = 0, with_weights: bool = False):
        self.cache = cache
        self.sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(DIM)
        self.device = cache.k_data.device
        _need(batch.q is not None and batch.q.dim() == 3 and batch.q.shape[2] == DIM, "q: expected [rows, heads, 128]")
        heads = int(batch.q.shape[1])
        rows = int(batch.total_rows)
        self.out = torch.empty((rows, heads, DIM), dtype=torch.bfloat16, device=self.device)
        self.lse = torch.empty((rows, heads), dtype=torch.float32, device=self.device) if with_lse else None
        self.rebind(batch)
        self.max_groups = int(max_groups)
        self.with_weights = bool(with_weights)
        n, more, most = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
        with torch.cuda.device(self.device):
            lib = _lib.load()
            _lib._check(lib.msa_kv8_attn_workspace_size(self._ref, ctypes.byref(n)), "msa_kv8_attn_workspace_size")
            if self.max_groups:
                _lib._check(lib.msa_kv8_attn_shared_workspace_size(self._ref, self.max_groups, ctypes.byref(more)),
                            "msa_kv8_attn_shared_workspace_size")
            if self.with_weights:
                _lib._check(lib.msa_kv8_attn_weights_workspace_size(self._ref, ctypes.byref(most)),
                            "msa_kv8_attn_weights_workspace_size")
            self.ws = torch.empty(max(n.value, more.value, most.value), dtype=torch.uint8, device=self.device)
            _lib.msa_workspace_init(self.ws[:256])   # the flags: a call on another stream may follow at once
        self._ws = (self.ws.data_ptr(), self.ws.numel())

    def rebind(self, batch: KV8Batch):
        """Point at another batch of the same sizes. One that does not fit raises, and what was bound
        stays bound."""
        cache_at = self.cache._pointers()
        dev, P, H, kd, ks, vd, vs = cache_at
        _need(dev == self.device, f"cache: expected it on {self.device}, got {dev}")
        batch_at = _geometry(batch, dev)
        B, total, most, M, lens, indptr, table = batch_at
        rows, heads = self.out.shape[:2]
        q = batch.q
        _need(q is not None and q.device == dev and q.shape == (rows, heads, DIM) and rows == total,
              f"q: expected [{rows}, {heads}, {DIM}] on {dev}")
        _need(q.dtype in _Q_TYPES, f"q: expected bfloat16 or E4M3 (uint8, float8_e4m3fn), got {q.dtype}")
        _need(heads % H == 0, f"q: {heads} heads do not divide among {H} KV heads")
        old = getattr(self, "args", None)
        _need(old is None or (old.num_reqs, old.max_rows_per_req, old.max_pages_per_req) == (B, most, M),
              "rebind: expected a batch of the same sizes")
        args = _lib.Kv8AttnArgs(B, total, most, P, M, H, heads // H, 0, _Q_TYPES[q.dtype], float(self.sm_scale),
                                _rows(q, heads, "q"), lens, indptr, table, None, q.data_ptr(), kd, ks, vd, vs,
                                self.out.data_ptr(), self.lse.data_ptr() if self.lse is not None else None)
        # Every check has passed. attend() compares these marks with the tensors: set earlier, they
        # would hide from the call after a refused one that its arguments are still the old ones.
        self._cache_at, self._batch_at = cache_at, batch_at
        self.batch, self._follows = batch, isinstance(batch, KV8Batch)
        c = self.cache
        self._held = (batch.q, batch.context_lens, batch.q_indptr, batch.block_table,   # as long as they are bound
                      c.k_data, c.k_scale, c.v_data, c.v_scale)
        self.args, self._ref = args, ctypes.byref(args)
        self._lse_of_all = False    # whether `lse` is that of the bound batch's rows over all keys they see

    def _batch_changed(self, batch) -> bool:
        """Whether a tensor or a size of the bound batch is another than the bound one."""
        a, held = self.args, self._held
        if batch.q is not held[0] or batch.q.data_ptr() != (a.q or 0):      # (no rows: the address is 0, which reads as None)
            return True
        if self._follows:
            return _geometry(batch, self.device) is not self._batch_at
        # a DecodeBatch keeps no marks of its own
        t = (batch.context_lens, batch.q_indptr, batch.block_table)
        return not (t[0] is held[1] and t[1] is held[2] and t[2] is held[3] and
                    batch.total_rows == a.total_rows and batch.max_rows_per_req == a.max_rows_per_req and
                    (t[0].data_ptr(), t[1].data_ptr(), t[2].data_ptr()) == self._batch_at[4:])

    def _current(self):
        """The arguments, marshalled again if a tensor was replaced."""
        moved = self._batch_changed(self.batch)
        if moved or self.cache._pointers() is not self._cache_at:
            of_all = self._lse_of_all and not moved     # (a cache that grew has the same keys)
            self.rebind(self.batch)
            self._lse_of_all = of_all
        return self.args

    def attend(self, block_ids: Optional[torch.Tensor] = None, stream=None, *, window: Optional[int] = None,
               sinks: int = 0) -> torch.Tensor:
        """softmax(sm_scale q k) v of every row over the keys it may see: of all blocks, or of
        those in block_ids (int32 [B, H, n <= 32], -1 = unused), e.g. the ones that
        MSADecoder.select_blocks chose; with a window, its last `window` keys (its own among them) and
        the first `sinks` ones. Returns `out`; `lse` has ln(sum(exp))."""
        a = self._current()
        if window is not None:
            _need(block_ids is None, "block_ids: not with a window")
            _need(0 < window <= _INT_MAX and 0 <= sinks <= _INT_MAX, f"window, sinks: expected at least 1 and 0, got {window}, {sinks}")
            a.block_ids, a.n_block_ids = None, 0
            _call(self.device, stream, _lib.load().msa_kv8_attn_window, "msa_kv8_attn_window", self._ref, window, sinks,
                  self._ws[0], self._ws[1])
            self._lse_of_all = window >= a.max_pages_per_req * BLOCK
            return self.out
        _need(sinks == 0, "sinks: only with a window")
        if block_ids is None:
            a.block_ids, a.n_block_ids = None, 0
        else:
            n = int(block_ids.shape[-1])
            _need(n >= 1, "block_ids: expected at least one id (None: all blocks)")
            a.block_ids = _plain(block_ids, torch.int32, (a.num_reqs, a.num_kv_heads, n), self.device, "block_ids")
            a.n_block_ids = n
        _call(self.device, stream, _lib.load().msa_kv8_attn, "msa_kv8_attn", self._ref, self._ws[0], self._ws[1])
        self._lse_of_all = block_ids is None
        return self.out

    def attend_shared(self, group_indptr: torch.Tensor, stream=None, *, min_saved: Optional[int] = None) -> torch.Tensor:
        """attend() to all keys, for requests whose block tables begin with the same pages: the leading pages
        that the requests group_indptr[g] .. group_indptr[g+1] - 1 (int32 on the GPU, at most
        max_groups groups) have in common are found and read for the rows of the group together, once for each item
        of them (128 / queries a KV head, 32 at most). min_saved: page reads, over all KV heads and groups, that this has to
        save, else requests are taken alone, as prompts are (None: the library's choice; where the sizes, the block
        table's width among them, leave little to save, the call is attend() itself)."""
        n = group_indptr.numel() - 1
        _need(min_saved is None or 0 <= min_saved <= _INT_MAX, f"min_saved: expected at least 0, got {min_saved}")
        _need(0 <= n <= self.max_groups, f"group_indptr: expected 1 to {self.max_groups + 1} entries (max_groups), got {n + 1}")
        a = self._current()
        at = _plain(group_indptr, torch.int32, (n + 1,), self.device, "group_indptr")
        a.block_ids, a.n_block_ids = None, 0
        _call(self.device, stream, _lib.load().msa_kv8_attn_shared, "msa_kv8_attn_shared", self._ref, n, at,
              -1 if min_saved is None else min_saved, self._ws[0], self._ws[1])
        self._lse_of_all = True
        return self.out

    def add_weights(self, old: Optional[torch.Tensor], new: torch.Tensor, keep: float = 1.0,
                    lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """new[b, h, t] = keep old[b, h, t] + the softmax weights that token t of request b got from this batch's rows, over the
        queries of KV head h; the batch's own tokens, whose slots are new, start from 0, and so does every token
        with old None. FP32 [B, H, L], L at least the block table's tokens; `new` may be `old`. Where PagePool.evict is to
        go by them, they are rows of the pool's [S, H, L]: a slice, or rows gathered before and copied back after. lse (FP32
        [rows, heads]) is what attend() to all keys left in `lse`, unless given: without it the last attention
        call has to be one to all keys of this batch (attend() or attend_shared()). Needs with_weights."""
        _need(self.with_weights, "add_weights: make the object with with_weights=True")
        a = self._current()
        if lse is None:
            lse = self.lse
            _need(lse is not None, "lse: expected one, as the object keeps none")
            _need(self._lse_of_all, "lse: expected one, as the object's is not that of this batch over all keys "
                                    "(attend() was not called, or last with a window or listed blocks)")
        shape = (a.num_reqs, a.num_kv_heads, int(new.shape[-1]) if new.dim() else 0)
        _need(shape[2] >= a.max_pages_per_req * BLOCK, f"new: expected at least {a.max_pages_per_req * BLOCK} tokens a head, got {shape[2]}")
        at = _plain(new, torch.float32, shape, self.device, "new")
        from_ = None if old is None else _plain(old, torch.float32, shape, self.device, "old")
        lse_at = _plain(lse, torch.float32, tuple(self.out.shape[:2]), self.device, "lse")
        a.block_ids, a.n_block_ids = None, 0
        _call(self.device, stream, _lib.load().msa_kv8_attn_weights, "msa_kv8_attn_weights", self._ref, lse_at, keep, from_, at,
              shape[2], self._ws[0], self._ws[1])
        return new

    def errors(self, stream=None) -> int:
        """Device error flags since the last read (synchronises the stream)."""
        with torch.cuda.device(self.device):
            return _lib.msa_get_error(self.ws, stream)
