"""The 8-bit paged cache (E4M3 codes, one FP32 scale for each 128-token page and KV head), the
append that fills it and the attention that reads it. All compute runs in libmsa's kernels
(msa_kv8_append, msa_kv8_attn in include/msa.h)."""
from __future__ import annotations

import ctypes
import dataclasses
import math
from typing import Optional

import torch

from . import _lib

DIM, BLOCK = 128, 128
_SRC_TYPES = {torch.bfloat16: _lib.TYPE_BF16, torch.float16: _lib.TYPE_F16, torch.float32: _lib.TYPE_F32}
_Q_TYPES = {torch.uint8: _lib.TYPE_E4M3, torch.float8_e4m3fn: _lib.TYPE_E4M3, torch.bfloat16: _lib.TYPE_BF16}


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _plain(t: torch.Tensor, dtype, shape, dev, name: str) -> int:
    """The address of a contiguous tensor of the given type and shape on `dev`."""
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    _need(t.is_cuda and t.device == dev, f"{name}: expected a tensor on {dev}, got {t.device}")
    _need(t.dtype in dtypes, f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    _need(tuple(t.shape) == tuple(shape), f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    _need(t.is_contiguous(), f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _rows(t: torch.Tensor, heads: int, name: str) -> int:
    """The stride between the rows of [rows, heads, 128] whose heads are contiguous."""
    _need(t.stride(2) == 1 and (heads == 1 or t.stride(1) == DIM),
          f"{name}: the heads of a row must be contiguous, got strides {t.stride()}")
    return t.stride(0) if t.shape[0] > 1 else heads * DIM


def _call(dev, stream, fn, what, *args):
    """fn(*args, stream) on the tensors' device; the stream is that device's current one unless given."""
    if torch.cuda.current_device() == dev.index:
        _lib._check(fn(*args, _lib._stream(stream)), what)
    else:
        with torch.cuda.device(dev):
            _lib._check(fn(*args, _lib._stream(stream)), what)


@dataclasses.dataclass
class KV8Batch:
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


def _geometry(a, cache: "KV8Cache", batch, dev):
    B = batch.num_reqs
    a.num_reqs, a.total_rows, a.max_rows_per_req = B, int(batch.total_rows), int(batch.max_rows_per_req)
    a.num_pages, a.num_kv_heads = cache.num_pages, cache.num_kv_heads
    a.max_pages_per_req = int(batch.block_table.shape[1])
    a.context_lens = _plain(batch.context_lens, torch.int32, (B,), dev, "context_lens")
    a.q_indptr = _plain(batch.q_indptr, torch.int32, (B + 1,), dev, "q_indptr")
    a.block_table = _plain(batch.block_table, torch.int32, (B, a.max_pages_per_req), dev, "block_table")


@dataclasses.dataclass
class KV8Cache:
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

    def _pointers(self, a, dev):
        P, H = self.num_pages, self.num_kv_heads
        for n in ("k", "v"):
            data, scale = getattr(self, n + "_data"), getattr(self, n + "_scale")
            setattr(a, n + "_data", _plain(data, (torch.uint8, torch.float8_e4m3fn), (P, H, BLOCK, DIM), dev, n + "_data"))
            setattr(a, n + "_scale", _plain(scale, torch.float32, (P, H), dev, n + "_scale"))

    def append(self, batch, k: Optional[torch.Tensor], v: Optional[torch.Tensor], ws: torch.Tensor, stream=None):
        """Quantise the batch's new tokens into their pages (msa_kv8_append): k and v
        [rows, H, 128] in bfloat16, float16 or float32 (one type for both; rows may be strided, as
        the parts of a fused projection are), either of them None; ws a zero-filled workspace
        of >= 256 bytes (error flags). `batch` is a KV8Batch or a DecodeBatch; its q is not read."""
        a = _lib.Kv8AppendArgs()
        dev = self.k_data.device
        _geometry(a, self, batch, dev)
        self._pointers(a, dev)
        types = {t.dtype for t in (k, v) if t is not None}
        _need(len(types) <= 1 and types <= _SRC_TYPES.keys(),
              f"k and v: expected one of bfloat16, float16, float32 for both, got {types}")
        a.src_type = _SRC_TYPES[types.pop()] if types else _lib.TYPE_BF16
        for name, t in (("k", k), ("v", v)):
            if t is None:
                continue
            _need(t.is_cuda and t.device == dev and tuple(t.shape) == (a.total_rows, a.num_kv_heads, DIM),
                  f"{name}: expected [{a.total_rows}, {a.num_kv_heads}, {DIM}] on {dev}, got {tuple(t.shape)} on {t.device}")
            setattr(a, name + "_token_stride", _rows(t, a.num_kv_heads, name))
            setattr(a, name, t.data_ptr())
        _need(ws.is_cuda and ws.device == dev and ws.is_contiguous(), f"ws: expected a contiguous tensor on {dev}")
        _call(dev, stream, _lib.load().msa_kv8_append, "msa_kv8_append", ctypes.byref(a),
              ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size())


class KV8Attention:
    """Attention over a KV8Cache for a batch; owns its workspace and outputs (`out` BF16
    [rows, heads, 128], `lse` FP32 [rows, heads]). Single tokens, speculative rows and prompts
    (causal) take the same call; a batch of the same sizes can be bound with `rebind`."""

    def __init__(self, cache: KV8Cache, batch: KV8Batch, sm_scale: Optional[float] = None, with_lse: bool = True):
        self.cache = cache
        self.sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(DIM)
        self.device = cache.k_data.device
        _need(batch.q is not None and batch.q.dim() == 3 and batch.q.shape[2] == DIM, "q: expected [rows, heads, 128]")
        heads = int(batch.q.shape[1])
        rows = int(batch.total_rows)
        self.out = torch.empty((rows, heads, DIM), dtype=torch.bfloat16, device=self.device)
        self.lse = torch.empty((rows, heads), dtype=torch.float32, device=self.device) if with_lse else None
        self.rebind(batch)
        n = ctypes.c_size_t(0)
        with torch.cuda.device(self.device):
            _lib._check(_lib.load().msa_kv8_attn_workspace_size(ctypes.byref(self.args), ctypes.byref(n)),
                        "msa_kv8_attn_workspace_size")
            self.ws = torch.empty(n.value, dtype=torch.uint8, device=self.device)
            _lib.msa_workspace_init(self.ws)

    def rebind(self, batch: KV8Batch):
        """Point at another batch of the same sizes."""
        a = _lib.Kv8AttnArgs()
        _geometry(a, self.cache, batch, self.device)
        self.cache._pointers(a, self.device)
        rows, heads = self.out.shape[:2]
        q = batch.q
        _need(q is not None and q.is_cuda and q.device == self.device and tuple(q.shape) == (rows, heads, DIM) and
              rows == a.total_rows, f"q: expected [{rows}, {heads}, {DIM}] on {self.device}")
        _need(q.dtype in _Q_TYPES, f"q: expected bfloat16 or E4M3 (uint8, float8_e4m3fn), got {q.dtype}")
        _need(heads % a.num_kv_heads == 0, f"q: {heads} heads do not divide among {a.num_kv_heads} KV heads")
        if getattr(self, "args", None) is not None:
            old = self.args
            _need((old.num_reqs, old.max_rows_per_req, old.max_pages_per_req) ==
                  (a.num_reqs, a.max_rows_per_req, a.max_pages_per_req), "rebind: expected a batch of the same sizes")
        a.q_per_kv = heads // a.num_kv_heads
        a.q_type, a.q_row_stride, a.q = _Q_TYPES[q.dtype], _rows(q, heads, "q"), q.data_ptr()
        a.sm_scale = float(self.sm_scale)
        a.out = self.out.data_ptr()
        a.lse = self.lse.data_ptr() if self.lse is not None else None
        self.batch, self.args = batch, a

    def attend(self, block_ids: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """softmax(sm_scale q k) v of every row over the keys it may see: of all blocks, or of
        those in block_ids (int32 [B, H, n <= 32], -1 = unused), e.g. the ones that
        MSADecoder.select_blocks chose. Returns `out`; `lse` has ln(sum(exp))."""
        a = self.args
        if block_ids is None:
            a.block_ids, a.n_block_ids = None, 0
        else:
            n = int(block_ids.shape[-1])
            a.block_ids = _plain(block_ids, torch.int32, (a.num_reqs, a.num_kv_heads, n), self.device, "block_ids")
            a.n_block_ids = n
        _call(self.device, stream, _lib.load().msa_kv8_attn, "msa_kv8_attn", ctypes.byref(a),
              ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel())
        return self.out

    def errors(self, stream=None) -> int:
        """Device error flags since the last read (synchronises the stream)."""
        with torch.cuda.device(self.device):
            return _lib.msa_get_error(self.ws, stream)
