"""The quantised key/value cache of one attention layer (include/gpt_ops.h: gpt_kv_cache and the
calls that take it) on torch tensors.

``KVCache`` bundles a layer's cache buffers; ``KVBatch`` describes the sequences of a call and their
new tokens and is shared by all layers.  A step of a layer is ``append`` (RoPE, QK-norm, quantise),
then ``attend``, over everything or over the blocks that ``select`` chose.  Nothing is read back to
the host, so a step can be captured into a CUDA graph and replayed with new contents.  Rows that belong
to no sequence are left as they are: in an output that a call makes itself they hold anything."""
from __future__ import annotations

import ctypes as C
import operator

import torch

from ._lib import KVBatchParams, KVCacheParams, call, check, lib

KV_BLOCK = 64  # tokens of a cache block
_INT_MAX = 2 ** 31 - 1  # (ctypes cuts a longer number off without a word)


def tile_bytes(bits: int, head_dim: int) -> int:
    """Bytes of one block and kv head: codes and scales of 64 keys and 64 values."""
    n = C.c_size_t()
    call("gpt_kv_tile_bytes", bits, head_dim, C.byref(n))
    return n.value


_device, _raw_stream = (getattr(torch._C, n, None) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))
_calls = {}  # library functions by name


def _launch(name: str, dev: torch.device, *args) -> None:
    """The library call ``name`` with ``dev``'s current stream as its last argument, launched on ``dev``
    whichever device is current.  A decoding step is a handful of calls of a few microseconds, so this
    path takes the raw stream handle and enters a device guard only where it changes something."""
    f = _calls.get(name)
    if f is None:
        f = _calls[name] = getattr(lib(), name)
    i = dev.index
    if _device() == i:
        rc = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(i))
    if rc:
        check(rc)


def _check(t: torch.Tensor, name: str, dtype, dev, shape=None) -> None:
    assert t.dtype == dtype, f"{name}: {dtype} needed, got {t.dtype}"
    assert t.device == dev, f"{name}: on {t.device}, the cache is on {dev}"
    assert t.is_contiguous(), f"{name}: must be contiguous"
    assert shape is None or t.shape == shape, f"{name}: shape {tuple(shape)} needed, got {tuple(t.shape)}"


def _out(t, name: str, shape, like: torch.Tensor) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one of ``like``'s type and device."""
    if t is None:
        return like.new_empty(*shape)  # (sizes one by one: parsed faster than a tuple)
    _check(t, name, like.dtype, like.device, shape)
    return t


def _frozen(*names):
    """Read-only attributes ``name``, held as ``_name``: the library's calls go by the pointers and sizes of
    the constructor, so an assignment would change nothing but let go of memory that they still use."""
    def deco(cls):
        for n in names:
            setattr(cls, n, property(operator.attrgetter("_" + n)))
        return cls
    return deco


@_frozen("block_table", "lens", "cu_new", "max_new", "device", "n_seq", "max_blocks")
class KVBatch:
    """Sequences and their new tokens (gpt_kv_batch): ``block_table`` int32 [n_seq, max_blocks], ``lens``
    int32 [n_seq] (new tokens included) and ``cu_new`` int32 [n_seq + 1], the first row of each
    sequence in the row tensors (None: one new token each, row b for sequence b); ``max_new``: the most
    new tokens a sequence has.  The tensors are kept, not copied: update them in place between steps
    (``batch.lens.add_(1)``, ``batch.lens.copy_(...)``); the attributes cannot be assigned to."""

    def __init__(self, block_table: torch.Tensor, lens: torch.Tensor, cu_new: torch.Tensor | None = None, *,
                 max_new: int = 1):
        dev = block_table.device
        assert block_table.dim() == 2, "block_table: [n_seq, max_blocks]"
        n, w = block_table.shape
        _check(block_table, "block_table", torch.int32, dev)
        _check(lens, "lens", torch.int32, dev, (n,))
        if cu_new is not None:
            _check(cu_new, "cu_new", torch.int32, dev, (n + 1,))
        assert 0 <= max_new <= _INT_MAX, "max_new: 32 bits, not negative"
        assert cu_new is not None or max_new == 1, "max_new: without cu_new it is 1"
        self._block_table, self._lens, self._cu_new, self._max_new, self._device = block_table, lens, cu_new, max_new, dev
        self._n_seq, self._max_blocks = n, w
        self._c = KVBatchParams(block_table.data_ptr(), lens.data_ptr(), cu_new.data_ptr() if cu_new is not None else None,
                                n, w, max_new)
        self._ref = C.byref(self._c)


@_frozen("n_blocks", "n_kv_head", "head_dim", "bits", "tiles", "bounds", "device")
class KVCache:
    """The cache of one attention layer: ``n_blocks`` blocks of 64 tokens for ``n_kv_head`` heads of
    ``head_dim`` (64 or 128) in ``bits`` (4 or 8).  ``bounds``: keep the elementwise key bounds of each
    block that ``select`` needs.  ``tiles`` and ``bounds`` may be given as tensors made earlier; like the
    sizes they cannot be assigned to later, their contents can."""

    def __init__(self, n_blocks: int, n_kv_head: int, head_dim: int, *, bits: int = 8, device="cuda:0",
                 tiles: torch.Tensor | None = None, bounds: torch.Tensor | bool = True):
        tb = tile_bytes(bits, head_dim)
        dev = tiles.device if tiles is not None else torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        if tiles is None:
            tiles = torch.zeros((n_blocks, n_kv_head, tb), dtype=torch.uint8, device=dev)
        _check(tiles, "tiles", torch.uint8, dev, (n_blocks, n_kv_head, tb))
        if bounds is True:
            bounds = torch.zeros((n_blocks, n_kv_head, 2, head_dim), dtype=torch.bfloat16, device=dev)
        elif bounds is False:
            bounds = None
        if bounds is not None:
            _check(bounds, "bounds", torch.bfloat16, dev, (n_blocks, n_kv_head, 2, head_dim))
        self._n_blocks, self._n_kv_head, self._head_dim, self._bits = n_blocks, n_kv_head, head_dim, bits
        self._tiles, self._bounds, self._device = tiles, bounds, dev
        self._scratch = {}
        # what outputs are made like: a new tensor of the same type takes less time than one by type and device
        self._bf16, self._f32, self._i32 = (torch.empty(0, dtype=t, device=dev)
                                            for t in (torch.bfloat16, torch.float32, torch.int32))
        self._c = KVCacheParams(tiles.data_ptr(), bounds.data_ptr() if bounds is not None else None, n_blocks,
                                n_kv_head, head_dim, bits)
        self._ref = C.byref(self._c)

    def append(self, batch: KVBatch, qkv: torch.Tensor, n_head: int, *, rope: bool = True, qk_norm: bool = True,
               rope_base: float = 10000.0, eps: float = 1e-5, q: torch.Tensor | None = None) -> torch.Tensor:
        """Writes the new tokens' keys and values (``qkv``: bf16 [M, (n_head + 2 n_kv_head) head_dim], raw)
        and returns their queries after RoPE and QK-norm, bf16 [M, n_head head_dim]."""
        M = qkv.shape[0]
        _check(qkv, "qkv", torch.bfloat16, self._device, (M, (n_head + 2 * self._n_kv_head) * self._head_dim))
        assert batch._device == self._device, "batch: on another device than the cache"
        q = _out(q, "q", (M, n_head * self._head_dim), self._bf16)
        _launch("gpt_op_kv_append", self._device, self._ref, batch._ref, qkv.data_ptr(), M, n_head, int(rope),
                int(qk_norm), rope_base, eps, q.data_ptr())
        return q

    def read(self, batch: KVBatch, M: int, *, k: torch.Tensor | None = None, v: torch.Tensor | None = None):
        """(k, v): bf16 [M, n_kv_head, head_dim], the values cached at the batch's new positions."""
        shape = (M, self._n_kv_head, self._head_dim)
        assert batch._device == self._device, "batch: on another device than the cache"
        k = _out(k, "k", shape, self._bf16)
        v = _out(v, "v", shape, self._bf16)
        _launch("gpt_op_kv_read", self._device, self._ref, batch._ref, M, k.data_ptr(), v.data_ptr())
        return k, v

    def _rows(self, batch: KVBatch, q: torch.Tensor):
        """Rows and heads of the queries, which are checked."""
        shape = q.shape
        assert len(shape) == 2 and shape[1] % self._head_dim == 0, "q: [M, n_head head_dim]"
        _check(q, "q", torch.bfloat16, self._device)
        assert batch._device == self._device, "batch: on another device than the cache"
        return shape[0], shape[1] // self._head_dim

    def select(self, batch: KVBatch, q: torch.Tensor, n_select: int, *, n_first: int = 1, n_last: int = 1,
               blocks: torch.Tensor | None = None, scores: torch.Tensor | None = None):
        """(blocks int32 [M, n_kv_head, n_select], scores fp32 [M, n_kv_head, max_blocks]): the blocks each
        new token attends to, by the bound of their keys' scores; the first ``n_first`` and last ``n_last``
        visible ones always."""
        M, H = self._rows(batch, q)
        assert max(abs(n_select), abs(n_first), abs(n_last)) <= _INT_MAX, "n_select, n_first, n_last: 32 bits"
        blocks = _out(blocks, "blocks", (M, self._n_kv_head, n_select), self._i32)
        scores = _out(scores, "scores", (M, self._n_kv_head, batch._max_blocks), self._f32)
        _launch("gpt_op_kv_select", self._device, self._ref, batch._ref, q.data_ptr(), M, H, n_select, n_first, n_last,
                blocks.data_ptr(), scores.data_ptr())
        return blocks, scores

    def scratch_bytes(self, batch: KVBatch, M: int, n_head: int, n_sel: int = 0) -> int:
        """Bytes of scratch that attend needs; it goes by the sizes alone, so it is asked for once a size."""
        key = (batch._n_seq, batch._max_new, batch._cu_new is None, M, n_head, n_sel > 0)
        n = self._scratch.get(key)
        if n is None:
            out = C.c_size_t()
            call("gpt_op_attention_kv_scratch_size", self._ref, batch._ref, M, n_head, n_sel, C.byref(out))
            n = self._scratch[key] = out.value
        return n

    def attend(self, batch: KVBatch, q: torch.Tensor, *, window: int = -1, blocks: torch.Tensor | None = None,
               o: torch.Tensor | None = None, lse: torch.Tensor | None = None, scratch: torch.Tensor | None = None):
        """(o bf16 [M, n_head head_dim], lse fp32 [M, n_head]): attention of the new tokens over the cache,
        over all earlier keys, over the last ``window`` and itself, or over the listed ``blocks`` (of each
        list the first min(length, visible blocks) entries are read: put the visible ones first).
        Made for a few new tokens a sequence: long chunks among single tokens are faster as a call of their own,
        prompts without earlier keys as ops.attention_fwd.
        ``scratch`` (uint8, scratch_bytes) may be passed in; calls that overlap need their own."""
        M, H = self._rows(batch, q)
        window = max(-2, min(int(window), _INT_MAX))  # beyond every length, or refused, all the same
        n_sel = 0
        if blocks is not None:
            n_sel = blocks.shape[-1]
            _check(blocks, "blocks", torch.int32, self._device, (M, self._n_kv_head, n_sel))
            assert n_sel > 0, "blocks: at least one entry a list"
        o = torch.empty_like(q) if o is None else _out(o, "o", q.shape, self._bf16)
        lse = _out(lse, "lse", (M, H), self._f32)
        if scratch is None:
            scratch = self._tiles.new_empty(self.scratch_bytes(batch, M, H, n_sel))
        else:
            _check(scratch, "scratch", torch.uint8, self._device)
        _launch("gpt_op_attention_kv", self._device, self._ref, batch._ref, q.data_ptr(), M, H, window,
                blocks.data_ptr() if blocks is not None else None, n_sel, o.data_ptr(), lse.data_ptr(),
                scratch.data_ptr(), scratch.numel())
        return o, lse
