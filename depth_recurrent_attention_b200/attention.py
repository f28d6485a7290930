"""Attention operators without a handle: causal attention over packed prompts, and a 4-bit cache of
keys and values (quantised as it is written, read back, attended by single tokens).

Every operator runs in libdreamer's CUDA kernels (include/dreamer.h); csrc/attention_py.cpp checks
arguments and passes pointers (in Python a small call's checks took longer than its kernel).
Tensors are CUDA tensors of one device, float32 or bfloat16; rows may be strided (a slice of a
fused projection), a row's heads lie densely.  Calls are asynchronous on `stream` (default: the
current stream of the tensors' device) and forward only: outputs carry no gradient.
"""
from __future__ import annotations

import ctypes as C

import torch

from .dreamer import KV4CacheC, _check, lib  # noqa: F401

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
BLOCK = 64  # tokens of a cache block
_fns = None


def _lib():
    """The C entry points with their types (KV4CacheC is dreamer_kv4_cache)."""
    global _fns
    if _fns is None:
        L = lib()
        vp, i, i64, f = C.c_void_p, C.c_int, C.c_int64, C.c_float
        L.dreamer_kv4_bytes.argtypes = [i, i, i, i]
        L.dreamer_kv4_bytes.restype = i64
        rows = [vp, vp, i64, vp, i64, vp, vp, i, i, vp, vp]
        L.dreamer_kv4_store.argtypes = rows
        L.dreamer_kv4_load.argtypes = rows[:9] + [i, vp, vp]
        L.dreamer_attn_kv4.argtypes = [vp, vp, i64, vp, i64, vp, i, i, f, vp, i64, vp, vp]
        L.dreamer_attn_kv4_workspace.argtypes = [vp, i]
        L.dreamer_attn_kv4_workspace.restype = i64
        L.dreamer_attn_packed.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i, i, i, i, i, i, f, vp, vp]
        for n in ("dreamer_kv4_store", "dreamer_kv4_load", "dreamer_attn_kv4", "dreamer_attn_packed"):
            getattr(L, n).restype = i
        _fns = L
    return _fns


def _fast():
    """The entry points that check arguments and call the library (csrc/attention_py.cpp)."""
    try:
        from . import _attention
    except ImportError as e:
        raise RuntimeError(f"_attention not built: run __graft_entry__.build() ({e})") from e
    return _attention


_ext = _fast()


def _done(rc, what):
    """An entry point's outputs, or its error code raised."""
    if type(rc) is int:
        _check(rc, what)
    return rc


def attn_packed(q, k, v, cu_seqlens, out=None, scale=None, status=None, stream=None):
    """Causal attention over packed prompts of different lengths, with grouped heads.

    q [tokens][n_heads][dim], k and v [tokens][n_kv_heads][dim]; cu_seqlens int32 [prompts + 1],
    not decreasing: prompt i holds rows cu_seqlens[i] .. cu_seqlens[i+1]-1.  Query head j uses key
    head j // (n_heads // n_kv_heads); scale (positive) defaults to 1 / sqrt(dim).  Returns
    `out`, [tokens][n_heads][dim], which must not overlap q, k or v (it may be other columns of their
    buffer).  Rows of no prompt are not written: they keep what `out` held, and without a given `out`
    what its new memory held.  bfloat16 takes dim 64 and 128, float32 also 16 and 32.  Boundaries out of
    order or outside the rows set `status`; rows that then lie in several prompts are undefined."""
    return _done(_ext.attn_packed(q, k, v, cu_seqlens, out, scale, status, stream), "dreamer_attn_packed")


class KV4Cache:
    """A 4-bit cache of keys and values for `batch` sequences, at `depth` depths.

    data: uint8 [depth][batch][n_kv_heads][capacity / 64][block bytes] (KV4Cache.alloc makes
    one); the layout of a block and the number format are those of dreamer_kv4_cache.  Outputs, and
    rows to be stored, must not lie in the cache's own memory."""

    def __init__(self, data, head_dim: int):
        self.depth, self.batch, self.n_kv_heads, self.capacity = _ext.kv4_sizes(data, head_dim)
        self.data, self.head_dim, self.device = data, head_dim, data.device

    @staticmethod
    def block_bytes(head_dim: int) -> int:
        """Bytes of 64 tokens of one head (0 for a head_dim that has no cache)."""
        return _lib().dreamer_kv4_bytes(1, 1, head_dim, BLOCK)

    @classmethod
    def alloc(cls, batch: int, n_kv_heads: int, head_dim: int, capacity: int, depth: int = 1,
              device="cuda"):
        """An empty cache; the capacity is rounded up to whole blocks of 64 tokens."""
        if min(batch, n_kv_heads, capacity, depth) < 1 or head_dim not in (64, 128):
            raise ValueError("positive sizes and a head_dim of 64 or 128")
        return cls(torch.zeros((depth, batch, n_kv_heads, -(-capacity // BLOCK),
                                cls.block_bytes(head_dim)), dtype=torch.uint8, device=device), head_dim)

    def store(self, k, v, cu_rows, start, depth: int = 0, status=None, stream=None):
        """Quantise rows: rows cu_rows[b] .. cu_rows[b+1]-1 of k and v ([rows][heads][dim])
        become positions start[b], start[b] + 1, ... of sequence b.  cu_rows int32 [batch + 1],
        not decreasing; start int32 [batch].  Rows of no sequence, and positions outside the
        cache (reported in `status`), are not stored."""
        _done(_ext.kv4_store(self.data, self.head_dim, depth, k, v, cu_rows, start, status, stream), "dreamer_kv4_store")

    def load(self, cu_rows, start, n_rows: int, dtype=torch.bfloat16, depth: int = 0, out=None,
             status=None, stream=None):
        """The rows that store() with the same cu_rows and start wrote, as (k, v) of `dtype`:
        [n_rows][heads][dim].  Rows of no sequence are left as they were in `out` (a pair of
        tensors), zeros where none is given."""
        if dtype not in _DTYPES:
            raise ValueError("dtype: torch.float32 or torch.bfloat16")
        k, v = (None, None) if out is None else out
        return _done(_ext.kv4_load(self.data, self.head_dim, depth, cu_rows, start, n_rows, _DTYPES[dtype], k, v,
                                   status, stream), "dreamer_kv4_load")

    def attend(self, q, lens, depth: int = 0, out=None, scale=None, status=None, stream=None):
        """Attention of one query token a sequence: q [batch][n_heads][dim] over the first
        lens[b] positions of sequence b (int32 [batch]; zeros where 0), query head j over key
        head j // (n_heads // n_kv_heads).  Returns [batch][n_heads][dim] (`out` may be q); scale
        defaults to 1 / sqrt(dim)."""
        return _done(_ext.kv4_attend(self.data, self.head_dim, depth, q, lens, out, scale, status, stream),
                     "dreamer_attn_kv4")
