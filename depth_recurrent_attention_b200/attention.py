"""Attention operators without a handle: causal attention over packed prompts, and a 4-bit cache of keys and values (quantised as it is
written, read back, attended by single tokens).

Every operator runs in libdreamer's CUDA kernels (include/dreamer.h); this module checks
arguments and passes pointers.  Tensors are CUDA tensors of one device, float32 or bfloat16;
rows may be strided (a slice of a fused projection), a row's heads lie densely.  Calls are
asynchronous on `stream` (default: the current stream of the tensors' device).
"""
from __future__ import annotations

import ctypes as C
import functools
import math

import torch

from .dreamer import KV4CacheC, _check, lib

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
BLOCK = 64  # tokens of a cache block
GROUP = 64  # channels that share a scale and an offset


_fns = None


def _lib():
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


try:  # the current stream's handle without a Stream object
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _rows(name, t, device, heads=None, dim=None, dtype=None, n=None):
    """A CUDA tensor [rows][heads][dim] whose rows are 16-byte aligned and whose heads lie
    densely; returns its row stride."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dim() != 3 or t.dtype not in _DTYPES:
        raise ValueError(f"{name}: a float32 or bfloat16 tensor [rows][heads][dim] on {device}")
    r, h, d = t.shape
    if (heads is not None and h != heads) or (dim is not None and d != dim) or \
            (n is not None and r != n) or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name}: {tuple(t.shape)} of {t.dtype} does not fit the other arguments")
    ld, sh, sd = t.stride()
    if r <= 1:
        ld = -(-h * d // 8) * 8
    if (sd != 1 and d > 1) or (sh != d and h > 1) or ld < h * d:
        raise ValueError(f"{name}: a row's heads have to lie densely (strides {t.stride()})")
    if r and (t.data_ptr() % 16 or ld * t.element_size() % 16):
        raise ValueError(f"{name}: rows have to be 16-byte aligned")
    return ld


def _ints(name, t, device, n):
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.int32 or \
            t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor of {n} on {device}")
    return t.data_ptr()


def _status(t, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.int32 or t.numel() < 1:
        raise ValueError(f"status: an int32 tensor on {device}")
    return t.data_ptr()


def _scale(scale, dim):
    scale = dim ** -0.5 if scale is None else float(scale)
    if not math.isfinite(scale):
        raise ValueError("scale: a finite number")
    return scale


def _empty(shape, dtype, device, stream):
    """New memory that belongs to the stream it is used on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(fn, what, device, stream, *args):
    if stream is None:
        handle = _raw_stream(device.index)
    elif stream.device != device:
        raise ValueError(f"stream: of {stream.device}, the tensors are on {device}")
    else:
        handle = stream.cuda_stream
    if device.index == torch.cuda.current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    _check(rc, what)


@functools.lru_cache(maxsize=256)
def _workspace(batch, kv_heads, dim, capacity, heads, index):
    with torch.cuda.device(index):
        return _lib().dreamer_attn_kv4_workspace(
            C.byref(KV4CacheC(None, batch, kv_heads, dim, capacity)), heads)


def attn_packed(q, k, v, cu_seqlens, out=None, scale=None, status=None, stream=None):
    """Causal attention over packed prompts of different lengths, with grouped heads.

    q [tokens][n_heads][dim], k and v [tokens][n_kv_heads][dim]; cu_seqlens int32 [prompts + 1],
    not decreasing: prompt i holds rows cu_seqlens[i] .. cu_seqlens[i+1]-1.  Query head j uses key
    head j // (n_heads // n_kv_heads); scale (positive) defaults to 1 / sqrt(dim).  Returns
    `out`, [tokens][n_heads][dim]; rows of no prompt are not written.  bfloat16 takes dim 64 and
    128, float32 also 16 and 32.  Boundaries out of order or outside the rows set `status`."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q: a CUDA tensor")
    dev = q.device
    ldq = _rows("q", q, dev)
    n, hq, d = q.shape
    ldk = _rows("k", k, dev, None, d, q.dtype, n)
    hk = k.shape[1]
    ldv = _rows("v", v, dev, hk, d, q.dtype, n)
    if hk < 1 or hq < 1 or hq % hk:
        raise ValueError(f"{hq} query heads over {hk} key heads")
    prompts = cu_seqlens.numel() - 1 if isinstance(cu_seqlens, torch.Tensor) else -1
    if prompts < 0:
        raise ValueError("cu_seqlens: int32 [prompts + 1]")
    cu = _ints("cu_seqlens", cu_seqlens, dev, prompts + 1)
    if out is None:
        out = _empty((n, hq, d), q.dtype, dev, stream)
    ldo = _rows("out", out, dev, hq, d, q.dtype, n)
    scale = _scale(scale, d)
    if not scale > 0:
        raise ValueError("scale: positive")
    if n:
        _call(_lib().dreamer_attn_packed, "dreamer_attn_packed", dev, stream, q.data_ptr(), ldq,
              k.data_ptr(), ldk, v.data_ptr(), ldv, out.data_ptr(), ldo, cu, prompts,
              n, hq, hk, d, _DTYPES[q.dtype], scale, _status(status, dev))
    return out


class KV4Cache:
    """A 4-bit cache of keys and values for `batch` sequences, at `depth` depths.

    data: uint8 [depth][batch][n_kv_heads][capacity / 64][block bytes] (KV4Cache.alloc makes
    one); the layout of a block and the number format are those of dreamer_kv4_cache."""

    def __init__(self, data, head_dim: int):
        if not isinstance(data, torch.Tensor) or not data.is_cuda or data.dtype != torch.uint8 or \
                data.dim() != 5 or not data.is_contiguous():
            raise ValueError("data: a contiguous CUDA uint8 tensor [depth][batch][heads][blocks][bytes]")
        if head_dim not in (64, 128):
            raise ValueError("head_dim: 64 or 128")
        if data.shape[4] != self.block_bytes(head_dim) or 0 in data.shape or data.data_ptr() % 16:
            raise ValueError(f"data: blocks of {self.block_bytes(head_dim)} bytes, 16-byte aligned")
        self.data, self.head_dim = data, head_dim
        self.depth, self.batch, self.n_kv_heads, blocks, _ = data.shape
        self.capacity = blocks * BLOCK
        self.device = data.device
        self._step = data.stride(0)
        self._base = data.data_ptr()

    @staticmethod
    def block_bytes(head_dim: int) -> int:
        return head_dim // GROUP * BLOCK * 2 * (32 + 4)

    @classmethod
    def alloc(cls, batch: int, n_kv_heads: int, head_dim: int, capacity: int, depth: int = 1,
              device="cuda"):
        """An empty cache; the capacity is rounded up to whole blocks of 64 tokens."""
        if min(batch, n_kv_heads, capacity, depth) < 1 or head_dim not in (64, 128):
            raise ValueError("positive sizes and a head_dim of 64 or 128")
        return cls(torch.zeros((depth, batch, n_kv_heads, -(-capacity // BLOCK),
                                cls.block_bytes(head_dim)), dtype=torch.uint8, device=device), head_dim)

    def _at(self, depth):
        if not 0 <= depth < self.depth:
            raise ValueError(f"depth: 0..{self.depth - 1}")
        return KV4CacheC(self._base + depth * self._step, self.batch, self.n_kv_heads,
                         self.head_dim, self.capacity)

    def store(self, k, v, cu_rows, start, depth: int = 0, status=None, stream=None):
        """Quantise rows: rows cu_rows[b] .. cu_rows[b+1]-1 of k and v ([rows][heads][dim])
        become positions start[b], start[b] + 1, ... of sequence b.  cu_rows int32 [batch + 1],
        not decreasing; start int32 [batch].  Rows of no sequence, and positions outside the
        cache (reported in `status`), are not stored."""
        dev = self.device
        ldk = _rows("k", k, dev, self.n_kv_heads, self.head_dim)
        ldv = _rows("v", v, dev, self.n_kv_heads, self.head_dim, k.dtype, k.shape[0])
        _call(_lib().dreamer_kv4_store, "dreamer_kv4_store", dev, stream, C.byref(self._at(depth)),
              k.data_ptr(), ldk, v.data_ptr(), ldv, _ints("cu_rows", cu_rows, dev, self.batch + 1),
              _ints("start", start, dev, self.batch), k.shape[0], _DTYPES[k.dtype],
              _status(status, dev)) if k.shape[0] else None

    def load(self, cu_rows, start, n_rows: int, dtype=torch.bfloat16, depth: int = 0, out=None,
             status=None, stream=None):
        """The rows that store() with the same cu_rows and start wrote, as (k, v) of `dtype`:
        [n_rows][heads][dim].  Rows of no sequence are left as they were in `out` (a pair of
        tensors), zeros where none is given."""
        dev = self.device
        if dtype not in _DTYPES:
            raise ValueError("dtype: torch.float32 or torch.bfloat16")
        if n_rows < 0:
            raise ValueError("n_rows: not negative")
        fresh = out is None
        if fresh:
            shape = (n_rows, self.n_kv_heads, self.head_dim)
            out = _empty(shape, dtype, dev, stream), _empty(shape, dtype, dev, stream)
        k, v = out
        ldk = _rows("out[0]", k, dev, self.n_kv_heads, self.head_dim, dtype, n_rows)
        ldv = _rows("out[1]", v, dev, self.n_kv_heads, self.head_dim, dtype, n_rows)
        if n_rows:
            _call(_lib().dreamer_kv4_load, "dreamer_kv4_load", dev, stream, C.byref(self._at(depth)),
                  k.data_ptr(), ldk, v.data_ptr(), ldv, _ints("cu_rows", cu_rows, dev, self.batch + 1),
                  _ints("start", start, dev, self.batch), n_rows, _DTYPES[dtype], int(fresh),
                  _status(status, dev))
        return k, v

    def attend(self, q, lens, depth: int = 0, out=None, scale=None, status=None, stream=None):
        """Attention of one query token a sequence: q [batch][n_heads][dim] over the first
        lens[b] positions of sequence b (int32 [batch]; zeros where 0), query head j over key
        head j // (n_heads // n_kv_heads).  Returns [batch][n_heads][dim]; scale defaults to
        1 / sqrt(dim)."""
        dev = self.device
        ldq = _rows("q", q, dev, None, self.head_dim, None, self.batch)
        hq = q.shape[1]
        if hq < 1 or hq % self.n_kv_heads:
            raise ValueError(f"q: a multiple of {self.n_kv_heads} heads")
        if out is None:
            out = _empty(q.shape, q.dtype, dev, stream)
        ldo = _rows("out", out, dev, hq, self.head_dim, q.dtype, self.batch)
        need = _workspace(self.batch, self.n_kv_heads, self.head_dim, self.capacity, hq, dev.index)
        ws = _empty((need,), torch.uint8, dev, stream) if need else None
        _call(_lib().dreamer_attn_kv4, "dreamer_attn_kv4", dev, stream, C.byref(self._at(depth)),
              q.data_ptr(), ldq, out.data_ptr(), ldo, _ints("lens", lens, dev, self.batch), hq,
              _DTYPES[q.dtype], _scale(scale, self.head_dim), ws.data_ptr() if need else None, need,
              _status(status, dev))
        return out
