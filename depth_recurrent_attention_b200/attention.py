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

Tensor = torch.Tensor
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_ALIGN = {torch.float32: 4, torch.bfloat16: 8}  # elements of 16 bytes
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


try:  # the current stream's handle without a Stream object, the current device without its checks
    from torch._C import _cuda_getCurrentRawStream as _raw_stream, _cuda_getDevice as _current_device
except ImportError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

    _current_device = torch.cuda.current_device


def _rows(name, t, index, heads=None, dim=None, dtype=None, n=None):
    """A CUDA tensor [rows][heads][dim] of device `index` whose rows are 16-byte aligned and whose
    heads lie densely; returns its pointer and row stride."""
    if not isinstance(t, Tensor) or t.dim() != 3 or t.get_device() != index or t.dtype not in _DTYPES:
        raise ValueError(f"{name}: a float32 or bfloat16 tensor [rows][heads][dim] on cuda:{index}")
    r, h, d = t.shape
    if (heads is not None and h != heads) or (dim is not None and d != dim) or \
            (n is not None and r != n) or (dtype is not None and t.dtype is not dtype):
        raise ValueError(f"{name}: {tuple(t.shape)} of {t.dtype} does not fit the other arguments")
    if t.is_contiguous():
        ld = h * d
    else:
        ld, sh, sd = t.stride()
        if (sd != 1 and d > 1) or (sh != d and h > 1) or ld < h * d:
            raise ValueError(f"{name}: a row's heads have to lie densely (strides {t.stride()})")
    p = t.data_ptr()
    if p % 16 or ld % _ALIGN[t.dtype]:
        if r > 1 or p % 16:
            raise ValueError(f"{name}: rows have to be 16-byte aligned")
        ld = -(-ld // 8) * 8  # one row has no stride
    return p, ld


def _ints(name, t, index, n):
    if not isinstance(t, Tensor) or t.dtype is not torch.int32 or t.get_device() != index or \
            t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor of {n} on cuda:{index}")
    return t.data_ptr()


def _status(t, index):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != index or t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError(f"status: an int32 tensor on cuda:{index}")
    return t.data_ptr()


def _scale(scale, dim):
    if scale is None:
        return dim ** -0.5
    scale = float(scale)
    if not math.isfinite(scale):
        raise ValueError("scale: a finite number")
    return scale


def _like(t, shape, stream, dtype=None):
    """New memory on t's device that belongs to the stream it is used on."""
    if stream is None:
        if dtype is None and t.shape == shape and t.is_contiguous():
            return torch.empty_like(t)
        return t.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return t.new_empty(shape, dtype=dtype)


def _call(fn, index, stream, *args):
    if stream is None:
        handle = _raw_stream(index)
    elif stream.device.index != index:
        raise ValueError(f"stream: of {stream.device}, the tensors are on cuda:{index}")
    else:
        handle = stream.cuda_stream
    if index == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc:
        _check(rc, fn.__name__)


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
    dev = q.get_device()
    qp, ldq = _rows("q", q, dev)
    dtype, (n, hq, d) = q.dtype, q.shape
    kp, ldk = _rows("k", k, dev, None, d, dtype, n)
    hk = k.shape[1]
    vp, ldv = _rows("v", v, dev, hk, d, dtype, n)
    if hk < 1 or hq < 1 or hq % hk:
        raise ValueError(f"{hq} query heads over {hk} key heads")
    prompts = cu_seqlens.numel() - 1 if isinstance(cu_seqlens, torch.Tensor) else -1
    if prompts < 0:
        raise ValueError("cu_seqlens: int32 [prompts + 1]")
    cu = _ints("cu_seqlens", cu_seqlens, dev, prompts + 1)
    scale = _scale(scale, d)
    if not scale > 0:
        raise ValueError("scale: positive")
    if out is None:
        out = _like(q, (n, hq, d), stream)
        op, ldo = out.data_ptr(), hq * d
    else:
        op, ldo = _rows("out", out, dev, hq, d, dtype, n)
    if n:
        _call(_lib().dreamer_attn_packed, dev, stream, qp, ldq, kp, ldk, vp, ldv, op, ldo, cu, prompts, n,
              hq, hk, d, _DTYPES[dtype], scale, _status(status, dev))
    return out


class KV4Cache:
    """A 4-bit cache of keys and values for `batch` sequences, at `depth` depths.

    data: uint8 [depth][batch][n_kv_heads][capacity / 64][block bytes] (KV4Cache.alloc makes
    one); the layout of a block and the number format are those of dreamer_kv4_cache."""

    def __init__(self, data, head_dim: int):
        if not isinstance(data, torch.Tensor) or data.dtype is not torch.uint8 or data.dim() != 5 or \
                not data.is_cuda or not data.is_contiguous():
            raise ValueError("data: a contiguous CUDA uint8 tensor [depth][batch][heads][blocks][bytes]")
        if head_dim not in (64, 128):
            raise ValueError("head_dim: 64 or 128")
        self.depth, self.batch, self.n_kv_heads, blocks, size = data.shape
        self._base = data.data_ptr()
        if size != self.block_bytes(head_dim) or not data.numel() or self._base % 16:
            raise ValueError(f"data: blocks of {self.block_bytes(head_dim)} bytes, 16-byte aligned")
        self.data, self.head_dim = data, head_dim
        self.capacity = blocks * BLOCK
        self.device = data.device
        self._index = data.get_device()

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
        return C.byref(KV4CacheC(self._base + depth * (self.data.numel() // self.depth) if depth else self._base,
                                 self.batch, self.n_kv_heads, self.head_dim, self.capacity))

    def store(self, k, v, cu_rows, start, depth: int = 0, status=None, stream=None):
        """Quantise rows: rows cu_rows[b] .. cu_rows[b+1]-1 of k and v ([rows][heads][dim])
        become positions start[b], start[b] + 1, ... of sequence b.  cu_rows int32 [batch + 1],
        not decreasing; start int32 [batch].  Rows of no sequence, and positions outside the
        cache (reported in `status`), are not stored."""
        dev = self._index
        kp, ldk = _rows("k", k, dev, self.n_kv_heads, self.head_dim)
        n = k.shape[0]
        vp, ldv = _rows("v", v, dev, self.n_kv_heads, self.head_dim, k.dtype, n)
        at, cu, st = self._at(depth), _ints("cu_rows", cu_rows, dev, self.batch + 1), _ints("start", start, dev, self.batch)
        if n:
            _call(_lib().dreamer_kv4_store, dev, stream, at, kp, ldk, vp, ldv, cu, st, n, _DTYPES[k.dtype],
                  _status(status, dev))

    def load(self, cu_rows, start, n_rows: int, dtype=torch.bfloat16, depth: int = 0, out=None,
             status=None, stream=None):
        """The rows that store() with the same cu_rows and start wrote, as (k, v) of `dtype`:
        [n_rows][heads][dim].  Rows of no sequence are left as they were in `out` (a pair of
        tensors), zeros where none is given."""
        dev = self._index
        if dtype not in _DTYPES:
            raise ValueError("dtype: torch.float32 or torch.bfloat16")
        if n_rows < 0:
            raise ValueError("n_rows: not negative")
        h, d = self.n_kv_heads, self.head_dim
        if out is None:
            k, v = _like(self.data, (2, n_rows, h, d), stream, dtype).unbind(0)
            kp, vp, ldk, ldv = k.data_ptr(), v.data_ptr(), h * d, h * d
        else:
            k, v = out
            kp, ldk = _rows("out[0]", k, dev, h, d, dtype, n_rows)
            vp, ldv = _rows("out[1]", v, dev, h, d, dtype, n_rows)
        at, cu, st = self._at(depth), _ints("cu_rows", cu_rows, dev, self.batch + 1), _ints("start", start, dev, self.batch)
        if n_rows:
            _call(_lib().dreamer_kv4_load, dev, stream, at, kp, ldk, vp, ldv, cu, st, n_rows, _DTYPES[dtype],
                  int(out is None), _status(status, dev))
        return k, v

    def attend(self, q, lens, depth: int = 0, out=None, scale=None, status=None, stream=None):
        """Attention of one query token a sequence: q [batch][n_heads][dim] over the first
        lens[b] positions of sequence b (int32 [batch]; zeros where 0), query head j over key
        head j // (n_heads // n_kv_heads).  Returns [batch][n_heads][dim]; scale defaults to
        1 / sqrt(dim)."""
        dev = self._index
        qp, ldq = _rows("q", q, dev, None, self.head_dim, None, self.batch)
        hq = q.shape[1]
        if hq < 1 or hq % self.n_kv_heads:
            raise ValueError(f"q: a multiple of {self.n_kv_heads} heads")
        if out is None:
            out = _like(q, q.shape, stream)
            op, ldo = out.data_ptr(), hq * self.head_dim
        else:
            op, ldo = _rows("out", out, dev, hq, self.head_dim, q.dtype, self.batch)
        need = _workspace(self.batch, self.n_kv_heads, self.head_dim, self.capacity, hq, dev)
        ws = _like(self.data, (need,), stream) if need else None
        _call(_lib().dreamer_attn_kv4, dev, stream, self._at(depth), qp, ldq, op, ldo,
              _ints("lens", lens, dev, self.batch), hq, _DTYPES[q.dtype], _scale(scale, self.head_dim),
              ws.data_ptr() if need else None, need, _status(status, dev))
        return out
