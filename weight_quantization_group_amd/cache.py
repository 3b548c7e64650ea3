"""Python binding of ``libhqq_cache.so`` (C ABI in include/hqq_cache.h): a key-value
cache held in the library's quantized format, and the attention of one new token a
sequence straight from its codes.

Argument checks and marshalling only, as in the package's other calls.  Keys, values
and queries are fp16 or bfloat16; each call runs on the current stream of the cache's
device.  workspace: an optional contiguous CUDA tensor of at least
hqq_cache_attention_workspace bytes; without one the call takes its own from torch's
allocator.  Calls that may run at the same time (two streams, two captured graphs) need a
workspace each.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from . import _U32, DTYPE_BF16, DTYPE_FP16, HQQError

CACHE_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhqq_cache.so")

# exported symbols, in include/hqq_cache.h order
CACHE_EXPORTS = ("hqq_cache_write", "hqq_cache_read", "hqq_cache_attention_workspace", "hqq_cache_attention",
                 "hqq_cache_strerror")


class HqqCacheSide(ctypes.Structure):
    """struct hqq_cache_side of include/hqq_cache.h"""
    _fields_ = [("packed", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p)]


class HqqCache(ctypes.Structure):
    """struct hqq_cache of include/hqq_cache.h"""
    _fields_ = [("k", HqqCacheSide), ("v", HqqCacheSide), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("nbits", ctypes.c_int32),
                ("group_size", ctypes.c_int32)]


class CacheError(HQQError):
    def __init__(self, fn: str, status: int):
        RuntimeError.__init__(self, f"{fn} failed: {hqq_cache_strerror(status)} (status {status})")
        self.status = status


_lib = None


def load_cache_library(path: str = CACHE_LIB_PATH):
    """Load libhqq_cache.so (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run `python -m weight_quantization_group_amd.build`")
    L = ctypes.CDLL(path)
    P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    for name, args, res in (
            ("hqq_cache_write", [P, P, i64, i64, P, i64, i64, i64, P, i32, P, P, P], i32),
            ("hqq_cache_read", [P, P, i64, i32, P, P, P], i32),
            ("hqq_cache_attention_workspace", [P, i64, i64, i64], i64),
            ("hqq_cache_attention", [P, P, i64, i64, i64, i64, P, i64, P, f32, i64, i32, P, P, P, i64, P], i32),
            ("hqq_cache_strerror", [i32], ctypes.c_char_p)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
    _lib = L
    return L


def hqq_cache_strerror(status: int) -> str:
    return load_cache_library().hqq_cache_strerror(int(status)).decode()


_DT = {torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16}
_F32, _I64, _I32 = (torch.float32,), (torch.int64,), (torch.int32,)


def _tensor(t, name: str, dtypes, shape, index: int) -> int:
    """The address of a contiguous CUDA tensor of this shape on device `index`, checked."""
    try:
        if t.get_device() == index and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, the cache is on cuda:{index}")


class QuantizedCache:
    """A paged key-value cache in the library's axis = 1 format.

    k, v: (packed, scale, zero) of the keys and of the values: int32
    [pages, heads, page_size, dim * nbits / 32] and float32 [pages, heads, page_size,
    dim / group_size], contiguous CUDA tensors on one device; kept alive by the object.
    nbits 2, 4 or 8; dim 64, 96, 128, 192 or 256; group_size 32 to 256, at most 4 groups a
    row; page_size a power of two from 16 to 1024.  QuantizedCache.empty allocates one.
    Slot s is place s % page_size of page s // page_size."""

    def __init__(self, k, v, nbits: int, group_size: int):
        self._lib = load_cache_library()
        self._k, self._v = tuple(k), tuple(v)
        packed = self._k[0]
        if not isinstance(packed, torch.Tensor) or not packed.is_cuda:
            raise TypeError("k must hold CUDA tensors")
        if packed.dim() != 4:
            raise ValueError(f"packed must be [pages, heads, page_size, words], got {list(packed.shape)}")
        if nbits not in (2, 4, 8):
            raise ValueError(f"nbits must be 2, 4 or 8, got {nbits}")
        self.nbits, self.group_size, self.device = int(nbits), int(group_size), packed.device
        self._index = packed.get_device()
        self.pages, self.heads, self.page_size, words = packed.shape
        self.dim = words * 32 // self.nbits
        meta = (self.pages, self.heads, self.page_size, self.dim // self.group_size if self.group_size > 0 else 0)
        sides = []
        for name, side in (("k", self._k), ("v", self._v)):
            if len(side) != 3:
                raise ValueError(f"{name} must be (packed, scale, zero)")
            sides.append(HqqCacheSide(_tensor(side[0], name + " packed", _U32, packed.shape, self._index),
                                      _tensor(side[1], name + " scale", _F32, meta, self._index),
                                      _tensor(side[2], name + " zero", _F32, meta, self._index)))
        # the library's layout checks, which need no device
        if min(packed.shape) < 1 or max(packed.shape) >= 1 << 31:
            raise ValueError(f"packed must not be empty, got {list(packed.shape)}")
        self._c = HqqCache(*sides, self.pages, self.page_size, self.heads, self.dim, self.nbits, self.group_size)
        self._ptr = ctypes.addressof(self._c)
        self._softmax_scale = 1.0 / math.sqrt(self.dim)
        self._room = None, 0          # the sizes last asked for, and their workspace's bytes
        _bytes(self, (1, self.heads, 1))

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, dim: int, nbits: int, group_size: int, device="cuda"):
        """A cache whose slots all hold zeros."""
        if nbits not in (2, 4, 8) or group_size <= 0 or dim % group_size:
            raise ValueError(f"nbits must be 2, 4 or 8 and group_size divide dim, got {nbits}, {group_size}, {dim}")
        at = (pages, heads, page_size)

        def side():
            return (torch.zeros(*at, dim * nbits // 32, dtype=torch.int32, device=device),
                    torch.ones(*at, dim // group_size, device=device), torch.zeros(*at, dim // group_size, device=device))

        return cls(side(), side(), nbits, group_size)

    @property
    def k(self):
        """(packed, scale, zero) of the keys."""
        return self._k

    @property
    def v(self):
        """(packed, scale, zero) of the values."""
        return self._v


def _bytes(cache: QuantizedCache, sizes) -> int:
    room = cache._room               # (one read: another thread's call may replace it)
    if room[0] == sizes:
        return room[1]
    n = cache._lib.hqq_cache_attention_workspace(cache._ptr, *sizes)
    if n < 0:
        raise CacheError("hqq_cache_attention_workspace", n)
    cache._room = sizes, n
    return n


def hqq_cache_attention_workspace(cache: QuantizedCache, batch: int, q_heads: int, table_width: int) -> int:
    """Bytes of workspace of hqq_cache_attention for these sizes."""
    return _bytes(cache, (batch, q_heads, table_width))


def _rows(t, name: str, cache: QuantizedCache):
    """(address, stride of the rows, stride of the heads, shape) of [rows, heads, dim] values of 16
    bits with any strides of rows and heads, checked."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DT:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != cache.dim:
        raise ValueError(f"{name} must be [rows, heads, {cache.dim}], got {list(shape)}")
    if t.get_device() != cache._index:
        raise ValueError(f"{name} is on {t.device}, the cache is on {cache.device}")
    a, b, c = t.stride()
    if c != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), a if shape[0] > 1 else 0, b if shape[1] > 1 else 0, shape


def _pair(t):
    # (empty_like costs the host half of what empty does)
    return t, torch.empty_like(t)


def _call(cache: QuantizedCache, f, *args) -> None:
    """Run the library's call f on the cache's device and its current stream."""
    index = cache._index
    # (torch's functions are looked up here: a torch without a GPU runtime imports the package)
    if torch._C._cuda_getDevice() == index:
        st = f(cache._ptr, *args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = f(cache._ptr, *args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise CacheError(f.__name__, st)


def hqq_cache_write(cache: QuantizedCache, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor,
                    values: bool = False):
    """Quantize K and V [tokens, heads, dim] into the cache at slots (int64 [tokens]), each
    group with the codes, scale and zero of hqq_quantize at iters = 0.  A slot outside the
    cache (-1, say) skips its token; the others must differ.  K and V may be parts of a
    wider tensor (strides multiples of 8, addresses of 16 bytes).  values: also return
    what the cache now stands for, (K_hat, V_hat), with zeros for skipped tokens."""
    pk, k_token, k_head, shape = _rows(K, "K", cache)
    pv, v_token, v_head, v_shape = _rows(V, "V", cache)
    tokens, dtype = shape[0], K.dtype
    if V.dtype != dtype:
        raise TypeError(f"K and V must have one dtype, got {dtype} and {V.dtype}")
    if shape[1] != cache.heads or v_shape != shape:
        raise ValueError(f"K and V must be [{tokens}, {cache.heads}, {cache.dim}], got {list(shape)} and {list(v_shape)}")
    at = _tensor(slots, "slots", _I64, (tokens,), cache._index)
    hat = to_k = to_v = None
    if values:
        hat = _pair(torch.empty_like(K, memory_format=torch.contiguous_format))
        to_k, to_v = hat[0].data_ptr(), hat[1].data_ptr()
    _call(cache, cache._lib.hqq_cache_write, pk, k_token, k_head, pv, v_token, v_head, tokens, at, _DT[dtype], to_k, to_v)
    return hat


def hqq_cache_read(cache: QuantizedCache, slots: torch.Tensor, dtype=torch.float16, out=None):
    """The keys and values at slots (int64 [tokens]) as (K, V), [tokens, heads, dim] of dtype
    (out's, where out = (K, V) is given); zeros at a slot outside the cache."""
    tokens = slots.numel() if isinstance(slots, torch.Tensor) else 0
    at = _tensor(slots, "slots", _I64, (tokens,), cache._index)
    shape = (tokens, cache.heads, cache.dim)
    if out is None:
        if dtype not in _DT:
            raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
        out = _pair(torch.empty(shape, dtype=dtype, device=cache.device))
        pk, pv = out[0].data_ptr(), out[1].data_ptr()
    else:
        K, V = out
        dtype = K.dtype if isinstance(K, torch.Tensor) else None
        if dtype not in _DT:
            raise TypeError("out must be float16 or bfloat16 tensors")
        pk, pv = _tensor(K, "out K", (dtype,), shape, cache._index), _tensor(V, "out V", (dtype,), shape, cache._index)
    _call(cache, cache._lib.hqq_cache_read, at, tokens, _DT[dtype], pk, pv)
    return tuple(out)


def hqq_cache_attention(cache: QuantizedCache, Q: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                        softmax_scale: float | None = None, window: int = 0, out=None, lse=None, workspace=None):
    """Attention of one new token a sequence over the cache: Q [batch, q_heads, dim] (it may be
    a part of a wider tensor), table (int32 [batch, pages of a sequence]) and lengths (int32
    [batch], the new token included) -> (out [batch, q_heads, dim], lse float32 [batch, q_heads]).
    q_heads is a multiple of the cache's heads; q heads that share a key-value head are
    neighbours.  softmax_scale: 1 / sqrt(dim) where not given.  window: only the last
    `window` tokens count (0: all).  A sequence of no tokens gives 0 and -inf; the tokens of a
    page outside the cache (-1, say) do not count."""
    pq, q_row, q_head, shape = _rows(Q, "Q", cache)
    batch, q_heads, _ = shape
    index, dtype, dev = cache._index, Q.dtype, cache.device
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [batch, pages of a sequence]")
    width = table.shape[1]
    pt = _tensor(table, "table", _I32, (batch, width), index)
    pl = _tensor(lengths, "lengths", _I32, (batch,), index)
    need = _bytes(cache, (batch, q_heads, width))
    if out is None:
        out = torch.empty_like(Q, memory_format=torch.contiguous_format)
        po = out.data_ptr()
    else:
        po = _tensor(out, "out", (dtype,), shape, index)
    if lse is None:
        lse = torch.empty((batch, q_heads), dtype=torch.float32, device=dev)
        pe = lse.data_ptr()
    else:
        pe = _tensor(lse, "lse", _F32, (batch, q_heads), index)
    given = workspace is not None
    if given:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous CUDA tensor")
        if workspace.get_device() != index:
            raise ValueError(f"workspace is on {workspace.device}, the cache is on {dev}")
        need = workspace.numel() * workspace.element_size()
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _call(cache, cache._lib.hqq_cache_attention, pq, q_row, q_head, batch, q_heads, pt, width, pl,
          cache._softmax_scale if softmax_scale is None else softmax_scale, window, _DT[dtype], po, pe,
          workspace.data_ptr() if need else None, need)
    if given and need and not torch.cuda.is_current_stream_capturing():
        # a workspace that belongs to another stream is not handed out again before this call's end
        workspace.record_stream(torch.cuda.current_stream(dev))
    return out, lse
