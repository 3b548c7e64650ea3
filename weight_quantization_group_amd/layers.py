"""Python binding of ``libhqq_layers.so`` (C ABI in include/hqq_layers.h): the gated
feed-forward block, the softmax cross entropy of a quantized output head, and the
backward passes through frozen quantized weights.

Argument checks and marshalling only, as in the package's other calls.  Weights are
(packed, scale, zero) of an axis = 1 weight [N, K], as hqq_quantize returns them; the
compute dtype is that of X (or dY), fp16 or bfloat16.  workspace: an optional
contiguous CUDA tensor of at least the bytes that the matching *_workspace function
returns; without one each call takes its own from torch's allocator.  Calls that may
run at the same time (two streams, two captured graphs) need a workspace each.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _U32, DTYPE_BF16, DTYPE_FP16, HQQError, _dev_ptr, _stream

LAYERS_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhqq_layers.so")

# exported symbols, in include/hqq_layers.h order
LAYERS_EXPORTS = ("hqq_linear_gated_workspace", "hqq_linear_gated", "hqq_linear_gated_backward_workspace",
                  "hqq_linear_gated_backward", "hqq_linear_batch_backward_workspace",
                  "hqq_linear_batch_backward", "hqq_linear_cross_entropy_workspace",
                  "hqq_linear_cross_entropy", "hqq_linear_cross_entropy_backward_workspace",
                  "hqq_linear_cross_entropy_backward", "hqq_layers_strerror")

# activations of the gated block (HQQ_ACT_*)
ACT_CODES = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
# weights per call of hqq_linear_batch_backward (HQQ_MAX_GRADS)
MAX_GRADS = 16


class HqqWeight(ctypes.Structure):
    """struct hqq_weight of include/hqq_layers.h"""
    _fields_ = [("packed", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p)]


class HqqLinearGrad(ctypes.Structure):
    """struct hqq_linear_grad of include/hqq_layers.h"""
    _fields_ = HqqWeight._fields_ + [("N", ctypes.c_int64), ("dY", ctypes.c_void_p)]


class LayersError(HQQError):
    def __init__(self, fn: str, status: int):
        RuntimeError.__init__(self, f"{fn} failed: {hqq_layers_strerror(status)} (status {status})")
        self.status = status


_lib = None


def load_layers_library(path: str = LAYERS_LIB_PATH):
    """Load libhqq_layers.so (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run `python -m weight_quantization_group_amd.build`")
    L = ctypes.CDLL(path)
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    sizes = [i64, i64, i64, i32, i32]
    for name, args in (
            ("hqq_linear_gated", [P, i64, i64, P, P, i64, i32, i32, i32, i32, P, P, i64, P]),
            ("hqq_linear_gated_backward", [P, P, i64, i64, P, P, i64, i32, i32, i32, i32, P, P, i64, P]),
            ("hqq_linear_batch_backward", [P, i32, i64, i64, i32, i32, i32, P, P, i64, P]),
            ("hqq_linear_cross_entropy", [P, i64, i64, P, i64, i32, i32, i32, P, P, P, P, i64, P]),
            ("hqq_linear_cross_entropy_backward",
             [P, P, i64, i64, P, i64, i32, i32, i32, P, P, P, P, i64, P])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, i32
        w = getattr(L, name + "_workspace")
        w.argtypes, w.restype = ([i64, i64, P, i32, i32, i32] if name == "hqq_linear_batch_backward" else sizes), i64
    L.hqq_layers_strerror.argtypes = [i32]
    L.hqq_layers_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


def hqq_layers_strerror(status: int) -> str:
    return load_layers_library().hqq_layers_strerror(int(status)).decode()


def _bytes(name: str, *args) -> int:
    n = getattr(load_layers_library(), name)(*args)
    if n < 0:
        raise LayersError(name, n)
    return int(n)


def hqq_linear_gated_workspace(M: int, K: int, N: int, nbits: int, group_size: int) -> int:
    """Bytes of workspace of hqq_linear_gated for these sizes."""
    return _bytes("hqq_linear_gated_workspace", M, K, N, nbits, group_size)


def hqq_linear_gated_backward_workspace(M: int, K: int, N: int, nbits: int, group_size: int) -> int:
    """Bytes of workspace of hqq_linear_gated_backward for these sizes."""
    return _bytes("hqq_linear_gated_backward_workspace", M, K, N, nbits, group_size)


def hqq_linear_batch_backward_workspace(M: int, K: int, Ns, nbits: int, group_size: int) -> int:
    """Bytes of workspace of hqq_linear_batch_backward for weights of output sizes Ns."""
    arr = (ctypes.c_int64 * max(1, len(Ns)))(*Ns)
    return _bytes("hqq_linear_batch_backward_workspace", M, K, arr, len(Ns), nbits, group_size)


def hqq_linear_cross_entropy_workspace(M: int, K: int, N: int, nbits: int, group_size: int) -> int:
    """Bytes of workspace of hqq_linear_cross_entropy for these sizes."""
    return _bytes("hqq_linear_cross_entropy_workspace", M, K, N, nbits, group_size)


def hqq_linear_cross_entropy_backward_workspace(M: int, K: int, N: int, nbits: int, group_size: int) -> int:
    """Bytes of workspace of hqq_linear_cross_entropy_backward for these sizes."""
    return _bytes("hqq_linear_cross_entropy_backward_workspace", M, K, N, nbits, group_size)


_DT = {torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16}


def _matrix(t, name: str, rows: int | None = None, cols: int | None = None, like=None):
    """Check a 16-bit [rows, cols] CUDA tensor (of like's dtype and device)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DT or (like is not None and t.dtype != like.dtype):
        raise TypeError(f"{name} must be float16 or bfloat16, the same in all arguments, got {t.dtype}")
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be [{'M' if rows is None else rows}, {'K' if cols is None else cols}], "
                         f"got {tuple(t.shape)}")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the other arguments are on {like.device}")
    return _dev_ptr(t, name, (t.dtype,))


def _array(t, name: str, dtypes, n: int, device):
    """Check a CUDA tensor of n values on device."""
    p = _dev_ptr(t, name, dtypes)
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got {t.numel()}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other arguments are on {device}")
    return p


def _weight(w, name: str, N: int, K: int, nbits: int, group_size: int, device):
    """The checked pointers (packed, scale, zero) of a weight [N, K]."""
    packed, scale, zero = w
    f32 = (torch.float32,)
    # sizes the library refuses are left to it
    words = N * K * nbits // 32 if nbits in (1, 2, 4, 8) else packed.numel()
    groups = N * (K // group_size) if group_size > 0 else scale.numel()
    return (_array(packed, f"{name} packed", _U32, words, device).value,
            _array(scale, f"{name} scale", f32, groups, device).value,
            _array(zero, f"{name} zero", f32, groups, device).value)


def _act(activation: str) -> int:
    if activation not in ACT_CODES:
        raise ValueError(f"activation must be one of {sorted(ACT_CODES)}, got {activation!r}")
    return ACT_CODES[activation]


def _call(name: str, device, workspace, need: int, *args):
    """Run the library's call `name` on device's current stream with a workspace."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    elif workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, the other arguments are on {device}")
    ptr = ctypes.c_void_p(workspace.data_ptr() if workspace is not None and workspace.numel() else None)
    size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    with torch.cuda.device(device):
        st = getattr(load_layers_library(), name)(*args, ptr, size, _stream(device))
    if st != 0:
        raise LayersError(name, st)


def hqq_linear_gated(X: torch.Tensor, gate, up, N: int, nbits: int, group_size: int,
                     activation: str = "silu", out=None, workspace=None) -> torch.Tensor:
    """Y = act(X . Wg_hat^T) * (X . Wu_hat^T) as a tensor [M, N]: the first half of a
    gated feed-forward block, for X [M, K] and the weights gate and up [N, K], each
    (packed, scale, zero).  activation: "silu", "gelu" or "gelu_tanh"."""
    px = _matrix(X, "X")
    M, K = X.shape
    act = _act(activation)
    g = HqqWeight(*_weight(gate, "gate", N, K, nbits, group_size, X.device))
    u = HqqWeight(*_weight(up, "up", N, K, nbits, group_size, X.device))
    need = hqq_linear_gated_workspace(M, K, N, nbits, group_size)
    if out is None:
        out = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _call("hqq_linear_gated", X.device, workspace, need, px, M, K, ctypes.byref(g), ctypes.byref(u), N, nbits,
          group_size, _DT[X.dtype], act, _matrix(out, "out", M, N, X))
    return out


def hqq_linear_gated_backward(dY: torch.Tensor, X: torch.Tensor, gate, up, N: int, nbits: int,
                              group_size: int, activation: str = "silu", out=None,
                              workspace=None) -> torch.Tensor:
    """The gradient dX [M, K] of hqq_linear_gated's input, from the gradient dY [M, N]
    of its output; the two projections are computed anew from X."""
    px = _matrix(X, "X")
    M, K = X.shape
    act = _act(activation)
    py = _matrix(dY, "dY", M, N, X)
    g = HqqWeight(*_weight(gate, "gate", N, K, nbits, group_size, X.device))
    u = HqqWeight(*_weight(up, "up", N, K, nbits, group_size, X.device))
    need = hqq_linear_gated_backward_workspace(M, K, N, nbits, group_size)
    if out is None:
        out = torch.empty((M, K), dtype=X.dtype, device=X.device)
    _call("hqq_linear_gated_backward", X.device, workspace, need, py, px, M, K, ctypes.byref(g), ctypes.byref(u), N,
          nbits, group_size, _DT[X.dtype], act, _matrix(out, "out", M, K, X))
    return out


def hqq_linear_batch_backward(dYs, weights, K: int, nbits: int, group_size: int, out=None,
                              workspace=None) -> torch.Tensor:
    """dX = sum_i dY_i . W_hat_i ([M, K]): the gradient of the input that several
    weights read (hqq_linear_batch), from the gradients dYs of their outputs.
    weights: [(packed, scale, zero, N), ...], at most MAX_GRADS."""
    dYs, weights = list(dYs), list(weights)
    if len(dYs) != len(weights) or not dYs:
        raise ValueError(f"one dY for each weight, at least one: got {len(dYs)} and {len(weights)}")
    if len(dYs) > MAX_GRADS:
        raise ValueError(f"at most {MAX_GRADS} weights, got {len(dYs)}")
    first = dYs[0]
    _matrix(first, "dYs[0]")
    M, dev = first.shape[0], first.device
    arr = (HqqLinearGrad * len(dYs))()
    for i, (dY, (packed, scale, zero, N)) in enumerate(zip(dYs, weights)):
        arr[i] = HqqLinearGrad(*_weight((packed, scale, zero), f"weights[{i}]", N, K, nbits, group_size, dev), N,
                               _matrix(dY, f"dYs[{i}]", M, N, first).value)
    need = hqq_linear_batch_backward_workspace(M, K, [w[3] for w in weights], nbits, group_size)
    if out is None:
        out = torch.empty((M, K), dtype=first.dtype, device=dev)
    _call("hqq_linear_batch_backward", dev, workspace, need, arr, len(dYs), M, K, nbits, group_size,
          _DT[first.dtype], _matrix(out, "out", M, K, first))
    return out


def hqq_linear_backward(dY: torch.Tensor, packed, scale, zero, K: int, nbits: int, group_size: int,
                        out=None, workspace=None) -> torch.Tensor:
    """dX = dY . W_hat ([M, K]): the gradient of hqq_linear's input."""
    N = dY.shape[1] if isinstance(dY, torch.Tensor) and dY.dim() == 2 else 0
    return hqq_linear_batch_backward([dY], [(packed, scale, zero, N)], K, nbits, group_size, out, workspace)


def hqq_linear_cross_entropy(X: torch.Tensor, targets: torch.Tensor, packed, scale, zero, N: int, nbits: int,
                             group_size: int, loss=None, lse=None, workspace=None):
    """Softmax cross entropy of the logits X . W_hat^T of a quantized head W [N, K]
    against targets (int64 [M]): (loss, lse), fp32 [M] each.  A row whose target lies
    outside [0, N) is ignored: its loss is 0.  The logits are never kept."""
    px = _matrix(X, "X")
    M, K = X.shape
    dev = X.device
    pt = _array(targets, "targets", (torch.int64,), M, dev)
    w = HqqWeight(*_weight((packed, scale, zero), "head", N, K, nbits, group_size, dev))
    need = hqq_linear_cross_entropy_workspace(M, K, N, nbits, group_size)
    loss = torch.empty(M, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(M, dtype=torch.float32, device=dev) if lse is None else lse
    _call("hqq_linear_cross_entropy", dev, workspace, need, px, M, K, ctypes.byref(w), N, nbits, group_size,
          _DT[X.dtype], pt, _array(loss, "loss", (torch.float32,), M, dev), _array(lse, "lse", (torch.float32,), M, dev))
    return loss, lse


def hqq_linear_cross_entropy_backward(dloss: torch.Tensor, X: torch.Tensor, targets: torch.Tensor,
                                      lse: torch.Tensor, packed, scale, zero, N: int, nbits: int,
                                      group_size: int, out=None, workspace=None) -> torch.Tensor:
    """The gradient dX [M, K] of hqq_linear_cross_entropy's input, from the gradient
    dloss (fp32 [M]) of its losses and the lse that it returned.  Ignored rows get 0."""
    px = _matrix(X, "X")
    M, K = X.shape
    dev = X.device
    f32 = (torch.float32,)
    pd, pl = _array(dloss, "dloss", f32, M, dev), _array(lse, "lse", f32, M, dev)
    pt = _array(targets, "targets", (torch.int64,), M, dev)
    w = HqqWeight(*_weight((packed, scale, zero), "head", N, K, nbits, group_size, dev))
    need = hqq_linear_cross_entropy_backward_workspace(M, K, N, nbits, group_size)
    if out is None:
        out = torch.empty((M, K), dtype=X.dtype, device=dev)
    _call("hqq_linear_cross_entropy_backward", dev, workspace, need, pd, px, M, K, ctypes.byref(w), N, nbits,
          group_size, _DT[X.dtype], pt, pl, _matrix(out, "out", M, K, X))
    return out
