"""The operators of include/moe_ops.h on torch tensors.

moe_linear, moe_grouped_linear, moe_group_slots and moe_combine_slots keep the
C names; LinearWeights holds the weights and the epilogue of a product. As in
the rest of the binding nothing is computed here: the functions check the
tensors, pass pointers and sizes to libmoe_decode.so, and turn status codes into
MoeError. Inference only: no gradients are recorded.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

from . import _abi

MOE_DTYPE_F16 = 2
MOE_EPI_NONE, MOE_EPI_SILU, MOE_EPI_GELU, MOE_EPI_GELU_TANH = range(4)
ACTIVATIONS = {"none": MOE_EPI_NONE, "silu": MOE_EPI_SILU, "gelu": MOE_EPI_GELU, "gelu_tanh": MOE_EPI_GELU_TANH}

OPS_EXPORTED = ("moe_linear", "moe_grouped_linear", "moe_group_slots", "moe_combine_slots", "moe_ops_check")


class moe_product(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("E", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("w", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("stride_e", ctypes.c_int64), ("bias", ctypes.c_void_p), ("bias_up", ctypes.c_void_p),
                ("activation", ctypes.c_int), ("act_limit", ctypes.c_float)]


_fns = None


def _lib():
    """The operators' C functions with their argument types."""
    global _fns
    if _fns is None:
        L = _abi.lib()
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.moe_linear.argtypes = [vp, vp, i64, i32, vp, i64, vp, i64, vp]
        L.moe_grouped_linear.argtypes = [vp, vp, vp, vp, i64, i32, i32, vp, i64, vp]
        L.moe_group_slots.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp]
        L.moe_combine_slots.argtypes = [i32, vp, i64, i32, vp, vp, i32, i32, i32, vp, i64, vp, i64, vp]
        L.moe_ops_check.argtypes = [vp]
        for name in OPS_EXPORTED:
            getattr(L, name).restype = i32
        _fns = L
    return _fns


def _dtype_code(dtype) -> int:
    import torch
    if dtype == torch.bfloat16:
        return _abi.MOE_DTYPE_BF16
    if dtype == torch.float16:
        return MOE_DTYPE_F16
    raise TypeError(f"{dtype} is not supported: bfloat16 or float16")


def _rows(t, what: str, cols: int, dtype, device, n: Optional[int] = None) -> int:
    """Check a [n, cols] tensor whose columns are adjacent; the distance of its rows."""
    if t.dim() != 2 or t.shape[1] != cols or (n is not None and t.shape[0] != n):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not [{'n' if n is None else n}, {cols}]")
    if t.dtype != dtype:
        raise TypeError(f"{what} is {t.dtype}, not {dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the columns of a row have to be adjacent")
    return t.stride(0) if t.shape[0] > 1 else cols


def _ints(t, what: str, shape, device):
    import torch
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype != torch.int32:
        raise TypeError(f"{what} is {t.dtype}, not int32")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} has to be contiguous and on {device}")


class _Launch:
    """The device and stream of a call: kernels go to `stream`, or to the current
    stream of the tensors' device, and outputs are allocated for that stream."""

    def __init__(self, device, stream):
        import torch
        self._on_device = self._on_stream = None
        if device.type != "cuda":
            raise ValueError(f"tensors have to be on a CUDA device, not on {device}")
        if torch.cuda.current_device() != device.index:
            self._on_device = torch.cuda.device(device)
        if stream is not None:
            s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
            self._on_stream = torch.cuda.stream(s)
        self._device = device

    def __enter__(self):
        import torch
        if self._on_device is not None:
            self._on_device.__enter__()
        if self._on_stream is not None:
            self._on_stream.__enter__()
        return torch.cuda.current_stream(self._device).cuda_stream

    def __exit__(self, *exc):
        if self._on_stream is not None:
            self._on_stream.__exit__(*exc)
        if self._on_device is not None:
            self._on_device.__exit__(*exc)


class LinearWeights:
    """The weights and the epilogue of a product (moe_product).

    w: [N, K], or [E, N, K] for one matrix per expert; bfloat16 or float16, inputs
    adjacent, rows (and experts) at any distance that is a multiple of 8 elements.
    w_up: the second matrix of a gated product, act(x w^T + bias) * (x w_up^T +
    bias_up), with w's shape and strides (the halves of one fused tensor have
    them). bias, bias_up: [N] or [E, N]. activation: "none", "silu", "gelu" or
    "gelu_tanh". act_limit: the clamp bound of a gated product, 0 for none.

    The tensors are referenced, not copied."""

    def __init__(self, w, w_up=None, bias=None, bias_up=None, activation: str = "none", act_limit: float = 0.0):
        if w.dim() not in (2, 3):
            raise ValueError(f"w has {w.dim()} dimensions, not 2 or 3")
        if activation not in ACTIVATIONS:
            raise ValueError(f"unknown activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
        self.grouped = w.dim() == 3
        self.E = w.shape[0] if self.grouped else 1
        self.N, self.K = w.shape[-2], w.shape[-1]
        self.dtype, self.device = w.dtype, w.device
        self.tensors = (w, w_up, bias, bias_up)
        if self.E < 1 or self.N < 1 or self.K < 1:
            raise ValueError(f"w is empty: {tuple(w.shape)}")
        if w.stride(-1) != 1 and self.K > 1:
            raise ValueError("w: the inputs of a row have to be adjacent")
        if w_up is not None and (w_up.shape != w.shape or w_up.stride() != w.stride() or w_up.dtype != w.dtype
                                 or w_up.device != w.device):
            raise ValueError("w_up needs the shape, strides, type and device of w")
        want = (self.E, self.N) if self.grouped else (self.N,)
        for name, b in (("bias", bias), ("bias_up", bias_up)):
            if b is not None and (tuple(b.shape) != want or b.dtype != w.dtype or b.device != w.device
                                  or not b.is_contiguous()):
                raise ValueError(f"{name} has to be contiguous {want} of {w.dtype} on {w.device}")
        ptr = _abi._ptr
        self.c = moe_product(_dtype_code(w.dtype), self.E, self.N, self.K, ptr(w), ptr(w_up),
                             w.stride(-2) if self.N > 1 else self.K,
                             w.stride(0) if self.grouped and self.E > 1 else 0, ptr(bias), ptr(bias_up),
                             ACTIVATIONS[activation], float(act_limit))
        self.ref = ctypes.addressof(self.c)


class SlotGroups(NamedTuple):
    """Rows grouped by expert (moe_group_slots): offsets [E + 1], slot_token and
    slot_k [n * top_k], slot_of [n, top_k]; all int32 on the device."""
    offsets: object
    slot_token: object
    slot_k: object
    slot_of: object


def _no_grad(x):
    import torch
    if x.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("x requires a gradient: the operators record none (use torch.no_grad())")


def moe_linear(x, weights: LinearWeights, residual=None, out=None, stream=None):
    """out [n, N] = epilogue(x [n, K]) (+ residual [n, N]); `out` may be `residual`."""
    import torch
    if weights.grouped:
        raise ValueError("moe_linear takes weights [N, K]; use moe_grouped_linear")
    _no_grad(x)
    dt, dev, n, N = weights.dtype, weights.device, x.shape[0], weights.N
    ldx = _rows(x, "x", weights.K, dt, dev)
    ldr = _rows(residual, "residual", N, dt, dev, n) if residual is not None else 0
    ldo = _rows(out, "out", N, dt, dev, n) if out is not None else N
    with _Launch(dev, stream) as st:
        if out is None:
            out = torch.empty((n, N), dtype=dt, device=dev)
        if n:
            _abi._check(_lib().moe_linear(weights.ref, x.data_ptr(), ldx, n,
                                          None if residual is None else residual.data_ptr(), ldr,
                                          out.data_ptr(), ldo, st), "moe_linear")
    return out


def moe_grouped_linear(x, weights: LinearWeights, offsets, row_token=None, out=None, stream=None):
    """out [rows, N]: row r of group e (offsets[e] <= r < offsets[e+1]) through
    expert e's matrix. x is [rows, K], or [tokens, K] with row_token [rows]. Rows
    outside every group are left as they were (unset in an `out` made here)."""
    import torch
    if not weights.grouped:
        raise ValueError("moe_grouped_linear takes weights [E, N, K]; use moe_linear")
    _no_grad(x)
    dt, dev, N = weights.dtype, weights.device, weights.N
    ldx = _rows(x, "x", weights.K, dt, dev)
    rows = x.shape[0] if row_token is None else row_token.numel()
    if row_token is not None:
        _ints(row_token, "row_token", (rows,), dev)
        if rows and not x.shape[0]:
            raise ValueError("x has no rows to take")
    _ints(offsets, "offsets", (weights.E + 1,), dev)
    ldo = _rows(out, "out", N, dt, dev, rows) if out is not None else N
    with _Launch(dev, stream) as st:
        if out is None:
            out = torch.empty((rows, N), dtype=dt, device=dev)
        if rows:
            _abi._check(_lib().moe_grouped_linear(weights.ref, offsets.data_ptr(),
                                                  None if row_token is None else row_token.data_ptr(),
                                                  x.data_ptr(), ldx, x.shape[0], rows, out.data_ptr(), ldo, st),
                        "moe_grouped_linear")
    return out


def moe_group_slots(topk_idx, E: int, experts: Optional[Tuple[int, int]] = None, stream=None) -> SlotGroups:
    """Group the slots of topk_idx [n, top_k] (int32) by expert. experts: (begin,
    end) of the ids that take part, all of them by default; other ids (another
    shard's, -1 for a dropped slot) belong to no group."""
    import torch
    if topk_idx.dim() != 2:
        raise ValueError(f"topk_idx has shape {tuple(topk_idx.shape)}, not [n, top_k]")
    n, k = topk_idx.shape
    dev = topk_idx.device
    _ints(topk_idx, "topk_idx", (n, k), dev)
    lo, hi = (0, E) if experts is None else experts
    with _Launch(dev, stream) as st:
        S = n * k
        buf = torch.empty(3 * S + E + 1, dtype=torch.int32, device=dev)
        # views of one allocation: offsets last, the three slot arrays in front
        token, rank, of, offsets = buf.split((S, S, S, E + 1))
        p = buf.data_ptr()
        # an empty tensor has no address: nothing of it is read
        _abi._check(_lib().moe_group_slots(topk_idx.data_ptr() or p, n, k, E, lo, hi, p + 12 * S, p, p + 4 * S,
                                           p + 8 * S, st), "moe_group_slots")
    return SlotGroups(offsets, token, rank, of.view(n, k))


def moe_combine_slots(y, slot_of, topk_w, residual=None, out=None, stream=None):
    """out [n, N] = sum_j topk_w[t, j] * y[slot_of[t, j]] (+ residual): y [rows, N],
    slot_of [n, top_k] int32 (a slot outside y's rows adds nothing), topk_w
    [n, top_k] float32; `out` may be `residual`."""
    import torch
    _no_grad(y)
    dt, dev = y.dtype, y.device
    code = _dtype_code(dt)
    if y.dim() != 2 or slot_of.dim() != 2:
        raise ValueError("y has to be [rows, N] and slot_of [n, top_k]")
    rows, N = y.shape
    n, k = slot_of.shape
    ldy = _rows(y, "y", N, dt, dev)
    _ints(slot_of, "slot_of", (n, k), dev)
    if topk_w.shape != slot_of.shape or topk_w.dtype != torch.float32 or topk_w.device != dev \
            or not topk_w.is_contiguous():
        raise ValueError(f"topk_w has to be contiguous float32 {tuple(slot_of.shape)} on {dev}")
    ldr = _rows(residual, "residual", N, dt, dev, n) if residual is not None else 0
    ldo = _rows(out, "out", N, dt, dev, n) if out is not None else N
    with _Launch(dev, stream) as st:
        if out is None:
            out = torch.empty((n, N), dtype=dt, device=dev)
        if n:
            _abi._check(_lib().moe_combine_slots(code, y.data_ptr() or None, ldy, rows, slot_of.data_ptr(),
                                                 topk_w.data_ptr(), n, k, N,
                                                 None if residual is None else residual.data_ptr(), ldr,
                                                 out.data_ptr(), ldo, st), "moe_combine_slots")
    return out


def moe_ops_check(stream=None) -> None:
    """Synchronise `stream` (the current one by default) and raise MoeError for a
    device-side wait of these operators that gave up since the last check."""
    _abi._check(_lib().moe_ops_check(_abi._stream(stream)), "moe_ops_check")
