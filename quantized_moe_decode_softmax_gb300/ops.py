"""The operators of include/moe_ops.h on torch tensors.

moe_linear, moe_grouped_linear, moe_group_slots and moe_combine_slots keep the
C names; LinearWeights holds the weights and the epilogue of a product. As in
the rest of the binding nothing is computed here: the functions check the
tensors, pass pointers and sizes to libmoe_decode.so, and turn status codes into
MoeError. Inference only: a call that autograd would have to record is refused.

`stream` is the stream that a call runs on (a torch stream, or a cudaStream_t as a
number), the current one by default. As everywhere in torch, another stream waits for
nothing by itself: what wrote the inputs is the caller's to order before it.

A usual call goes through the torch_calls module (csrc/torch_calls.cpp), which does
the same checks in less time and returns None for whatever is not usual; the
functions here then take over, with their messages.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings
from typing import NamedTuple, Optional, Tuple

from . import _abi, build

MOE_DTYPE_F16 = 2
MOE_EPI_NONE, MOE_EPI_SILU, MOE_EPI_GELU, MOE_EPI_GELU_TANH = range(4)
ACTIVATIONS = {"none": MOE_EPI_NONE, "silu": MOE_EPI_SILU, "gelu": MOE_EPI_GELU, "gelu_tanh": MOE_EPI_GELU_TANH}

OPS_EXPORTED = ("moe_linear", "moe_grouped_linear", "moe_group_slots", "moe_combine_slots", "moe_ops_check")


class moe_product(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("E", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("w", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("stride_e", ctypes.c_int64), ("bias", ctypes.c_void_p), ("bias_up", ctypes.c_void_p),
                ("activation", ctypes.c_int), ("act_limit", ctypes.c_float)]


torch = None   # bound by _bind: importing the package does not import torch
_c = None      # the operators' C functions
_calls = None  # the torch_calls module, where it has been built for this torch


def _bind():
    """Bind torch and the C functions (first use; raises if the library is not built)."""
    global torch, _c, _calls
    L = _abi.lib()
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.moe_linear.argtypes = [vp, vp, i64, i32, vp, i64, vp, i64, vp]
    L.moe_grouped_linear.argtypes = [vp, vp, vp, vp, i64, i32, i32, vp, i64, vp]
    L.moe_group_slots.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp]
    L.moe_combine_slots.argtypes = [i32, vp, i64, i32, vp, vp, i32, i32, i32, vp, i64, vp, i64, vp]
    L.moe_ops_check.argtypes = [vp]
    for name in OPS_EXPORTED:
        getattr(L, name).restype = i32
    import torch as t
    torch = t
    path = build.calls_path()
    if path is not None and os.path.exists(path):
        loader = importlib.machinery.ExtensionFileLoader("_torch_calls", path)
        try:
            m = importlib.util.module_from_spec(
                importlib.util.spec_from_file_location("_torch_calls", path, loader=loader))
            m.bind(*[ctypes.cast(getattr(L, f), vp).value for f in
                     ("moe_linear", "moe_grouped_linear", "moe_group_slots", "moe_combine_slots")])
            _calls = m
        except (ImportError, OSError) as e:  # every call has its way through ctypes
            warnings.warn(f"{path} cannot be loaded ({e}): calls of the operators go through ctypes")
    _c = L
    return L


def _lib():
    return _c or _bind()


def _dtype_code(dtype) -> int:
    if dtype == torch.bfloat16:
        return _abi.MOE_DTYPE_BF16
    if dtype == torch.float16:
        return MOE_DTYPE_F16
    raise TypeError(f"{dtype} is not supported: bfloat16 or float16")


def _rows(t, what: str, cols: int, dtype, device, n: int = -1) -> int:
    """Check a [n, cols] tensor (any n: -1) whose columns are adjacent on CUDA device
    number `device`; the distance of its rows. A call spends about as long here as
    on the GPU for a few tokens, so that each property is asked for once."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (n >= 0 and shape[0] != n):
        raise ValueError(f"{what} has shape {tuple(shape)}, not [{'n' if n < 0 else n}, {cols}]")
    if t.dtype is not dtype:
        raise TypeError(f"{what} is {t.dtype}, not {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{what} is on {t.device}, not on CUDA device {device}")
    if t.is_contiguous():
        return cols
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError(f"{what}: the columns of a row have to be adjacent")
    return row if shape[0] > 1 else cols


def _ints(t, what: str, shape, device):
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype is not torch.int32:
        raise TypeError(f"{what} is {t.dtype}, not int32")
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what} has to be contiguous and on CUDA device {device}")


class _Elsewhere:
    """The device (by its number) and stream of a call that names a stream or whose
    tensors are not on the current device: outputs are allocated there, kernels go
    there. The tensors of the call are recorded on a named stream, so that memory that the
    caller lets go of right afterwards is not given out again before the call has run
    there. (Not on a stream that torch does not own: it may be destroyed first. Its
    caller keeps the tensors.)"""

    def __init__(self, device: int, stream, tensors=()):
        if device < 0:
            raise ValueError("tensors have to be on a CUDA device")
        self._device = device
        self._on_device = torch.cuda.device(device)
        self._recorded = ()
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        elif stream is not None:
            if stream.device.index != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors are on CUDA device {device}")
            if not isinstance(stream, torch.cuda.ExternalStream):
                self._recorded = tensors
        self._stream = stream
        self._on_stream = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self._on_device.__enter__()
        if self._on_stream is not None:
            self._on_stream.__enter__()
        return torch.cuda.current_stream(self._device).cuda_stream

    def __exit__(self, *exc):
        for t in self._recorded:
            if t is not None:
                t.record_stream(self._stream)
        if self._on_stream is not None:
            self._on_stream.__exit__(*exc)
        self._on_device.__exit__(*exc)


def _here(device: int, stream) -> bool:
    """Whether a call needs neither another device nor another stream."""
    return stream is None and device >= 0 and torch._C._cuda_getDevice() == device


class LinearWeights:
    """The weights and the epilogue of a product (moe_product).

    w: [N, K], or [E, N, K] for one matrix per expert; bfloat16 or float16, inputs
    adjacent, rows (and experts) at any distance that is a multiple of 8 elements.
    w_up: the second matrix of a gated product, act(x w^T + bias) * (x w_up^T +
    bias_up), with w's shape and strides (the halves of one fused tensor have
    them). bias, bias_up: [N] or [E, N]. activation: "none", "silu", "gelu" or
    "gelu_tanh". act_limit: the clamp bound of a gated product, 0 for none.

    The tensors are referenced, not copied. One that is given another storage (`w.data =
    other`, as offloading does) is followed: a call goes by the tensors as they are then (a
    captured graph by what they were at its capture). Their shapes and type have to stay."""

    def __init__(self, w, w_up=None, bias=None, bias_up=None, activation: str = "none", act_limit: float = 0.0):
        _lib()
        if w.dim() not in (2, 3):
            raise ValueError(f"w has {w.dim()} dimensions, not 2 or 3")
        if activation not in ACTIVATIONS:
            raise ValueError(f"unknown activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
        self.grouped = w.dim() == 3
        self.E = w.shape[0] if self.grouped else 1
        self.N, self.K = w.shape[-2], w.shape[-1]
        self.dtype = w.dtype
        self.tensors = (w, w_up, bias, bias_up)
        if self.E < 1 or self.N < 1 or self.K < 1:
            raise ValueError(f"w is empty: {tuple(w.shape)}")
        self._epilogue = ACTIVATIONS[activation], float(act_limit)
        self.c = moe_product()
        self.ref = ctypes.addressof(self.c)
        self._bind()

    def _layout(self):
        return [None if t is None else (t.data_ptr(), t.shape, t.stride(), t.dtype, t.device) for t in self.tensors]

    def _bind(self):
        """Check the tensors and write their addresses and strides into the struct."""
        w, w_up, bias, bias_up = self.tensors
        layout = self._layout()
        lead = (self.E,) if self.grouped else ()
        if tuple(w.shape) != lead + (self.N, self.K) or w.dtype != self.dtype:
            raise ValueError(f"w has become {tuple(w.shape)} of {w.dtype}: it was {lead + (self.N, self.K)} of {self.dtype}")
        if w.stride(-1) != 1 and self.K > 1:
            raise ValueError("w: the inputs of a row have to be adjacent")
        if w_up is not None and (w_up.shape != w.shape or w_up.stride() != w.stride() or w_up.dtype != w.dtype
                                 or w_up.device != w.device):
            raise ValueError("w_up needs the shape, strides, type and device of w")
        want = lead + (self.N,)
        for name, b in (("bias", bias), ("bias_up", bias_up)):
            if b is not None and (tuple(b.shape) != want or b.dtype != w.dtype or b.device != w.device
                                  or not b.is_contiguous()):
                raise ValueError(f"{name} has to be contiguous {want} of {w.dtype} on {w.device}")
        ptr = _abi._ptr
        if w.is_cuda and not all(t is None or ptr(t) for t in self.tensors):
            raise ValueError("the storage of a weight has been freed")
        c = moe_product(_dtype_code(w.dtype), self.E, self.N, self.K, ptr(w), ptr(w_up),
                        w.stride(-2) if self.N > 1 else self.K,
                        w.stride(0) if self.grouped and self.E > 1 else 0, ptr(bias), ptr(bias_up), *self._epilogue)
        # in one piece and in place: a call of another thread has read `ref`, or copies `c`
        (ctypes.c_char * ctypes.sizeof(c)).from_buffer(self.c).raw = bytes(c)
        self.device, self.device_index = w.device, w.get_device()
        self._bound = layout

    def current(self) -> moe_product:
        """A copy of the struct that describes the tensors as they are now."""
        if self._layout() != self._bound:
            self._bind()
        return moe_product.from_buffer_copy(self.c)


class SlotGroups(NamedTuple):
    """Rows grouped by expert (moe_group_slots): offsets [E + 1], slot_token and
    slot_k [n * top_k], slot_of [n, top_k]; all int32 on the device, and parts of
    one allocation: they are not to be resized in place."""
    offsets: object
    slot_token: object
    slot_k: object
    slot_of: object


def _no_grad(*tensors):
    """Refuse a call that autograd would have to record: every floating-point input, the
    weights and the output count."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise RuntimeError("an input requires a gradient: the operators record none (use torch.no_grad())")
    fw = torch.autograd.forward_ad
    if fw._current_level >= 0 and any(t is not None and fw.unpack_dual(t).tangent is not None for t in tensors):
        raise RuntimeError("an input carries a forward-mode tangent: the operators propagate none")


def _raise(status: int, what: str):
    raise _abi.MoeError(status, what)


def moe_linear(x, weights: LinearWeights, residual=None, out=None, stream=None):
    """out [n, N] = epilogue(x [n, K]) (+ residual [n, N]); `out` may be `residual`."""
    if stream is None and _calls is not None and not weights.grouped:
        r = _calls.linear(weights.ref, weights.device_index, x, residual, out, weights.tensors)
        if r is not None:
            return r if r.__class__ is not int else _raise(r, "moe_linear")
    if weights.grouped:
        raise ValueError("moe_linear takes weights [N, K]; use moe_grouped_linear")
    _no_grad(x, residual, out, *weights.tensors)
    c = weights.current()
    dt, dev, N = weights.dtype, weights.device_index, weights.N
    ldx = _rows(x, "x", weights.K, dt, dev)
    n = x.shape[0]
    ldr = ldo = N
    if residual is not None:
        ldr = _rows(residual, "residual", N, dt, dev, n)
    if out is not None:
        ldo = _rows(out, "out", N, dt, dev, n)
    if _here(dev, stream):
        return _linear(c, x, ldx, n, weights, residual, ldr, out, ldo, torch._C._cuda_getCurrentRawStream(dev))
    with _Elsewhere(dev, stream, (x, residual, out, *weights.tensors)) as st:
        return _linear(c, x, ldx, n, weights, residual, ldr, out, ldo, st)


def _written(out):
    """An output that was given counts as written, for whoever keeps it for a backward pass."""
    if not out.is_inference():
        torch.autograd.graph.increment_version(out)


def _linear(c, x, ldx, n, weights, residual, ldr, out, ldo, st):
    if out is None:
        out = torch.empty((n, weights.N), dtype=weights.dtype, device=weights.device)
    else:
        _written(out)
    if n:
        status = _c.moe_linear(ctypes.addressof(c), x.data_ptr(), ldx, n, None if residual is None else residual.data_ptr(),
                               ldr, out.data_ptr(), ldo, st)
        if status:
            _raise(status, "moe_linear")
    return out


def moe_grouped_linear(x, weights: LinearWeights, offsets, row_token=None, out=None, stream=None):
    """out [rows, N]: row r of group e (offsets[e] <= r < offsets[e+1]) through
    expert e's matrix. x is [rows, K], or [tokens, K] with row_token [rows]. Rows
    outside every group are left as they were (unset in an `out` made here)."""
    if stream is None and _calls is not None and weights.grouped:
        r = _calls.grouped(weights.ref, weights.device_index, x, offsets, row_token, out, weights.tensors)
        if r is not None:
            return r if r.__class__ is not int else _raise(r, "moe_grouped_linear")
    if not weights.grouped:
        raise ValueError("moe_grouped_linear takes weights [E, N, K]; use moe_linear")
    _no_grad(x, out, *weights.tensors)
    c = weights.current()
    dt, dev, N = weights.dtype, weights.device_index, weights.N
    ldx = _rows(x, "x", weights.K, dt, dev)
    rows = x.shape[0]
    if row_token is not None:
        tokens, rows = rows, row_token.numel()
        _ints(row_token, "row_token", (rows,), dev)
        if rows and not tokens:
            raise ValueError("x has no rows to take")
    _ints(offsets, "offsets", (weights.E + 1,), dev)
    ldo = N if out is None else _rows(out, "out", N, dt, dev, rows)
    if _here(dev, stream):
        return _grouped(c, x, ldx, rows, weights, offsets, row_token, out, ldo,
                        torch._C._cuda_getCurrentRawStream(dev))
    with _Elsewhere(dev, stream, (x, offsets, row_token, out, *weights.tensors)) as st:
        return _grouped(c, x, ldx, rows, weights, offsets, row_token, out, ldo, st)


def _grouped(c, x, ldx, rows, weights, offsets, row_token, out, ldo, st):
    if out is None:
        out = torch.empty((rows, weights.N), dtype=weights.dtype, device=weights.device)
    else:
        _written(out)
    if rows:
        status = _c.moe_grouped_linear(ctypes.addressof(c), offsets.data_ptr(),
                                       None if row_token is None else row_token.data_ptr(), x.data_ptr(), ldx,
                                       x.shape[0], rows, out.data_ptr(), ldo, st)
        if status:
            _raise(status, "moe_grouped_linear")
    return out


def moe_group_slots(topk_idx, E: int, experts: Optional[Tuple[int, int]] = None, stream=None) -> SlotGroups:
    """Group the slots of topk_idx [n, top_k] (int32) by expert. experts: (begin,
    end) of the ids that take part, all of them by default; other ids (another
    shard's, -1 for a dropped slot) belong to no group."""
    _lib()
    lo, hi = (0, E) if experts is None else experts
    if stream is None and _calls is not None:
        r = _calls.slots(topk_idx, E, lo, hi)
        if r is not None:
            return SlotGroups._make(r) if r.__class__ is not int else _raise(r, "moe_group_slots")
    shape, dev = topk_idx.shape, topk_idx.get_device()
    if len(shape) != 2:
        raise ValueError(f"topk_idx has shape {tuple(shape)}, not [n, top_k]")
    _ints(topk_idx, "topk_idx", shape, dev)
    if _here(dev, stream):
        return _slots(topk_idx, shape, E, lo, hi, torch._C._cuda_getCurrentRawStream(dev))
    with _Elsewhere(dev, stream, (topk_idx,)) as st:
        return _slots(topk_idx, shape, E, lo, hi, st)


def _slots(topk_idx, shape, E, lo, hi, st):
    n, k = shape
    dev = topk_idx.device
    E, lo, hi = int(E), int(lo), int(hi)
    int32 = torch.int32
    # four allocations: from Python, views of one cost more time
    offsets = torch.empty(max(E, 0) + 1, dtype=int32, device=dev)
    token = torch.empty(n * k, dtype=int32, device=dev)
    rank = torch.empty(n * k, dtype=int32, device=dev)
    of = torch.empty(shape, dtype=int32, device=dev)
    p = offsets.data_ptr()  # stands in for empty tensors, which have no address: nothing of them is used
    status = _c.moe_group_slots(topk_idx.data_ptr() or p, n, k, E, lo, hi, p, token.data_ptr() or p,
                                rank.data_ptr() or p, of.data_ptr() or p, st)
    if status:
        _raise(status, "moe_group_slots")
    return SlotGroups(offsets, token, rank, of)


def moe_combine_slots(y, slot_of, topk_w, residual=None, out=None, stream=None):
    """out [n, N] = sum_j topk_w[t, j] * y[slot_of[t, j]] (+ residual): y [rows, N],
    slot_of [n, top_k] int32 (a slot outside y's rows adds nothing), topk_w
    [n, top_k] float32; `out` may be `residual`."""
    _lib()
    if stream is None and _calls is not None:
        r = _calls.combine(y, slot_of, topk_w, residual, out)
        if r is not None:
            return r if r.__class__ is not int else _raise(r, "moe_combine_slots")
    _no_grad(y, topk_w, residual, out)
    dt, dev = y.dtype, y.get_device()
    code = _dtype_code(dt)
    shape, ys = slot_of.shape, y.shape
    if len(shape) != 2 or len(ys) != 2:
        raise ValueError("y has to be [rows, N] and slot_of [n, top_k]")
    n, N = shape[0], ys[1]
    ldy = _rows(y, "y", N, dt, dev)
    _ints(slot_of, "slot_of", shape, dev)
    if topk_w.shape != shape or topk_w.dtype is not torch.float32 or topk_w.get_device() != dev \
            or not topk_w.is_contiguous():
        raise ValueError(f"topk_w has to be contiguous float32 {tuple(shape)} on CUDA device {dev}")
    ldr = ldo = N
    if residual is not None:
        ldr = _rows(residual, "residual", N, dt, dev, n)
    if out is not None:
        ldo = _rows(out, "out", N, dt, dev, n)
    if _here(dev, stream):
        return _combine(code, y, ldy, slot_of, topk_w, residual, ldr, out, ldo,
                        torch._C._cuda_getCurrentRawStream(dev))
    with _Elsewhere(dev, stream, (y, slot_of, topk_w, residual, out)) as st:
        return _combine(code, y, ldy, slot_of, topk_w, residual, ldr, out, ldo, st)


def _combine(code, y, ldy, slot_of, topk_w, residual, ldr, out, ldo, st):
    n, k = slot_of.shape
    rows, N = y.shape
    if out is None:
        out = torch.empty((n, N), dtype=y.dtype, device=y.device)
    else:
        _written(out)
    if n:
        status = _c.moe_combine_slots(code, y.data_ptr() or None, ldy, rows, slot_of.data_ptr(), topk_w.data_ptr(), n,
                                      k, N, None if residual is None else residual.data_ptr(), ldr, out.data_ptr(),
                                      ldo, st)
        if status:
            _raise(status, "moe_combine_slots")
    return out


def moe_ops_check(stream=None) -> None:
    """Synchronise `stream` (the current one by default) and raise MoeError for a
    device-side wait of these operators on its device (a stream given as a number: on the
    current device) that gave up since the last check, on any stream."""
    lib = _lib()
    if stream is None or isinstance(stream, int):
        return _abi._check(lib.moe_ops_check(_abi._stream(stream)), "moe_ops_check")
    with torch.cuda.device(stream.device):
        _abi._check(lib.moe_ops_check(stream.cuda_stream), "moe_ops_check")
