"""Convenience wrappers over the C ABI: resident layer weights and a layer
object that owns a plan, and the 16-bit expert layers that run beside it.
Argument marshalling only."""
from __future__ import annotations

from typing import Any, Optional

import numpy as np

from . import _abi
from .ops import (LinearWeights, _no_grad, moe_combine_slots, moe_group_slots, moe_grouped_linear, moe_linear,
                  moe_ops_check)

_DT = {"f32": _abi.MOE_DTYPE_F32, "bf16": _abi.MOE_DTYPE_BF16}


def _to_torch(a: np.ndarray, device, torch):
    """numpy storage array -> device tensor with the same bytes.
    uint32 -> int32, uint16 (bf16 bits) -> bfloat16, uint8 -> uint8 (6-bit
    down codes), float32 -> float32."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint32:
        return torch.from_numpy(a.view(np.int32)).to(device)
    if a.dtype == np.uint8:
        return torch.from_numpy(a).to(device)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    if a.dtype == np.float32:
        return torch.from_numpy(a).to(device)
    raise TypeError(a.dtype)


class DeviceLayer:
    """One MoE layer's weights resident on a CUDA device.

    router_w: [E, D] float32 or bf16; router_bias: [E] float32 or None;
    planes: the nine quantised arrays (see include/moe_decode.h)."""

    def __init__(self, router_w, router_bias, planes: dict, E: int, top_k: int, D: int, Dff: int):
        self.router_w = router_w
        self.router_bias = router_bias
        self.planes = planes
        self.E, self.top_k, self.D, self.Dff = E, top_k, D, Dff
        self.c_planes = _abi.make_planes(planes)

    @classmethod
    def from_host(cls, router_w_storage: np.ndarray, router_bias: Optional[np.ndarray], planes: Any,
                  top_k: int, device="cuda"):
        import torch
        arrs = {f: _to_torch(getattr(planes, f), device, torch) for f in _abi.PLANE_FIELDS}
        rw = _to_torch(router_w_storage, device, torch)
        rb = None if router_bias is None else _to_torch(router_bias.astype(np.float32), device, torch)
        E, Dff, D8 = arrs["gate_q"].shape
        return cls(rw, rb, arrs, E, top_k, D8 * 8, Dff)

    @property
    def plane_bytes_per_expert(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.planes.values()) // self.E


class MoeDecodeLayer:
    """Owns one plan (workspace sized for max_tokens) on the current device."""

    def __init__(self, E: int, top_k: int, D: int, Dff: int, max_tokens: int = 64,
                 act_dtype: str = "bf16", out_dtype: Optional[str] = None, flags: int = 0,
                 mma_min_tokens: int = 0, activation: int = _abi.MOE_ACT_SWIGLU,
                 act_limit: float = 0.0, down_bits: int = 0, experts=None):
        """experts: (begin, end) of the experts this plan owns (an expert-parallel
        shard), or None for all of them."""
        eb, ee = (0, 0) if experts is None else (int(experts[0]), int(experts[1]))
        self.cfg = _abi.make_config(E, top_k, D, Dff, max_tokens, x_dtype=_DT[act_dtype],
                                    router_dtype=_DT[act_dtype],
                                    out_dtype=_DT[out_dtype or act_dtype], flags=flags,
                                    mma_min_tokens=mma_min_tokens, activation=activation,
                                    act_limit=act_limit, down_bits=down_bits,
                                    expert_begin=eb, expert_end=ee)
        self.act_dtype = act_dtype
        self.out_dtype = out_dtype or act_dtype
        self.plan = _abi.moe_plan_create(self.cfg)
        self._shared_stream = None  # of the last step with a shared expert

    def _out_torch_dtype(self):
        import torch
        return torch.float32 if self.out_dtype == "f32" else torch.bfloat16

    def forward(self, x, w: DeviceLayer, out=None, stream=None, shared=None):
        """One step. shared: a SharedExpert whose output is added to the routed
        experts' (16-bit activations and output: its type)."""
        import torch
        n = x.shape[0]
        if shared is not None and {x.dtype, out.dtype if out is not None else self._out_torch_dtype()} != {shared.dtype}:
            raise TypeError(f"the shared expert is {shared.dtype}: x and the step's output have to be, too")
        if shared is not None:
            shared.refuse(x, out, w.D)
        if out is None:
            out = torch.empty((n, w.D), dtype=self._out_torch_dtype(), device=x.device)
        _abi.moe_decode_forward(self.plan, x, w.router_w, w.router_bias, w.c_planes, n,
                                self.cfg.top_k, out, stream)
        if shared is not None:
            self._shared_stream = torch.cuda.current_stream() if stream is None else stream
            shared.forward(x, residual=out, out=out, stream=stream)
        return out

    def forward_layers(self, steps, stream=None):
        """steps: sequence of (x, DeviceLayer, out), run in order as one chain
        (moe_decode_forward_layers); returns the outs."""
        _abi.moe_decode_forward_layers(
            self.plan, [(x, w.router_w, w.router_bias, w.c_planes, out) for x, w, out in steps],
            steps[0][0].shape[0], self.cfg.top_k, stream)
        return [out for _, _, out in steps]

    def forward_host(self, x_host, w: DeviceLayer, out_host, stream=None):
        n = x_host.shape[0]
        _abi.moe_decode_forward_host(self.plan, x_host, w.router_w, w.router_bias, w.c_planes, n,
                                     self.cfg.top_k, out_host, stream)
        return out_host

    def routing(self, n_tokens: int):
        return _abi.moe_get_routing(self.plan, n_tokens, self.cfg.E, self.cfg.top_k)

    def check(self):
        """Raise MoeError for a device-side wait that gave up: of the plan's steps, and of
        the shared experts that ran beside them."""
        _abi.moe_plan_check(self.plan)
        if self._shared_stream is not None:
            moe_ops_check(self._shared_stream)

    def close(self):
        if getattr(self, "plan", None):
            _abi.moe_plan_free(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SharedExpert:
    """A 16-bit expert that every token takes: down(act(x gate^T) * (x up^T)).
    gate, up [F, D], down [D, F]; two launches (moe_linear)."""

    def __init__(self, gate, up, down, activation: str = "silu", act_limit: float = 0.0):
        self.gate_up = LinearWeights(gate, w_up=up, activation=activation, act_limit=act_limit)
        self.down = LinearWeights(down)
        if (self.down.N, self.down.K) != (self.gate_up.K, self.gate_up.N):
            raise ValueError(f"down {tuple(down.shape)} does not fit gate {tuple(gate.shape)}")
        self.dtype = self.down.dtype

    def refuse(self, x, out, width: int):
        """Raise for a step `width` wide on x that this expert cannot run beside."""
        if self.down.N != width:
            raise ValueError(f"the shared expert is {self.down.N} wide, the step {width}")
        _no_grad(x, out, *self.gate_up.tensors, *self.down.tensors)

    def forward(self, x, residual=None, out=None, stream=None):
        """[n, D] -> [n, D], plus `residual` (which `out` may be)."""
        h = moe_linear(x, self.gate_up, stream=stream)
        return moe_linear(h, self.down, residual=residual, out=out, stream=stream)

    def check(self, stream=None):
        """moe_ops_check: raise MoeError for a device-side wait that gave up."""
        moe_ops_check(stream)


class RoutedExperts:
    """Experts with 16-bit weights under any router: gate, up [E, F, D], down
    [E, D, F]. The router's top-k ids and weights are arguments of forward, which
    groups the slots, runs the two grouped products and combines. experts: (begin,
    end) of the expert ids whose slots are run (the weights cover all E ids)."""

    def __init__(self, gate, up, down, activation: str = "silu", act_limit: float = 0.0, experts=None):
        self.gate_up = LinearWeights(gate, w_up=up, activation=activation, act_limit=act_limit)
        self.down = LinearWeights(down)
        if (self.down.E, self.down.N, self.down.K) != (self.gate_up.E, self.gate_up.K, self.gate_up.N):
            raise ValueError(f"down {tuple(down.shape)} does not fit gate {tuple(gate.shape)}")
        self.experts = experts

    def forward(self, x, topk_idx, topk_w, residual=None, out=None, stream=None):
        """x [n, D], topk_idx [n, k] int32, topk_w [n, k] float32 -> [n, D]."""
        if x.dim() != 2 or topk_idx.dim() != 2 or x.shape[0] != topk_idx.shape[0]:
            raise ValueError(f"x {tuple(x.shape)} and topk_idx {tuple(topk_idx.shape)} have to be [n, D] and [n, k]")
        g = moe_group_slots(topk_idx, self.gate_up.E, experts=self.experts, stream=stream)
        h = moe_grouped_linear(x, self.gate_up, g.offsets, row_token=g.slot_token, stream=stream)
        y = moe_grouped_linear(h, self.down, g.offsets, stream=stream)
        return moe_combine_slots(y, g.slot_of, topk_w, residual=residual, out=out, stream=stream)

    def check(self, stream=None):
        """moe_ops_check: raise MoeError for a device-side wait that gave up."""
        moe_ops_check(stream)
