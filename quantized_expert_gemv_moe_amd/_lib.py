"""ctypes binding of ``libmoe_decode.so`` (include/moe_decode.h).

Argument marshalling only: every step of the decode block runs in the HIP
kernels behind the C ABI.  torch is used for device memory and the current
HIP stream.  There is no fallback: if the library is not built, or a call
returns an error status, this module raises.
"""

from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass
from typing import Optional

import torch

from . import build as _build

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_DEVICE = range(5)
MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_F16 = 0, 1, 2
MOE_DOWN_ROWS, MOE_DOWN_COLS = 0, 1
MOE_ACT_SWIGLU, MOE_ACT_GEGLU = 0, 1
_ACTIVATIONS = {"swiglu": MOE_ACT_SWIGLU, "geglu": MOE_ACT_GEGLU}
MOE_FN_NONE, MOE_FN_RELU, MOE_FN_SILU, MOE_FN_GELU, MOE_FN_GELU_TANH = range(5)
_FNS = {"none": MOE_FN_NONE, "relu": MOE_FN_RELU, "silu": MOE_FN_SILU, "gelu": MOE_FN_GELU,
        "gelu_tanh": MOE_FN_GELU_TANH}
MOE_ROWS_TOKEN, MOE_ROWS_SLOT, MOE_ROWS_SORTED = range(3)
_ROWS = {"token": MOE_ROWS_TOKEN, "slot": MOE_ROWS_SLOT, "sorted": MOE_ROWS_SORTED}
_DTYPES = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16}
MOE_MAX_EXPERTS = 1024
MOE_MAX_TOP_K = 16
MOE_MAX_TOKENS = 65535
MOE_STATIC_SCRATCH_BYTES = 8 << 20


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


class LayerStruct(C.Structure):
    _fields_ = [
        ("hidden", C.c_int32), ("dff", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
        ("bits", C.c_int32), ("group_size", C.c_int32), ("act_dtype", C.c_int32),
        ("clamp_limit", C.c_float),
        ("gate_q", C.c_void_p), ("up_q", C.c_void_p),
        ("gate_s", C.c_void_p), ("gate_b", C.c_void_p), ("up_s", C.c_void_p), ("up_b", C.c_void_p),
        ("down_q", C.c_void_p), ("down_s", C.c_void_p), ("down_b", C.c_void_p),
        ("expert_scale", C.c_void_p),
        ("down_layout", C.c_int32), ("down_scale", C.c_void_p), ("activation", C.c_int32),
        ("down_bits", C.c_int32),
    ]


class PlanStruct(C.Structure):
    _fields_ = [("counts", C.c_void_p), ("offsets", C.c_void_p), ("sorted_slots", C.c_void_p),
                ("unique_experts", C.c_void_p), ("n_unique", C.c_void_p), ("work", C.c_void_p)]


class LinearStruct(C.Structure):
    _fields_ = [
        ("in_features", C.c_int32), ("out_features", C.c_int32), ("n_groups", C.c_int32), ("dtype", C.c_int32),
        ("out_dtype", C.c_int32), ("fn", C.c_int32), ("clamp_limit", C.c_float), ("reserved", C.c_int32),
        ("w", C.c_void_p), ("w_up", C.c_void_p), ("bias", C.c_void_p), ("bias_up", C.c_void_p),
        ("row_stride", C.c_int64), ("group_stride", C.c_int64), ("bias_stride", C.c_int64),
    ]


_lib = None

EXPORTS = ("moe_router_logits", "moe_route_topk", "moe_expert_plan", "moe_route_plan", "moe_workspace_size",
           "moe_decode_step", "moe_decode_step_residual",
           "moe_decode_layer", "moe_decode_layer_static", "moe_route_gate_up", "moe_expert_gate_up", "moe_expert_down_combine", "moe_pack_down",
           "moe_layer_check", "moe_status_str", "moe_abi_version",
           "moe_linear_check", "moe_matmul_workspace_size", "moe_grouped_workspace_size", "moe_matmul",
           "moe_grouped_matmul", "moe_combine")


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> C.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"HIP library {path} is not built; run __graft_entry__.build() "
                "or python -m quantized_expert_gemv_moe_amd.build")
        L = C.CDLL(path)
        vp, i32 = C.c_void_p, C.c_int32
        L.moe_router_logits.argtypes = [vp, i32, i32, C.c_int, vp, i32, vp, vp]
        L.moe_router_logits.restype = C.c_int
        L.moe_route_topk.argtypes = [vp, i32, i32, i32, vp, vp, vp]
        L.moe_route_topk.restype = C.c_int
        L.moe_expert_plan.argtypes = [vp, i32, i32, i32, C.POINTER(PlanStruct), vp]
        L.moe_expert_plan.restype = C.c_int
        L.moe_route_plan.argtypes = [vp, i32, i32, i32, vp, vp, C.POINTER(PlanStruct), vp]
        L.moe_route_plan.restype = C.c_int
        L.moe_workspace_size.argtypes = [C.POINTER(LayerStruct), i32]
        L.moe_workspace_size.restype = C.c_size_t
        L.moe_decode_step.argtypes = [C.POINTER(LayerStruct), vp, i32, vp, vp, C.POINTER(PlanStruct),
                                      vp, vp, C.c_size_t, vp]
        L.moe_decode_step.restype = C.c_int
        L.moe_decode_step_residual.argtypes = [C.POINTER(LayerStruct), vp, i32, vp, vp, C.POINTER(PlanStruct),
                                               vp, vp, vp, C.c_size_t, vp]
        L.moe_decode_step_residual.restype = C.c_int
        L.moe_decode_layer.argtypes = [C.POINTER(LayerStruct), vp, vp, i32, vp, vp, C.POINTER(PlanStruct),
                                       vp, vp, vp, C.c_size_t, vp]
        L.moe_decode_layer.restype = C.c_int
        L.moe_decode_layer_static.argtypes = [C.POINTER(LayerStruct), vp, vp, i32, vp, vp, C.POINTER(PlanStruct),
                                              vp, vp, vp]
        L.moe_decode_layer_static.restype = C.c_int
        L.moe_route_gate_up.argtypes = [C.POINTER(LayerStruct), vp, vp, i32, vp, vp, C.POINTER(PlanStruct),
                                        vp, C.c_size_t, vp]
        L.moe_route_gate_up.restype = C.c_int
        L.moe_expert_gate_up.argtypes = [C.POINTER(LayerStruct), vp, i32, C.POINTER(PlanStruct), vp,
                                         C.c_size_t, vp]
        L.moe_expert_gate_up.restype = C.c_int
        L.moe_expert_down_combine.argtypes = [C.POINTER(LayerStruct), i32, vp, vp, C.POINTER(PlanStruct), vp,
                                              vp, vp, C.c_size_t, vp]
        L.moe_expert_down_combine.restype = C.c_int
        L.moe_pack_down.argtypes = [C.POINTER(LayerStruct), vp, vp, vp, vp]
        L.moe_pack_down.restype = C.c_int
        L.moe_layer_check.argtypes = [C.POINTER(LayerStruct)]
        L.moe_layer_check.restype = C.c_int
        i64, lp = C.c_int64, C.POINTER(LinearStruct)
        L.moe_linear_check.argtypes = [lp]
        L.moe_linear_check.restype = C.c_int
        L.moe_matmul_workspace_size.argtypes = [lp, i32]
        L.moe_matmul_workspace_size.restype = C.c_size_t
        L.moe_grouped_workspace_size.argtypes = [lp, i32]
        L.moe_grouped_workspace_size.restype = C.c_size_t
        L.moe_matmul.argtypes = [lp, vp, i64, i32, vp, i32, i64, vp, i64, vp, C.c_size_t, vp]
        L.moe_matmul.restype = C.c_int
        L.moe_grouped_matmul.argtypes = [lp, vp, i64, i32, i32, i32, C.POINTER(PlanStruct), vp, i64, vp, C.c_size_t,
                                         vp]
        L.moe_grouped_matmul.restype = C.c_int
        L.moe_combine.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, i32, vp, i32, vp]
        L.moe_combine.restype = C.c_int
        L.moe_status_str.argtypes = [C.c_int]
        L.moe_status_str.restype = C.c_char_p
        L.moe_abi_version.argtypes = []
        L.moe_abi_version.restype = C.c_int32
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().moe_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


# ------------------------------------------------------- argument checks
# The C ABI validates everything it can see on the host (shapes in the layer
# struct, alignment, workspace size); the extents and dtypes of the device
# buffers it is handed are the caller's contract.  These checks hold every
# tensor to that contract before the call, so a wrong-sized buffer raises
# here instead of reaching a kernel.
def _act_dtype(layer: "DeviceLayer"):
    return torch.bfloat16 if layer.act_dtype == MOE_DTYPE_BF16 else torch.float32


def _need(t: Optional[torch.Tensor], name: str, dtype, shape):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous {dtype} device tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _check_x(layer: "DeviceLayer", x: torch.Tensor, name: str = "x") -> int:
    if x is None or x.dim() != 2:
        raise ValueError(f"{name} must be a [B, hidden] tensor")
    _need(x, name, _act_dtype(layer), (x.shape[0], layer.hidden))
    return x.shape[0]


def _check_routing(layer: "DeviceLayer", B: int, idx: torch.Tensor, w: torch.Tensor):
    _need(idx, "idx", torch.int32, (B, layer.top_k))
    _need(w, "w", torch.float32, (B, layer.top_k))


def _check_plan_buffers(plan: "Plan", n_experts: int, n_slots: int):
    E = n_experts
    if (plan.counts.numel() < E or plan.offsets.numel() < E + 1 or plan.unique_experts.numel() < E
            or plan.work.numel() < 4 * E or plan.sorted_slots.numel() < n_slots or plan.n_unique.numel() < 1):
        raise ValueError("plan buffers are too small for this layer and batch")
    for t in (plan.counts, plan.offsets, plan.sorted_slots, plan.unique_experts, plan.n_unique, plan.work):
        if t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("plan buffers must be contiguous int32 device tensors")


def _check_plan(layer: "DeviceLayer", plan: "Plan", B: int):
    _check_plan_buffers(plan, layer.n_experts, B * layer.top_k)


def _check_logits(logits: torch.Tensor):
    if (logits is None or logits.dtype != torch.float32 or logits.dim() != 2 or not logits.is_contiguous()
            or not logits.is_cuda):
        raise ValueError("logits must be a contiguous fp32 [B, E] device tensor")


def _check_out(layer: "DeviceLayer", B: int, out: torch.Tensor, residual: Optional[torch.Tensor]):
    _need(out, "out", _act_dtype(layer), (B, layer.hidden))
    if residual is not None:
        _need(residual, "residual", _act_dtype(layer), (B, layer.hidden))


def _check_workspace(layer: "DeviceLayer", B: int, workspace: torch.Tensor):
    if workspace is None or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    need = workspace_size(layer, B)
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace holds {have} bytes, {need} needed for {B} tokens")


# ------------------------------------------------------------------- layer
@dataclass
class DeviceLayer:
    """Device tensors of one layer plus the ABI descriptor pointing at them."""

    hidden: int
    dff: int
    n_experts: int
    top_k: int
    act_dtype: int
    clamp_limit: float
    tensors: dict
    struct: LayerStruct
    down_layout: int = MOE_DOWN_ROWS
    activation: str = "swiglu"
    bits: int = 4
    down_bits: int = 4
    group_size: int = 64

    @staticmethod
    def from_tensors(hidden, dff, n_experts, top_k, act: str, clamp_limit: float, tensors: dict,
                     down_layout: int = MOE_DOWN_ROWS, activation: str = "swiglu", bits: int = 4,
                     down_bits: int = 4, group_size: int = 64):
        """``tensors``: gate_q/up_q/down_q (int32 or uint32 words), *_s/*_b (fp16 bits as
        int16/uint16), optional 'sidecar' (fp32 [E], on gate and up) and 'down_sidecar'
        (fp32 [E], on the down output); all on the same device.  ``activation`` is
        "swiglu" or "geglu"; ``bits`` (gate/up) and ``down_bits`` are 4, 6 or 8,
        ``group_size`` 32, 64 or 128."""
        if activation not in _ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}")
        t = {k: v for k, v in tensors.items() if v is not None}
        for k, v in t.items():
            if not v.is_contiguous():
                raise ValueError(f"{k} must be contiguous")
        st = LayerStruct(hidden=hidden, dff=dff, n_experts=n_experts, top_k=top_k, bits=bits,
                         group_size=group_size, act_dtype=MOE_DTYPE_BF16 if act == "bf16" else MOE_DTYPE_F32,
                         clamp_limit=float(clamp_limit), down_layout=down_layout,
                         activation=_ACTIVATIONS[activation], down_bits=down_bits)
        for name in ("gate_q", "up_q", "down_q", "gate_s", "gate_b", "up_s", "up_b", "down_s", "down_b"):
            setattr(st, name, t[name].data_ptr())
        sc = t.get("sidecar")
        st.expert_scale = None if sc is None else sc.data_ptr()
        ds = t.get("down_sidecar")
        st.down_scale = None if ds is None else ds.data_ptr()
        return DeviceLayer(hidden, dff, n_experts, top_k, st.act_dtype, float(clamp_limit), t, st, down_layout,
                           activation, bits, down_bits, group_size)

    def pack_down(self, stream=None, free_rows: bool = False) -> "DeviceLayer":
        """A copy of this layer whose down projection is regrouped to MOE_DOWN_COLS
        (moe_pack_down); gate/up and the sidecars are shared."""
        if self.down_layout != MOE_DOWN_ROWS:
            raise ValueError("the down projection is already packed")
        t = dict(self.tensors)
        q = torch.empty_like(t["down_q"])
        s = torch.empty_like(t["down_s"])
        b = torch.empty_like(t["down_b"])
        _check(lib().moe_pack_down(C.byref(self.struct), _ptr(q), _ptr(s), _ptr(b), _stream(stream)),
               "moe_pack_down")
        if free_rows:
            torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()
        t["down_q"], t["down_s"], t["down_b"] = q, s, b
        act = "bf16" if self.act_dtype == MOE_DTYPE_BF16 else "f32"
        return DeviceLayer.from_tensors(self.hidden, self.dff, self.n_experts, self.top_k, act, self.clamp_limit,
                                        t, down_layout=MOE_DOWN_COLS, activation=self.activation, bits=self.bits,
                                        down_bits=self.down_bits, group_size=self.group_size)

    @staticmethod
    def from_host(layer, device="cuda"):
        """Copy a ``moe_workloads.Layer`` (numpy) to the device."""
        import numpy as np

        def dev(a, dt):
            return torch.from_numpy(np.ascontiguousarray(a).view(dt)).to(device)

        sh = layer.shape
        t = {}
        for n in ("gate_q", "up_q", "down_q"):
            t[n] = dev(getattr(layer, n), np.int32)
        for n in ("gate_s", "gate_b", "up_s", "up_b", "down_s", "down_b"):
            t[n] = dev(getattr(layer, n), np.int16)
        t["sidecar"] = None if layer.sidecar is None else dev(layer.sidecar.astype(np.float32), np.float32)
        t["down_sidecar"] = (None if layer.down_sidecar is None
                             else dev(layer.down_sidecar.astype(np.float32), np.float32))
        return DeviceLayer.from_tensors(sh.hidden, sh.dff, sh.n_experts, sh.top_k, sh.act,
                                        layer.clamp or 0.0, t, activation=layer.activation, bits=sh.bits,
                                        down_bits=sh.down_bits, group_size=sh.group_size)

    def check(self) -> int:
        return lib().moe_layer_check(C.byref(self.struct))


# -------------------------------------------------------------------- plan
@dataclass
class Plan:
    counts: torch.Tensor
    offsets: torch.Tensor
    sorted_slots: torch.Tensor
    unique_experts: torch.Tensor
    n_unique: torch.Tensor
    work: torch.Tensor
    struct: PlanStruct

    @staticmethod
    def allocate(n_experts: int, max_slots: int, device="cuda") -> "Plan":
        i32 = dict(dtype=torch.int32, device=device)
        p = [torch.empty(n_experts, **i32), torch.empty(n_experts + 1, **i32),
             torch.empty(max(max_slots, 1), **i32), torch.empty(n_experts, **i32), torch.empty(1, **i32),
             torch.empty((n_experts, 4), **i32)]
        st = PlanStruct(*[x.data_ptr() for x in p])
        return Plan(*p, st)


# ------------------------------------------------------------- entry points
def router_logits(x: torch.Tensor, w_router: torch.Tensor, logits: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """moe_router_logits: x [B,H] (bf16 or fp32), w_router bf16 [E,H] -> fp32 logits [B,E]."""
    if x.dim() != 2 or not x.is_contiguous() or x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be a contiguous bf16 or fp32 [B, H] tensor")
    if w_router.dim() != 2 or not w_router.is_contiguous() or w_router.dtype != torch.bfloat16:
        raise ValueError("w_router must be a contiguous bf16 [E, H] tensor")
    B, H = x.shape
    E = w_router.shape[0]
    if w_router.shape[1] != H:
        raise ValueError("x and w_router disagree on hidden")
    if logits is None:
        logits = torch.empty((B, E), dtype=torch.float32, device=x.device)
    act = MOE_DTYPE_BF16 if x.dtype == torch.bfloat16 else MOE_DTYPE_F32
    _check(lib().moe_router_logits(_ptr(x), B, H, act, _ptr(w_router), E, _ptr(logits), _stream(stream)),
           "moe_router_logits")
    return logits


def route_topk(logits: torch.Tensor, top_k: int, idx: Optional[torch.Tensor] = None,
               w: Optional[torch.Tensor] = None, stream=None):
    """moe_route_topk: fp32 logits [B,E] -> (int32 idx [B,k], fp32 w [B,k])."""
    _check_logits(logits)
    B, E = logits.shape
    if idx is None:
        idx = torch.empty((B, top_k), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((B, top_k), dtype=torch.float32, device=logits.device)
    _need(idx, "idx", torch.int32, (B, top_k))
    _need(w, "w", torch.float32, (B, top_k))
    _check(lib().moe_route_topk(_ptr(logits), B, E, top_k, _ptr(idx), _ptr(w), _stream(stream)),
           "moe_route_topk")
    return idx, w


def expert_plan(idx: torch.Tensor, n_experts: int, plan: Optional[Plan] = None, stream=None) -> Plan:
    """moe_expert_plan over int32 idx [B,k]."""
    if idx.dtype != torch.int32 or idx.dim() != 2 or not idx.is_contiguous() or not idx.is_cuda:
        raise ValueError("idx must be a contiguous int32 [B, k] device tensor")
    B, k = idx.shape
    if plan is None:
        plan = Plan.allocate(n_experts, B * k, device=idx.device)
    _check_plan_buffers(plan, n_experts, B * k)
    _check(lib().moe_expert_plan(_ptr(idx), B, n_experts, k, C.byref(plan.struct), _stream(stream)),
           "moe_expert_plan")
    return plan


def route_plan(logits: torch.Tensor, top_k: int, plan: Optional[Plan] = None, idx: Optional[torch.Tensor] = None,
               w: Optional[torch.Tensor] = None, stream=None):
    """moe_route_plan: router and planner in one launch; returns (idx, w, plan)."""
    _check_logits(logits)
    B, E = logits.shape
    if idx is None:
        idx = torch.empty((B, top_k), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((B, top_k), dtype=torch.float32, device=logits.device)
    if plan is None:
        plan = Plan.allocate(E, B * top_k, device=logits.device)
    _need(idx, "idx", torch.int32, (B, top_k))
    _need(w, "w", torch.float32, (B, top_k))
    _check_plan_buffers(plan, E, B * top_k)
    _check(lib().moe_route_plan(_ptr(logits), B, E, top_k, _ptr(idx), _ptr(w), C.byref(plan.struct),
                                _stream(stream)), "moe_route_plan")
    return idx, w, plan


def workspace_size(layer: DeviceLayer, max_tokens: int) -> int:
    return int(lib().moe_workspace_size(C.byref(layer.struct), int(max_tokens)))


def alloc_workspace(layer: DeviceLayer, max_tokens: int, device="cuda") -> torch.Tensor:
    n = workspace_size(layer, max_tokens)
    if n == 0 and max_tokens > 0:
        raise MoeError(layer.check() or MOE_ERR_INVALID_ARG, "moe_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def decode_step(layer: DeviceLayer, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, plan: Plan,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_decode_step: x [B,H] (bf16 or fp32 per the layer) -> out [B,H];
    with a residual, moe_decode_step_residual (out = residual + the block)."""
    B = _check_x(layer, x)
    _check_routing(layer, B, idx, w)
    _check_plan(layer, plan, B)
    if out is None:
        out = torch.empty_like(x)
    _check_out(layer, B, out, residual)
    if workspace is None:
        workspace = alloc_workspace(layer, B, device=x.device)
    _check_workspace(layer, B, workspace)
    if residual is None:
        _check(lib().moe_decode_step(C.byref(layer.struct), _ptr(x), B, _ptr(idx), _ptr(w), C.byref(plan.struct),
                                     _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
               "moe_decode_step")
    else:
        _check(lib().moe_decode_step_residual(C.byref(layer.struct), _ptr(x), B, _ptr(idx), _ptr(w),
                                              C.byref(plan.struct), _ptr(residual), _ptr(out), _ptr(workspace),
                                              workspace.numel(), _stream(stream)), "moe_decode_step_residual")
    return out


def route_gate_up(layer: DeviceLayer, x: torch.Tensor, logits: torch.Tensor, idx: torch.Tensor, w: torch.Tensor,
                  plan: Plan, workspace: torch.Tensor, stream=None):
    """moe_route_gate_up: first half of decode_layer (routing, plan, h into the workspace)."""
    B = _check_x(layer, x)
    _need(logits, "logits", torch.float32, (B, layer.n_experts))
    _check_routing(layer, B, idx, w)
    _check_plan(layer, plan, B)
    _check_workspace(layer, B, workspace)
    _check(lib().moe_route_gate_up(C.byref(layer.struct), _ptr(logits), _ptr(x), x.shape[0], _ptr(idx), _ptr(w),
                                   C.byref(plan.struct), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_route_gate_up")
    return idx, w, plan


def expert_gate_up(layer: DeviceLayer, x: torch.Tensor, plan: Plan, workspace: torch.Tensor, stream=None):
    """moe_expert_gate_up: first half of decode_step (h into the workspace)."""
    B = _check_x(layer, x)
    _check_plan(layer, plan, B)
    _check_workspace(layer, B, workspace)
    _check(lib().moe_expert_gate_up(C.byref(layer.struct), _ptr(x), x.shape[0], C.byref(plan.struct),
                                    _ptr(workspace), workspace.numel(), _stream(stream)), "moe_expert_gate_up")


def expert_down_combine(layer: DeviceLayer, n_tokens: int, idx: torch.Tensor, w: torch.Tensor, plan: Plan,
                        out: torch.Tensor, workspace: torch.Tensor, residual: Optional[torch.Tensor] = None,
                        stream=None):
    """moe_expert_down_combine: second half of decode_step."""
    B = int(n_tokens)
    _check_routing(layer, B, idx, w)
    _check_plan(layer, plan, B)
    _check_out(layer, B, out, residual)
    _check_workspace(layer, B, workspace)
    _check(lib().moe_expert_down_combine(C.byref(layer.struct), n_tokens, _ptr(idx), _ptr(w), C.byref(plan.struct),
                                         _ptr(residual), _ptr(out), _ptr(workspace), workspace.numel(),
                                         _stream(stream)), "moe_expert_down_combine")
    return out


def decode_layer(layer: DeviceLayer, x: torch.Tensor, logits: torch.Tensor, plan: Optional[Plan] = None,
                 workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 residual: Optional[torch.Tensor] = None, bufs: Optional[dict] = None, stream=None):
    """moe_decode_layer: one layer step from router logits (router, planner,
    expert block); returns (out, idx, w, plan)."""
    B = _check_x(layer, x)
    E = layer.n_experts
    _need(logits, "logits", torch.float32, (B, E))
    bufs = bufs or {}
    k = layer.top_k
    idx = bufs.get("idx")
    w = bufs.get("w")
    if idx is None:
        idx = torch.empty((B, k), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((B, k), dtype=torch.float32, device=logits.device)
    if plan is None:
        plan = Plan.allocate(E, B * k, device=logits.device)
    _check_routing(layer, B, idx, w)
    _check_plan(layer, plan, B)
    if out is None:
        out = torch.empty_like(x)
    _check_out(layer, B, out, residual)
    if workspace is None:
        workspace = alloc_workspace(layer, B, device=x.device)
    _check_workspace(layer, B, workspace)
    _check(lib().moe_decode_layer(C.byref(layer.struct), _ptr(logits), _ptr(x), B, _ptr(idx), _ptr(w),
                                  C.byref(plan.struct), _ptr(residual), _ptr(out), _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "moe_decode_layer")
    return out, idx, w, plan


def decode_layer_static(layer: DeviceLayer, x: torch.Tensor, logits: torch.Tensor, plan: Plan, out: torch.Tensor,
                        idx: torch.Tensor, w: torch.Tensor, residual: Optional[torch.Tensor] = None, stream=None):
    """moe_decode_layer_static: moe_decode_layer without a workspace (the library's
    per-device scratch array holds h and y).  Every buffer is the caller's:
    nothing is allocated here either."""
    B = _check_x(layer, x)
    _need(logits, "logits", torch.float32, (B, layer.n_experts))
    _check_routing(layer, B, idx, w)
    _check_plan(layer, plan, B)
    _check_out(layer, B, out, residual)
    _check(lib().moe_decode_layer_static(C.byref(layer.struct), _ptr(logits), _ptr(x), B, _ptr(idx), _ptr(w),
                                         C.byref(plan.struct), _ptr(residual), _ptr(out), _stream(stream)),
           "moe_decode_layer_static")
    return out


# --------------------------------------------------- unquantised products
# These run on the current stream of the tensors' own device (or on `stream`),
# whichever device is current, and what they allocate belongs to that stream.
# They sit on the path of every decoded token, where the host's time per call
# is longer than a small product's on the device: the checks of a call that fits are
# one pass of comparisons, and a message is put together only for one that does not.
@dataclass
class Linear:
    """Weights of a product plus the ABI descriptor (moe_linear_t) pointing at them."""

    w: torch.Tensor
    w_up: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]
    bias_up: Optional[torch.Tensor]
    in_features: int
    out_features: int
    n_groups: int
    out_dtype: torch.dtype
    struct: LinearStruct

    def __post_init__(self):
        self.dtype, self.device, self.index = self.w.dtype, self.w.device, self.w.get_device()
        self._ref = C.byref(self.struct)

    @staticmethod
    def from_tensors(w: torch.Tensor, bias: Optional[torch.Tensor] = None, w_up: Optional[torch.Tensor] = None,
                     bias_up: Optional[torch.Tensor] = None, activation: str = "none",
                     out_dtype: Optional[torch.dtype] = None, clamp_limit: float = 0.0) -> "Linear":
        """``w``: [out, in], or [experts, out, in] for grouped_matmul, bf16, fp16 or fp32, each
        row contiguous; ``w_up`` (same shape and strides) makes the product gated.  ``bias`` and
        ``bias_up``: [out] or [experts, out].  ``activation``: none, relu, silu, gelu or
        gelu_tanh.  ``out_dtype`` defaults to the weights' type.  The tensors are used in place
        and kept alive by this object."""
        if activation not in _FNS:
            raise ValueError(f"activation must be one of {sorted(_FNS)}")
        if clamp_limit > 0 and C.c_float(clamp_limit).value == 0:
            raise ValueError("clamp_limit is too small for fp32, where it would be zero and mean none")
        if w is None or w.dim() not in (2, 3) or w.dtype not in _DTYPES or not w.is_cuda or w.numel() == 0:
            raise ValueError("w must be a non-empty [out, in] or [experts, out, in] bf16, fp16 or fp32 device tensor")
        out_dtype = w.dtype if out_dtype is None else out_dtype
        if out_dtype not in _DTYPES:
            raise ValueError("out_dtype must be bf16, fp16 or fp32")
        if (bias_up is not None) != (bias is not None and w_up is not None):
            raise ValueError("bias_up goes with bias and w_up")
        N, K = w.shape[-2:]
        E = w.shape[0] if w.dim() == 3 else 1
        if max(N, K, E) > _INT32_MAX:
            raise ValueError("the sizes of w must fit 32 bits")
        if K > 1 and w.stride(-1) != 1:
            raise ValueError("the rows of w must be contiguous")
        if w_up is not None and (w_up.shape != w.shape or w_up.dtype != w.dtype or w_up.device != w.device
                                 or any(n > 1 and a != b for n, a, b in zip(w.shape, w.stride(), w_up.stride()))):
            raise ValueError("w_up must match w in shape, type, device and strides")
        for b in (bias, bias_up):
            if b is None:
                continue
            if b.shape != w.shape[:-1] or b.dtype != w.dtype or b.device != w.device or (N > 1 and b.stride(-1) != 1):
                raise ValueError("a bias must be [out] or [experts, out] of w's type and device, rows contiguous")
            if b.dim() == 2 and E > 1 and b.stride(0) != bias.stride(0):
                raise ValueError("bias and bias_up must have the same strides")
        row = w.stride(-2) if N > 1 else K
        group = w.stride(0) if E > 1 else 0
        bias_group = bias.stride(0) if bias is not None and E > 1 else 0
        if row < K or (E > 1 and group <= 0) or (bias is not None and E > 1 and bias_group <= 0):
            raise ValueError("expanded (broadcast) weights have no layout here")
        st = LinearStruct(in_features=K, out_features=N, n_groups=E, dtype=_DTYPES[w.dtype],
                          out_dtype=_DTYPES[out_dtype], fn=_FNS[activation], clamp_limit=float(clamp_limit),
                          w=w.data_ptr(), w_up=None if w_up is None else w_up.data_ptr(),
                          bias=None if bias is None else bias.data_ptr(),
                          bias_up=None if bias_up is None else bias_up.data_ptr(),
                          row_stride=row, group_stride=group, bias_stride=bias_group)
        lin = Linear(w, w_up, bias, bias_up, K, N, E, out_dtype, st)
        _check(lin.check(), "moe_linear_check")
        return lin

    def check(self) -> int:
        return lib().moe_linear_check(C.byref(self.struct))


def matmul_workspace_size(linear: Linear, max_rows: int) -> int:
    return int(lib().moe_matmul_workspace_size(C.byref(linear.struct), _int32("max_rows", max_rows)))


def grouped_workspace_size(linear: Linear, max_slots: int) -> int:
    return int(lib().moe_grouped_workspace_size(C.byref(linear.struct), _int32("max_slots", max_slots)))


def _alloc_bytes(n: int, device) -> Optional[torch.Tensor]:
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def alloc_matmul_workspace(linear: Linear, max_rows: int) -> Optional[torch.Tensor]:
    """The workspace matmul needs for up to max_rows rows; None when it needs none."""
    return _alloc_bytes(matmul_workspace_size(linear, max_rows), linear.w.device)


def alloc_grouped_workspace(linear: Linear, max_slots: int) -> Optional[torch.Tensor]:
    """The workspace grouped_matmul needs for up to max_slots slots; None when it needs none."""
    return _alloc_bytes(grouped_workspace_size(linear, max_slots), linear.w.device)


# The calls beneath torch.cuda's own, for the path of every call; builds of torch without a
# GPU lack them, and only calls on device tensors get to use either.
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _on(device: torch.device, stream, call):
    """call(stream handle) with `device` current and `stream` (default: that device's
    current one) the stream that allocations belong to."""
    if stream is None:
        with torch.cuda.device(device):
            return call(_raw_stream(device.index))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _strides(t: torch.Tensor, rows: int, cols: int, name: str) -> int:
    """Elements between the rows of a [rows, cols] tensor with contiguous rows, 0 when it has one row."""
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if rows <= 1:
        return 0
    if s0 < cols:
        raise ValueError(f"the rows of {name} overlap (an expanded tensor?)")
    return s0


# The ABI's sizes are 32 bits wide, and ctypes would pass the low 32 of a longer one.
_INT32_MAX = 0x7FFFFFFF


def _int32(name: str, n: int) -> int:
    n = int(n)
    if not -_INT32_MAX <= n <= _INT32_MAX:
        raise ValueError(f"{name} must fit 32 bits")
    return n


def _refuse(name: str, t: torch.Tensor, rows, cols: int, dtype, device):
    raise ValueError(f"{name} must be a {dtype} [{rows}, {cols}] tensor on {device}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _workspace(workspace: Optional[torch.Tensor], need, linear: Linear, rows: int):
    """The caller's workspace, or one allocated for the call where it needs one."""
    if workspace is None:
        return _alloc_bytes(need(linear._ref, rows), linear.device)
    if workspace.device != linear.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {linear.device}")
    return workspace


def matmul(linear: Linear, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_matmul: x [rows, in] -> out [rows, out] = residual + f(x w^T + bias), f gated when the
    linear has w_up.  Rows of x, residual and out may be strided; residual is any of the three
    types; out may be residual itself."""
    if stream is not None or _get_device() != linear.index:
        return _on(linear.device, stream, lambda handle: _matmul(linear, x, residual, out, workspace, handle))
    return _matmul(linear, x, residual, out, workspace, _raw_stream(linear.index))


def _matmul(linear, x, residual, out, workspace, handle):
    device, index, K, N = linear.device, linear.index, linear.in_features, linear.out_features
    if x.dim() != 2 or x.shape[1] != K or x.dtype is not linear.dtype or x.get_device() != index:
        _refuse("x", x, "rows", K, linear.dtype, device)
    rows = x.shape[0]
    if rows > _INT32_MAX:
        raise ValueError(f"x has {rows} rows, more than fit 32 bits")
    res = None
    res_type = res_stride = 0
    if residual is not None:
        res_type = _DTYPES.get(residual.dtype)
        if residual.shape != (rows, N) or residual.get_device() != index or res_type is None:
            _refuse("residual", residual, rows, N, "bf16, fp16 or fp32", device)
        res, res_stride = residual.data_ptr(), _strides(residual, rows, N, "residual")
    if out is None:
        out = torch.empty((rows, N), dtype=linear.out_dtype, device=device)
    elif out.shape != (rows, N) or out.dtype is not linear.out_dtype or out.get_device() != index:
        _refuse("out", out, rows, N, linear.out_dtype, device)
    L = lib()
    ws = _workspace(workspace, L.moe_matmul_workspace_size, linear, rows)
    st = L.moe_matmul(linear._ref, x.data_ptr(), _strides(x, rows, K, "x"), rows, res, res_type, res_stride,
                      out.data_ptr(), _strides(out, rows, N, "out"), None if ws is None else ws.data_ptr(),
                      0 if ws is None else ws.numel() * ws.element_size(), handle)
    if st:
        raise MoeError(st, "moe_matmul")
    return out


def grouped_matmul(linear: Linear, x: torch.Tensor, plan: Plan, n_slots: int, top_k: int = 1, rows: str = "token",
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """moe_grouped_matmul over a plan of n_slots slots: out [n_slots, out].  ``rows``: "token" (x has a
    row per token, slot s reads row s // top_k), "slot" (x has a row per slot) or "sorted"
    (rows of x and out lie grouped by expert, in the plan's order).  Rows of slots that the
    plan does not list are left as they are (unset when out is allocated here)."""
    n_slots, top_k = int(n_slots), int(top_k)
    if stream is not None or _get_device() != linear.index:
        return _on(linear.device, stream,
                   lambda handle: _grouped(linear, x, plan, n_slots, top_k, rows, out, workspace, handle))
    return _grouped(linear, x, plan, n_slots, top_k, rows, out, workspace, _raw_stream(linear.index))


def _grouped(linear, x, plan, n_slots, top_k, rows, out, workspace, handle):
    device, index, K, N = linear.device, linear.index, linear.in_features, linear.out_features
    mode = _ROWS.get(rows)
    if mode is None:
        raise ValueError(f"rows must be one of {sorted(_ROWS)}")
    if not 0 <= n_slots <= _INT32_MAX or not 1 <= top_k <= _INT32_MAX:
        raise ValueError("n_slots must be at least 0 and top_k at least 1, and both fit 32 bits")
    if x.dim() != 2 or x.shape[1] != K or x.dtype is not linear.dtype or x.get_device() != index:
        _refuse("x", x, "rows", K, linear.dtype, device)
    x_rows = x.shape[0]
    if x_rows != (-(-n_slots // top_k) if mode == MOE_ROWS_TOKEN else n_slots):
        raise ValueError(f"x has {x_rows} rows, which does not fit {n_slots} slots with rows={rows!r}, top_k={top_k}")
    work, slots = plan.work, plan.sorted_slots
    if work.numel() < 4 * min(linear.n_groups, max(n_slots, 1)) or work.get_device() != index:
        raise ValueError(f"the plan's records are too few for {linear.n_groups} experts or not on {device}")
    if mode != MOE_ROWS_SORTED and (slots.numel() < n_slots or slots.get_device() != index):
        raise ValueError(f"the plan's sorted_slots are fewer than {n_slots} or not on {device}")
    if out is None:
        out = torch.empty((n_slots, N), dtype=linear.out_dtype, device=device)
    elif out.shape != (n_slots, N) or out.dtype is not linear.out_dtype or out.get_device() != index:
        _refuse("out", out, n_slots, N, linear.out_dtype, device)
    L = lib()
    ws = _workspace(workspace, L.moe_grouped_workspace_size, linear, n_slots)
    st = L.moe_grouped_matmul(linear._ref, x.data_ptr(), _strides(x, x_rows, K, "x"), n_slots, top_k, mode,
                              C.byref(plan.struct), out.data_ptr(), _strides(out, n_slots, N, "out"),
                              None if ws is None else ws.data_ptr(),
                              0 if ws is None else ws.numel() * ws.element_size(), handle)
    if st:
        raise MoeError(st, "moe_grouped_matmul")
    return out


def combine(y: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, n_experts: int,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """moe_combine: y [B * k, H], idx int32 [B, k], w fp32 [B, k] -> out [B, H] =
    residual + the weighted sum of each token's k rows.  out_dtype defaults to out's type, else
    the residual's, else y's."""
    index = y.get_device()
    if index < 0:
        raise ValueError("y must be a contiguous bf16, fp16 or fp32 [slots, hidden] device tensor")
    if stream is not None or _get_device() != index:
        return _on(y.device, stream, lambda handle: _combine(y, idx, w, n_experts, residual, out, out_dtype, handle))
    return _combine(y, idx, w, n_experts, residual, out, out_dtype, _raw_stream(index))


def _combine(y, idx, w, n_experts, residual, out, out_dtype, handle):
    device, index, y_type = y.device, y.get_device(), _DTYPES.get(y.dtype)
    if y.dim() != 2 or y_type is None or not y.is_contiguous():
        raise ValueError("y must be a contiguous bf16, fp16 or fp32 [slots, hidden] device tensor")
    H = y.shape[1]
    if idx.dim() != 2 or idx.dtype is not torch.int32 or not idx.is_contiguous() or idx.get_device() != index:
        raise ValueError(f"idx must be a contiguous int32 [B, k] tensor on {device}")
    B, k = idx.shape
    if max(B, k, H, n_experts) > _INT32_MAX or n_experts < -_INT32_MAX:
        raise ValueError("the sizes of y and idx and n_experts must fit 32 bits")
    if w.dtype is not torch.float32 or w.shape != idx.shape or not w.is_contiguous() or w.get_device() != index:
        _refuse("w", w, B, k, "contiguous fp32", device)
    if y.shape[0] != B * k:
        raise ValueError(f"y has {y.shape[0]} rows, {B * k} needed for {B} tokens of {k} slots")
    res, res_type = None, 0
    if residual is not None:
        res_type = _DTYPES.get(residual.dtype)
        if residual.shape != (B, H) or residual.get_device() != index or res_type is None or not residual.is_contiguous():
            _refuse("residual", residual, B, H, "contiguous bf16, fp16 or fp32", device)
        res = residual.data_ptr()
    if out is None:
        if out_dtype is None:
            out_dtype = y.dtype if residual is None else residual.dtype
        out = torch.empty((B, H), dtype=out_dtype, device=device)
    out_type = _DTYPES.get(out.dtype)
    if (out.shape != (B, H) or out.get_device() != index or out_type is None or not out.is_contiguous()
            or (out_dtype is not None and out.dtype is not out_dtype)):
        _refuse("out", out, B, H, f"contiguous {out_dtype or 'bf16, fp16 or fp32'}", device)
    st = lib().moe_combine(y.data_ptr(), y_type, idx.data_ptr(), w.data_ptr(), B, H, k, int(n_experts), res, res_type,
                           out.data_ptr(), out_type, handle)
    if st:
        raise MoeError(st, "moe_combine")
    return out
