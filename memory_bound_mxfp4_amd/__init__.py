"""Python binding of libmoe_mxfp4.so, the MI355X MXFP4 MoE decode-layer library.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Tensors are torch tensors on the GPU (bf16 data may be
torch.bfloat16 or int16/uint16 bit patterns); work goes on the current torch
stream unless a stream is given.  If the library is not built, loading
raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from operator import index as _index
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_mxfp4.so")

MOE_OK, MOE_ERR_INVALID_ARGUMENT, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_DTYPE_BF16, MOE_DTYPE_F32, MOE_DTYPE_F16, MOE_DTYPE_I8, MOE_DTYPE_F8 = 0, 1, 2, 3, 4
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_EXPERTS_CANONICAL, MOE_EXPERTS_PACKED = 0, 1
MAX_BATCH = 64

# Symbols the C header declares (checked by tests/test_abi.py).
EXPORTS = ("moe_expert_bytes", "moe_workspace_size", "moe_router_workspace_size", "router_topk",
           "expert_gemv_mxfp4", "moe_decode_layer", "moe_decode_layer_kernel_count",
           "moe_decode_layer_kernel_name", "moe_decode_layer_timed", "moe_workspace_init", "moe_pack_experts",
           "moe_unpack_experts", "rmsnorm_bf16", "dense_gemv_bf16", "residual_add_bf16", "residual_add_rmsnorm_bf16",
           "moe_workspace_status", "moe_stream_read_probe", "moe_decode_layer_noalloc", "moe_decode_layer_mxfp8",
           "moe_prefetch", "moe_set_max_workgroups", "moe_status_string", "moe_route", "quant_rows_i8",
           "gemm_i8_workspace_size", "gemm_i8", "moe_slot_groups_size", "moe_group_slots",
           "experts_gemm_i8_workspace_size", "experts_gemm_i8", "moe_combine", "quant_rows_f8", "gemm_f8_workspace_size",
           "gemm_f8", "experts_gemm_f8_workspace_size", "experts_gemm_f8", "residual_add_rmsnorm_f8",
           "residual_add_rmsnorm_i8")


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class LayerWeightsC(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("shared_inter", ctypes.c_int32),
                ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("shared_gate", ctypes.c_void_p), ("shared_up", ctypes.c_void_p),
                ("shared_down", ctypes.c_void_p), ("experts", ctypes.c_void_p), ("expert_layout", ctypes.c_int32)]


_lib = None


def load():
    """Load the built library (raises if it is missing: no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run memory_bound_mxfp4_amd.build.build() "
                          "or __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    sig = {
        "moe_expert_bytes": (Z, [I, I]),
        "moe_workspace_size": (I, [P, I, ctypes.POINTER(Z)]),
        "moe_router_workspace_size": (Z, [I, I]),
        "router_topk": (I, [P, I, I, P, P, I, I, P, P, P, P, Z, P]),
        "expert_gemv_mxfp4": (I, [P, P, I, I, P, I, I, P, P]),
        "moe_decode_layer": (I, [P, P, P, I, P, P, P, Z, P]),
        "moe_decode_layer_kernel_count": (I, []),
        "moe_decode_layer_kernel_name": (ctypes.c_char_p, [I]),
        "moe_decode_layer_timed": (I, [P, P, P, I, P, P, P, Z, P, P, I]),
        "moe_workspace_init": (I, [P, Z, P]),
        "moe_pack_experts": (I, [P, I, I, I, P, Z, P]),
        "moe_unpack_experts": (I, [P, I, I, I, P, Z, P]),
        "rmsnorm_bf16": (I, [P, I, I, F, P, P]),
        "dense_gemv_bf16": (I, [P, I, I, P, I, P, P]),
        "residual_add_bf16": (I, [P, P, I, I, P]),
        "residual_add_rmsnorm_bf16": (I, [P, P, I, I, F, P, P]),
        "moe_workspace_status": (I, [P, Z, P, P]),
        "moe_decode_layer_noalloc": (I, [P, P, P, I, P, P, P, P]),
        "moe_decode_layer_mxfp8": (I, [P, P, P, I, P, P, P, Z, P]),
        "moe_prefetch": (I, [P, I, I, P]),
        "moe_set_max_workgroups": (I, [I]),
        "moe_stream_read_probe": (I, [P, Z, I, P, P]),
        "moe_status_string": (ctypes.c_char_p, [I]),
        "moe_route": (I, [P, I, Z, I, P, P, P, P, P]),
        "quant_rows_i8": (I, [P, I, Z, I, I, P, P, P]),
        "gemm_i8_workspace_size": (Z, [I, I, I, I, I]),
        "gemm_i8": (I, [P, I, Z, P, I, I, P, P, I, I, P, I, P, Z, P]),
        "moe_slot_groups_size": (Z, [I, I, I]),
        "moe_group_slots": (I, [P, I, I, I, P, Z, P]),
        "experts_gemm_i8_workspace_size": (Z, [I, I, I, I, I, I, I, I]),
        "experts_gemm_i8": (I, [P, I, Z, P, I, I, P, Z, I, I, I, P, P, I, I, P, I, P, Z, P]),
        "moe_combine": (I, [P, I, P, I, I, I, P, P, P]),
        "quant_rows_f8": (I, [P, I, Z, I, I, P, P, P]),
        "gemm_f8_workspace_size": (Z, [I, I, I, I, I]),
        "gemm_f8": (I, [P, I, Z, P, I, I, P, P, I, I, P, I, P, Z, P]),
        "experts_gemm_f8_workspace_size": (Z, [I, I, I, I, I, I, I, I]),
        "experts_gemm_f8": (I, [P, I, Z, P, I, I, P, Z, I, I, I, P, P, I, I, P, I, P, Z, P]),
        "residual_add_rmsnorm_f8": (I, [P, Z, P, I, Z, P, I, I, F, P, P, P, P, P]),
        "residual_add_rmsnorm_i8": (I, [P, Z, P, I, Z, P, I, I, F, P, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


def _check(rc: int, what: str):
    if rc != MOE_OK:
        raise MoeError(rc, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def expert_bytes(hidden: int, inter: int) -> int:
    return int(load().moe_expert_bytes(hidden, inter))


@dataclass
class LayerWeights:
    """One layer's weights (device tensors) and shape."""
    hidden: int
    inter: int
    num_experts: int
    top_k: int
    shared_inter: int
    router_w: object
    experts: object
    router_bias: Optional[object] = None
    shared_gate: Optional[object] = None
    shared_up: Optional[object] = None
    shared_down: Optional[object] = None
    expert_layout: int = MOE_EXPERTS_CANONICAL

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_cs":
            object.__setattr__(self, "_cs", None)

    def c_struct(self) -> LayerWeightsC:
        cs = getattr(self, "_cs", None)
        if cs is not None:
            return cs
        cs = LayerWeightsC(self.hidden, self.inter, self.num_experts, self.top_k, self.shared_inter,
                             _ptr(self.router_w), _ptr(self.router_bias), _ptr(self.shared_gate),
                             _ptr(self.shared_up), _ptr(self.shared_down), _ptr(self.experts), self.expert_layout)
        object.__setattr__(self, "_cs", cs)
        return cs


def _pack(experts, num_experts: int, hidden: int, inter: int, to_packed: bool, scratch=None, stream=None):
    import torch
    nb = expert_bytes(hidden, inter)
    scratch = torch.empty(nb, dtype=torch.uint8, device=experts.device) if scratch is None else scratch
    f = load().moe_pack_experts if to_packed else load().moe_unpack_experts
    _check(f(_ptr(experts), num_experts, hidden, inter, _ptr(scratch), scratch.numel(), _stream(stream)),
           "moe_pack_experts" if to_packed else "moe_unpack_experts")
    return experts


def pack_experts(experts, num_experts: int, hidden: int, inter: int, scratch=None, stream=None):
    """Rewrite canonical expert blobs in place into the packed layout (moe_pack_experts)."""
    return _pack(experts, num_experts, hidden, inter, True, scratch, stream)


def unpack_experts(experts, num_experts: int, hidden: int, inter: int, scratch=None, stream=None):
    """Inverse of pack_experts (moe_unpack_experts)."""
    return _pack(experts, num_experts, hidden, inter, False, scratch, stream)


def pack_layer(w: LayerWeights, stream=None) -> LayerWeights:
    """Pack a layer's experts in place (once, at load time) and mark them packed."""
    if w.expert_layout != MOE_EXPERTS_PACKED:
        pack_experts(w.experts, w.num_experts, w.hidden, w.inter, stream=stream)
        w.expert_layout = MOE_EXPERTS_PACKED
    return w


def workspace_size(w: LayerWeights, batch: int) -> int:
    n = ctypes.c_size_t(0)
    cs = w.c_struct()
    _check(load().moe_workspace_size(ctypes.byref(cs), batch, ctypes.byref(n)), "moe_workspace_size")
    return int(n.value)


WS_STATUS_OFFSET = 28


def workspace_init(ws, stream=None):
    """Clear a workspace before its first use (moe_workspace_init)."""
    _check(load().moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "moe_workspace_init")
    return ws


def alloc_workspace(w: LayerWeights, batch: int, device=None):
    """A cleared workspace for `w` at `batch` rows."""
    import torch
    ws = torch.empty(workspace_size(w, batch), dtype=torch.uint8, device=device or w.router_w.device)
    return workspace_init(ws)


WS_ACTIVE_EXPERTS_OFFSET = 384


def workspace_status(ws, stream=None) -> int:
    """The workspace's sticky status word (0 = every wait completed), read
    through moe_workspace_status. Synchronises the stream."""
    import torch
    out = torch.zeros(1, dtype=torch.int32, device=ws.device)
    _check(load().moe_workspace_status(_ptr(ws), ws.numel(), _ptr(out), _stream(stream)), "moe_workspace_status")
    torch.cuda.synchronize(ws.device)
    return int(out.item()) & 0xFFFFFFFF


def workspace_active_experts(ws) -> int:
    """Batch > 1: distinct experts the last call on `ws` routed to, as counted
    on the device (low half of the word at WS_ACTIVE_EXPERTS_OFFSET). Synchronises."""
    import numpy as np
    off = WS_ACTIVE_EXPERTS_OFFSET
    return int(ws[off:off + 4].cpu().numpy().view(np.uint32)[0])


def set_max_workgroups(n: int) -> None:
    """Cap the layer kernel's grid at n workgroups (0: the default) -- moe_set_max_workgroups."""
    _check(load().moe_set_max_workgroups(int(n)), "moe_set_max_workgroups")


def stream_read_probe(buf, blocks_per_cu: int = 4, sink=None, stream=None):
    """Enqueue one streaming read of all of `buf` (moe_stream_read_probe)."""
    import torch
    sink = torch.zeros(1, dtype=torch.int32, device=buf.device) if sink is None else sink
    _check(load().moe_stream_read_probe(_ptr(buf), buf.numel() * buf.element_size(), blocks_per_cu, _ptr(sink),
                                        _stream(stream)), "moe_stream_read_probe")
    return sink


def router_topk(x, router_w, top_k: int, bias=None, idx=None, gate=None, logits=None, ws=None, stream=None):
    """Router GEMV + top-k + renormalised gates. Returns (idx int32 [B][k], gate fp32 [B][k])."""
    import torch
    B, H = x.shape
    E = router_w.shape[0]
    dev = x.device
    idx = torch.empty((B, top_k), dtype=torch.int32, device=dev) if idx is None else idx
    gate = torch.empty((B, top_k), dtype=torch.float32, device=dev) if gate is None else gate
    if logits is None and ws is None:
        ws = torch.empty(load().moe_router_workspace_size(B, E), dtype=torch.uint8, device=dev)
    _check(load().router_topk(_ptr(x), B, H, _ptr(router_w), _ptr(bias), E, top_k, _ptr(idx), _ptr(gate),
                              _ptr(logits), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "router_topk")
    return idx, gate


def expert_gemv_mxfp4(codes, scales, x, n: int, k: int, y=None, stream=None):
    """y[b][n] = dequant(codes, scales) . x[b]; x bf16 or fp32 [B][k]. Returns y fp32 [B][n]."""
    import torch
    B = x.shape[0]
    y = torch.empty((B, n), dtype=torch.float32, device=x.device) if y is None else y
    xdt = MOE_DTYPE_F32 if x.dtype == torch.float32 else MOE_DTYPE_BF16
    _check(load().expert_gemv_mxfp4(_ptr(codes), _ptr(scales), n, k, _ptr(x), xdt, B, _ptr(y), _stream(stream)),
           "expert_gemv_mxfp4")
    return y


def moe_decode_layer(w: LayerWeights, x, residual, idx=None, gate=None, ws=None, stream=None, mxfp8=False):
    """The whole layer; `residual` (fp32 [B][H]) is updated in place. Returns (idx, gate).
    mxfp8: the routed experts' FP4 x MXFP8 variant (moe_decode_layer_mxfp8)."""
    import torch
    B = x.shape[0]
    dev = x.device
    idx = torch.empty((B, w.top_k), dtype=torch.int32, device=dev) if idx is None else idx
    gate = torch.empty((B, w.top_k), dtype=torch.float32, device=dev) if gate is None else gate
    ws = alloc_workspace(w, B, dev) if ws is None else ws
    cs = w.c_struct()
    f, name = (load().moe_decode_layer_mxfp8, "moe_decode_layer_mxfp8") if mxfp8 else \
        (load().moe_decode_layer, "moe_decode_layer")
    _check(f(ctypes.byref(cs), _ptr(x), _ptr(residual), B, _ptr(idx), _ptr(gate), _ptr(ws), ws.numel(),
             _stream(stream)), name)
    return idx, gate


NOALLOC_SCRATCH_BYTES = 24 << 20


def moe_decode_layer_noalloc(w: LayerWeights, x, residual, idx, gate, status=None, stream=None):
    """moe_decode_layer on the library's own static device workspace
    (moe_decode_layer_noalloc): nothing is allocated by the call.  idx, gate
    and the optional status word (int32 [1]) are caller-provided device tensors."""
    B = x.shape[0]
    cs = w.c_struct()
    _check(load().moe_decode_layer_noalloc(ctypes.byref(cs), _ptr(x), _ptr(residual), B, _ptr(idx), _ptr(gate),
                                           _ptr(status), _stream(stream)), "moe_decode_layer_noalloc")
    return idx, gate


def layer_kernel_names():
    lib = load()
    return [lib.moe_decode_layer_kernel_name(i).decode() for i in range(lib.moe_decode_layer_kernel_count())]


def moe_decode_layer_timed(w: LayerWeights, x, residual, idx, gate, ws, events, stream=None):
    """moe_decode_layer recording torch.cuda.Event objects around each kernel
    (len(events) == len(layer_kernel_names()) + 1) on `stream`."""
    B = x.shape[0]
    cs = w.c_struct()
    for e in events:  # torch creates the underlying hipEvent_t lazily, on first record
        if not e.cuda_event:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(load().moe_decode_layer_timed(ctypes.byref(cs), _ptr(x), _ptr(residual), B, _ptr(idx), _ptr(gate),
                                         _ptr(ws), ws.numel(), _stream(stream), arr, len(events)),
           "moe_decode_layer_timed")
    return idx, gate


class RangeC(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


PREFETCH_MAX_RANGES = 8


def prefetch(tensors, blocks: int = 256, stream=None):
    """Read device tensors once into the last-level cache (moe_prefetch)."""
    tensors = [t for t in tensors if t is not None]
    arr = (RangeC * len(tensors))(*[RangeC(t.data_ptr(), t.numel() * t.element_size()) for t in tensors])
    _check(load().moe_prefetch(arr, len(tensors), blocks, _stream(stream)), "moe_prefetch")


def rmsnorm_bf16(h, eps: float = 1e-6, out=None, stream=None):
    import torch
    B, H = h.shape
    out = torch.empty((B, H), dtype=torch.bfloat16, device=h.device) if out is None else out
    _check(load().rmsnorm_bf16(_ptr(h), B, H, float(eps), _ptr(out), _stream(stream)), "rmsnorm_bf16")
    return out


def dense_gemv_bf16(w, x, y=None, stream=None):
    import torch
    n, k = w.shape
    B = x.shape[0]
    y = torch.empty((B, n), dtype=torch.bfloat16, device=x.device) if y is None else y
    _check(load().dense_gemv_bf16(_ptr(w), n, k, _ptr(x), B, _ptr(y), _stream(stream)), "dense_gemv_bf16")
    return y


def residual_add_bf16(h, t, stream=None):
    B, H = h.shape
    _check(load().residual_add_bf16(_ptr(h), _ptr(t), B, H, _stream(stream)), "residual_add_bf16")
    return h


def residual_add_rmsnorm_bf16(h, t, eps: float = 1e-6, out=None, stream=None):
    """h += t (in place), then out = bf16(RMSNorm(h)), as one launch."""
    import torch
    B, H = h.shape
    out = torch.empty((B, H), dtype=torch.bfloat16, device=h.device) if out is None else out
    _check(load().residual_add_rmsnorm_bf16(_ptr(h), _ptr(t), B, H, float(eps), _ptr(out), _stream(stream)),
           "residual_add_rmsnorm_bf16")
    return out


# ---- routing, slots by expert, 8-bit products ---------------------------------------------------------------
#
# With `stream` (a torch stream or its address) a call runs there, and the outputs and workspaces it makes belong to
# that stream; what it is given has to be ready there, and what it returns is used elsewhere as any tensor of another
# stream is: behind a wait, and with record_stream if it may be freed while in use.


class RouteParamsC(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


@functools.lru_cache(maxsize=256)
def _route_params(*fields):
    """The C struct of a routing, by reference; a decode step routes the same way again and again. The fields are
    plain numbers: kept by value, not by the identity of what held them."""
    for v in fields[:-1]:
        _int(v, "a parameter of the routing")
    return ctypes.byref(RouteParamsC(*fields))


_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_dtypes: dict = {}


_module = None


def _torch():
    """torch, imported when it is first needed; a statement in each call would cost as much as its checks."""
    global _module
    if _module is None:
        import torch
        _dtypes.update({torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32, torch.float16: MOE_DTYPE_F16})
        _module = torch
    return _module


def _dtype_code(dtype, what: str, int8: bool = False) -> int:
    torch = _torch()
    code = _dtypes.get(dtype)
    if code is not None:
        return code
    if int8 and dtype == torch.int8:
        return MOE_DTYPE_I8
    raise ValueError(f"{what} must be bfloat16, float16 or float32{' or int8' if int8 else ''}, not {dtype}")


def _want(t, shape: tuple, dtype, device, what: str):
    """Checks a tensor that a kernel takes by address: shape, type, device, dense rows one after another."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {shape} on {device}, not "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t


_MAX_INT = 0x7FFFFFFF


def _int(v: int, what: str) -> int:
    """Sizes go to the C interface as 32-bit integers, and a longer one would lose its upper bits on the way."""
    if not -_MAX_INT <= v <= _MAX_INT:
        raise ValueError(f"{what} is out of range: {v}")
    return v


def _rows(t, what: str):
    """Checks a matrix whose rows may lie apart; returns rows, columns and the row stride."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be a matrix")
    rows, cols = t.shape
    if rows > _MAX_INT or cols > _MAX_INT:
        raise ValueError(f"{what} is out of range: {rows} x {cols}")
    if t.is_contiguous():
        return rows, cols, cols
    stride = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or stride < cols:
        raise ValueError(f"{what} must have consecutive elements in a row and rows that do not overlap")
    return rows, cols, stride


def _addr(t):
    return None if t is None else t.data_ptr()


def _empty(shape, dtype, device, stream):
    """Memory for a call on `stream`, from that stream's own pool: what is freed there is used again only behind the
    call, and nothing of another stream still works on it."""
    import torch
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream):
        return torch.empty(shape, dtype=dtype, device=device)


_current: tuple = ()  # torch's raw current stream of a device, and its current device


def _launch(what: str, device, stream, *args):
    """Calls an entry point with `device` current, on the given stream or on that device's current one."""
    global _current
    if device.type != "cuda":
        raise ValueError(f"{what} takes tensors on the GPU, not on {device}")
    if not _current:
        # as current_stream(device) and current_device(), without building a Stream
        _current = (_torch()._C._cuda_getCurrentRawStream, _torch()._C._cuda_getDevice)
    index = device.index
    if stream is None:
        s = _current[0](index)
    else:
        s = stream if isinstance(stream, int) else stream.cuda_stream
    f = getattr(_lib or load(), what)
    if index == _current[1]():
        rc = f(*args, s)
    else:
        with _torch().cuda.device(device):
            rc = f(*args, s)
    if rc != MOE_OK:
        raise MoeError(rc, what)


def moe_route(logits, top_k: int, bias=None, score: str = "softmax", groups: int = 1, top_groups: int = 1,
              group_top: int = 1, renorm: bool = True, scale: float = 1.0, idx=None, gate=None, stream=None):
    """Router logits [rows][E] to experts and gates (moe_route): softmax or sigmoid scores, a bias for the
    selection, groups of experts, renormalised gates. A scale held in a tensor is read in every call, which waits for
    the GPU if it is there. Returns (idx int32 [rows][k], gate fp32 [rows][k])."""
    torch = _torch()
    rows, E, stride = _rows(logits, "logits")
    dev = logits.device
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    code = _dtype_code(logits.dtype, "logits")
    if bias is not None:
        _want(bias, (E,), torch.float32, dev, "bias")
    top_k = _index(top_k)
    p = _route_params(E, top_k, _SCORES[score], _index(groups), _index(top_groups), _index(group_top), int(bool(renorm)),
                      ctypes.c_float(scale).value + 0.0)  # + 0.0: no -0.0, which is the same key as 0.0
    shape = (rows, top_k)
    idx = _empty(shape, torch.int32, dev, stream) if idx is None else _want(idx, shape, torch.int32, dev, "idx")
    gate = _empty(shape, torch.float32, dev, stream) if gate is None else _want(gate, shape, torch.float32, dev, "gate")
    _launch("moe_route", dev, stream, _addr(logits), code, stride, rows, _addr(bias), p, _addr(idx), _addr(gate))
    return idx, gate


def quant_rows_i8(x, q=None, scale=None, stream=None):
    """Rows of x [rows][k] to 8-bit codes with one scale each (quant_rows_i8). Returns (q int8, scale fp32 [rows])."""
    torch = _torch()
    rows, k, stride = _rows(x, "x")
    dev = x.device
    code = _dtype_code(x.dtype, "x")
    q = _empty((rows, k), torch.int8, dev, stream) if q is None else _want(q, (rows, k), torch.int8, dev, "q")
    scale = _empty((rows,), torch.float32, dev, stream) if scale is None else \
        _want(scale, (rows,), torch.float32, dev, "scale")
    _launch("quant_rows_i8", dev, stream, _addr(x), code, stride, rows, k, _addr(q), _addr(scale))
    return q, scale


def gemm_i8_workspace_size(m: int, n: int, k: int, swiglu: bool, x_dtype) -> int:
    for v, what in ((m, "m"), (n, "n"), (k, "k")):
        _int(v, what)
    return int(load().gemm_i8_workspace_size(m, n, k, int(bool(swiglu)), _dtype_code(x_dtype, "x", int8=True)))


def _i8_operands(x, x_scale, w, w_scale, swiglu: bool, lead: tuple):
    """Shape checks shared by the two products; w is lead + [2][n][k] with swiglu, else lead + [n][k]."""
    torch = _torch()
    rows, k, stride = _rows(x, "x")
    dev = x.device
    parts = (2,) if swiglu else ()
    if w.dim() != len(lead) + len(parts) + 2:
        raise ValueError(f"w has {w.dim()} dimensions, not {len(lead) + len(parts) + 2}")
    n = _int(w.shape[-2], "the rows of w")
    _want(w, lead + parts + (n, k), torch.int8, dev, "w")
    _want(w_scale, lead + parts + (n,), torch.float32, dev, "w_scale")
    if (x_scale is not None) != (x.dtype == torch.int8):
        raise ValueError("x_scale goes with int8 rows, and only with them")
    if x_scale is not None:
        _want(x_scale, (rows,), torch.float32, dev, "x_scale")
    return rows, k, stride, n, _dtype_code(x.dtype, "x", int8=True)


def _out(out, shape, out_dtype, device, stream):
    torch = _torch()
    if out is None:
        return _empty(shape, torch.bfloat16 if out_dtype is None else out_dtype, device, stream)
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out is {out.dtype}, not {out_dtype}")
    return _want(out, shape, out.dtype, device, "out")


def _workspace(ws, need: int, device, stream):
    torch = _torch()
    if ws is None:
        return _empty(need, torch.uint8, device, stream) if need else None
    return _want(ws, tuple(ws.shape), torch.uint8, device, "ws")


def gemm_i8(x, w, w_scale, x_scale=None, swiglu: bool = False, out=None, out_dtype=None, ws=None, stream=None):
    """y = x w^T in 8-bit integers (gemm_i8): x [m][k] float rows, quantised on the way, or int8 codes with
    x_scale [m]; w int8 [n][k] with w_scale [n], or [2][n][k] and [2][n] with swiglu. Returns y [m][n] in out's
    type, out_dtype or bfloat16; neither out nor ws overlaps an input."""
    m, k, stride, n, code = _i8_operands(x, x_scale, w, w_scale, swiglu, ())
    dev = x.device
    y = _out(out, (m, n), out_dtype, dev, stream)
    ws = _workspace(ws, 0 if ws is not None else load().gemm_i8_workspace_size(m, n, k, int(bool(swiglu)), code), dev, stream)
    _launch("gemm_i8", dev, stream, _addr(x), code, stride, _addr(x_scale), m, k, _addr(w), _addr(w_scale), n, int(bool(swiglu)),
            _addr(y), _dtype_code(y.dtype, "out"), _addr(ws), 0 if ws is None else ws.numel())
    return y


@dataclass
class SlotGroups:
    """The slots of a routing by expert (moe_group_slots): `order` int32 [tokens * top_k] and `offsets` int32
    [num_experts + 2] are views of `buffer`, which also holds what experts_gemm_i8 works through."""
    tokens: int
    top_k: int
    num_experts: int
    buffer: object
    order: object
    offsets: object


def alloc_slot_groups(tokens: int, top_k: int, num_experts: int, device=None, stream=None) -> SlotGroups:
    import torch
    for v, what in ((tokens, "tokens"), (top_k, "top_k"), (num_experts, "num_experts")):
        _int(v, what)
    size = int(load().moe_slot_groups_size(tokens, top_k, num_experts))
    if not size:
        raise ValueError(f"slot groups of {tokens} tokens, {top_k} slots each and {num_experts} experts are out of range")
    buf = _empty(size, torch.uint8, torch.device("cuda" if device is None else device), stream)
    slots = tokens * top_k
    at = (4 * slots + 255) // 256 * 256
    return SlotGroups(tokens, top_k, num_experts, buf, buf[:4 * slots].view(torch.int32),
                      buf[at:at + 4 * (num_experts + 2)].view(torch.int32))


def moe_group_slots(idx, num_experts: int, groups: Optional[SlotGroups] = None, stream=None) -> SlotGroups:
    """Sort the slots of idx (int32 [tokens][k]) by expert (moe_group_slots)."""
    torch = _torch()
    if idx.dim() != 2:
        raise ValueError("idx must be a matrix")
    tokens, top_k = idx.shape
    _want(idx, (tokens, top_k), torch.int32, idx.device, "idx")
    if groups is None:
        groups = alloc_slot_groups(tokens, top_k, num_experts, idx.device, stream)
    elif (groups.tokens, groups.top_k, groups.num_experts) != (tokens, top_k, num_experts) or \
            groups.buffer.device != idx.device:
        raise ValueError("groups were allocated for another shape or device")
    _launch("moe_group_slots", idx.device, stream, _addr(idx), tokens, top_k, num_experts, _addr(groups.buffer),
            groups.buffer.numel())
    return groups


def experts_gemm_i8_workspace_size(groups: SlotGroups, x_rows: int, n: int, k: int, swiglu: bool, x_dtype) -> int:
    for v, what in ((x_rows, "x_rows"), (n, "n"), (k, "k")):
        _int(v, what)
    return int(load().experts_gemm_i8_workspace_size(groups.tokens, groups.top_k, groups.num_experts, x_rows, n, k,
                                                     int(bool(swiglu)), _dtype_code(x_dtype, "x", int8=True)))


def experts_gemm_i8(x, groups: SlotGroups, w, w_scale, x_scale=None, swiglu: bool = False, out=None, out_dtype=None,
                    ws=None, stream=None):
    """gemm_i8 of every slot with its expert's matrix (experts_gemm_i8): x has a row per token or per slot, w is
    int8 [num_experts][n][k] (or [num_experts][2][n][k] with swiglu). Returns y [tokens * top_k][n]."""
    E = groups.num_experts
    rows, k, stride, n, code = _i8_operands(x, x_scale, w, w_scale, swiglu, (E,))
    dev = x.device
    if rows != groups.tokens and rows != groups.tokens * groups.top_k:
        raise ValueError(f"x has {rows} rows, neither the tokens nor the slots of the groups")
    if groups.buffer.device != dev:
        raise ValueError("groups are on another device")
    y = _out(out, (groups.tokens * groups.top_k, n), out_dtype, dev, stream)
    need = 0 if ws is not None else load().experts_gemm_i8_workspace_size(groups.tokens, groups.top_k, E, rows, n, k,
                                                                          int(bool(swiglu)), code)
    ws = _workspace(ws, need, dev, stream)
    _launch("experts_gemm_i8", dev, stream, _addr(x), code, stride, _addr(x_scale), rows, k, _addr(groups.buffer),
            groups.buffer.numel(), groups.tokens, groups.top_k, E, _addr(w), _addr(w_scale), n, int(bool(swiglu)), _addr(y),
            _dtype_code(y.dtype, "out"), _addr(ws), 0 if ws is None else ws.numel())
    return y


def moe_combine(y, gate, residual=None, out=None, stream=None):
    """out[t] = residual[t] + sum_j gate[t][j] * y[t * k + j] (moe_combine), fp32 [tokens][hidden]; out may be
    residual itself. Returns out."""
    torch = _torch()
    tokens, top_k = gate.shape
    hidden = y.shape[-1]
    if tokens > _MAX_INT or hidden > _MAX_INT:
        raise ValueError(f"{tokens} tokens of {hidden} columns are out of range")
    dev = y.device
    _want(gate, (tokens, top_k), torch.float32, dev, "gate")
    _want(y, (tokens * top_k, hidden), y.dtype, dev, "y")
    shape = (tokens, hidden)
    if residual is not None:
        _want(residual, shape, torch.float32, dev, "residual")
    out = _empty(shape, torch.float32, dev, stream) if out is None else _want(out, shape, torch.float32, dev, "out")
    _launch("moe_combine", dev, stream, _addr(y), _dtype_code(y.dtype, "y"), _addr(gate), tokens, top_k, hidden,
            _addr(residual), _addr(out))
    return out


# ---- 8-bit floating point: e4m3 codes with a scale for each block of 128 -----------------------------------------------

BLOCK = 128


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _f8_code(dtype) -> int:
    return MOE_DTYPE_F8 if dtype == _torch().float8_e4m3fn else _dtype_code(dtype, "x")


def quant_rows_f8(x, q=None, scale=None, stream=None):
    """Rows of x [rows][k] to e4m3 codes with a scale for each block of 128 (quant_rows_f8). Returns (q float8_e4m3fn
    [rows][k], scale fp32 [ceil(k / 128)][rows])."""
    rows, k, stride = _rows(x, "x")
    dev = x.device
    code = _dtype_code(x.dtype, "x")
    q, scale = _codes_out(q, scale, rows, k, True, dev, stream)
    _launch("quant_rows_f8", dev, stream, _addr(x), code, stride, rows, k, _addr(q), _addr(scale))
    return q, scale


def _codes_out(q, scale, rows: int, k: int, f8: bool, device, stream):
    torch = _module or _torch()
    dtype = torch.float8_e4m3fn if f8 else torch.int8
    shape = (_blocks(k), rows) if f8 else (rows,)
    q = _empty((rows, k), dtype, device, stream) if q is None else _want(q, (rows, k), dtype, device, "q")
    scale = _empty(shape, torch.float32, device, stream) if scale is None else \
        _want(scale, shape, torch.float32, device, "scale")
    return q, scale


def _norm_q(what: str, f8: bool, h, t, gain, eps, h_out, out, q, scale, stream):
    torch = _module or _torch()
    rows, hidden, stride = _rows(h, "h")
    dev, shape, f32 = h.device, h.shape, torch.float32
    if h.dtype != f32:
        raise ValueError(f"h must be float32, not {h.dtype}")
    at = h.data_ptr()
    t_at = out_at = gain_at = None
    code = t_stride = 0
    if t is not None:
        if t.shape != shape or t.device != dev:
            raise ValueError(f"t must have the shape of h on its device, not {tuple(t.shape)} on {t.device}")
        t_stride = hidden if t.is_contiguous() else _rows(t, "t")[2]
        code, t_at = _dtype_code(t.dtype, "t"), t.data_ptr()
        h_out = _want(h if h_out is None else h_out, shape, f32, dev, "h_out").data_ptr()
    elif h_out is not None:
        raise ValueError("h_out goes with t, and only with it")
    if gain is not None:
        gain_at = _want(gain, (hidden,), f32, dev, "gain").data_ptr()
    if out is not None:
        out_at = _want(out, shape, torch.bfloat16, dev, "out").data_ptr()
    q, scale = _codes_out(q, scale, rows, hidden, f8, dev, stream)
    _launch(what, dev, stream, at, stride, t_at, code, t_stride, gain_at, rows, hidden, float(eps), h_out, out_at,
            q.data_ptr(), scale.data_ptr())
    return q, scale


def residual_add_rmsnorm_f8(h, t=None, gain=None, eps: float = 1e-6, h_out=None, out=None, q=None, scale=None,
                            stream=None):
    """h + t to h_out (h itself if none is given; without t nothing is added), then RMSNorm of it times gain as e4m3
    codes with a scale for each block of 128, as one launch (residual_add_rmsnorm_f8); the normalised rows also in
    bfloat16 to out, if given. Returns (q float8_e4m3fn [rows][hidden], scale fp32 [ceil(hidden / 128)][rows])."""
    return _norm_q("residual_add_rmsnorm_f8", True, h, t, gain, eps, h_out, out, q, scale, stream)


def residual_add_rmsnorm_i8(h, t=None, gain=None, eps: float = 1e-6, h_out=None, out=None, q=None, scale=None,
                            stream=None):
    """residual_add_rmsnorm_f8 with int8 codes and one scale a row, as gemm_i8 takes them. Returns (q int8
    [rows][hidden], scale fp32 [rows])."""
    return _norm_q("residual_add_rmsnorm_i8", False, h, t, gain, eps, h_out, out, q, scale, stream)


def gemm_f8_workspace_size(m: int, n: int, k: int, swiglu: bool, x_dtype) -> int:
    for v, what in ((m, "m"), (n, "n"), (k, "k")):
        _int(v, what)
    return int(load().gemm_f8_workspace_size(m, n, k, int(bool(swiglu)), _f8_code(x_dtype)))


def _f8_operands(x, x_scale, w, w_scale, swiglu: bool, lead: tuple):
    """Shape checks shared by the two products; w is lead + [2][n][k] with swiglu, else lead + [n][k]."""
    torch = _torch()
    rows, k, stride = _rows(x, "x")
    dev = x.device
    parts = (2,) if swiglu else ()
    if w.dim() != len(lead) + len(parts) + 2:
        raise ValueError(f"w has {w.dim()} dimensions, not {len(lead) + len(parts) + 2}")
    n = _int(w.shape[-2], "the rows of w")
    _want(w, lead + parts + (n, k), torch.float8_e4m3fn, dev, "w")
    _want(w_scale, lead + parts + (_blocks(n), _blocks(k)), torch.float32, dev, "w_scale")
    code = _f8_code(x.dtype)
    if (x_scale is not None) != (code == MOE_DTYPE_F8):
        raise ValueError("x_scale goes with float8_e4m3fn rows, and only with them")
    if x_scale is not None:
        _want(x_scale, (_blocks(k), rows), torch.float32, dev, "x_scale")
    return rows, k, stride, n, code


def gemm_f8(x, w, w_scale, x_scale=None, swiglu: bool = False, out=None, out_dtype=None, ws=None, stream=None):
    """y = x w^T in 8-bit floating point (gemm_f8): x [m][k] float rows, quantised on the way, or float8_e4m3fn codes
    with x_scale [ceil(k / 128)][m]; w float8_e4m3fn [n][k] with w_scale [ceil(n / 128)][ceil(k / 128)], or [2][..][..]
    both with swiglu. Returns y [m][n] in out's type, out_dtype or bfloat16; neither out nor ws overlaps an input. The
    products are summed in fp32 where y is float32 or has up to 16 rows; other 16-bit outputs may lose what lies below
    2^-13 of the largest of 8 neighbouring products, which matters where large ones cancel."""
    m, k, stride, n, code = _f8_operands(x, x_scale, w, w_scale, swiglu, ())
    dev = x.device
    y = _out(out, (m, n), out_dtype, dev, stream)
    ws = _workspace(ws, 0 if ws is not None else load().gemm_f8_workspace_size(m, n, k, int(bool(swiglu)), code), dev, stream)
    _launch("gemm_f8", dev, stream, _addr(x), code, stride, _addr(x_scale), m, k, _addr(w), _addr(w_scale), n, int(bool(swiglu)),
            _addr(y), _dtype_code(y.dtype, "out"), _addr(ws), 0 if ws is None else ws.numel())
    return y


def experts_gemm_f8_workspace_size(groups: SlotGroups, x_rows: int, n: int, k: int, swiglu: bool, x_dtype) -> int:
    for v, what in ((x_rows, "x_rows"), (n, "n"), (k, "k")):
        _int(v, what)
    return int(load().experts_gemm_f8_workspace_size(groups.tokens, groups.top_k, groups.num_experts, x_rows, n, k,
                                                     int(bool(swiglu)), _f8_code(x_dtype)))


def experts_gemm_f8(x, groups: SlotGroups, w, w_scale, x_scale=None, swiglu: bool = False, out=None, out_dtype=None,
                    ws=None, stream=None):
    """gemm_f8 of every slot with its expert's matrix (experts_gemm_f8): x has a row per token or per slot, w is
    float8_e4m3fn [num_experts][n][k] (or [num_experts][2][n][k] with swiglu). Returns y [tokens * top_k][n]; its sums are
    those of gemm_f8, in fp32 where y is float32."""
    E = groups.num_experts
    rows, k, stride, n, code = _f8_operands(x, x_scale, w, w_scale, swiglu, (E,))
    dev = x.device
    if rows != groups.tokens and rows != groups.tokens * groups.top_k:
        raise ValueError(f"x has {rows} rows, neither the tokens nor the slots of the groups")
    if groups.buffer.device != dev:
        raise ValueError("groups are on another device")
    y = _out(out, (groups.tokens * groups.top_k, n), out_dtype, dev, stream)
    need = 0 if ws is not None else load().experts_gemm_f8_workspace_size(groups.tokens, groups.top_k, E, rows, n, k,
                                                                          int(bool(swiglu)), code)
    ws = _workspace(ws, need, dev, stream)
    _launch("experts_gemm_f8", dev, stream, _addr(x), code, stride, _addr(x_scale), rows, k, _addr(groups.buffer),
            groups.buffer.numel(), groups.tokens, groups.top_k, E, _addr(w), _addr(w_scale), n, int(bool(swiglu)), _addr(y),
            _dtype_code(y.dtype, "out"), _addr(ws), 0 if ws is None else ws.numel())
    return y
