"""quantized_moe_ffn_amd — routed MoE FFN over GGUF block-quantized experts on MI355X.

A thin Python binding over ``libmoe.so`` (C ABI in ``include/moe.h``).  Every
function here only marshals arguments: torch tensors supply device memory and
the current HIP stream, and every step of the path runs in the library's HIP
kernels.  There is no CPU fallback: if ``libmoe.so`` is missing or cannot be
loaded, the first call raises.

Entry points keep the C names: ``moe_route_topk``, ``moe_quantize_act``,
``moe_router_logits``, ``moe_expert_ffn_q``, ``moe_combine``, ``moe_combine_ep``, ``moe_shared_gate``,
``moe_forward``, ``moe_forward_ep``, ``moe_forward_noalloc``, ``moe_forward_router``, ``moe_dequant_q``,
``moe_check_device_errors``, ``moe_last_error``, ``moe_abi_version``,
``moe_route_workspace_bytes``, ``moe_ffn_workspace_bytes``,
``moe_forward_workspace_bytes``; and for routing by a score rule and experts in
8-bit floats ``moe_route_scored``, ``moe_quantize_fp8``, ``moe_matmul_fp8``,
``moe_expert_ffn_fp8``, ``moe_forward_fp8``, ``moe_ffn_fp8_workspace_bytes``,
``moe_forward_fp8_workspace_bytes``.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_Q8_0 = 8
MOE_Q4_K = 12
MOE_Q5_K = 13
MOE_Q5_1 = 7
MOE_ROUTE_RENORM = 1
MOE_FFN_AUTO = 0
AUTO_DECODE_MAX_T = 8   # MOE_FFN_AUTO takes the fp-activation path up to this many tokens
MOE_FFN_DECODE = 1
MOE_FFN_INT8 = 2
MOE_FFN_PAIR_BF16 = 16  # layer calls: per-pair outputs stay in the workspace (bf16 on the MFMA GEMMs)

MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_F32 = 0
MOE_F16 = 1
MOE_BF16 = 30
MOE_FP8_BLOCK = 128

BLOCK_WEIGHTS = {MOE_Q4_K: 256, MOE_Q5_K: 256, MOE_Q8_0: 32, MOE_Q5_1: 32}
BLOCK_BYTES = {MOE_Q4_K: 144, MOE_Q5_K: 176, MOE_Q8_0: 34, MOE_Q5_1: 24}

EXPORTS = (
    "moe_abi_version", "moe_last_error", "moe_route_workspace_bytes", "moe_route_topk",
    "moe_quantize_act", "moe_ffn_workspace_bytes", "moe_expert_ffn_q", "moe_combine",
    "moe_dequant_q", "moe_check_device_errors", "moe_forward_workspace_bytes", "moe_forward",
    "moe_router_logits", "moe_combine_ep", "moe_shared_gate", "moe_forward_ep", "moe_forward_noalloc",
    "moe_forward_router",
    "moe_route_scored", "moe_quantize_fp8", "moe_matmul_fp8", "moe_ffn_fp8_workspace_bytes", "moe_expert_ffn_fp8",
    "moe_forward_fp8_workspace_bytes", "moe_forward_fp8",
)

MOE_NOALLOC_SCRATCH_BYTES = 8 << 20   # the static workspace of moe_forward_noalloc, per GPU


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__("%s failed with status %d: %s" % (where, status, message))
        self.status = status


class moe_qmatrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("qtype", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("row_bytes", ctypes.c_int64), ("expert_bytes", ctypes.c_int64)]


class moe_layer(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("has_shared", ctypes.c_int32), ("gate", moe_qmatrix), ("up", moe_qmatrix),
                ("down", moe_qmatrix), ("sh_gate", moe_qmatrix), ("sh_up", moe_qmatrix),
                ("sh_down", moe_qmatrix)]


class moe_epilogue(ctypes.Structure):
    _fields_ = [("residual", ctypes.c_void_p), ("shared_gate", ctypes.c_void_p)]


class moe_routing(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("idx", "w", "count", "offset", "pair", "active", "n_active")]


class moe_route_spec(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float),
                ("bias", ctypes.c_void_p)]


class moe_fp8_matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("row_stride", ctypes.c_int64), ("expert_stride", ctypes.c_int64)]


class moe_fp8_layer(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("has_shared", ctypes.c_int32), ("gate", moe_fp8_matrix), ("up", moe_fp8_matrix),
                ("down", moe_fp8_matrix), ("sh_gate", moe_fp8_matrix), ("sh_up", moe_fp8_matrix),
                ("sh_down", moe_fp8_matrix)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libmoe.so and declares its signatures (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libmoe.so not found at %s: build it first (python -m quantized_moe_ffn_amd.build "
                           "or __graft_entry__.build())" % path)
    lib = ctypes.CDLL(path)
    P, i32, i64, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
    st = ctypes.c_int
    lib.moe_abi_version.restype = i32
    lib.moe_last_error.restype = ctypes.c_char_p
    lib.moe_route_workspace_bytes.argtypes = [i32, i32, i32]
    lib.moe_route_workspace_bytes.restype = sz
    lib.moe_route_topk.argtypes = [P, i32, i32, i32, u32, ctypes.POINTER(moe_routing), P, sz, P]
    lib.moe_route_topk.restype = st
    lib.moe_quantize_act.argtypes = [P, i32, i32, P, P, P]
    lib.moe_quantize_act.restype = st
    lib.moe_router_logits.argtypes = [P, i32, i32, P, i32, P, P]
    lib.moe_router_logits.restype = st
    lib.moe_ffn_workspace_bytes.argtypes = [ctypes.POINTER(moe_layer), i32, i32, u32]
    lib.moe_ffn_workspace_bytes.restype = sz
    lib.moe_expert_ffn_q.argtypes = [ctypes.POINTER(moe_layer), ctypes.POINTER(moe_routing), i32, i32, P, P, P,
                                     u32, P, P, P, sz, P]
    lib.moe_expert_ffn_q.restype = st
    lib.moe_combine.argtypes = [P, P, P, P, i32, i32, i32, P, P]
    lib.moe_combine.restype = st
    lib.moe_dequant_q.argtypes = [P, i32, i64, P, P]
    lib.moe_dequant_q.restype = st
    lib.moe_forward_workspace_bytes.argtypes = [ctypes.POINTER(moe_layer), i32, i32, u32]
    lib.moe_forward_workspace_bytes.restype = sz
    lib.moe_forward.argtypes = [ctypes.POINTER(moe_layer), P, P, i32, i32, u32, u32, ctypes.POINTER(moe_routing),
                                P, P, P, P, P, sz, P]
    lib.moe_forward.restype = st
    lib.moe_forward_ep.argtypes = [ctypes.POINTER(moe_layer), P, P, i32, i32, u32, u32,
                                   ctypes.POINTER(moe_routing), P, P, P, ctypes.POINTER(moe_epilogue), P, P, sz, P]
    lib.moe_forward_ep.restype = st
    lib.moe_forward_noalloc.argtypes = [ctypes.POINTER(moe_layer), P, P, i32, i32, u32, u32,
                                        ctypes.POINTER(moe_routing), P, P, P, P, P]
    lib.moe_forward_noalloc.restype = st
    lib.moe_forward_router.argtypes = [ctypes.POINTER(moe_layer), P, P, P, i32, i32, u32, u32,
                                       ctypes.POINTER(moe_routing), P, P, P, P, P, sz, P]
    lib.moe_forward_router.restype = st
    lib.moe_combine_ep.argtypes = [P, P, P, P, P, P, i32, i32, i32, P, P]
    lib.moe_combine_ep.restype = st
    lib.moe_shared_gate.argtypes = [P, i32, i32, P, P, P]
    lib.moe_shared_gate.restype = st
    lib.moe_route_scored.argtypes = [P, i32, i32, i32, ctypes.POINTER(moe_route_spec), ctypes.POINTER(moe_routing), P,
                                     sz, P]
    lib.moe_route_scored.restype = st
    lib.moe_quantize_fp8.argtypes = [P, i32, i64, i32, i32, P, P, P]
    lib.moe_quantize_fp8.restype = st
    lib.moe_matmul_fp8.argtypes = [P, P, i32, ctypes.POINTER(moe_fp8_matrix), P, i32, i64, P]
    lib.moe_matmul_fp8.restype = st
    lib.moe_ffn_fp8_workspace_bytes.argtypes = [ctypes.POINTER(moe_fp8_layer), i32, i32]
    lib.moe_ffn_fp8_workspace_bytes.restype = sz
    lib.moe_expert_ffn_fp8.argtypes = [ctypes.POINTER(moe_fp8_layer), ctypes.POINTER(moe_routing), i32, i32, P, P, P,
                                       P, P, sz, P]
    lib.moe_expert_ffn_fp8.restype = st
    lib.moe_forward_fp8_workspace_bytes.argtypes = [ctypes.POINTER(moe_fp8_layer), i32, i32, u32]
    lib.moe_forward_fp8_workspace_bytes.restype = sz
    lib.moe_forward_fp8.argtypes = [ctypes.POINTER(moe_fp8_layer), ctypes.POINTER(moe_route_spec), P, P, i32, i32, i32,
                                    u32, ctypes.POINTER(moe_routing), P, P, P, sz, P]
    lib.moe_forward_fp8.restype = st
    lib.moe_check_device_errors.argtypes = [P]
    lib.moe_check_device_errors.restype = st
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where, moe_last_error())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ----------------------------------------------------------------------------- descriptors

class QMatrix:
    """A device bank of quantized matrices: uint8 tensor [n_experts][rows][row_bytes]."""

    def __init__(self, data, qtype: int, cols: int):
        assert data.dtype.itemsize == 1 and data.dim() == 3 and data.is_contiguous()
        self.data, self.qtype, self.cols = data, int(qtype), int(cols)
        self.rows = data.shape[1]
        self.row_bytes = cols // BLOCK_WEIGHTS[qtype] * BLOCK_BYTES[qtype]
        assert data.shape[2] == self.row_bytes, (data.shape, self.row_bytes)

    def struct(self) -> moe_qmatrix:
        return moe_qmatrix(self.data.data_ptr(), self.qtype, self.rows, self.cols, 0, self.row_bytes,
                           self.data.shape[1] * self.data.shape[2])


class Layer:
    """One MoE layer: routed banks gate/up [E][I][.], down [E][H][.], optional shared expert."""

    def __init__(self, gate: QMatrix, up: QMatrix, down: QMatrix, shared=None):
        self.gate, self.up, self.down, self.shared = gate, up, down, shared
        self.n_experts = gate.data.shape[0]
        self.hidden = gate.cols
        self.inter = gate.rows
        s = moe_layer()
        s.n_experts, s.hidden, s.inter = self.n_experts, self.hidden, self.inter
        s.gate, s.up, s.down = gate.struct(), up.struct(), down.struct()
        if shared is not None:
            s.has_shared = 1
            s.sh_gate, s.sh_up, s.sh_down = (m.struct() for m in shared)
        self._s = s

    def struct(self) -> moe_layer:
        return self._s


class Routing:
    """Device buffers written by moe_route_topk for T tokens, E experts, top-k."""

    def __init__(self, T: int, E: int, k: int, device="cuda"):
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        self.T, self.E, self.k = T, E, k
        self.idx = torch.empty((T, k), **i32)
        self.w = torch.empty((T, k), dtype=torch.float32, device=device)
        self.count = torch.empty(E, **i32)
        self.offset = torch.empty(E + 1, **i32)
        self.pair = torch.empty(T * k, **i32)
        self.active = torch.empty(max(1, min(E, T * k)), **i32)
        self.n_active = torch.empty(1, **i32)
        self._s = moe_routing(*(t.data_ptr() for t in (self.idx, self.w, self.count, self.offset, self.pair,
                                                        self.active, self.n_active)))

    def struct(self) -> moe_routing:
        return self._s


# ----------------------------------------------------------------------------- C entry points

def moe_abi_version() -> int:
    return int(load_library().moe_abi_version())


def moe_last_error() -> str:
    return load_library().moe_last_error().decode()


def moe_route_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(load_library().moe_route_workspace_bytes(T, E, k))


def moe_route_topk(logits, k: int, routing: Routing, renorm: bool = True, workspace=None, stream=None):
    T, E = logits.shape
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().moe_route_topk(_ptr(logits), T, E, k, MOE_ROUTE_RENORM if renorm else 0,
                                       ctypes.byref(routing.struct()), _ptr(workspace), nbytes, _stream(stream))
    _check(st, "moe_route_topk")


def moe_router_logits(x, w_router, logits, stream=None):
    """logits[t][e] = sum_h w_router[e][h] * x[t][h] (fp32 device tensors)."""
    T, H = x.shape
    E = w_router.shape[0]
    assert w_router.shape[1] == H and tuple(logits.shape) == (T, E)
    _check(load_library().moe_router_logits(_ptr(x), T, H, _ptr(w_router), E, _ptr(logits), _stream(stream)),
           "moe_router_logits")


def moe_quantize_act(x, xq, xd, stream=None):
    T, H = x.shape
    _check(load_library().moe_quantize_act(_ptr(x), T, H, _ptr(xq), _ptr(xd), _stream(stream)),
           "moe_quantize_act")


def moe_ffn_workspace_bytes(layer: Layer, T: int, k: int, flags: int = MOE_FFN_AUTO) -> int:
    return int(load_library().moe_ffn_workspace_bytes(ctypes.byref(layer.struct()), T, k, flags))


def moe_expert_ffn_q(layer: Layer, routing: Routing, T: int, k: int, y_pair, x=None, xq=None, xd=None,
                     flags: int = MOE_FFN_AUTO, y_shared=None, workspace=None, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().moe_expert_ffn_q(ctypes.byref(layer.struct()), ctypes.byref(routing.struct()), T, k,
                                         _ptr(x), _ptr(xq), _ptr(xd), flags, _ptr(y_pair), _ptr(y_shared),
                                         _ptr(workspace), nbytes, _stream(stream))
    _check(st, "moe_expert_ffn_q")


def moe_combine(y_pair, w, out, y_shared=None, shared_scale=None, stream=None):
    T, k = w.shape
    H = out.shape[1]
    _check(load_library().moe_combine(_ptr(y_pair), _ptr(w), _ptr(y_shared), _ptr(shared_scale), T, k, H,
                                      _ptr(out), _stream(stream)), "moe_combine")


def moe_combine_ep(y_pair, w, out, y_shared=None, shared_scale=None, shared_gate_s=None, residual=None,
                   stream=None):
    T, k = w.shape
    H = out.shape[1]
    _check(load_library().moe_combine_ep(_ptr(y_pair), _ptr(w), _ptr(y_shared), _ptr(shared_scale),
                                         _ptr(shared_gate_s), _ptr(residual), T, k, H, _ptr(out),
                                         _stream(stream)), "moe_combine_ep")


def moe_shared_gate(x, gate_w, s, stream=None):
    """s[t] = sigmoid(gate_w . x[t]) (fp32 device tensors)."""
    T, H = x.shape
    _check(load_library().moe_shared_gate(_ptr(x), T, H, _ptr(gate_w), _ptr(s), _stream(stream)),
           "moe_shared_gate")


def moe_dequant_q(blocks, qtype: int, n_weights: int, out, stream=None):
    _check(load_library().moe_dequant_q(_ptr(blocks), qtype, n_weights, _ptr(out), _stream(stream)),
           "moe_dequant_q")


def moe_forward_workspace_bytes(layer: Layer, T: int, k: int, flags: int = MOE_FFN_AUTO) -> int:
    return int(load_library().moe_forward_workspace_bytes(ctypes.byref(layer.struct()), T, k, flags))


def moe_forward(layer: Layer, logits, x, k: int, routing: Routing, y_pair, out, y_shared=None, shared_scale=None,
                renorm: bool = True, flags: int = MOE_FFN_AUTO, workspace=None, stream=None):
    T = x.shape[0]
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().moe_forward(ctypes.byref(layer.struct()), _ptr(logits), _ptr(x), T, k,
                                    MOE_ROUTE_RENORM if renorm else 0, flags, ctypes.byref(routing.struct()),
                                    _ptr(y_pair), _ptr(y_shared), _ptr(shared_scale), _ptr(out), _ptr(workspace),
                                    nbytes, _stream(stream))
    _check(st, "moe_forward")


def moe_forward_ep(layer: Layer, logits, x, k: int, routing: Routing, y_pair, out, y_shared=None,
                   shared_scale=None, residual=None, shared_gate=None, renorm: bool = True,
                   flags: int = MOE_FFN_AUTO, workspace=None, stream=None):
    T = x.shape[0]
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ep = moe_epilogue(_ptr(residual), _ptr(shared_gate))
    st = load_library().moe_forward_ep(ctypes.byref(layer.struct()), _ptr(logits), _ptr(x), T, k,
                                       MOE_ROUTE_RENORM if renorm else 0, flags, ctypes.byref(routing.struct()),
                                       _ptr(y_pair), _ptr(y_shared), _ptr(shared_scale), ctypes.byref(ep), _ptr(out),
                                       _ptr(workspace), nbytes, _stream(stream))
    _check(st, "moe_forward_ep")


def moe_forward_noalloc(layer: Layer, logits, x, k: int, routing: Routing, y_pair, out, y_shared=None,
                        shared_scale=None, renorm: bool = True, flags: int = MOE_FFN_AUTO, stream=None):
    """moe_forward with the library's static per-GPU scratch as its workspace (no allocation)."""
    T = x.shape[0]
    st = load_library().moe_forward_noalloc(ctypes.byref(layer.struct()), _ptr(logits), _ptr(x), T, k,
                                            MOE_ROUTE_RENORM if renorm else 0, flags, ctypes.byref(routing.struct()),
                                            _ptr(y_pair), _ptr(y_shared), _ptr(shared_scale), _ptr(out),
                                            _stream(stream))
    _check(st, "moe_forward_noalloc")


def moe_forward_router(layer: Layer, x, w_router, logits, k: int, routing: Routing, y_pair, out, workspace,
                       y_shared=None, shared_scale=None, renorm: bool = True, flags: int = MOE_FFN_AUTO, stream=None):
    """The layer from x and the router matrix (logits written); moe_forward's workspace."""
    T = x.shape[0]
    nbytes = workspace.numel() * workspace.element_size()
    st = load_library().moe_forward_router(ctypes.byref(layer.struct()), _ptr(x), _ptr(w_router), _ptr(logits), T, k,
                                           MOE_ROUTE_RENORM if renorm else 0, flags, ctypes.byref(routing.struct()),
                                           _ptr(y_pair), _ptr(y_shared), _ptr(shared_scale), _ptr(out),
                                           _ptr(workspace), nbytes, _stream(stream))
    _check(st, "moe_forward_router")


def moe_check_device_errors(stream=None):
    _check(load_library().moe_check_device_errors(_stream(stream)), "moe_check_device_errors")


# ----------------------------------------------------------------------------- scored routing, 8-bit floats

_elem_ids = None
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _elem_id(t) -> int:
    """MOE_F32 / MOE_F16 / MOE_BF16 of a tensor (raises ValueError for another type)."""
    global _elem_ids
    if _elem_ids is None:
        import torch
        _elem_ids = {torch.float32: MOE_F32, torch.float16: MOE_F16, torch.bfloat16: MOE_BF16}
    i = _elem_ids.get(t.dtype)
    if i is None:
        raise ValueError("dtype %s: supported are float32, float16 and bfloat16" % t.dtype)
    return i


def _need(name: str, t, dtype, shape, device):
    """Checks a tensor argument: type, shape, contiguity and device (kept light: it runs at every call)."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError("%s: %s %s on %s%s, expected %s %s on %s, contiguous"
                         % (name, t.dtype, tuple(t.shape), t.device, "" if t.is_contiguous() else " (not contiguous)",
                            dtype, tuple(shape), device))


def _fp8_codes(name: str, t):
    if t.dtype is not _torch().float8_e4m3fn and t.dtype is not _torch().uint8:
        raise ValueError("%s has dtype %s: e4m3 codes are float8_e4m3fn or uint8" % (name, t.dtype))


def _launch_stream(device, stream) -> int:
    """The stream of a call on tensors of `device`, which has to be the current one."""
    if device.type != "cuda":
        raise ValueError("tensors must be on a GPU, got %s" % device)
    torch = _torch()
    cur = torch._C._cuda_getDevice()
    if device.index != cur:
        raise ValueError("tensors are on %s, the current device is cuda:%d" % (device, cur))
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(cur)
    return _stream(stream)


class RouteSpec:
    """Score rule of moe_route_scored: score "softmax" or "sigmoid", n_group groups of which
    topk_group stay (group score: the sum of the group_top largest biased scores), renormalised
    weights times scale; bias fp32 [E] on the device, or None."""

    def __init__(self, score: str = "softmax", n_group: int = 1, topk_group: int = 1, group_top: int = 1,
                 renorm: bool = True, scale: float = 1.0, bias=None):
        if score not in ("softmax", "sigmoid"):
            raise ValueError("score = %r: use 'softmax' or 'sigmoid'" % (score,))
        if bias is not None:
            _need("bias", bias, _torch().float32, (bias.numel(),), bias.device)
        self.bias = bias
        self._s = moe_route_spec(MOE_SCORE_SIGMOID if score == "sigmoid" else MOE_SCORE_SOFTMAX, n_group, topk_group,
                                 group_top, 1 if renorm else 0, scale, _ptr(bias))

    def struct(self) -> moe_route_spec:
        return self._s

    def check(self, E: int, device):
        if self.bias is not None and (self.bias.numel() != E or self.bias.device != device):
            raise ValueError("bias has %d entries on %s, expected %d on %s"
                             % (self.bias.numel(), self.bias.device, E, device))


class Fp8Matrix:
    """A device bank of e4m3 matrices: codes [n][rows][cols] (float8_e4m3fn or uint8, columns contiguous,
    rows and experts at any 16-byte multiple) and scales fp32 [n][ceil(rows/128)][ceil(cols/128)]."""

    def __init__(self, data, scale):
        _fp8_codes("data", data)
        if data.dim() != 3:
            raise ValueError("data has shape %s, expected [n][rows][cols]" % (tuple(data.shape),))
        n, rows, cols = data.shape
        if cols > 1 and data.stride(2) != 1:
            raise ValueError("data: columns must be contiguous")
        b = MOE_FP8_BLOCK
        _need("scale", scale, _torch().float32, (n, (rows + b - 1) // b, (cols + b - 1) // b), data.device)
        self.data, self.scale, self.n, self.rows, self.cols = data, scale, n, rows, cols
        self._s = moe_fp8_matrix(data.data_ptr(), scale.data_ptr(), rows, cols,
                                 data.stride(1) if rows > 1 else (cols + 15) // 16 * 16,
                                 data.stride(0) if n > 1 else (rows * max(cols, data.stride(1)) + 15) // 16 * 16)

    def struct(self) -> moe_fp8_matrix:
        return self._s


class Fp8Layer:
    """One MoE layer over e4m3 experts: gate/up [E][I][H], down [E][H][I], optional shared expert
    (three one-expert matrices)."""

    def __init__(self, gate: Fp8Matrix, up: Fp8Matrix, down: Fp8Matrix, shared=None):
        mats = (gate, up, down) + (tuple(shared) if shared is not None else ())
        if len(mats) not in (3, 6):
            raise ValueError("shared: expected (gate, up, down)")
        self.gate, self.up, self.down, self.shared = gate, up, down, shared
        self.n_experts, self.inter, self.hidden = gate.n, gate.rows, gate.cols
        self.device = gate.data.device
        for m, n in zip(mats, (self.n_experts,) * 3 + (1,) * 3):
            if m.n != n or m.data.device != self.device:
                raise ValueError("a matrix bank holds %d experts on %s, expected %d on %s"
                                 % (m.n, m.data.device, n, self.device))
        s = moe_fp8_layer()
        s.n_experts, s.hidden, s.inter = self.n_experts, self.hidden, self.inter
        s.gate, s.up, s.down = gate.struct(), up.struct(), down.struct()
        if shared is not None:
            s.has_shared = 1
            s.sh_gate, s.sh_up, s.sh_down = (m.struct() for m in shared)
        self._s = s

    def struct(self) -> moe_fp8_layer:
        return self._s


def _check_routing(routing: Routing, T: int, E: int, k: int, device):
    if routing.T != T or routing.E != E or routing.k != k or routing.idx.device != device:
        raise ValueError("routing buffers are for T, E, k = %d, %d, %d on %s, expected %d, %d, %d on %s"
                         % (routing.T, routing.E, routing.k, routing.idx.device, T, E, k, device))


def _ws(workspace, device):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("workspace must be contiguous and on %s" % device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def moe_route_scored(logits, k: int, routing: Routing, spec: RouteSpec, workspace=None, stream=None):
    """Expert selection by a score rule, with moe_route_topk's buffers and workspace (fp32 logits [T][E])."""
    T, E = logits.shape
    _need("logits", logits, _torch().float32, (T, E), logits.device)
    _check_routing(routing, T, E, k, logits.device)
    spec.check(E, logits.device)
    wp, wn = _ws(workspace, logits.device)
    st = load_library().moe_route_scored(logits.data_ptr(), T, E, k, ctypes.byref(spec.struct()),
                                         ctypes.byref(routing.struct()), wp, wn, _launch_stream(logits.device, stream))
    _check(st, "moe_route_scored")


def moe_quantize_fp8(x, xq, xs, stream=None):
    """x [T][H] (float32, float16 or bfloat16; columns contiguous, rows at any 16-byte multiple) to e4m3
    codes xq [T][H] and scales xs fp32 [T][ceil(H/128)]."""
    T, H = x.shape
    if x.stride(1) != 1 and H > 1:
        raise ValueError("x: columns must be contiguous")
    d = x.device
    _fp8_codes("xq", xq)
    _need("xq", xq, xq.dtype, (T, H), d)
    _need("xs", xs, _torch().float32, (T, (H + MOE_FP8_BLOCK - 1) // MOE_FP8_BLOCK), d)
    _check(load_library().moe_quantize_fp8(x.data_ptr(), _elem_id(x), x.stride(0) if T > 1 else H, T, H,
                                           xq.data_ptr(), xs.data_ptr(), _launch_stream(d, stream)),
           "moe_quantize_fp8")


def moe_matmul_fp8(xq, xs, w: Fp8Matrix, y, stream=None):
    """y [T][N] = block-scaled product of xq [T][K], xs (from moe_quantize_fp8) with one matrix [1][N][K];
    y float32, float16 or bfloat16, columns contiguous, rows at any distance."""
    T, K = xq.shape
    _fp8_codes("xq", xq)
    d = w.data.device
    _need("xq", xq, xq.dtype, (T, w.cols), d)
    _need("xs", xs, _torch().float32, (T, w.scale.shape[2]), d)
    if w.n != 1:
        raise ValueError("w holds %d matrices, expected one" % w.n)
    if y.shape != (T, w.rows) or (y.stride(1) != 1 and w.rows > 1) or y.device != d:
        raise ValueError("y has shape %s, strides %s on %s: expected %s, contiguous columns, on %s"
                         % (tuple(y.shape), y.stride(), y.device, (T, w.rows), d))
    _check(load_library().moe_matmul_fp8(xq.data_ptr(), xs.data_ptr(), T, ctypes.byref(w.struct()), y.data_ptr(),
                                         _elem_id(y), y.stride(0) if T > 1 else w.rows,
                                         _launch_stream(d, stream)), "moe_matmul_fp8")


def moe_ffn_fp8_workspace_bytes(layer: Fp8Layer, T: int, k: int) -> int:
    return int(load_library().moe_ffn_fp8_workspace_bytes(ctypes.byref(layer.struct()), T, k))


def moe_expert_ffn_fp8(layer: Fp8Layer, routing: Routing, T: int, k: int, y_pair, xq, xs, y_shared=None,
                       workspace=None, stream=None):
    H, d = layer.hidden, layer.device
    _check_routing(routing, T, layer.n_experts, k, d)
    _fp8_codes("xq", xq)
    f32 = _torch().float32
    _need("xq", xq, xq.dtype, (T, H), d)
    _need("xs", xs, f32, (T, H // MOE_FP8_BLOCK), d)
    _need("y_pair", y_pair, f32, (T * k, H), d)
    if y_shared is not None:
        _need("y_shared", y_shared, f32, (T, H), d)
    wp, wn = _ws(workspace, d)
    st = load_library().moe_expert_ffn_fp8(ctypes.byref(layer.struct()), ctypes.byref(routing.struct()), T, k,
                                           xq.data_ptr(), xs.data_ptr(), y_pair.data_ptr(), _ptr(y_shared), wp, wn,
                                           _launch_stream(d, stream))
    _check(st, "moe_expert_ffn_fp8")


def moe_forward_fp8_workspace_bytes(layer: Fp8Layer, T: int, k: int, flags: int = 0) -> int:
    return int(load_library().moe_forward_fp8_workspace_bytes(ctypes.byref(layer.struct()), T, k, flags))


def moe_forward_fp8(layer: Fp8Layer, logits, x, k: int, routing: Routing, spec: RouteSpec, out, shared_scale=None,
                    flags: int = 0, workspace=None, stream=None):
    """The whole layer over e4m3 experts from fp32 logits [T][E] and x [T][H] (out has x's type; it may be x)."""
    T, E = logits.shape
    d = layer.device
    f32 = _torch().float32
    _need("logits", logits, f32, (T, layer.n_experts), d)
    xt = _elem_id(x)
    _need("x", x, x.dtype, (T, layer.hidden), d)
    _need("out", out, x.dtype, (T, layer.hidden), d)
    if shared_scale is not None:
        _need("shared_scale", shared_scale, f32, (T,), d)
    _check_routing(routing, T, E, k, d)
    spec.check(E, d)
    wp, wn = _ws(workspace, d)
    st = load_library().moe_forward_fp8(ctypes.byref(layer.struct()), ctypes.byref(spec.struct()), logits.data_ptr(),
                                        x.data_ptr(), xt, T, k, flags, ctypes.byref(routing.struct()),
                                        _ptr(shared_scale), out.data_ptr(), wp, wn, _launch_stream(d, stream))
    _check(st, "moe_forward_fp8")


# ----------------------------------------------------------------------------- whole layer

class LayerBuffers:
    """Routing, workspace and output buffers for one (T, k) shape of a layer."""

    def __init__(self, layer: Layer, T: int, k: int, flags: int = MOE_FFN_AUTO, device="cuda"):
        import torch
        H, E = layer.hidden, layer.n_experts
        self.T, self.k, self.flags = T, k, flags
        self.routing = Routing(T, E, k, device)
        rw = moe_route_workspace_bytes(T, E, k)
        self.route_ws = torch.empty(max(rw, 1), dtype=torch.uint8, device=device)
        fw = moe_ffn_workspace_bytes(layer, T, k, flags & ~MOE_FFN_PAIR_BF16)
        self.ffn_ws = torch.empty(max(fw, 256), dtype=torch.uint8, device=device)
        self.y_pair = torch.empty((T * k, H), dtype=torch.float32, device=device)
        self.y_shared = torch.empty((T, H), dtype=torch.float32, device=device) if layer.shared else None
        self.xq = torch.empty((T, H), dtype=torch.int8, device=device)
        self.xd = torch.empty((T, H // 256), dtype=torch.float32, device=device)
        self.out = torch.empty((T, H), dtype=torch.float32, device=device)
        self.gate_s = torch.empty(T, dtype=torch.float32, device=device)
        fwd = moe_forward_workspace_bytes(layer, T, k, flags)
        self.fwd_ws = torch.empty(max(fwd, 256), dtype=torch.uint8, device=device)


def forward(layer: Layer, logits, x, k: int, bufs: LayerBuffers | None = None, flags: int = MOE_FFN_AUTO,
            renorm: bool = True, shared_scale=None, stream=None, fused: bool = True, residual=None,
            shared_gate=None) -> LayerBuffers:
    """The whole layer on one stream.  fused=True: one moe_forward call (two kernels
    for decode batches), moe_forward_ep when an epilogue (residual, shared-expert
    gate vector) is given; fused=False: the separate calls route -> (quantize) ->
    expert FFN -> (shared gate) -> combine."""
    T = x.shape[0]
    if bufs is None:
        bufs = LayerBuffers(layer, T, k, flags, device=x.device)
    epilogue = residual is not None or shared_gate is not None
    if fused:
        if epilogue:
            moe_forward_ep(layer, logits, x, k, bufs.routing, bufs.y_pair, bufs.out, bufs.y_shared, shared_scale,
                           residual, shared_gate, renorm, flags, bufs.fwd_ws, stream)
        else:
            moe_forward(layer, logits, x, k, bufs.routing, bufs.y_pair, bufs.out, bufs.y_shared, shared_scale,
                        renorm, flags, bufs.fwd_ws, stream)
        return bufs
    sel = flags & ~MOE_FFN_PAIR_BF16   # the separate stages hand fp32 y_pair to the combine
    path = sel if sel != MOE_FFN_AUTO else (MOE_FFN_DECODE if T <= AUTO_DECODE_MAX_T else MOE_FFN_INT8)
    moe_route_topk(logits, k, bufs.routing, renorm, bufs.route_ws, stream)
    if path == MOE_FFN_INT8:
        moe_quantize_act(x, bufs.xq, bufs.xd, stream)
    moe_expert_ffn_q(layer, bufs.routing, T, k, bufs.y_pair, x=x if path == MOE_FFN_DECODE else None,
                     xq=bufs.xq if path == MOE_FFN_INT8 else None, xd=bufs.xd if path == MOE_FFN_INT8 else None,
                     flags=path, y_shared=bufs.y_shared, workspace=bufs.ffn_ws, stream=stream)
    if epilogue:
        sg = None
        if shared_gate is not None:
            sg = bufs.gate_s
            moe_shared_gate(x, shared_gate, sg, stream)
        moe_combine_ep(bufs.y_pair, bufs.routing.w, bufs.out, bufs.y_shared, shared_scale, sg, residual, stream)
    else:
        moe_combine(bufs.y_pair, bufs.routing.w, bufs.out, bufs.y_shared, shared_scale, stream)
    return bufs
