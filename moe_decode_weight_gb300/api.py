"""Python binding of the C-ABI library ``libmdw.so`` (argument marshalling only).

Every function here has the name of the C entry point it calls and does no arithmetic of
its own: torch tensors supply device memory and the current CUDA stream, and every step of
the decode path runs in the library's kernels. If the library is missing or fails to load
this module raises; there is no CPU fallback.
"""

from __future__ import annotations

import ctypes as C
import importlib.machinery
import importlib.util
import os
from dataclasses import dataclass, field

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmdw.so")

MDW_MAGIC = 0x3157444D
FMT_BF16, FMT_FP8, FMT_MXFP4, FMT_INT4_GROUP, FMT_KV_PAGED, FMT_LINEAR_STATE = 1, 2, 3, 4, 5, 6
DT_BF16, DT_F16, DT_F32, DT_E4M3 = 1, 2, 3, 4
STATUS = {0: "MDW_OK", 1: "MDW_ERR_INVALID_ARG", 2: "MDW_ERR_UNSUPPORTED_SHAPE",
          3: "MDW_ERR_FORMAT_MISMATCH", 4: "MDW_ERR_WORKSPACE_TOO_SMALL", 5: "MDW_ERR_CUDA",
          6: "MDW_ERR_TIMEOUT", 7: "MDW_ERR_DEVICE_BOUNDS"}
HIDDEN, INTER = 2560, 768
MAX_M, MAX_TOPK, MAX_VOCAB_TOPK, MAX_EXPERTS = 32, 8, 32, 512
MAX_REQUESTS, MAX_TREE, MAX_GROUP, MAX_NORM_WIDTH = 4096, 64, 64, 16384
GATES = {"none": 0, "mul": 1, "sigmoid": 2, "silu": 3}

# exported symbols declared in include/moe_decode_weight.h
SYMBOLS = ["mdw_status_string", "mdw_version", "mdw_moe_workspace_bytes", "mdw_moe_workspace_layout",
           "moe_decode_layer", "quantize_lm_head_fp8", "mdw_lm_head_bf16_init",
           "mdw_lm_head_workspace_bytes", "lm_head_fp8", "lm_head_bf16", "lm_head_fp8_rmsnorm",
           "mdw_stack_workspace_bytes",
           "moe_decode_stack", "mdw_device_status", "moe_decode_layer_noalloc", "mdw_sample_topk",
           "lm_head_fp8_sample", "moe_decode_stack_routed", "mdw_debug_set_spin_budget",
           "w4_linear", "mdw_kv_plan", "mdw_kv_write", "mdw_tree_attention_workspace_bytes",
           "mdw_tree_attention", "mdw_linear_attention_workspace_bytes", "mdw_linear_attention",
           "mdw_linear_tree_attention", "mdw_linear_state_advance", "mdw_block_norm"]


class MdwError(RuntimeError):
    def __init__(self, fn: str, code: int, detail: str = ""):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}" + (f": {detail}" if detail else ""))
        self.code = code


class MoeWeightsC(C.Structure):
    _fields_ = [("magic", C.c_uint32), ("fmt", C.c_int32), ("num_experts", C.c_int32),
                ("top_k", C.c_int32), ("hidden", C.c_int32), ("inter", C.c_int32),
                ("router_w", C.c_void_p), ("w13_q", C.c_void_p), ("w13_s", C.c_void_p),
                ("w2_q", C.c_void_p), ("w2_s", C.c_void_p), ("sh_w13_q", C.c_void_p),
                ("sh_w13_s", C.c_void_p), ("sh_w2_q", C.c_void_p), ("sh_w2_s", C.c_void_p)]


class LMHeadC(C.Structure):
    _fields_ = [("magic", C.c_uint32), ("fmt", C.c_int32), ("vocab", C.c_int64),
                ("hidden", C.c_int32), ("reserved", C.c_int32), ("w", C.c_void_p),
                ("row_scale", C.c_void_p)]


class MoeWsLayoutC(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("header", "xq", "sx", "logits", "ids", "gates",
                                          "slot_expert", "pair_token", "pair_slot", "pair_gate",
                                          "h", "hq", "sh", "total")]


class W4WeightsC(C.Structure):
    _fields_ = [("magic", C.c_uint32), ("fmt", C.c_int32), ("n", C.c_int32), ("k", C.c_int32),
                ("group", C.c_int32), ("dtype", C.c_int32), ("q", C.c_void_p), ("scale", C.c_void_p),
                ("zero", C.c_void_p)]


class KVCacheC(C.Structure):
    _fields_ = [("magic", C.c_uint32), ("fmt", C.c_int32), ("dtype", C.c_int32), ("num_pages", C.c_int32),
                ("page_size", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("reserved", C.c_int32), ("page_stride", C.c_int64), ("k", C.c_void_p), ("v", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p)]


class LinearStateC(C.Structure):
    _fields_ = [("magic", C.c_uint32), ("fmt", C.c_int32), ("num_slots", C.c_int32), ("heads", C.c_int32),
                ("head_dim", C.c_int32), ("reserved", C.c_int32), ("slot_stride", C.c_int64), ("s", C.c_void_p)]


_lib = None


def lib() -> C.CDLL:
    """Load libmdw.so (once) and declare its signatures. Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with moe_decode_weight_gb300.build.build()")
    L = C.CDLL(LIB_PATH)
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    L.mdw_status_string.restype = C.c_char_p
    L.mdw_status_string.argtypes = [C.c_int]
    L.mdw_version.restype = i32
    L.mdw_debug_set_spin_budget.restype = i64
    L.mdw_debug_set_spin_budget.argtypes = [i64]
    L.mdw_moe_workspace_bytes.restype = sz
    L.mdw_moe_workspace_bytes.argtypes = [C.POINTER(MoeWeightsC), i32]
    L.mdw_moe_workspace_layout.restype = C.c_int
    L.mdw_moe_workspace_layout.argtypes = [C.POINTER(MoeWeightsC), i32, C.POINTER(MoeWsLayoutC)]
    L.moe_decode_layer.restype = C.c_int
    L.moe_decode_layer.argtypes = [C.POINTER(MoeWeightsC), i32, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    L.quantize_lm_head_fp8.restype = C.c_int
    L.quantize_lm_head_fp8.argtypes = [vp, i64, i32, vp, vp, C.POINTER(LMHeadC), vp]
    L.mdw_lm_head_bf16_init.restype = C.c_int
    L.mdw_lm_head_bf16_init.argtypes = [vp, i64, i32, C.POINTER(LMHeadC)]
    L.mdw_lm_head_workspace_bytes.restype = sz
    L.mdw_lm_head_workspace_bytes.argtypes = [C.POINTER(LMHeadC), i32, i32]
    for name in ("lm_head_fp8", "lm_head_bf16", "lm_head_fp8_rmsnorm"):
        f = getattr(L, name)
        f.restype = C.c_int
        f.argtypes = [C.POINTER(LMHeadC), i32, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    L.mdw_stack_workspace_bytes.restype = sz
    L.mdw_stack_workspace_bytes.argtypes = [C.POINTER(MoeWeightsC), i32, C.POINTER(LMHeadC), i32, i32]
    L.moe_decode_stack.restype = C.c_int
    L.moe_decode_stack.argtypes = [C.POINTER(MoeWeightsC), i32, C.POINTER(LMHeadC), i32, vp, vp, vp, vp,
                                   i32, vp, vp, vp, sz, vp]
    L.moe_decode_stack_routed.restype = C.c_int
    L.moe_decode_stack_routed.argtypes = [C.POINTER(MoeWeightsC), i32, C.POINTER(LMHeadC), i32, vp, vp, vp, vp,
                                          i32, vp, vp, vp, vp, sz, vp]
    L.mdw_device_status.restype = C.c_int
    L.mdw_device_status.argtypes = [vp, vp]
    L.moe_decode_layer_noalloc.restype = C.c_int
    L.moe_decode_layer_noalloc.argtypes = [C.POINTER(MoeWeightsC), i32, vp, vp, i32, vp, vp, vp, vp, vp, vp]
    f64 = C.c_double
    L.mdw_sample_topk.restype = C.c_int
    L.mdw_sample_topk.argtypes = [i32, i32, vp, vp, f64, f64, vp, vp, vp]
    L.lm_head_fp8_sample.restype = C.c_int
    L.lm_head_fp8_sample.argtypes = [C.POINTER(LMHeadC), i32, vp, i32, i32, f64, f64, vp, vp, vp, vp, vp, sz, vp]
    f32 = C.c_float
    L.w4_linear.restype = C.c_int
    L.w4_linear.argtypes = [C.POINTER(W4WeightsC), i32, vp, i64, vp, i64, i32, vp, vp, i64, vp, vp]
    L.mdw_kv_plan.restype = C.c_int
    L.mdw_kv_plan.argtypes = [i32, vp, vp, i32, i32, vp, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp]
    L.mdw_kv_write.restype = C.c_int
    L.mdw_kv_write.argtypes = [C.POINTER(KVCacheC), i32, vp, i64, vp, i64, i32, vp, vp, vp]
    L.mdw_tree_attention_workspace_bytes.restype = sz
    L.mdw_tree_attention_workspace_bytes.argtypes = [C.POINTER(KVCacheC), i32, i32, i32, i32]
    L.mdw_tree_attention.restype = C.c_int
    L.mdw_tree_attention.argtypes = [C.POINTER(KVCacheC), i32, i32, i32, i32, vp, i64, i32, vp, i64, vp, vp, i32,
                                     vp, vp, vp, f32, vp, vp, sz, vp]
    L.mdw_linear_attention_workspace_bytes.restype = sz
    L.mdw_linear_attention_workspace_bytes.argtypes = [C.POINTER(LinearStateC), i32, i32, i32, i32]
    L.mdw_linear_attention.restype = C.c_int
    L.mdw_linear_attention.argtypes = [C.POINTER(LinearStateC), i32, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                       vp, vp, vp, f32, vp, vp, sz, vp]
    L.mdw_linear_tree_attention.restype = C.c_int
    L.mdw_linear_tree_attention.argtypes = [C.POINTER(LinearStateC), i32, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                            vp, vp, vp, f32, vp, vp]
    L.mdw_linear_state_advance.restype = C.c_int
    L.mdw_linear_state_advance.argtypes = [C.POINTER(LinearStateC), i32, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp]
    L.mdw_block_norm.restype = C.c_int
    L.mdw_block_norm.argtypes = [i32, i32, i32, vp, i64, i32, vp, i32, vp, i64, i32, f32, vp, i64, f32, vp, i64, i32, vp, vp, i64, f32, vp]
    _lib = L
    return L


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _check(fn: str, code: int):
    if code != 0:
        raise MdwError(fn, code)


# ----------------------------------------------------------------------------- handles


@dataclass
class MoeWeights:
    """One layer's device tensors and the C descriptor that points at them."""
    router_w: torch.Tensor
    w13_q: torch.Tensor
    w13_s: torch.Tensor
    w2_q: torch.Tensor
    w2_s: torch.Tensor
    shared: tuple | None
    top_k: int = 8
    c: MoeWeightsC = field(init=False)

    def __post_init__(self):
        sh = self.shared if self.shared is not None else (None,) * 4
        self.c = MoeWeightsC(MDW_MAGIC, FMT_MXFP4, self.w13_q.shape[0], self.top_k, HIDDEN, INTER,
                             *(t.data_ptr() if t is not None else None for t in
                               (self.router_w, self.w13_q, self.w13_s, self.w2_q, self.w2_s, *sh)))


@dataclass
class LMHead:
    """A head descriptor plus the tensors it points at (kept alive here)."""
    c: LMHeadC
    tensors: tuple


def mdw_status_string(code: int) -> str:
    return lib().mdw_status_string(code).decode()


def mdw_version() -> int:
    return lib().mdw_version()


def mdw_debug_set_spin_budget(cycles: int) -> int:
    """Test hook: bound of the kernels' inter-block waits in clock64 cycles (<= 0: the
    default); returns the previous bound."""
    return lib().mdw_debug_set_spin_budget(int(cycles))


def mdw_moe_workspace_bytes(w: MoeWeights, m: int) -> int:
    return lib().mdw_moe_workspace_bytes(C.byref(w.c), m)


def mdw_moe_workspace_layout(w: MoeWeights, m: int) -> dict:
    out = MoeWsLayoutC()
    _check("mdw_moe_workspace_layout", lib().mdw_moe_workspace_layout(C.byref(w.c), m, C.byref(out)))
    return {n: getattr(out, n) for n, _ in MoeWsLayoutC._fields_}


def moe_decode_layer(w: MoeWeights, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
                     residual=None, topk_override=None, topk_ids_out=None, topk_w_out=None,
                     stream=None) -> None:
    m = x.shape[0]
    code = lib().moe_decode_layer(C.byref(w.c), m, _ptr(x), _ptr(y), int(y.dtype == torch.float32),
                                  _ptr(residual), _ptr(topk_override), _ptr(topk_ids_out),
                                  _ptr(topk_w_out), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream))
    _check("moe_decode_layer", code)


def moe_decode_layer_noalloc(w: MoeWeights, x: torch.Tensor, y: torch.Tensor, residual=None,
                             topk_override=None, topk_ids_out=None, topk_w_out=None,
                             device_status_out=None, stream=None) -> None:
    """moe_decode_layer for callers that cannot allocate device memory: the library's own
    fixed scratch array replaces the workspace (see the C declaration for its limits)."""
    code = lib().moe_decode_layer_noalloc(C.byref(w.c), x.shape[0], _ptr(x), _ptr(y),
                                          int(y.dtype == torch.float32), _ptr(residual),
                                          _ptr(topk_override), _ptr(topk_ids_out), _ptr(topk_w_out),
                                          _ptr(device_status_out), _stream(stream))
    _check("moe_decode_layer_noalloc", code)


def quantize_lm_head_fp8(w_bf16: torch.Tensor, q_out: torch.Tensor, scale_out: torch.Tensor,
                         stream=None) -> LMHead:
    head = LMHeadC()
    code = lib().quantize_lm_head_fp8(_ptr(w_bf16), w_bf16.shape[0], w_bf16.shape[1], _ptr(q_out),
                                      _ptr(scale_out), C.byref(head), _stream(stream))
    _check("quantize_lm_head_fp8", code)
    return LMHead(head, (q_out, scale_out))


def mdw_lm_head_bf16_init(w_bf16: torch.Tensor) -> LMHead:
    head = LMHeadC()
    _check("mdw_lm_head_bf16_init",
           lib().mdw_lm_head_bf16_init(_ptr(w_bf16), w_bf16.shape[0], w_bf16.shape[1], C.byref(head)))
    return LMHead(head, (w_bf16,))


def mdw_lm_head_workspace_bytes(head: LMHead, m: int, topk: int) -> int:
    return lib().mdw_lm_head_workspace_bytes(C.byref(head.c), m, topk)


def _head(fn: str, head: LMHead, h: torch.Tensor, argmax_out, ws, logits=None, topk=1, topk_idx=None,
          topk_val=None, stream=None):
    code = getattr(lib(), fn)(C.byref(head.c), h.shape[0], _ptr(h), _ptr(logits), _ptr(argmax_out), topk,
                              _ptr(topk_idx), _ptr(topk_val), _ptr(ws), ws.numel() * ws.element_size(),
                              _stream(stream))
    _check(fn, code)


def lm_head_fp8(head: LMHead, h: torch.Tensor, argmax_out: torch.Tensor, ws: torch.Tensor, logits=None,
                topk: int = 1, topk_idx=None, topk_val=None, stream=None) -> None:
    _head("lm_head_fp8", head, h, argmax_out, ws, logits, topk, topk_idx, topk_val, stream)


def lm_head_bf16(head: LMHead, h: torch.Tensor, argmax_out: torch.Tensor, ws: torch.Tensor, logits=None,
                 topk: int = 1, topk_idx=None, topk_val=None, stream=None) -> None:
    _head("lm_head_bf16", head, h, argmax_out, ws, logits, topk, topk_idx, topk_val, stream)


def lm_head_fp8_rmsnorm(head: LMHead, r: torch.Tensor, argmax_out: torch.Tensor, ws: torch.Tensor,
                        logits=None, topk: int = 1, topk_idx=None, topk_val=None, stream=None) -> None:
    _head("lm_head_fp8_rmsnorm", head, r, argmax_out, ws, logits, topk, topk_idx, topk_val, stream)


def mdw_sample_topk(topk_val: torch.Tensor, topk_idx: torch.Tensor, temperature: float, top_p: float,
                    u: torch.Tensor, token_out: torch.Tensor, stream=None) -> None:
    """Draw one token per row of the [M, k] candidates (u: float64 [M] uniforms in [0, 1))."""
    m, k = topk_val.shape
    _check("mdw_sample_topk", lib().mdw_sample_topk(m, k, _ptr(topk_val), _ptr(topk_idx), float(temperature),
                                                      float(top_p), _ptr(u), _ptr(token_out), _stream(stream)))


def lm_head_fp8_sample(head: LMHead, h: torch.Tensor, token_out: torch.Tensor, ws: torch.Tensor, u: torch.Tensor,
                       temperature: float, top_p: float, topk: int, norm_input: bool = False, topk_idx=None,
                       topk_val=None, stream=None) -> None:
    """FP8 head (optionally on bf16(RMSNorm(h))) and the draw on its top-k, in one launch per
    16 tokens."""
    _check("lm_head_fp8_sample",
           lib().lm_head_fp8_sample(C.byref(head.c), h.shape[0], _ptr(h), 1 if norm_input else 0, topk,
                                    float(temperature), float(top_p), _ptr(u), _ptr(token_out), _ptr(topk_idx),
                                    _ptr(topk_val), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def _layer_array(layers):
    """ctypes array of layer descriptors (a prebuilt array is passed through unchanged)."""
    if isinstance(layers, C.Array):
        return layers
    arr = (MoeWeightsC * len(layers))()
    for i, w in enumerate(layers):
        arr[i] = w.c
    return arr


def mdw_stack_workspace_bytes(layers, head, m: int, topk: int) -> int:
    hc = C.byref(head.c) if head is not None else None
    return lib().mdw_stack_workspace_bytes(_layer_array(layers), len(layers), hc, m, topk)


def moe_decode_stack(layers, head, r0: torch.Tensor, argmax_out, ws: torch.Tensor,
                     resid_out=None, logits=None, topk: int = 1, topk_idx=None, topk_val=None,
                     stream=None) -> None:
    """head=None runs the layers only (resid_out required); lm_head_fp8_rmsnorm finishes."""
    arr = _layer_array(layers)
    hc = C.byref(head.c) if head is not None else None
    code = lib().moe_decode_stack(arr, len(layers), hc, r0.shape[0], _ptr(r0), _ptr(resid_out),
                                  _ptr(logits), _ptr(argmax_out), topk, _ptr(topk_idx), _ptr(topk_val),
                                  _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check("moe_decode_stack", code)


def moe_decode_stack_routed(layers, head, r0: torch.Tensor, argmax_out, ws: torch.Tensor, topk_override,
                            resid_out=None, logits=None, topk: int = 1, topk_idx=None, topk_val=None,
                            stream=None) -> None:
    """moe_decode_stack with imposed routing: topk_override int32 [L, M, K] on the device (or None)."""
    arr = _layer_array(layers)
    hc = C.byref(head.c) if head is not None else None
    code = lib().moe_decode_stack_routed(arr, len(layers), hc, r0.shape[0], _ptr(r0), _ptr(resid_out),
                                         _ptr(logits), _ptr(argmax_out), topk, _ptr(topk_idx), _ptr(topk_val),
                                         _ptr(topk_override), _ptr(ws), ws.numel() * ws.element_size(),
                                         _stream(stream))
    _check("moe_decode_stack_routed", code)


def mdw_device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns the device status word of the workspace."""
    return lib().mdw_device_status(_ptr(ws), _stream(stream))


# ------------------------------------------------------- the attention sub-layer of a window

_DT = {torch.bfloat16: DT_BF16, torch.float16: DT_F16, torch.float32: DT_F32}
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_bound = None


def _binding():
    """The extension that reads the tensors of the calls below and makes them (loaded once)."""
    global _bound
    if _bound is not None:
        return _bound
    path = os.path.join(_PKG, "_binding.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with moe_decode_weight_gb300.build.build()")
    L = lib()
    loader = importlib.machinery.ExtensionFileLoader("_binding", path)
    m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_binding", path, loader=loader))
    loader.exec_module(m)
    # the raw handles: the objects that torch.cuda.current_stream() builds cost as much as a launch
    device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
    m.setup((torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.uint8, torch.int32, torch.int64, torch.uint64),
            MdwError, device, stream, tuple(C.cast(f, C.c_void_p).value for f in
                                            (L.w4_linear, L.mdw_kv_plan, L.mdw_kv_write, L.mdw_tree_attention, L.mdw_linear_attention,
                                             L.mdw_linear_tree_attention, L.mdw_linear_state_advance, L.mdw_block_norm)))
    _bound = m
    return m


def _call(fn, *args):
    """fn(*args); it answers with a device where its tensors are on another one than the current."""
    device = fn(*args)
    if device is not None:
        with torch.cuda.device(device):
            fn(*args)


def _packed_rows(shape, stride) -> bool:
    """Whether a tensor is contiguous from its second dimension on."""
    width = 1
    for n, step in zip(reversed(shape[1:]), reversed(stride[1:])):
        if n != 1 and step != width:
            return False
        width *= n
    return True


def _address(fn: str, t: torch.Tensor, name: str, dtypes, device, shape=None) -> int:
    """Address of a handle's tensor, contiguous from its second dimension on."""
    if not t.is_cuda or t.device != device or (shape is not None and t.shape != shape) or not _packed_rows(t.shape, t.stride()):
        raise MdwError(fn, 1, f"{name}: {tuple(t.shape)} on {t.device}, strides {t.stride()}; wanted {shape or 'its'} shape on {device}")
    if t.dtype not in dtypes:
        raise MdwError(fn, 3, f"{name} has type {t.dtype}")
    return t.data_ptr()


@dataclass
class W4Weights:
    """A dense weight in int4 with group scales (descriptor and the tensors it points at): q uint8
    [N, K/2], scale bf16 or f16 [N, K/group], zero uint8 [N, K/group] or None (8 everywhere)."""
    q: torch.Tensor
    scale: torch.Tensor
    zero: torch.Tensor | None = None
    c: W4WeightsC = field(init=False)
    address: int = field(init=False)
    device_index: int = field(init=False)

    def __post_init__(self):
        fn, q, scale = "W4Weights", self.q, self.scale
        if q.dim() != 2 or scale.dim() != 2 or scale.shape[0] != q.shape[0]:
            raise MdwError(fn, 1, "q is [N, K/2], scale [N, K/group]")
        n, k, groups = q.shape[0], 2 * q.shape[1], scale.shape[1]
        if n < 1 or groups < 1 or k % groups != 0 or k // groups not in (32, 64, 128):
            raise MdwError(fn, 2, f"{k} input features in {groups} groups: groups are 32, 64 or 128 wide")
        for t in (q, scale, self.zero):
            if t is not None and not t.is_contiguous():
                raise MdwError(fn, 1, "weights are contiguous")
        self.c = W4WeightsC(MDW_MAGIC, FMT_INT4_GROUP, n, k, k // groups, _DT.get(scale.dtype, 0),
                            _address(fn, q, "q", (torch.uint8,), q.device),
                            _address(fn, scale, "scale", (torch.bfloat16, torch.float16), q.device),
                            None if self.zero is None else _address(fn, self.zero, "zero", (torch.uint8,), q.device, scale.shape))
        self.address = C.addressof(self.c)
        self.device_index = q.get_device()


def w4_linear(w: W4Weights, x: torch.Tensor, y: torch.Tensor, bias=None, residual=None, status=None,
              stream=None) -> None:
    """y = x . W^T (+ bias) (+ residual) for x [M, K], M <= 32; y [M, N] in x's type or float32."""
    _call((_bound or _binding()).w4_linear, w, x, y, bias, residual, status, stream)


@dataclass
class KVCache:
    """A paged key/value cache (descriptor and its tensors): k, v [pages, kv heads, page size, head dim] in
    bf16, f16 or E4M3 (float8_e4m3fn or uint8, with k_scale, v_scale float32 [kv heads]); the pages
    may be strided, what is inside one is contiguous."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None
    c: KVCacheC = field(init=False)
    address: int = field(init=False)
    device_index: int = field(init=False)

    def __post_init__(self):
        fn, k, v = "KVCache", self.k, self.v
        if k.dim() != 4:
            raise MdwError(fn, 1, "k and v are [pages, kv heads, page size, head dim]")
        fp8 = k.dtype in _E4M3
        pk = _address(fn, k, "k", _E4M3 if fp8 else (torch.bfloat16, torch.float16), k.device)
        pv = _address(fn, v, "v", (k.dtype,), k.device, k.shape)
        strides = {k.stride(0), v.stride(0)} if k.shape[0] > 1 else {k.shape[1] * k.shape[2] * k.shape[3]}
        if len(strides) > 1:
            raise MdwError(fn, 1, f"k and v have page strides {strides}")
        if fp8 != (self.k_scale is not None) or fp8 != (self.v_scale is not None):
            raise MdwError(fn, 1, "k_scale and v_scale belong to E4M3 caches, and to no other")
        scales = [None, None]
        if fp8:
            scales = [_address(fn, t.view(1, -1), n, (torch.float32,), k.device, (1, k.shape[1]))
                      for t, n in ((self.k_scale, "k_scale"), (self.v_scale, "v_scale"))]
        self.c = KVCacheC(MDW_MAGIC, FMT_KV_PAGED, DT_E4M3 if fp8 else _DT[k.dtype], k.shape[0], k.shape[2],
                          k.shape[1], k.shape[3], 0, strides.pop(), pk, pv, *scales)
        self.address = C.addressof(self.c)
        self.device_index = k.get_device()


def mdw_kv_plan(ctx_len: torch.Tensor, new_len: torch.Tensor, page_size: int, num_pages: int,
                block_table: torch.Tensor, free_pages: torch.Tensor, row_start: torch.Tensor,
                slot_map: torch.Tensor, positions: torch.Tensor, pages_taken: torch.Tensor, parents=None,
                tree_mask=None, status=None, stream=None) -> None:
    """Block tables, slot map, positions and tree masks from request lengths (see the C declaration):
    ctx_len, new_len int32 [B]; block_table int32 [B, max pages]; free_pages int32 [F]; row_start int32
    [B + 1]; slot_map int64 [T]; positions, parents int32 [T]; tree_mask int64 or uint64 [T];
    pages_taken, status int32 [1]."""
    _call((_bound or _binding()).kv_plan, ctx_len, new_len, page_size, num_pages, block_table, free_pages, row_start, slot_map,
          positions, pages_taken, parents, tree_mask, status, stream)


def mdw_kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, status=None,
                 stream=None) -> None:
    """Rows k, v [T, kv heads, head dim] (rows may be strided) to the cache's slots slot_map int64 [T]."""
    _call((_bound or _binding()).kv_write, cache, k, v, slot_map, status, stream)


def mdw_tree_attention_workspace_bytes(cache: KVCache, b: int, t: int, q_heads: int, max_new: int) -> int:
    if cache.k.get_device() == torch.cuda.current_device():
        return lib().mdw_tree_attention_workspace_bytes(cache.c, b, t, q_heads, max_new)
    with torch.cuda.device(cache.k.device):
        return lib().mdw_tree_attention_workspace_bytes(cache.c, b, t, q_heads, max_new)


def mdw_tree_attention(cache: KVCache, q: torch.Tensor, out: torch.Tensor, block_table: torch.Tensor,
                       ctx_len: torch.Tensor, row_start: torch.Tensor, max_new: int, ws: torch.Tensor,
                       tree_mask=None, lse=None, scale: float | None = None, status=None, stream=None) -> None:
    """Attention of the drafted rows q [T, query heads, head dim] over the paged cache (see the C
    declaration); out like q, lse float32 [T, query heads] or None, scale head_dim ** -0.5 by default, ws
    uint8 of at least mdw_tree_attention_workspace_bytes."""
    _call((_bound or _binding()).tree_attention, cache, q, out, block_table, ctx_len, row_start, max_new, ws, tree_mask, lse,
          scale, status, stream)


# ------------------------------------------- the linear-attention sub-layer, and between sub-layers


@dataclass
class LinearState:
    """The states of a linear-attention layer (descriptor and its tensor): s float32 [slots, value heads, head
    dim, head dim]; the slots may be strided, what is inside one is contiguous."""
    s: torch.Tensor
    c: LinearStateC = field(init=False)
    address: int = field(init=False)
    device_index: int = field(init=False)

    def __post_init__(self):
        fn, s = "LinearState", self.s
        if s.dim() != 4 or s.shape[2] != s.shape[3]:
            raise MdwError(fn, 1, "s is [slots, value heads, head dim, head dim]")
        p = _address(fn, s, "s", (torch.float32,), s.device)
        stride = s.stride(0) if s.shape[0] > 1 else s.shape[1] * s.shape[2] * s.shape[3]
        self.c = LinearStateC(MDW_MAGIC, FMT_LINEAR_STATE, s.shape[0], s.shape[1], s.shape[2], 0, stride, p)
        self.address = C.addressof(self.c)
        self.device_index = s.get_device()


def mdw_linear_attention_workspace_bytes(state: LinearState, b: int, t: int, qk_heads: int, max_new: int) -> int:
    if state.s.get_device() == torch.cuda.current_device():
        return lib().mdw_linear_attention_workspace_bytes(state.c, b, t, qk_heads, max_new)
    with torch.cuda.device(state.s.device):
        return lib().mdw_linear_attention_workspace_bytes(state.c, b, t, qk_heads, max_new)


def mdw_linear_attention(state: LinearState, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                         out: torch.Tensor, row_start: torch.Tensor, slot_in: torch.Tensor, slot_out: torch.Tensor,
                         max_new: int, ws: torch.Tensor, scale: float | None = None, status=None, stream=None) -> None:
    """Linear attention with a decay for each head over the rows of B requests, from the states slot_in to the
    states slot_out (see the C declaration): q, k bf16 [T, key heads, head dim], v, out bf16 [T, value heads, head
    dim] (rows may be strided), log_decay float32 [T, value heads] or [value heads], row_start int32 [B + 1],
    slot_in, slot_out int32 [B], scale head_dim ** -0.5 by default, ws uint8 of at least
    mdw_linear_attention_workspace_bytes."""
    _call((_bound or _binding()).linear_attention, state, q, k, v, log_decay, out, row_start, slot_in, slot_out, max_new, ws,
          scale, status, stream)


def mdw_linear_tree_attention(state: LinearState, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                              out: torch.Tensor, row_start: torch.Tensor, slot_in: torch.Tensor, max_new: int,
                              tree_mask=None, scale: float | None = None, status=None, stream=None) -> None:
    """The same for trees of drafted tokens (tree_mask int64 or uint64 [T], as mdw_kv_plan gives it; None: chains); the
    states stay as they are."""
    _call((_bound or _binding()).linear_tree_attention, state, q, k, v, log_decay, out, row_start, slot_in, max_new, tree_mask,
          scale, status, stream)


def mdw_linear_state_advance(state: LinearState, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                             row_start: torch.Tensor, accepted: torch.Tensor, slot_in: torch.Tensor, slot_out: torch.Tensor,
                             max_new: int, status=None, stream=None) -> None:
    """The states after the accepted rows of each request: accepted int64 or uint64 [B], a bit per row."""
    _call((_bound or _binding()).linear_state_advance, state, k, v, log_decay, row_start, accepted, slot_in, slot_out, max_new,
          status, stream)


def mdw_block_norm(y: torch.Tensor, sum: torch.Tensor | None, post_weight=None, group: int | None = None, gate=None,
                   gate_kind: str = "none", residual=None, pre_weight=None, x=None, branch_scale: float = 1.0,
                   residual_scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """Norm after a sub-layer, gate, scaled residual and norm before the next (see the C declaration): y [T, W];
    sum = residual_scale * residual + branch_scale * act(gate) * norm(y) and x = norm(sum) * pre_weight, both [T, W], x of the
    sum as rounded to sum's type (without sum to residual's, without either to float32);
    post_weight [group] (W by default), gate [T, W] or [W], gate_kind "none", "mul", "sigmoid" or "silu"."""
    if gate_kind not in GATES:
        raise MdwError("mdw_block_norm", 1, f"gate_kind {gate_kind!r} is none of {sorted(GATES)}")
    _call((_bound or _binding()).block_norm, y, sum, post_weight, group, gate, GATES[gate_kind], residual, pre_weight, x,
          branch_scale, residual_scale, eps, stream)
