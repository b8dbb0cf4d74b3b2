"""Python binding of libhfq4moe.so: the routed-expert HFQ4 MoE layer on B200.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Functions carry the C ABI's names (see include/hfq4moe.h) and take
torch tensors, numpy arrays, raw integer addresses or None for pointers, and
a torch stream, a raw cudaStream_t integer or None (= torch's current stream)
for streams.  A failed call raises HfqError with the library's message.

The library must be built (``python -m expert_offload_b200.build``); there is
no fallback of any kind when it is missing.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libhfq4moe.so")

HFQ_OK = 0
STATUS = {0: "HFQ_OK", -1: "HFQ_ERR_ARG", -2: "HFQ_ERR_ALIGN", -3: "HFQ_ERR_UNSUPPORTED",
          -4: "HFQ_ERR_NOFIT", -5: "HFQ_ERR_CUDA", -6: "HFQ_ERR_TIMEOUT", -7: "HFQ_ERR_ALLOC",
          -8: "HFQ_ERR_WORKSPACE"}
HFQ_F32, HFQ_BF16 = 0, 1
PATH_AUTO, PATH_GEMV, PATH_TC = 0, 1, 2
ARENA_HUGEPAGE = 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_FULL = 0, 1, 2, 3
GATE_LINEAR, GATE_SIGMOID = 0, 1
ACT_NONE, ACT_SWIGLU = 0, 1
BLOCK, BLOCK_BYTES = 256, 136
MAX_EXPERTS, MAX_TOPK, MAX_STACK_LAYERS = 512, 16, 64
MAX_GROUPS, Q8_MAX_K = 32, 16384


class HfqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


class hfq4_layer(ctypes.Structure):
    _fields_ = [("expert_ptr", ctypes.c_void_p), ("expert_loc", ctypes.c_void_p),
                ("n_experts", ctypes.c_int), ("hidden", ctypes.c_int), ("inter", ctypes.c_int)]


class moe_route_rule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int),
                ("group_top", ctypes.c_int), ("renormalise", ctypes.c_int), ("scale", ctypes.c_float)]


class moe_norm_rule(ctypes.Structure):
    _fields_ = [("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p), ("w_dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("w_offset", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("gate_kind", ctypes.c_int), ("gate_act", ctypes.c_int)]


_vp, _i, _sz, _u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64

# name -> (restype, argtypes)
_SIGS = {
    "hfq_last_error": (ctypes.c_char_p, []),
    "hfq_version": (_i, []),
    "hfq4_matrix_bytes": (_sz, [_i, _i]),
    "hfq4_expert_bytes": (_sz, [_i, _i]),
    "hfq4_pack_experts": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _sz]),
    "hfq4_pack_experts_device": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _sz, _vp]),
    "hfq4_dequant": (_i, [_vp, _i, _i, _vp, _vp]),
    "hfq_route_workspace_bytes": (_sz, [_i, _i, _i]),
    "moe_route": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_route_scored_workspace_bytes": (_sz, [_i, _i, _i]),
    "moe_route_scored": (_i, [_vp, _i, _i, _i, _i, _vp, ctypes.POINTER(moe_route_rule), _i, _vp, _vp, _vp,
                              _vp, _vp, _vp, _sz, _vp]),
    "moe_norm_residual": (_i, [ctypes.POINTER(moe_norm_rule), _i, _i, _vp, _i, _i, _vp, _vp, _i, _i, _vp,
                               _vp, _vp, _vp, _i, _vp, _vp, _vp]),
    "q8_quantize_rows": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _i, _vp, _vp]),
    "q8_matmul": (_i, [_vp, _i, _vp, _i, _i, _vp, _i, _vp, _i, _vp, _i, _i, _vp]),
    "q8_linear_workspace_bytes": (_sz, [_i, _i, _i]),
    "q8_linear": (_i, [_vp, _i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _i, _i, _vp, _sz, _vp]),
    "hfq4_moe_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "hfq4_moe_forward": (_i, [ctypes.POINTER(hfq4_layer), _vp, _i, _i, _vp, _vp, _i, _vp, _vp,
                              _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "hfq4_moe_forward_noalloc": (_i, [ctypes.POINTER(hfq4_layer), _vp, _i, _i, _vp, _vp, _i,
                                      _vp, _vp, _vp]),
    "hfq4_stack_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "hfq4_stack_launches": (_i, [_i, _i, _i, _i, _i]),
    "hfq4_moe_decode_stack": (_i, [ctypes.POINTER(hfq4_layer), _i, _vp, _i, _vp, _i, _vp, _vp,
                                   _vp, _vp, _i, _vp, _sz, _vp]),
    "moe_router_logits": (_i, [_vp, _i, _i, _i, _vp, _i, _i, _vp, _vp]),
    "hfq4_moe_decode_stack_routed": (_i, [ctypes.POINTER(hfq4_layer), _i, _vp, _i, _i, _vp, _i,
                                          _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "hfq_workspace_status": (_i, [_vp, _sz, _vp]),
    "hfq_set_option": (_i, [_i, ctypes.c_longlong]),
    "hfq_host_arena_create": (_i, [_sz, _i, ctypes.POINTER(_vp), ctypes.POINTER(_vp)]),
    "hfq_host_arena_destroy": (_i, [_vp]),
    "hfq_placement_build": (_i, [_i, _i, _sz, _vp, _i, _i, _sz, _vp, _vp,
                                 ctypes.POINTER(_sz), ctypes.POINTER(_sz)]),
    "hfq_placement_pointers": (_i, [_i, _i, _sz, _vp, _vp, _vp, _vp, _vp]),
    "hfq_probe_read": (_i, [_vp, _sz, _i, _vp, _vp]),
    "hfq_cache_create": (_i, [_i, _i, _sz, _i, _vp, _vp, _vp, _vp, _sz, _vp, _vp, _vp,
                              ctypes.POINTER(_vp)]),
    "hfq_cache_observe": (_i, [_vp, _i, _vp, _i, _i, _vp]),
    "hfq_cache_flush": (_i, [_vp, _vp]),
    "hfq_cache_slot_of": (_i, [_vp, _i, _i, ctypes.POINTER(_i)]),
    "hfq_cache_stats": (_i, [_vp, ctypes.POINTER(_u64), ctypes.POINTER(_u64), ctypes.POINTER(_u64),
                             ctypes.POINTER(_u64)]),
    "hfq_cache_destroy": (_i, [_vp]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m expert_offload_b200.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype, f.argtypes = res, args
        _lib = l
    return _lib


def symbols():
    """Names of the C entry points this binding declares."""
    return list(_SIGS)


def last_error() -> str:
    return lib().hfq_last_error().decode()


def _check(status: int) -> None:
    if status != HFQ_OK:
        raise HfqError(status, last_error())


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if hasattr(a, "data_ptr"):
        return a.data_ptr()
    if hasattr(a, "ctypes"):
        return a.ctypes.data
    raise TypeError(f"cannot take the address of {type(a)}")


def _nbytes(a, name: str = "workspace") -> int:
    if isinstance(a, int):
        raise HfqError(-1, f"{name} must be a tensor or an array: an address does not say its size")
    if hasattr(a, "nbytes") and not callable(a.nbytes):
        return int(a.nbytes)
    return int(a.numel() * a.element_size())


_I32, _I8, _ANY = 2, 3, 4                 # operand kinds besides HFQ_F32 and HFQ_BF16
_ROUTE, _NORM, _QUANTIZE, _MATMUL, _LINEAR = range(5)
_call = None


def _dense(name, t, n) -> None:
    """n elements without a gap."""
    if not t.is_contiguous():
        raise HfqError(-1, f"{name} has gaps between its elements, which the call takes as neighbours")
    if t.numel() < n:
        raise HfqError(-1, f"{name} holds fewer elements than the call reads or writes")


def _layout(name, t, rows, cols, ld, whole) -> None:
    """Rows of cols elements that start ld apart, in a tensor that is not exactly
    rows * ld elements without a gap.  A row is what some of the last dimensions
    hold without a gap; all others count rows.  A flat buffer has no rows of its
    own, and one row has no distance."""
    dims = [(n, s) for n, s in zip(t.shape, t.stride()) if n != 1]
    have, at = 1, len(dims)              # elements of a row, from dimension `at` on
    while at and dims[at - 1][1] == have and have < ld:
        at -= 1
        have *= dims[at][0]
    if at == 0:                          # without a gap up to ld or the tensor's end
        flat = len(dims) <= 1 or rows == 1 or have == ld
        ok = flat and have >= (rows - 1) * ld + cols
    elif rows == 1:
        ok = have >= cols
    else:
        count, step = 1, ld
        for n, s in reversed(dims[:at]):
            if s != step:
                break
            count, step = count * n, step * n
        ok = have >= cols and have <= ld and count >= rows
    if not ok:
        raise HfqError(-1, f"{name} does not hold {rows} rows of {cols} elements that start {ld} apart")
    if whole > cols and (t.untyped_storage().nbytes() // t.element_size() - t.storage_offset() <
                         (rows - 1) * ld + whole):
        raise HfqError(-1, f"{name} needs {whole} elements of memory for its last row")


def _bind(*args) -> None:
    """Loads and sets up the native module at the first call that finds torch."""
    global _call
    lib()
    path = os.path.join(PKG, "lib", "_bind.so")
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m expert_offload_b200.build`")
    spec = importlib.util.spec_from_file_location("_bind", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    torch = sys.modules.get("torch")
    if torch is None:
        mod.setup(HfqError, _layout, None, None, {})
    else:
        mod.setup(HfqError, _layout, torch.Tensor, torch._C._cuda_getDevice if torch.cuda.is_available() else None,
                  {HFQ_F32: (torch.float32,), HFQ_BF16: (torch.bfloat16, torch.int16, torch.uint16),
                   _I32: (torch.int32,), _I8: (torch.int8,),
                   _ANY: (torch.uint8, torch.int8, torch.int16, torch.int32, torch.int64, torch.float32)})
        _call = mod.call
    mod.call(*args)


def _stream(s):
    if s is None:
        torch = sys.modules.get("torch")
        if torch is None:
            return None
        if torch.cuda.is_initialized():
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        if torch.cuda.is_available():
            return torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


# ------------------------------------------------------------------ sizes

def hfq4_matrix_bytes(rows: int, cols: int) -> int:
    return lib().hfq4_matrix_bytes(rows, cols)


def hfq4_expert_bytes(hidden: int, inter: int) -> int:
    return lib().hfq4_expert_bytes(hidden, inter)


# ---------------------------------------------------------------- packing

def hfq4_pack_experts(gate, up, down, out, n_experts: int, hidden: int, inter: int) -> None:
    """Host packer: numpy f32 gate/up [E,I,H], down [E,H,I] -> out uint8 bytes."""
    _check(lib().hfq4_pack_experts(_ptr(gate), _ptr(up), _ptr(down), n_experts, hidden, inter,
                                   _ptr(out), _nbytes(out, "out")))


def hfq4_pack_experts_device(gate, up, down, out, n_experts: int, hidden: int, inter: int,
                             stream=None) -> None:
    _check(lib().hfq4_pack_experts_device(_ptr(gate), _ptr(up), _ptr(down), n_experts, hidden,
                                          inter, _ptr(out), _nbytes(out, "out"), _stream(stream)))


def hfq4_dequant(blocks, rows: int, cols: int, out, stream=None) -> None:
    _check(lib().hfq4_dequant(_ptr(blocks), rows, cols, _ptr(out), _stream(stream)))


# ------------------------------------------------------------------ route

def hfq_route_workspace_bytes(T: int, E: int, k: int) -> int:
    return lib().hfq_route_workspace_bytes(T, E, k)


def moe_route(logits, T: int, E: int, k: int, idx, wts, cnt=None, off=None, perm=None,
              workspace=None, stream=None) -> None:
    ws_bytes = _nbytes(workspace) if workspace is not None else 0
    _check(lib().moe_route(_ptr(logits), T, E, k, _ptr(idx), _ptr(wts), _ptr(cnt), _ptr(off),
                           _ptr(perm), _ptr(workspace), ws_bytes, _stream(stream)))


def moe_router_logits(x, x_dtype: int, T: int, hidden: int, router, router_dtype: int,
                      n_experts: int, logits, stream=None) -> None:
    """logits [T, E] f32 = x Wr^T on the device."""
    _check(lib().moe_router_logits(_ptr(x), x_dtype, T, hidden, _ptr(router), router_dtype,
                                   n_experts, _ptr(logits), _stream(stream)))


class RouteRule:
    """How moe_route_scored scores, groups and weighs (a moe_route_rule)."""

    def __init__(self, score: int = SCORE_SOFTMAX, n_groups: int = 1, topk_groups: int = 1,
                 group_top: int = 1, renormalise: bool = True, scale: float = 1.0):
        self.struct = moe_route_rule(score, n_groups, topk_groups, group_top, int(renormalise), scale)
        self.address = ctypes.addressof(self.struct)


def moe_route_scored_workspace_bytes(T: int, E: int, k: int) -> int:
    return lib().moe_route_scored_workspace_bytes(T, E, k)


def moe_route_scored(logits, logits_dtype: int, T: int, E: int, k: int, rule: RouteRule, idx, wts,
                     bias=None, cnt=None, off=None, perm=None, workspace=None, ld: int = 0,
                     stream=None) -> None:
    """Top-k routing by scores and a bias, with groups; lists as moe_route's."""
    (_call or _bind)(_ROUTE, ("logits", logits, logits_dtype, T, E, ld or E, E), logits_dtype, ld, T, E,
                     bias if bias is None else ("bias", bias, HFQ_F32, 1, E), rule.address, k,
                     ("idx", idx, _I32, T, k), ("wts", wts, HFQ_F32, T, k),
                     cnt if cnt is None else ("cnt", cnt, _I32, 1, E),
                     off if off is None else ("off", off, _I32, 1, E + 1),
                     perm if perm is None else ("perm", perm, _I32, T, k),
                     workspace if workspace is None else ("workspace", workspace, _ANY, 0, 0),
                     0 if workspace is None else _nbytes(workspace), _stream(stream))


# ---------------------------------------------------- norm, gate, residual

class NormRule:
    """What moe_norm_residual does to every row (a moe_norm_rule); keeps the
    weights it points to alive."""

    def __init__(self, w_post=None, w_pre=None, w_dtype: int = HFQ_BF16, eps: float = 1e-6,
                 w_offset: float = 0.0, residual_scale: float = 1.0, branch_scale: float = 1.0,
                 gate_kind: int = GATE_NONE, gate_act: int = GATE_LINEAR):
        self.w_post, self.w_pre, self.w_dtype, self.gate_kind = w_post, w_pre, w_dtype, gate_kind
        self.struct = moe_norm_rule(_ptr(w_post), _ptr(w_pre), w_dtype, eps, w_offset, residual_scale,
                                    branch_scale, gate_kind, gate_act)
        self.address = ctypes.addressof(self.struct)
        self.tensors = any(w is not None and type(w) is not int for w in (w_post, w_pre))
        self.checked = 0                 # elements that the weights are known to have ...
        self.device = None               # ... on this device

    def check(self, H: int) -> None:
        """The weights hold H elements of their type on the current device; they
        are the rule's own, so once is enough for each length and device."""
        for name, w in (("w_post", self.w_post), ("w_pre", self.w_pre)):
            if w is None or type(w) is int:
                continue
            torch = sys.modules.get("torch")
            kinds = (torch.float32,) if self.w_dtype == HFQ_F32 else (torch.bfloat16, torch.int16, torch.uint16)
            if not w.is_cuda or w.get_device() != torch._C._cuda_getDevice() or w.dtype not in kinds:
                raise HfqError(-1, f"{name} is not a tensor of the current CUDA device of the rule's w_dtype")
            _dense(name, w, H)
            self.device = w.get_device()
        self.checked = H


def moe_norm_residual(rule: NormRule, T: int, H: int, x, x_dtype: int, y=None, y_dtype: int = HFQ_F32,
                      y2=None, y2_gate=None, gate=None, x_out=None, xn=None, xn_dtype: int = HFQ_BF16,
                      xq=None, xq_scale=None, ldx: int = 0, ldy: int = 0, stream=None) -> None:
    """x' = residual_scale x + branch_scale gate norm(y + y2), xn = norm(x')."""
    if rule.tensors and (rule.checked < H or rule.device != sys.modules["torch"]._C._cuda_getDevice()):
        rule.check(H)
    lx, ly, kind = ldx or H, ldy or H, rule.gate_kind
    (_call or _bind)(_NORM, rule.address, T, H, ("x", x, x_dtype, T, H, lx, H), x_dtype, ldx,
                     y if y is None else ("y", y, y_dtype, T, H, ly, H),
                     y2 if y2 is None else ("y2", y2, y_dtype, T, H, ly, H), y_dtype, ldy,
                     y2_gate if y2_gate is None else ("y2_gate", y2_gate, HFQ_F32, T, 1),
                     gate if gate is None else
                     ("gate", gate, HFQ_F32, 1 if kind == GATE_CHANNEL else T, 1 if kind == GATE_TOKEN else H),
                     x_out if x_out is None else ("x_out", x_out, x_dtype, T, H, lx, H),
                     xn if xn is None else ("xn", xn, xn_dtype, T, H), xn_dtype,
                     xq if xq is None else ("xq", xq, _I8, T, -(-H // 16) * 16),
                     xq_scale if xq_scale is None else ("xq_scale", xq_scale, HFQ_F32, T, 1), _stream(stream))


# --------------------------------------------------- products in 8 bits

def q8_quantize_rows(x, x_dtype: int, rows: int, cols: int, q, scale, act: int = ACT_NONE, ldx: int = 0,
                     ldq: int = 0, stream=None) -> None:
    """int8 rows and their f32 scales; act ACT_SWIGLU quantises silu(gate) * up."""
    width = 2 * cols if act == ACT_SWIGLU else cols
    c16 = -(-cols // 16) * 16
    (_call or _bind)(_QUANTIZE, ("x", x, x_dtype, rows, width, ldx or width, width), x_dtype, ldx, rows, cols, act,
                     ("q", q, _I8, rows, c16, ldq or c16, c16), ldq, ("scale", scale, HFQ_F32, rows, 1),
                     _stream(stream))


def q8_matmul(xq, xs, T: int, K: int, wq, ws, N: int, y, y_dtype: int, ldxq: int = 0, ldw: int = 0,
              ldy: int = 0, stream=None) -> None:
    """y = (xq wq^T) * xs * ws for quantised rows xq and channels wq."""
    k16 = -(-K // 16) * 16
    (_call or _bind)(_MATMUL, ("xq", xq, _I8, T, K, ldxq or k16, k16), ldxq, ("xs", xs, HFQ_F32, T, 1), T, K,
                     ("wq", wq, _I8, N, K, ldw or k16, k16), ldw, ("ws", ws, HFQ_F32, N, 1), N,
                     ("y", y, y_dtype, T, N, ldy or N, N), y_dtype, ldy, _stream(stream))


def q8_linear_workspace_bytes(T: int, K: int, N: int) -> int:
    return lib().q8_linear_workspace_bytes(T, K, N)


def q8_linear(x, x_dtype: int, T: int, K: int, wq, ws, N: int, y, y_dtype: int, workspace=None, ldx: int = 0,
              ldw: int = 0, ldy: int = 0, stream=None) -> None:
    """y = x W^T with x quantised on the way: q8_quantize_rows, then q8_matmul."""
    k16 = -(-K // 16) * 16
    (_call or _bind)(_LINEAR, ("x", x, x_dtype, T, K, ldx or K, K), x_dtype, ldx, T, K,
                     ("wq", wq, _I8, N, K, ldw or k16, k16), ldw, ("ws", ws, HFQ_F32, N, 1), N,
                     ("y", y, y_dtype, T, N, ldy or N, N), y_dtype, ldy,
                     workspace if workspace is None else ("workspace", workspace, _ANY, 0, 0),
                     0 if workspace is None else _nbytes(workspace), _stream(stream))


# ---------------------------------------------------------------- forward

class Layer:
    """Keeps an hfq4_layer struct and the device tensors it points to alive."""

    def __init__(self, expert_ptr, n_experts: int, hidden: int, inter: int, expert_loc=None):
        self.expert_ptr, self.expert_loc = expert_ptr, expert_loc
        self.struct = hfq4_layer(_ptr(expert_ptr), _ptr(expert_loc), n_experts, hidden, inter)


def hfq4_moe_workspace_bytes(T: int, k: int, hidden: int, inter: int, n_experts: int) -> int:
    return lib().hfq4_moe_workspace_bytes(T, k, hidden, inter, n_experts)


def hfq4_moe_forward(layer: Layer, x, x_dtype: int, T: int, idx, wts, k: int, y, workspace,
                     y_bf16=None, cnt=None, off=None, perm=None, path: int = PATH_AUTO,
                     stream=None) -> None:
    _check(lib().hfq4_moe_forward(ctypes.byref(layer.struct), _ptr(x), x_dtype, T, _ptr(idx),
                                  _ptr(wts), k, _ptr(cnt), _ptr(off), _ptr(perm), _ptr(y),
                                  _ptr(y_bf16), path, _ptr(workspace), _nbytes(workspace),
                                  _stream(stream)))


def hfq4_moe_forward_noalloc(layer: Layer, x, x_dtype: int, T: int, idx, wts, k: int, y,
                             y_bf16=None, stream=None) -> None:
    """hfq4_moe_forward without a workspace: for callers that cannot allocate
    device memory (scratch is a fixed array inside the library)."""
    _check(lib().hfq4_moe_forward_noalloc(ctypes.byref(layer.struct), _ptr(x), x_dtype, T,
                                          _ptr(idx), _ptr(wts), k, _ptr(y), _ptr(y_bf16),
                                          _stream(stream)))


def hfq4_stack_workspace_bytes(T: int, k: int, hidden: int, inter: int, n_experts: int) -> int:
    return lib().hfq4_stack_workspace_bytes(T, k, hidden, inter, n_experts)


def hfq4_stack_launches(n_layers: int, T: int, k: int, hidden: int, inter: int) -> int:
    return lib().hfq4_stack_launches(n_layers, T, k, hidden, inter)


def layer_array(layers):
    arr = (hfq4_layer * len(layers))()
    for i, l in enumerate(layers):
        arr[i] = l.struct
    return arr


def hfq4_moe_decode_stack(layers, logits, k: int, x0, T: int, x_out, workspace, y_all=None,
                          idx_all=None, wts_all=None, path: int = PATH_AUTO, stream=None,
                          _layer_array=None) -> None:
    arr = _layer_array if _layer_array is not None else layer_array(layers)
    _check(lib().hfq4_moe_decode_stack(arr, len(layers), _ptr(logits), k, _ptr(x0), T, _ptr(x_out),
                                       _ptr(y_all), _ptr(idx_all), _ptr(wts_all), path,
                                       _ptr(workspace), _nbytes(workspace), _stream(stream)))


def hfq4_moe_decode_stack_routed(layers, router, router_dtype: int, k: int, x0, T: int, x_out,
                                 workspace, y_all=None, idx_all=None, wts_all=None,
                                 logits_all=None, stream=None, _layer_array=None) -> None:
    arr = _layer_array if _layer_array is not None else layer_array(layers)
    _check(lib().hfq4_moe_decode_stack_routed(arr, len(layers), _ptr(router), router_dtype, k,
                                              _ptr(x0), T, _ptr(x_out), _ptr(y_all),
                                              _ptr(idx_all), _ptr(wts_all), _ptr(logits_all),
                                              _ptr(workspace), _nbytes(workspace),
                                              _stream(stream)))


OPT_WAIT_TIMEOUT_NS, OPT_TEST_MISSING_ARRIVALS, OPT_TIMELINE_BUFFER = 1, 2, 3


def hfq_set_option(option: int, value: int) -> None:
    _check(lib().hfq_set_option(option, value))


def hfq_workspace_status(workspace, stream=None) -> None:
    """Raises HfqError for a device-side error recorded in the workspace; None
    reads the array of hfq4_moe_forward_noalloc on the current device."""
    nbytes = 0 if workspace is None else _nbytes(workspace)
    _check(lib().hfq_workspace_status(_ptr(workspace), nbytes, _stream(stream)))


# --------------------------------------------------------- offload plumbing

def hfq_host_arena_create(nbytes: int, flags: int = 0):
    """Returns (host_address, device_address) of a pinned, mapped arena."""
    h, d = ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib().hfq_host_arena_create(nbytes, flags, ctypes.byref(h), ctypes.byref(d)))
    return h.value, d.value


def hfq_host_arena_destroy(host: int) -> None:
    _check(lib().hfq_host_arena_destroy(host))


def hfq_placement_build(counts, expert_bytes: int, resident_layers: int, hot_per_layer: int,
                        hbm_budget: int):
    """Returns (loc uint8 [L,E], slot int64 [L,E], hbm_needed, host_needed)."""
    import numpy as np
    counts = np.ascontiguousarray(counts, dtype=np.uint32)
    L, E = counts.shape
    loc = np.zeros((L, E), dtype=np.uint8)
    slot = np.zeros((L, E), dtype=np.int64)
    hn, hs = ctypes.c_size_t(), ctypes.c_size_t()
    st = lib().hfq_placement_build(L, E, expert_bytes, counts.ctypes.data, resident_layers,
                                   hot_per_layer, hbm_budget, loc.ctypes.data, slot.ctypes.data,
                                   ctypes.byref(hn), ctypes.byref(hs))
    if st != HFQ_OK:
        err = HfqError(st, last_error())
        err.hbm_needed, err.host_needed = hn.value, hs.value
        raise err
    return loc, slot, hn.value, hs.value


def hfq_placement_pointers(loc, slot, expert_bytes: int, hbm_base: int, host_dev_base: int):
    import numpy as np
    L, E = loc.shape
    out = np.zeros((L, E), dtype=np.uint64)
    _check(lib().hfq_placement_pointers(L, E, expert_bytes, _ptr(np.ascontiguousarray(loc)),
                                        _ptr(np.ascontiguousarray(slot)), hbm_base, host_dev_base,
                                        out.ctypes.data))
    return out


def hfq_probe_read(src, nbytes: int, iters: int, sink, stream=None) -> None:
    _check(lib().hfq_probe_read(_ptr(src), nbytes, iters, _ptr(sink), _stream(stream)))


# ------------------------------------------------------------ expert cache

class ExpertCache:
    """hfq_cache_* over the pointer (and location) tables of L layers.

    home, host_src: uint64 [L, E] numpy arrays (see include/hfq4moe.h);
    home_loc: uint8 [L, E]; slot_mem, table_dev, loc_dev: device tensors or
    None (table_dev None: bookkeeping only)."""

    def __init__(self, L: int, E: int, expert_bytes: int, slots: int, home, host_src, home_loc,
                 slot_mem=None, table_dev=None, loc_dev=None, stream=None):
        import numpy as np
        self._keep = [np.ascontiguousarray(home, np.uint64), np.ascontiguousarray(host_src, np.uint64),
                      np.ascontiguousarray(home_loc, np.uint8)]
        h = ctypes.c_void_p()
        _check(lib().hfq_cache_create(L, E, expert_bytes, slots, self._keep[0].ctypes.data,
                                      self._keep[1].ctypes.data, self._keep[2].ctypes.data,
                                      _ptr(slot_mem), _nbytes(slot_mem, "slot_mem") if slot_mem is not None else 0,
                                      _ptr(table_dev), _ptr(loc_dev), _stream(stream), ctypes.byref(h)))
        self.handle = h.value

    def observe(self, layer: int, ids, max_admit: int, stream=None) -> None:
        import numpy as np
        a = np.ascontiguousarray(ids, np.int32).ravel()
        _check(lib().hfq_cache_observe(self.handle, layer, a.ctypes.data, a.size, max_admit,
                                       _stream(stream)))

    def flush(self, stream=None) -> None:
        """Names the slots of the refills still in flight."""
        _check(lib().hfq_cache_flush(self.handle, _stream(stream)))

    def slot_of(self, layer: int, expert: int) -> int:
        s = ctypes.c_int()
        _check(lib().hfq_cache_slot_of(self.handle, layer, expert, ctypes.byref(s)))
        return s.value

    def stats(self):
        v = [ctypes.c_uint64() for _ in range(4)]
        _check(lib().hfq_cache_stats(self.handle, *[ctypes.byref(x) for x in v]))
        return dict(zip(("hits", "misses", "admitted", "evicted"), (x.value for x in v)))

    def close(self) -> None:
        if self.handle:
            _check(lib().hfq_cache_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except (HfqError, AttributeError, TypeError):
            pass
