"""ctypes binding of the C ABI in include/moe_gb300.h (argument marshalling only).

Every function keeps the C name and argument order.  Array arguments accept a
torch tensor (its data_ptr() is passed), a raw integer device address, or
None for a nullable pointer; `stream` defaults to torch's current CUDA stream.
A non-MOE_OK status raises MoeError with the library's own message.  Nothing
here computes any part of the layer: if the CUDA library cannot be loaded,
every call fails loudly.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
HEADER = os.path.join(os.path.dirname(HERE), "include", "moe_gb300.h")

(MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_DEVICE_CHECK,
 MOE_ERR_TIMEOUT) = range(7)
MOE_F32, MOE_BF16, MOE_Q8_0, MOE_Q4_K, MOE_Q8_0_R, MOE_Q5_K, MOE_Q6_K, MOE_Q3_K, MOE_MXFP4, MOE_F16 = range(10)
MOE_W_OUT_IN, MOE_W_IN_OUT = range(2)
MOE_GROUPED_ROWS, MOE_GROUPED_TENSOR = range(2)
MOE_LINEAR_SPLIT, MOE_LINEAR_PAIRS = range(2)
MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_SILU = range(5)
MOE_ROUTE_SOFTMAX, MOE_ROUTE_SIGMOID_GROUP = range(2)

STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
                4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_CHECK", 6: "MOE_ERR_TIMEOUT"}


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class moe_route_cfg(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int),
                ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int), ("routed_scale", ctypes.c_float),
                ("renormalize", ctypes.c_int)]


class moe_qmat(ctypes.Structure):
    _fields_ = [("qtype", ctypes.c_int), ("data", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("expert_stride_bytes", ctypes.c_int64)]


class moe_layer_desc(ctypes.Structure):
    _fields_ = [("route", moe_route_cfg), ("hidden", ctypes.c_int), ("intermediate", ctypes.c_int),
                ("x_type", ctypes.c_int), ("W_router", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("gate", moe_qmat), ("up", moe_qmat), ("down", moe_qmat),
                ("shared_intermediate", ctypes.c_int), ("s_gate", moe_qmat), ("s_up", moe_qmat),
                ("s_down", moe_qmat), ("accumulate", ctypes.c_int), ("tc_min_tokens", ctypes.c_int),
                ("decode_chain_off", ctypes.c_int), ("norm_gamma", ctypes.c_void_p), ("norm_eps", ctypes.c_float),
                ("expert_counts", ctypes.c_void_p)]


class moe_grouped_desc(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("y_type", ctypes.c_int), ("order", ctypes.c_int), ("n_experts", ctypes.c_int),
                ("n_out", ctypes.c_int), ("n_in", ctypes.c_int), ("w", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("row_stride", ctypes.c_int64), ("expert_stride", ctypes.c_int64)]


class moe_w4_desc(ctypes.Structure):
    _fields_ = [("x_type", ctypes.c_int), ("y_type", ctypes.c_int), ("scale_type", ctypes.c_int),
                ("group", ctypes.c_int), ("n_experts", ctypes.c_int), ("n_out", ctypes.c_int), ("n_in", ctypes.c_int),
                ("q", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("q_up", ctypes.c_void_p), ("scales_up", ctypes.c_void_p), ("zeros_up", ctypes.c_void_p)]


class moe_norm_desc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("x_type", ctypes.c_int), ("y_type", ctypes.c_int), ("u_type", ctypes.c_int),
                ("gamma_post", ctypes.c_void_p), ("gamma_pre", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float), ("scale", ctypes.c_float)]


def _c_int(v, name):
    """v as it is, if it is a C int: ctypes would cut off what lies above 32 bits without a word."""
    if not -(1 << 31) <= v < 1 << 31:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name} = {v} too large")
    return v


class _Desc(ctypes.Structure):
    """A description whose whole numbers fit their fields."""

    def __init__(self, *values, **named):
        super().__init__(*values, **named)
        given = {**dict(zip((name for name, _ in self._fields_), values)), **named}
        for name, kind in self._fields_:
            if kind is ctypes.c_int and name in given:
                _c_int(given[name], name)


class moe_linear_desc(_Desc):
    _fields_ = [("type", ctypes.c_int), ("y_type", ctypes.c_int), ("order", ctypes.c_int), ("n_out", ctypes.c_int),
                ("n_in", ctypes.c_int), ("w", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("bias", ctypes.c_void_p),
                ("bias_type", ctypes.c_int), ("act", ctypes.c_int), ("scale", ctypes.c_float), ("res_scale", ctypes.c_float)]


class moe_layer_norm_desc(_Desc):
    _fields_ = [("H", ctypes.c_int), ("x_type", ctypes.c_int), ("y_type", ctypes.c_int), ("gamma", ctypes.c_void_p),
                ("beta", ctypes.c_void_p), ("eps", ctypes.c_float)]


class moe_balance_desc(_Desc):
    _fields_ = [("mode", ctypes.c_int), ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int), ("coef", ctypes.c_float),
                ("accumulate", ctypes.c_int)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return os.path.join(HERE, "_build", "libmoe_gb300.so")


def load(build_if_missing: bool = True):
    """The loaded CUDA library (built in-tree on first use when missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if build_if_missing:
                from . import build as _build
                path = _build.build()
            if not os.path.exists(path):
                raise OSError(f"the CUDA library {path} is missing; run __graft_entry__.build()")
            _lib = _declare(ctypes.CDLL(path))
    return _lib


def _declare(lib):
    P, I, I64, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    PS = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "moe_route": [ctypes.POINTER(moe_route_cfg), P, I, I, I, P, P, P, P, P, P, P],
        "moe_permute_workspace_size": [I, I, I, PS],
        "moe_permute": [P, I, I, I, P, P, P, P, S, P],
        "moe_permute_noalloc": [P, I, I, I, P, P, P, P],
        "moe_expert_counts_add": [P, I, P, P],
        "moe_expert_ffn_workspace_size": [I, I, I, I, I, PS],
        "moe_expert_ffn": [ctypes.POINTER(moe_qmat)] * 3 + [I, P, I, I, I, I, P, P, I, P, P, S, P],
        "moe_expert_gateup": [ctypes.POINTER(moe_qmat)] * 2 + [I, P, I, I, I, I, P, P, I, P, P],
        "moe_expert_down": [ctypes.POINTER(moe_qmat), I, P, I, I, I, P, P, I, P, P],
        "moe_combine": [P, P, P, I, I, I, P, I, P, P],
        "moe_rmsnorm_bf16": [P, P, I, I, F, P, P],
        "moe_layer_plan_create": [ctypes.POINTER(moe_layer_desc), ctypes.POINTER(P)],
        "moe_layer_plan_destroy": [P],
        "moe_layer_workspace_size": [P, I, PS],
        "moe_layer_path": [P, I, ctypes.POINTER(ctypes.c_int)],
        "moe_layer": [P, P, I, P, P, S, P],
        "moe_layer_timed": [P, P, I, P, P, S, P, P, P],
        "moe_layer_debug_views": [P, I, P, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.POINTER(P)],
        "moe_read_device_status": [P, I, P, ctypes.POINTER(ctypes.c_int32), P],
        "moe_permute_read_device_status": [I, I, I, P, ctypes.POINTER(ctypes.c_int32), P],
        "moe_debug_set_waits": [ctypes.c_uint64, I],
        "moe_debug_set_stamps": [P, S],
        "moe_weights_prepare_size": [ctypes.POINTER(moe_qmat), I, PS],
        "moe_weights_prepare": [ctypes.POINTER(moe_qmat), I, P, S, P],
        "moe_grouped_plan_create": [ctypes.POINTER(moe_grouped_desc), ctypes.POINTER(P)],
        "moe_grouped_plan_destroy": [P],
        "moe_grouped_path": [P, I, I, ctypes.POINTER(ctypes.c_int)],
        "moe_grouped_matmul": [P, P, I64, I, I, P, P, P, I64, P, P],
        "moe_w4_plan_create": [ctypes.POINTER(moe_w4_desc), ctypes.POINTER(P)],
        "moe_w4_plan_destroy": [P],
        "moe_w4_matmul": [P, P, I64, I, I, P, P, P, I64, P, P],
        "moe_norm_residual": [ctypes.POINTER(moe_norm_desc), P, I64, P, I64, P, I64, I64, I, P, I64, P, I64, P],
        "moe_linear_plan_create": [ctypes.POINTER(moe_linear_desc), ctypes.POINTER(P)],
        "moe_linear_plan_destroy": [P],
        "moe_linear_path": [P, I, ctypes.POINTER(ctypes.c_int)],
        "moe_linear": [P, P, I64, I, P, I, I64, P, I64, P, P],
        "moe_layer_norm": [ctypes.POINTER(moe_layer_norm_desc), P, I64, I, P, I64, P, P, P],
        "moe_layer_norm_backward_workspace_size": [I, I, PS],
        "moe_layer_norm_backward": [ctypes.POINTER(moe_layer_norm_desc), P, I64, P, I64, P, P, P, I64, I, P, I64, P, P, I, P, S,
                                    P],
        "moe_balance_workspace_size": [I, I, I, PS],
        "moe_balance_loss": [ctypes.POINTER(moe_balance_desc), P, I64, P, I, P, I, P, P, P, P, P, I64, P, P, S, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.moe_last_error.argtypes = []
    lib.moe_last_error.restype = ctypes.c_char_p
    lib.moe_version.argtypes = []
    lib.moe_version.restype = ctypes.c_char_p
    return lib


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current_stream = None


def _stream(stream):
    if stream is None:
        global _current_stream
        if _current_stream is None:
            import torch
            # the address alone: torch.cuda.current_stream() makes a stream object, about 3 us of host time
            raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            _current_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int):
    if status != MOE_OK:
        msg = load().moe_last_error().decode(errors="replace")
        raise MoeError(status, msg)


def qmat(qtype: int, data, rows: int, cols: int, expert_stride_bytes: int = 0) -> moe_qmat:
    return moe_qmat(qtype, _p(data), rows, cols, expert_stride_bytes)


def route_cfg(mode: int, n_experts: int, top_k: int, n_groups: int = 1, topk_groups: int = 1,
              routed_scale: float = 1.0, renormalize: bool = True) -> moe_route_cfg:
    return moe_route_cfg(mode, n_experts, top_k, n_groups, topk_groups, routed_scale, int(renormalize))


# ------------------------------------------------------------------ calls (C names)

def moe_route(cfg, x, x_type, T, H, W_router, bias, logits_in, logits_out, topk_ids, topk_w, stream=None):
    _check(load().moe_route(ctypes.byref(cfg), _p(x), x_type, T, H, _p(W_router), _p(bias), _p(logits_in),
                            _p(logits_out), _p(topk_ids), _p(topk_w), _stream(stream)))


def moe_permute_workspace_size(T, k, E) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_permute_workspace_size(T, k, E, ctypes.byref(n)))
    return n.value


def moe_permute(topk_ids, T, k, E, sorted_pairs, offsets, pair_pos, workspace, ws_bytes, stream=None):
    _check(load().moe_permute(_p(topk_ids), T, k, E, _p(sorted_pairs), _p(offsets), _p(pair_pos),
                              _p(workspace), ws_bytes, _stream(stream)))


def moe_expert_counts_add(offsets, E, counts, stream=None):
    """counts[e] += offsets[e+1] - offsets[e] (counts: int64 [E] on the device, a running histogram)."""
    _check(load().moe_expert_counts_add(_p(offsets), E, _p(counts), _stream(stream)))


def moe_permute_noalloc(topk_ids, T, k, E, sorted_pairs, offsets, pair_pos, stream=None):
    """moe_permute without a workspace (fixed library scratch; T*k <= 65536)."""
    _check(load().moe_permute_noalloc(_p(topk_ids), T, k, E, _p(sorted_pairs), _p(offsets), _p(pair_pos),
                                      _stream(stream)))


def moe_expert_ffn_workspace_size(T, k, E, H, I) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_expert_ffn_workspace_size(T, k, E, H, I, ctypes.byref(n)))
    return n.value


def moe_expert_ffn(gate, up, down, E, x, x_type, T, H, I, sorted_pairs, offsets, k, y_pairs, workspace,
                   ws_bytes, stream=None):
    _check(load().moe_expert_ffn(ctypes.byref(gate), ctypes.byref(up), ctypes.byref(down), E, _p(x), x_type,
                                 T, H, I, _p(sorted_pairs), _p(offsets), k, _p(y_pairs), _p(workspace),
                                 ws_bytes, _stream(stream)))


def moe_expert_gateup(gate, up, E, x, x_type, T, H, I, sorted_pairs, offsets, k, h, stream=None):
    _check(load().moe_expert_gateup(ctypes.byref(gate), ctypes.byref(up), E, _p(x), x_type, T, H, I,
                                    _p(sorted_pairs), _p(offsets), k, _p(h), _stream(stream)))


def moe_expert_down(down, E, h, T, H, I, sorted_pairs, offsets, k, y_pairs, stream=None):
    _check(load().moe_expert_down(ctypes.byref(down), E, _p(h), T, H, I, _p(sorted_pairs), _p(offsets), k,
                                  _p(y_pairs), _stream(stream)))


def moe_combine(y_pairs, topk_w, pair_pos, T, k, H, shared_out, accumulate, out, stream=None):
    _check(load().moe_combine(_p(y_pairs), _p(topk_w), _p(pair_pos), T, k, H, _p(shared_out),
                              int(accumulate), _p(out), _stream(stream)))


def moe_rmsnorm_bf16(x, gamma, T, H, eps, u, stream=None):
    _check(load().moe_rmsnorm_bf16(_p(x), _p(gamma), T, H, float(eps), _p(u), _stream(stream)))


def moe_grouped_plan_create(desc: moe_grouped_desc) -> int:
    h = ctypes.c_void_p(0)
    _check(load().moe_grouped_plan_create(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def moe_grouped_plan_destroy(plan: int):
    _check(load().moe_grouped_plan_destroy(plan))


def moe_grouped_path(plan, T, k) -> int:
    """Which kernel moe_grouped_matmul runs for T tokens of k experts: a MOE_GROUPED_* value."""
    v = ctypes.c_int(-1)
    _check(load().moe_grouped_path(plan, T, k, ctypes.byref(v)))
    return v.value


def moe_grouped_matmul(plan, x, x_stride, T, k, sorted_pairs, offsets, y, y_stride, status=None, stream=None):
    _check(load().moe_grouped_matmul(plan, _p(x), x_stride, T, k, _p(sorted_pairs), _p(offsets), _p(y), y_stride,
                                     _p(status), _stream(stream)))


def moe_w4_plan_create(desc: moe_w4_desc) -> int:
    h = ctypes.c_void_p(0)
    _check(load().moe_w4_plan_create(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def moe_w4_plan_destroy(plan: int):
    _check(load().moe_w4_plan_destroy(plan))


def moe_w4_matmul(plan, x, x_stride, T, k, sorted_pairs, offsets, y, y_stride, status=None, stream=None):
    _check(load().moe_w4_matmul(plan, _p(x), x_stride, T, k, _p(sorted_pairs), _p(offsets), _p(y), y_stride,
                                _p(status), _stream(stream)))


def moe_norm_residual(desc: moe_norm_desc, x, x_stride, y, y_stride, gate, gate_row, gate_col, T, x_out, x_out_stride,
                      u, u_stride, stream=None):
    _check(load().moe_norm_residual(ctypes.byref(desc), _p(x), x_stride, _p(y), y_stride, _p(gate), gate_row, gate_col,
                                    T, _p(x_out), x_out_stride, _p(u), u_stride, _stream(stream)))


def moe_linear_plan_create(desc: moe_linear_desc) -> int:
    h = ctypes.c_void_p(0)
    _check(load().moe_linear_plan_create(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def moe_linear_plan_destroy(plan: int):
    _check(load().moe_linear_plan_destroy(plan))


def moe_linear_path(plan, T) -> int:
    """Which kernel moe_linear runs for T rows: a MOE_LINEAR_* value."""
    v = ctypes.c_int(-1)
    _check(load().moe_linear_path(plan, _c_int(T, "T"), ctypes.byref(v)))
    return v.value


def moe_linear(plan, x, x_stride, T, r, r_type, r_stride, y, y_stride, status=None, stream=None):
    _check(load().moe_linear(plan, _p(x), x_stride, _c_int(T, "T"), _p(r), r_type, r_stride, _p(y), y_stride, _p(status),
                             _stream(stream)))


def moe_layer_norm(desc: moe_layer_norm_desc, x, x_stride, T, y, y_stride, mean, rstd, stream=None):
    _check(load().moe_layer_norm(ctypes.byref(desc), _p(x), x_stride, _c_int(T, "T"), _p(y), y_stride, _p(mean), _p(rstd),
                                 _stream(stream)))


def moe_layer_norm_backward_workspace_size(H, T) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_layer_norm_backward_workspace_size(_c_int(H, "H"), _c_int(T, "T"), ctypes.byref(n)))
    return n.value


def moe_layer_norm_backward(desc: moe_layer_norm_desc, dy, dy_stride, x, x_stride, mean, rstd, add, add_stride, T, dx, dx_stride,
                            dgamma, dbeta, accumulate, workspace, ws_bytes, stream=None):
    _check(load().moe_layer_norm_backward(ctypes.byref(desc), _p(dy), dy_stride, _p(x), x_stride, _p(mean), _p(rstd), _p(add),
                                          add_stride, _c_int(T, "T"), _p(dx), dx_stride, _p(dgamma), _p(dbeta), int(accumulate),
                                          _p(workspace), ws_bytes, _stream(stream)))


def moe_balance_workspace_size(E, T, n_seqs=1) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_balance_workspace_size(_c_int(E, "n_experts"), _c_int(T, "T"), _c_int(n_seqs, "n_seqs"), ctypes.byref(n)))
    return n.value


def moe_balance_loss(desc: moe_balance_desc, logits, stride, ids, T, seq_offsets, n_seqs, mask, upstream, loss, counts, dlogits,
                     dstride, status, workspace, ws_bytes, stream=None):
    _check(load().moe_balance_loss(ctypes.byref(desc), _p(logits), stride, _p(ids), _c_int(T, "T"), _p(seq_offsets),
                                   _c_int(n_seqs, "n_seqs"), _p(mask), _p(upstream), _p(loss), _p(counts),
                                   _p(dlogits), dstride, _p(status), _p(workspace), ws_bytes, _stream(stream)))


def moe_layer_plan_create(desc: moe_layer_desc) -> int:
    h = ctypes.c_void_p(0)
    _check(load().moe_layer_plan_create(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def moe_layer_plan_destroy(plan: int):
    _check(load().moe_layer_plan_destroy(plan))


def moe_layer_workspace_size(plan: int, T: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_layer_workspace_size(plan, T, ctypes.byref(n)))
    return n.value


MOE_PATH_GEMV, MOE_PATH_DECODE_CHAIN, MOE_PATH_TENSOR = 0, 1, 2
PATH_NAMES = {MOE_PATH_GEMV: "gemv", MOE_PATH_DECODE_CHAIN: "decode_chain", MOE_PATH_TENSOR: "tensor"}


def moe_layer_path(plan, T):
    """Which kernels moe_layer runs for T tokens: one of the MOE_PATH_* values."""
    v = ctypes.c_int(-1)
    _check(load().moe_layer_path(plan, T, ctypes.byref(v)))
    return v.value


def moe_layer(plan, x, T, out, workspace, ws_bytes, stream=None):
    _check(load().moe_layer(plan, _p(x), T, _p(out), _p(workspace), ws_bytes, _stream(stream)))


def moe_layer_timed(plan, x, T, out, workspace, ws_bytes, stream=None, ev_before=None, ev_after=None):
    """moe_layer recording torch.cuda.Event objects around the routed gate/up kernel."""
    eb = ev_before.cuda_event if ev_before is not None else None
    ea = ev_after.cuda_event if ev_after is not None else None
    _check(load().moe_layer_timed(plan, _p(x), T, _p(out), _p(workspace), ws_bytes, _stream(stream), eb, ea))


def moe_layer_debug_views(plan, T, workspace):
    a, b, c = ctypes.c_void_p(0), ctypes.c_void_p(0), ctypes.c_void_p(0)
    _check(load().moe_layer_debug_views(plan, T, _p(workspace), ctypes.byref(a), ctypes.byref(b),
                                        ctypes.byref(c)))
    return a.value, b.value, c.value


def moe_read_device_status(plan, T, workspace, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(load().moe_read_device_status(plan, T, _p(workspace), ctypes.byref(code), _stream(stream)))
    return code.value


def moe_permute_read_device_status(T, k, E, workspace, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(load().moe_permute_read_device_status(T, k, E, _p(workspace), ctypes.byref(code), _stream(stream)))
    return code.value


def moe_weights_prepare_size(m: moe_qmat, n_experts: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_weights_prepare_size(ctypes.byref(m), n_experts, ctypes.byref(n)))
    return n.value


def moe_weights_prepare(m: moe_qmat, n_experts: int, dst, dst_bytes: int, stream=None) -> moe_qmat:
    """Repacks m (Q8_0) into dst; returns the moe_qmat that describes the prepared tensor."""
    out = moe_qmat(m.qtype, m.data, m.rows, m.cols, m.expert_stride_bytes)
    _check(load().moe_weights_prepare(ctypes.byref(out), n_experts, _p(dst), dst_bytes, _stream(stream)))
    return out


def moe_debug_set_stamps(buf, nbytes: int):
    _check(load().moe_debug_set_stamps(_p(buf), int(nbytes)))


def moe_debug_set_waits(limit_ns: int, stall: int):
    _check(load().moe_debug_set_waits(int(limit_ns), int(stall)))


def moe_last_error() -> str:
    return load().moe_last_error().decode(errors="replace")


def moe_version() -> str:
    return load().moe_version().decode()
