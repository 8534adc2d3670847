"""Device-resident MoE layer: torch tensors in, one moe_layer call out.

A convenience wrapper over the C ABI for callers that hold their weights in
torch tensors.  It fills a moe_layer_desc from the tensors, creates the plan
once, keeps a workspace buffer (torch memory) sized for the largest T seen,
and calls moe_layer.  All arithmetic runs in the CUDA library.
"""
from __future__ import annotations

import threading

import torch

from . import _native as N

_QT = {"q8_0": N.MOE_Q8_0, "q4_k": N.MOE_Q4_K, "q8_0_r": N.MOE_Q8_0_R, "q5_k": N.MOE_Q5_K, "q6_k": N.MOE_Q6_K,
       "q3_k": N.MOE_Q3_K, "mxfp4": N.MOE_MXFP4}


def row_bytes(qtype: int, cols: int) -> int:
    if qtype == N.MOE_Q8_0_R:                     # quants, then fp16 scales padded to 16 bytes
        nb = cols // 32
        return 32 * nb + (2 * nb + 15) // 16 * 16
    if qtype == N.MOE_Q8_0:
        return cols // 32 * 34
    if qtype == N.MOE_MXFP4:
        return cols // 32 * 17
    return cols // 256 * {N.MOE_Q4_K: 144, N.MOE_Q5_K: 176, N.MOE_Q6_K: 210, N.MOE_Q3_K: 110}[qtype]


def prepare_q8_0(t, rows: int, cols: int, n_experts: int = 1):
    """A Q8_0 tensor (uint8, [n_experts, rows, rb] or [rows, rb] on the GPU) repacked by
    moe_weights_prepare into a new uint8 tensor of the MOE_Q8_0_R layout (qtype "q8_0_r")."""
    m = N.qmat(N.MOE_Q8_0, t, rows, cols, rows * row_bytes(N.MOE_Q8_0, cols))
    nbytes = N.moe_weights_prepare_size(m, n_experts)
    dst = torch.empty(nbytes, dtype=torch.uint8, device=t.device)
    N.moe_weights_prepare(m, n_experts, dst, nbytes)
    shape = (n_experts, rows, row_bytes(N.MOE_Q8_0_R, cols)) if t.dim() == 3 else (rows, row_bytes(N.MOE_Q8_0_R, cols))
    return dst.view(*shape)


def _stream_object(stream, device):
    """The torch stream of a stream's handle (0 and 1 are two names of the default stream)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = N._stream(stream)
    return torch.cuda.ExternalStream(handle, device) if handle > 1 else torch.cuda.default_stream(device)


def _empty(shape, dtype, device, stream):
    """Memory for what a call on `stream` writes, in the order of that stream: from the current stream's memory it could
    be a block that kernels waiting there have yet to read, and would go back there while `stream` still writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream, device)):
        return torch.empty(shape, dtype=dtype, device=device)


class MoeLayer:
    """gate/up: uint8 [E, I, rb(H)], down: uint8 [E, H, rb(I)] on the GPU (qtype, or
    qtype_down for down); shared expert matrices in shared_qtype."""

    def __init__(self, *, mode: str, E: int, k: int, H: int, I: int, qtype: str, gate, up, down, W_router,
                 bias=None, n_groups: int = 1, topk_groups: int = 1, scale: float = 1.0,
                 renormalize: bool = True, x_dtype: str = "bf16", I_s: int = 0, shared_qtype: str = "q8_0",
                 s_gate=None, s_up=None, s_down=None, accumulate: bool = False, tc_min_tokens: int = 0,
                 decode_chain: bool = True, norm_gamma=None, norm_eps: float = 1e-6, qtype_down: str | None = None,
                 expert_counts=None):
        self.E, self.k, self.H, self.I = E, k, H, I
        self.x_dtype = x_dtype
        qt = _QT[qtype]
        qd = _QT[qtype_down] if qtype_down else qt      # the down matrix may be stored in another type
        self._keep = [gate, up, down, W_router, bias, s_gate, s_up, s_down, norm_gamma, expert_counts]
        d = N.moe_layer_desc()
        d.route = N.route_cfg(N.MOE_ROUTE_SIGMOID_GROUP if mode == "sigmoid_group" else N.MOE_ROUTE_SOFTMAX,
                              E, k, n_groups, topk_groups, scale, renormalize)
        d.hidden, d.intermediate = H, I
        d.x_type = N.MOE_BF16 if x_dtype == "bf16" else N.MOE_F32
        d.W_router = W_router.data_ptr()
        d.bias = bias.data_ptr() if bias is not None else None
        d.gate = N.qmat(qt, gate, I, H, I * row_bytes(qt, H))
        d.up = N.qmat(qt, up, I, H, I * row_bytes(qt, H))
        d.down = N.qmat(qd, down, H, I, H * row_bytes(qd, I))
        d.shared_intermediate = I_s
        if I_s > 0:
            sq = _QT[shared_qtype]
            d.s_gate = N.qmat(sq, s_gate, I_s, H, 0)
            d.s_up = N.qmat(sq, s_up, I_s, H, 0)
            d.s_down = N.qmat(sq, s_down, H, I_s, 0)
        d.accumulate = int(accumulate)
        d.tc_min_tokens = tc_min_tokens
        d.decode_chain_off = 0 if decode_chain else 1
        if norm_gamma is not None:       # pre-norm: x is the fp32 residual stream
            d.norm_gamma = norm_gamma.data_ptr()
            d.norm_eps = norm_eps
        if expert_counts is not None:    # running routing histogram: int64 [E] on the device
            if expert_counts.dtype != torch.int64 or expert_counts.numel() != E or not expert_counts.is_cuda:
                raise ValueError("expert_counts must be an int64 CUDA tensor of E entries")
            d.expert_counts = expert_counts.data_ptr()
        self.desc = d
        self.plan = N.moe_layer_plan_create(d)
        self.ws = None
        self.ws_T, self.ws_stream = -1, 0

    def path(self, T: int) -> str:
        """Which kernels a call with T tokens runs: "gemv", "decode_chain" or "tensor"."""
        return N.PATH_NAMES[N.moe_layer_path(self.plan, T)]

    def workspace_bytes(self, T: int) -> int:
        return N.moe_layer_workspace_size(self.plan, T)

    def ensure_workspace(self, T: int, device=None, stream=None):
        if self.ws is None or T > self.ws_T:
            nbytes = self.workspace_bytes(T)
            self.ws = _empty(nbytes, torch.uint8, device or "cuda", stream)
            self.ws_T, self.ws_stream = T, N._stream(stream)
        return self.ws

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """An output that is not given is made in the order of `stream`, as under torch.cuda.stream(stream)."""
        T = x.shape[0]
        if out is None:
            out = _empty((T, self.H), torch.float32, x.device, stream)
        ws = self.ensure_workspace(T, x.device, stream)
        handle = N._stream(stream)
        if handle != self.ws_stream:     # (a workspace of another stream's memory, which a larger one may replace meanwhile)
            ws.record_stream(_stream_object(handle, x.device))
        N.moe_layer(self.plan, x, T, out, ws, ws.numel(), handle)
        return out

    def debug_views(self, T: int):
        """(ids [T,k] int32, gates [T,k] fp32, offsets [E+1] int32) of the last call, copied to the host."""
        pi, pw, po = N.moe_layer_debug_views(self.plan, T, self.ws)
        base = self.ws.data_ptr()
        def view(ptr, n, dtype):
            off = ptr - base
            return self.ws[off:off + n * 4].view(dtype).clone().cpu()
        return (view(pi, T * self.k, torch.int32).view(T, self.k), view(pw, T * self.k, torch.float32).view(T, self.k),
                view(po, self.E + 1, torch.int32))

    def rebuild_plan(self):
        """Re-create the plan after editing self.desc."""
        N.moe_layer_plan_destroy(self.plan)
        self.plan = N.moe_layer_plan_create(self.desc)
        self.ws, self.ws_T = None, -1   # the workspace layout may have changed

    def device_status(self, T: int) -> int:
        return N.moe_read_device_status(self.plan, T, self.ws)

    def __del__(self):
        try:
            if getattr(self, "plan", None):
                N.moe_layer_plan_destroy(self.plan)
                self.plan = None
        except Exception:
            pass


_VT = {torch.float32: N.MOE_F32, torch.bfloat16: N.MOE_BF16, torch.float16: N.MOE_F16}


def _cuda(t, name, dtypes=None, dim=None, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on device {t.get_device()}, not on device {device}")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {[str(d) for d in dtypes]}, not {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")


def _on_current(device, **tensors):
    """Refuse a call whose tensors are not all on `device`, or whose device is not the current one: the kernel
    runs there, and an address of another device is nothing that it may read."""
    if device != torch.cuda.current_device():
        raise ValueError(f"device {device} of the call is not the current one ({torch.cuda.current_device()})")
    for name, t in tensors.items():
        if t is not None and t.get_device() != device:
            raise ValueError(f"{name} is on device {t.get_device()}, not on device {device}")


def _row_stride(t, name):
    """Elements between the rows of a 2-D tensor whose rows are dense."""
    n, width = t.shape
    row, col = t.stride()
    if col != 1 and width != 1:
        raise ValueError(f"the last dimension of {name} must be dense")
    return row if n > 1 else (width + 7) // 8 * 8        # (one row: its stride is never used)


_words: dict = {}                    # device: [words, how many are given away]
_all_words: list = []
_words_lock = threading.Lock()


def _status_word(device):
    """A status word (int32 [1], MOE_OK) that lives as long as the program: calls in flight and captured graphs may raise it after
    the object that they were made with is gone.  None during a capture that would have to make the words."""
    with _words_lock:
        held = _words.get(device)
        if held is None or held[1] == held[0].numel():
            if device.type == "cuda" and torch.cuda.is_current_stream_capturing():
                return None
            held = _words[device] = [torch.zeros(1024, dtype=torch.int32, device=device), 0]
            _all_words.append(held[0])
            if device.type == "cuda":                    # (zero before a call on any stream raises one)
                torch.cuda.current_stream(device).synchronize()
        held[1] += 1
        return held[0][held[1] - 1: held[1]]


class _Products:
    """What GroupedExperts and W4Experts share: the rows of a call, checked and passed on."""

    plan = None

    def device_status(self, clear: bool = False) -> int:
        """What the calls without a status of their own have raised so far, once all of them are done: MOE_OK,
        MOE_ERR_DEVICE_CHECK or MOE_ERR_TIMEOUT.  clear: back to MOE_OK."""
        word = self._status
        if word is None:
            raise RuntimeError("made during the first capture on its device, without a status word: pass status")
        if word.is_cuda:
            torch.cuda.synchronize(word.device)
        code = int(word.item())
        if clear:
            word.zero_()
            if word.is_cuda:
                torch.cuda.synchronize(word.device)
        return code

    def __call__(self, x: torch.Tensor, offsets: torch.Tensor | None = None, sorted_pairs: torch.Tensor | None = None,
                 k: int = 1, out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
        """y [T*k, n_out]: row i is the product of sorted position i's row of x with its expert's matrix.

        With sorted_pairs (int32 [T*k], moe_permute's) x holds the T tokens, row i being that of token
        sorted_pairs[i] // k; without, x holds the T*k rows in sorted order.  offsets (int32 [E+1], moe_permute's) may
        be left out for one expert.  status: int32 [1], raised when a device-side check fails (None: a word of
        this object's own, which device_status() reads).  All of them are on the weights' device, which has to be the
        current one.  stream (None: the current one) has to come after what wrote the inputs; without out, y is made
        in the order of that stream, as under torch.cuda.stream(stream).
        """
        if k < 1:
            raise ValueError(f"k = {k}: a token has at least one expert")
        n, width = x.shape
        T = n if sorted_pairs is not None else n // k
        P = T * k
        if x.dtype is not self.x_dtype or width != self.n_in or not x.is_cuda:
            raise ValueError(f"x must be a {self.x_dtype} CUDA tensor [rows, {self.n_in}]")
        if sorted_pairs is None and P != n:
            raise ValueError(f"{n} rows of x are not a multiple of k = {k}")
        if sorted_pairs is not None and (sorted_pairs.dtype is not torch.int32 or sorted_pairs.numel() != P
                                         or not sorted_pairs.is_contiguous() or not sorted_pairs.is_cuda):
            raise ValueError(f"sorted_pairs must be a dense int32 CUDA tensor of {P} entries")
        if offsets is not None and (offsets.dtype is not torch.int32 or offsets.numel() != self.n_experts + 1
                                    or not offsets.is_contiguous() or not offsets.is_cuda):
            raise ValueError(f"offsets must be a dense int32 CUDA tensor of {self.n_experts + 1} entries")
        if status is not None and (status.dtype is not torch.int32 or status.numel() < 1 or not status.is_cuda):
            raise ValueError("status must be an int32 CUDA tensor")
        if out is None:
            out = _empty((P, self.n_out), self.y_dtype, x.device, stream)
        elif out.dtype is not self.y_dtype or out.shape != (P, self.n_out) or not out.is_cuda:
            raise ValueError(f"out must be a {self.y_dtype} CUDA tensor [{P}, {self.n_out}]")
        _on_current(self.device, x=x, offsets=offsets, sorted_pairs=sorted_pairs, out=out, status=status)
        self._matmul(self.plan, x, _row_stride(x, "x"), T, k, sorted_pairs, offsets, out, _row_stride(out, "out"),
                     self._status if status is None else status, stream)
        return out

    def __del__(self):
        try:
            if self.plan:
                self._destroy(self.plan)
                self.plan = None
        except Exception:
            pass


class GroupedExperts(_Products):
    """Products of each expert's rows with its bf16 / fp16 matrix (moe_grouped_matmul).

    w: [E, n_out, n_in] (order "out_in") or [E, n_in, n_out] ("in_out") on the GPU, last dimension dense, the
    other strides multiples of 8 elements; w_up (same shape and strides): the call gives
    silu(w x) * (w_up x).  y_dtype: fp32 (what moe_combine reads), bf16 or fp16.
    """

    _matmul = staticmethod(N.moe_grouped_matmul)
    _destroy = staticmethod(N.moe_grouped_plan_destroy)

    def __init__(self, w: torch.Tensor, w_up: torch.Tensor | None = None, *, order: str = "out_in",
                 y_dtype: torch.dtype = torch.float32):
        if order not in ("out_in", "in_out"):
            raise ValueError(f"order must be 'out_in' or 'in_out', not {order!r}")
        if y_dtype not in _VT:
            raise ValueError(f"y_dtype must be one of {[str(d) for d in _VT]}")
        _cuda(w, "w", (torch.bfloat16, torch.float16), 3)
        if w.stride(2) != 1 and w.shape[2] != 1:
            raise ValueError("the last dimension of w must be dense")
        if w_up is not None:
            _cuda(w_up, "w_up", (w.dtype,), 3, w.get_device())
            if w_up.shape != w.shape or w_up.stride() != w.stride():
                raise ValueError("w_up must have w's shape and strides")
        self.n_experts = w.shape[0]
        self.n_out, self.n_in = (w.shape[1], w.shape[2]) if order == "out_in" else (w.shape[2], w.shape[1])
        self.x_dtype, self.y_dtype, self.device = w.dtype, y_dtype, w.get_device()
        self._keep = (w, w_up)
        self._status = _status_word(w.device)
        self.plan = N.moe_grouped_plan_create(N.moe_grouped_desc(
            _VT[w.dtype], _VT[y_dtype], N.MOE_W_OUT_IN if order == "out_in" else N.MOE_W_IN_OUT, self.n_experts,
            self.n_out, self.n_in, w.data_ptr(), w_up.data_ptr() if w_up is not None else None,
            _row_stride(w[0], "w"), w.stride(0)))

    def path(self, T: int, k: int = 1) -> str:
        """Which kernel a call with T tokens of k experts runs: "rows" or "tensor"."""
        return ("rows", "tensor")[N.moe_grouped_path(self.plan, T, k)]


class W4Experts(_Products):
    """The same products over 4-bit weights with group scales (moe_w4_matmul).

    q: uint8 [E, n_out, n_in // 2] (weight 2j in the low nibble of byte j), scales: fp16 or bf16
    [E, n_out, n_in // group], zeros: uint8 like scales, or None for 8 everywhere; up: (q, scales, zeros) of
    the gated pair's other matrix.  All dense, on the GPU.
    """

    _matmul = staticmethod(N.moe_w4_matmul)
    _destroy = staticmethod(N.moe_w4_plan_destroy)

    def __init__(self, q: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None, *, up=None,
                 group: int = 128, x_dtype: torch.dtype = torch.bfloat16, y_dtype: torch.dtype = torch.float32):
        if x_dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("x_dtype must be torch.bfloat16 or torch.float16")
        if y_dtype not in _VT:
            raise ValueError(f"y_dtype must be one of {[str(d) for d in _VT]}")
        if group not in (32, 64, 128):
            raise ValueError(f"group must be 32, 64 or 128, not {group}")
        up = (None, None, None) if up is None else tuple(up) + (None,) * (3 - len(up))
        if (up[0] is not None) and (up[2] is None) != (zeros is None):
            raise ValueError("both matrices have zero points, or neither")
        _cuda(q, "q", (torch.uint8,), 3)
        E, n_out, n_in = q.shape[0], q.shape[1], 2 * q.shape[2]
        if n_in % group:
            raise ValueError(f"n_in = {n_in} is not a multiple of the group {group}")
        for name, t, dtypes, width in (("scales", scales, (torch.float16, torch.bfloat16), n_in // group),
                                       ("zeros", zeros, (torch.uint8,), n_in // group),
                                       ("q_up", up[0], (torch.uint8,), n_in // 2),
                                       ("scales_up", up[1], (scales.dtype,), n_in // group),
                                       ("zeros_up", up[2], (torch.uint8,), n_in // group), ("q", q, None, n_in // 2)):
            if t is None:
                if name in ("scales",) or (name == "scales_up" and up[0] is not None):
                    raise ValueError(f"{name} is missing")
                continue
            _cuda(t, name, dtypes, 3, q.get_device())
            if tuple(t.shape) != (E, n_out, width) or not t.is_contiguous():
                raise ValueError(f"{name} must be dense [{E}, {n_out}, {width}]")
        self.n_experts, self.n_out, self.n_in = E, n_out, n_in
        self.x_dtype, self.y_dtype, self.device = x_dtype, y_dtype, q.get_device()
        self._keep = (q, scales, zeros, up)
        self._status = _status_word(q.device)
        p = [t.data_ptr() if t is not None else None for t in (q, scales, zeros) + up]
        self.plan = N.moe_w4_plan_create(N.moe_w4_desc(_VT[x_dtype], _VT[y_dtype], _VT[scales.dtype], group, E, n_out,
                                                       n_in, *p))


class NormResidual:
    """The norm behind a block, its gate and residual scale, and the next block's norm (moe_norm_residual).

    gamma_post, gamma_pre: fp32 [H] on the GPU (gamma_post None: no norm behind the block; gamma_pre None: no u).
    """

    def __init__(self, H: int, *, gamma_post: torch.Tensor | None = None, gamma_pre: torch.Tensor | None = None,
                 eps: float = 1e-6, res_scale: float = 1.0, scale: float = 1.0):
        self.device = None               # the gains'; without any, each call's own
        for name, g in (("gamma_post", gamma_post), ("gamma_pre", gamma_pre)):
            if g is not None:
                _cuda(g, name, (torch.float32,), 1, self.device)
                self.device = g.get_device()
                if g.numel() != H or not g.is_contiguous():
                    raise ValueError(f"{name} must be dense [{H}]")
        self.H = H
        self._keep = (gamma_post, gamma_pre)
        self._scales = (eps, res_scale, scale)
        self._desc = {}                  # the call's description, by the types of its tensors

    def __call__(self, x: torch.Tensor | None, y: torch.Tensor, gate: torch.Tensor | None = None,
                 x_out: torch.Tensor | None = None, u: torch.Tensor | None = None, stream=None):
        """(x_out, u): the residual stream behind the block (in x's type; x_out may be x) and its norm.

        x (None: 0), y: [T, H].  gate: fp32, broadcastable to [T, H] ([H], [1, H], [T, 1] or [T, H]).
        Outputs that are not given are made: x_out like x (or y), u in bf16 when gamma_pre was given.  All tensors are
        on one device, which has to be the current one; stream as in the products' calls.
        """
        shape = y.shape
        T, H = shape
        if H != self.H:
            raise ValueError(f"y must be [T, {self.H}]")
        if x_out is None:
            x_out = _empty((T, H), (x if x is not None else y).dtype, y.device, stream)
        if u is None and self._keep[1] is not None:
            u = _empty((T, H), torch.bfloat16, y.device, stream)
        xs = us = gate_row = gate_col = 0
        ys = self._rows(y, "y", shape)
        os = self._rows(x_out, "x_out", shape)
        if x is not None:
            xs = self._rows(x, "x", shape)
            if x.dtype is not x_out.dtype:
                raise ValueError("x_out must have x's type")
        if u is not None:
            us = self._rows(u, "u", shape)
        if gate is not None:
            gs, st = gate.shape, gate.stride()
            if len(gs) == 1:
                gs, st = (1,) + tuple(gs), (0,) + st
            if gate.dtype is not torch.float32 or not gate.is_cuda or len(gs) != 2 or gs[0] not in (1, T) or gs[1] not in (1, H):
                raise ValueError(f"gate must be an fp32 CUDA tensor broadcastable to [{T}, {H}]")
            gate_row, gate_col = st[0] if gs[0] != 1 else 0, st[1] if gs[1] != 1 else 0
        device = y.get_device()
        if self.device is not None and device != self.device:
            raise ValueError(f"y is on device {device}, gamma_post / gamma_pre on device {self.device}")
        _on_current(device, x=x, gate=gate, x_out=x_out, u=u)
        types = (x_out.dtype, y.dtype, u.dtype if u is not None else torch.float32)
        desc = self._desc.get(types)
        if desc is None:
            g = [t.data_ptr() if t is not None else None for t in self._keep]
            desc = self._desc[types] = N.moe_norm_desc(H, *(_VT[t] for t in types), *g, *self._scales)
        N.moe_norm_residual(desc, x, xs, y, ys, gate, gate_row, gate_col, T, x_out, os, u, us, stream)
        return x_out, u

    def _rows(self, t, name, shape):
        """Elements between the rows of t, a [T, H] tensor of the call."""
        if t.shape != shape or t.dtype not in _VT or not t.is_cuda:
            raise ValueError(f"{name} must be an fp32, bf16 or fp16 CUDA tensor {list(shape)}")
        row, col = t.stride()
        if col != 1 and shape[1] != 1:
            raise ValueError(f"the last dimension of {name} must be dense")
        return row if shape[0] > 1 else (shape[1] + 7) // 8 * 8
