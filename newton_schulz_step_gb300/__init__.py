"""Muon optimizer step on GB300 (sm_103a): Python binding of libmuon_gb300.so.

This module only marshals arguments: it checks torch tensors (device,
dtype, contiguity, shape), takes their device pointers and the current CUDA
stream, and calls the C ABI declared in include/muon_gb300.h.  Every step of
the computation runs in the library's CUDA kernels.  There is no fallback:
if the library is not built, or no sm_103a GPU is current, calls raise.

Entry points mirror the C ABI:
  ns5(G)                         the quintic Newton-Schulz iteration on a stack of matrices
  step(p, g, buf, ...)           one Muon step on a stack of same-shape weights
  step_grouped([(p, g, buf)...]) one Muon step on every group of a model
  adam_step([(p, g, m, v)...])   one DistAdam step on the non-matrix parameters
  qk_norm_rope(q, k, cos, sin)   RMS norm and rotary positions of the query and key heads
  attention(q, k, v, cu_seqlens) causal attention over packed sequences, grouped heads
with qk_norm_rope_backward and attention_backward for their gradients.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading

import torch

__all__ = [
    "COEFFS", "EPS", "MuonError", "load_library", "library_path", "workspace_bytes",
    "grouped_workspace_bytes", "Workspace", "ns5", "step", "step_noalloc", "step_grouped",
    "GroupedStep", "AdamStep", "adam_step", "ADAM_LR", "ADAM_BETAS", "ADAM_EPS",
    "workspace_status", "noalloc_status", "selftest_wait_timeout", "status_string",
    "kernel_launch_count", "trace_begin", "trace_end",
    "set_fused_ns", "fused_ns", "set_persistent_rounds", "persistent_rounds",
    "set_streamed_apply", "streamed_apply", "KERNEL_KINDS",
    "ROPE_EPS", "rope_tables", "qk_norm_rope", "qk_norm_rope_backward",
    "norm_rope_workspace_bytes", "attention", "attention_backward", "attention_workspace_bytes",
]

# Quintic coefficients and rounds as printed in "Muon Custom Sizing 实战", section 2.3.
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7

# DistAdam settings printed in "Muon Custom Sizing 实战", section 四.
ADAM_LR = 0.008
ADAM_BETAS = (0.8, 0.95)
ADAM_EPS = 1e-8

KERNEL_KINDS = {0: "prologue", 1: "small_ns", 2: "gram", 3: "poly", 4: "update", 5: "apply",
                6: "adam", 7: "fused_ns", 8: "rounds", 9: "norm_rope", 10: "norm_rope_backward",
                11: "attention", 12: "attention_dq", 13: "attention_dkv"}
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error", 4: "timeout",
           5: "workspace"}

_LIB_NAME = "libmuon_gb300.so"
_lib = None


def library_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), _LIB_NAME)


class MuonError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


class _Group(ctypes.Structure):
    _fields_ = [("params", ctypes.c_void_p), ("grads", ctypes.c_void_p),
                ("momentum_buf", ctypes.c_void_p), ("g_dtype", ctypes.c_int),
                ("batch", ctypes.c_int), ("rows", ctypes.c_int), ("cols", ctypes.c_int),
                ("lr_scale", ctypes.c_float)]


class _AdamTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("numel", ctypes.c_longlong), ("g_dtype", ctypes.c_int),
                ("lr_scale", ctypes.c_float), ("wd_scale", ctypes.c_float)]


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong)]


class _NormRope(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("tokens", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("k_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("norm", ctypes.c_int), ("interleaved", ctypes.c_int), ("eps", ctypes.c_float),
                ("table_len", ctypes.c_int), ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p)]


class _AttentionSpec(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int), ("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("cu_seqlens", ctypes.c_void_p), ("scale", ctypes.c_float)]


class _TraceRecord(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("round", ctypes.c_int), ("ms", ctypes.c_float),
                ("flops", ctypes.c_double), ("bytes", ctypes.c_double)]


def load_library():
    """Load libmuon_gb300.so from this package directory (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m newton_schulz_step_gb300.build`")
    L = ctypes.CDLL(path)
    vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.muon_workspace_bytes.argtypes = [ci, ci, ci]
    L.muon_workspace_bytes.restype = sz
    L.muon_grouped_workspace_bytes.argtypes = [ctypes.POINTER(_Group), ci]
    L.muon_grouped_workspace_bytes.restype = sz
    L.muon_ns5.argtypes = [vp, ci, vp, ci, ci, ci, ci, cf, cf, cf, cf, vp, sz, vp]
    L.muon_ns5.restype = ci
    L.muon_step.argtypes = [vp, vp, ci, vp, ci, ci, ci, cf, ci, cf, cf, cf, ci, cf, cf, cf, cf,
                            vp, sz, vp]
    L.muon_step.restype = ci
    L.muon_step_noalloc.argtypes = [vp, vp, ci, vp, ci, ci, ci, cf, ci, cf, cf, cf, ci, cf, cf,
                                    cf, cf, vp]
    L.muon_step_noalloc.restype = ci
    L.muon_step_grouped.argtypes = [ctypes.POINTER(_Group), ci, cf, ci, cf, cf, ci, cf, cf, cf,
                                    cf, vp, sz, vp]
    L.muon_step_grouped.restype = ci
    L.muon_workspace_status.argtypes = [vp, sz, vp, ci]
    L.muon_workspace_status.restype = ci
    L.muon_noalloc_status.argtypes = [vp, ci]
    L.muon_noalloc_status.restype = ci
    L.muon_selftest_wait_timeout.argtypes = [vp, sz, ci, vp]
    L.muon_selftest_wait_timeout.restype = ci
    L.muon_adam_step.argtypes = [ctypes.POINTER(_AdamTensor), ci, ci, cf, cf, cf, cf, cf, vp]
    L.muon_adam_step.restype = ci
    rope, spec, hd = ctypes.POINTER(_NormRope), ctypes.POINTER(_AttentionSpec), _Heads
    L.muon_qk_norm_rope.argtypes = [rope, hd, hd, hd, hd, vp]
    L.muon_qk_norm_rope.restype = ci
    L.muon_norm_rope_workspace_bytes.argtypes = [ci]
    L.muon_norm_rope_workspace_bytes.restype = sz
    L.muon_qk_norm_rope_backward.argtypes = [rope, hd, hd, hd, hd, hd, hd, vp, vp, vp, sz, vp]
    L.muon_qk_norm_rope_backward.restype = ci
    L.muon_attention_workspace_bytes.argtypes = [ci, ci, ci, ci]
    L.muon_attention_workspace_bytes.restype = sz
    L.muon_attention.argtypes = [spec, hd, hd, hd, hd, vp, vp, sz, vp]
    L.muon_attention.restype = ci
    L.muon_attention_backward.argtypes = [spec, hd, hd, hd, hd, hd, vp, hd, hd, hd, vp, sz, vp]
    L.muon_attention_backward.restype = ci
    L.muon_set_persistent_rounds.argtypes = [ci]
    L.muon_set_persistent_rounds.restype = ci
    L.muon_set_fused_ns.argtypes = [ci]
    L.muon_set_fused_ns.restype = ci
    L.muon_set_streamed_apply.argtypes = [ci]
    L.muon_set_streamed_apply.restype = ci
    L.muon_status_string.argtypes = [ci]
    L.muon_status_string.restype = ctypes.c_char_p
    L.muon_kernel_launch_count.argtypes = []
    L.muon_kernel_launch_count.restype = ctypes.c_ulonglong
    L.muon_trace_begin.argtypes = [ci]
    L.muon_trace_begin.restype = ci
    L.muon_trace_end.argtypes = [ctypes.POINTER(_TraceRecord), ci, ctypes.POINTER(ci)]
    L.muon_trace_end.restype = ci
    _lib = L
    return L


def status_string(code: int) -> str:
    try:
        return load_library().muon_status_string(code).decode()
    except ImportError:
        return _STATUS.get(code, "unknown status")


def _raise(code: int, where: str):
    if code != 0:
        raise MuonError(code, where)


def _gdt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return 0
    if t.dtype == torch.bfloat16:
        return 1
    raise TypeError(f"gradients must be float32 or bfloat16, got {t.dtype}")


def _as3d(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dim() == 2:
        t = t.unsqueeze(0)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, cols] or [batch, rows, cols], got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream_handle(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return int(getattr(stream, "cuda_stream", stream))


def workspace_bytes(batch: int, rows: int, cols: int) -> int:
    return int(load_library().muon_workspace_bytes(batch, rows, cols))


def _groups_array(groups):
    arr = (_Group * max(1, len(groups)))()
    for i, (p, g, b, s) in enumerate(groups):
        arr[i].params = p.data_ptr() if p is not None else None
        arr[i].grads = g.data_ptr() if g is not None else None
        arr[i].momentum_buf = b.data_ptr() if b is not None else None
        arr[i].g_dtype = _gdt(g) if g is not None else 1
        arr[i].batch, arr[i].rows, arr[i].cols = (int(x) for x in g.shape)
        arr[i].lr_scale = float(s)
    return arr


def grouped_workspace_bytes(shapes) -> int:
    """shapes: iterable of (batch, rows, cols)."""
    shapes = list(shapes)
    arr = (_Group * max(1, len(shapes)))()
    for i, (b, r, c) in enumerate(shapes):
        arr[i].batch, arr[i].rows, arr[i].cols, arr[i].g_dtype = b, r, c, 1
    return int(load_library().muon_grouped_workspace_bytes(arr, len(shapes)))


class Workspace:
    """Zero-filled device scratch owned by the caller (one per concurrent stream)."""

    def __init__(self, nbytes: int, device=None):
        self.tensor = torch.zeros(max(256, int(nbytes)), dtype=torch.uint8,
                                  device=device if device is not None else "cuda")
        if self.tensor.data_ptr() % 256:
            raise RuntimeError("workspace allocation is not 256-byte aligned")

    @property
    def ptr(self) -> int:
        return self.tensor.data_ptr()

    @property
    def nbytes(self) -> int:
        return self.tensor.numel()

    def ensure(self, nbytes: int):
        if nbytes > self.nbytes:
            self.__init__(nbytes, self.tensor.device)
        return self


_default_ws = {}


def _workspace(ws, need: int, device) -> Workspace:
    if ws is not None:
        return ws
    key = torch.device(device).index if torch.device(device).index is not None else \
        torch.cuda.current_device()
    w = _default_ws.get(key)
    if w is None:
        w = _default_ws[key] = Workspace(need, device)
    return w.ensure(need)


def ns5(G: torch.Tensor, out: torch.Tensor | None = None, steps: int = STEPS, coeffs=COEFFS,
        eps: float = EPS, workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """The quintic Newton-Schulz iteration of every matrix of G ([b, r, c] or [r, c]); bf16 result."""
    L = load_library()
    squeeze = G.dim() == 2
    G3 = _as3d(G, "G")
    _gdt(G3)
    if out is None:
        out = torch.empty(G3.shape, dtype=torch.bfloat16, device=G3.device)
    out3 = _as3d(out, "out")
    if out3.dtype != torch.bfloat16 or out3.shape != G3.shape:
        raise ValueError("out must be bfloat16 with G's shape")
    b, r, c = G3.shape
    ws = _workspace(workspace, L.muon_workspace_bytes(b, r, c), G3.device)
    a_, b_, c_ = coeffs
    _raise(L.muon_ns5(G3.data_ptr(), _gdt(G3), out3.data_ptr(), b, r, c, steps, a_, b_, c_, eps,
                      ws.ptr, ws.nbytes, _stream_handle(stream)), "muon_ns5")
    return out3[0] if squeeze else out3


def step(params, grads, momentum_buf, *, momentum: float, lr: float, weight_decay: float,
         nesterov: bool = True, lr_scale: float = 0.0, steps: int = STEPS, coeffs=COEFFS,
         eps: float = EPS, workspace: Workspace | None = None, stream=None):
    """One Muon step, in place on params and momentum_buf (fp32, [b, r, c] or [r, c])."""
    L = load_library()
    p3, g3, m3 = _as3d(params, "params"), _as3d(grads, "grads"), _as3d(momentum_buf, "momentum_buf")
    if p3.dtype != torch.float32 or m3.dtype != torch.float32:
        raise TypeError("params and momentum_buf must be float32")
    if not (p3.shape == g3.shape == m3.shape):
        raise ValueError("params, grads and momentum_buf must have the same shape")
    b, r, c = g3.shape
    ws = _workspace(workspace, L.muon_workspace_bytes(b, r, c), g3.device)
    a_, b_, c_ = coeffs
    _raise(L.muon_step(p3.data_ptr(), g3.data_ptr(), _gdt(g3), m3.data_ptr(), b, r, c,
                       momentum, int(bool(nesterov)), lr, weight_decay, lr_scale, steps,
                       a_, b_, c_, eps, ws.ptr, ws.nbytes, _stream_handle(stream)), "muon_step")


def step_noalloc(params, grads, momentum_buf, *, momentum: float, lr: float,
                 weight_decay: float, nesterov: bool = True, lr_scale: float = 0.0,
                 steps: int = STEPS, coeffs=COEFFS, eps: float = EPS, stream=None):
    """step() without a workspace, for callers that may not allocate device memory:
    the library's built-in 64 MiB device scratch (of the tensors' GPU) is used
    instead.  The call runs with the tensors' device current, so the scratch and
    the kernels are on that device."""
    L = load_library()
    p3, g3, m3 = _as3d(params, "params"), _as3d(grads, "grads"), _as3d(momentum_buf, "momentum_buf")
    if p3.dtype != torch.float32 or m3.dtype != torch.float32:
        raise TypeError("params and momentum_buf must be float32")
    if not (p3.shape == g3.shape == m3.shape):
        raise ValueError("params, grads and momentum_buf must have the same shape")
    if not (p3.device == g3.device == m3.device):
        raise ValueError("params, grads and momentum_buf must be on the same device")
    b, r, c = g3.shape
    a_, b_, c_ = coeffs
    with torch.cuda.device(p3.device):
        _raise(L.muon_step_noalloc(p3.data_ptr(), g3.data_ptr(), _gdt(g3), m3.data_ptr(), b, r, c,
                                   momentum, int(bool(nesterov)), lr, weight_decay, lr_scale,
                                   steps, a_, b_, c_, eps, _stream_handle(stream)),
               "muon_step_noalloc")


def _normalise_groups(groups):
    out = []
    for grp in groups:
        if len(grp) == 3:
            p, g, b = grp
            s = 0.0
        else:
            p, g, b, s = grp
        p3, g3, b3 = _as3d(p, "params"), _as3d(g, "grads"), _as3d(b, "momentum_buf")
        if p3.dtype != torch.float32 or b3.dtype != torch.float32:
            raise TypeError("params and momentum_buf must be float32")
        if not (p3.shape == g3.shape == b3.shape):
            raise ValueError("params, grads and momentum_buf must have the same shape")
        _gdt(g3)
        out.append((p3, g3, b3, s))
    return out


class GroupedStep:
    """A prepared muon_step_grouped call: the group table is marshalled once.

    Calling it enqueues one Muon step over every group on the current (or
    given) stream.  The tensors must stay alive and in place between calls.
    """

    def __init__(self, groups, *, momentum: float, lr: float, weight_decay: float,
                 nesterov: bool = True, steps: int = STEPS, coeffs=COEFFS, eps: float = EPS,
                 workspace: Workspace | None = None):
        L = load_library()
        self._groups = _normalise_groups(groups)
        self._arr = _groups_array(self._groups)
        self._n = len(self._groups)
        need = int(L.muon_grouped_workspace_bytes(self._arr, self._n))
        if need == 0 and self._n:
            raise ValueError("invalid group shapes")
        dev = self._groups[0][1].device if self._n else torch.device("cuda")
        self.workspace = workspace.ensure(need) if workspace is not None else Workspace(need, dev)
        self._scalars = (float(momentum), int(bool(nesterov)), float(lr), float(weight_decay),
                         int(steps), *(float(x) for x in coeffs), float(eps))

    def __call__(self, stream=None):
        L = load_library()
        mom, nest, lr, wd, steps, a_, b_, c_, eps = self._scalars
        _raise(L.muon_step_grouped(self._arr, self._n, mom, nest, lr, wd, steps, a_, b_, c_, eps,
                                   self.workspace.ptr, self.workspace.nbytes,
                                   _stream_handle(stream)), "muon_step_grouped")


def step_grouped(groups, *, momentum: float, lr: float, weight_decay: float,
                 nesterov: bool = True, steps: int = STEPS, coeffs=COEFFS, eps: float = EPS,
                 workspace: Workspace | None = None, stream=None):
    """One Muon step over every group: groups = [(params, grads, bufs[, lr_scale]), ...]."""
    GroupedStep(groups, momentum=momentum, lr=lr, weight_decay=weight_decay, nesterov=nesterov,
                steps=steps, coeffs=coeffs, eps=eps, workspace=workspace)(stream)


class AdamStep:
    """A prepared muon_adam_step call over tensors = [(param, grad, exp_avg, exp_avg_sq
    [, lr_scale[, wd_scale]]), ...]; param and the moments are fp32, grad fp32 or bf16,
    all contiguous CUDA tensors of one numel per entry (any shape).  Calling it with
    the step count t (>= 1, after the increment) enqueues one update."""

    def __init__(self, tensors, *, lr: float = ADAM_LR, betas=ADAM_BETAS, eps: float = ADAM_EPS,
                 weight_decay: float = 0.0):
        load_library()
        self._keep = []
        self._arr = (_AdamTensor * max(1, len(tensors)))()
        for i, ent in enumerate(tensors):
            p, g, m, v = ent[:4]
            ls = float(ent[4]) if len(ent) > 4 else 1.0
            ws = float(ent[5]) if len(ent) > 5 else 1.0
            for t, name in ((p, "param"), (g, "grad"), (m, "exp_avg"), (v, "exp_avg_sq")):
                if not t.is_cuda or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous CUDA tensor")
            if p.dtype != torch.float32 or m.dtype != torch.float32 or v.dtype != torch.float32:
                raise TypeError("param, exp_avg and exp_avg_sq must be float32")
            if not (p.numel() == g.numel() == m.numel() == v.numel()):
                raise ValueError("param, grad, exp_avg and exp_avg_sq must have the same numel")
            a = self._arr[i]
            a.param, a.grad, a.exp_avg, a.exp_avg_sq = (t.data_ptr() for t in (p, g, m, v))
            a.numel, a.g_dtype, a.lr_scale, a.wd_scale = p.numel(), _gdt(g), ls, ws
            self._keep.append((p, g, m, v))
        self._n = len(tensors)
        self._scalars = (float(lr), float(betas[0]), float(betas[1]), float(eps),
                         float(weight_decay))

    def __call__(self, step: int, stream=None):
        lr, b1, b2, eps, wd = self._scalars
        _raise(load_library().muon_adam_step(self._arr, self._n, int(step), lr, b1, b2, eps, wd,
                                             _stream_handle(stream)), "muon_adam_step")


def adam_step(tensors, step: int, *, lr: float = ADAM_LR, betas=ADAM_BETAS, eps: float = ADAM_EPS,
              weight_decay: float = 0.0, stream=None):
    """One DistAdam update, in place, of every (param, grad, exp_avg, exp_avg_sq[, lr_scale
    [, wd_scale]]) entry at step count `step` (>= 1)."""
    AdamStep(tensors, lr=lr, betas=betas, eps=eps, weight_decay=weight_decay)(step, stream)


# ------------------------------------------------------------ attention path
ROPE_EPS = 1e-6


def rope_tables(length: int, rot_dim: int, *, base: float = 10000.0, scale: float = 1.0,
                device=None):
    """cos and sin of the angles (position / scale) base^(-2i / rot_dim), i < rot_dim / 2, for
    the positions 0..length-1: two [length, rot_dim / 2] fp32 tensors.  scale > 1 spreads the
    angles of a context it times as long over the trained range."""
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / max(1, rot_dim))
    ang = (torch.arange(length, dtype=torch.float64) / scale)[:, None] * inv[None, :]
    device = device if device is not None else "cuda"
    return ang.cos().float().to(device), ang.sin().float().to(device)


def _cuda_device(t, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


# The checks below compare device indices, -1 for CPU tensors, and cost the host of a call
# about 100 ns for each property of a tensor that they read.
def _refuse_heads(t, name, shape, dtype, index):
    """Says what is wrong with a [tokens, heads, head_dim] argument."""
    device = torch.device("cuda", index)
    _cuda_device(t, name)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous along head_dim")


def _heads(t, name: str, shape, dtype, index) -> _Heads:
    """The view of a [tokens, heads, head_dim] tensor of the given shape, dtype and device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and len(shape) == 3:
        st, sh, sd = t.stride()
        if sd == 1 or shape[2] <= 1:
            return _Heads(t.data_ptr(), st, sh)
    _refuse_heads(t, name, shape, dtype, index)


def _out_heads(t, name: str, like):
    """(tensor, view) of an output shaped like `like`: the caller's, or a new contiguous one."""
    if t is None:
        t = torch.empty_like(like)        # (half the time of new_empty)
        if not t.is_contiguous():         # it takes the strides of a dense tensor
            t = like.new_empty(like.shape)
        _, heads, dim = like.shape
        return t, _Heads(t.data_ptr(), heads * dim, dim)
    return t, _heads(t, name, like.shape, like.dtype, like.get_device())


def _ptr(t, name: str, index, dtype, shape=None):
    """Pointer of a contiguous tensor argument of one dtype (None passes)."""
    if t is None:
        return None
    if (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    device = torch.device("cuda", index)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


@contextlib.contextmanager
def _launch_on(device, stream):
    """Makes `device` and the stream of the call current, so that what the call allocates
    belongs to that stream."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            yield


# (the public current_stream() builds a Stream object, 2 us a call; current_device() looks
# whether CUDA is up, which it is where there is a CUDA tensor)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

# (device index, stream handle) -> (pointer, bytes, Workspace, the entry it outgrew)
_stream_ws = {}
_stream_ws_lock = threading.Lock()


def _stream_workspace(ws, need: int, index: int, handle: int):
    """Pointer, size and owner of the caller's workspace, or of one kept for each device and
    stream: calls on different streams may overlap, and must not share one.  A workspace that is
    outgrown stays allocated, for another thread may be about to launch with its pointer; sizes
    double, so that all of them together are less than twice the last.
    A call that is being captured gets a workspace of its graph alone, which may be replayed on
    any stream and in any order; clearing its status block is a node of that graph."""
    if ws is not None:
        return ws.ptr, ws.nbytes, ws
    if torch.cuda.is_current_stream_capturing():
        own = torch.empty(max(256, need), dtype=torch.uint8, device=torch.device("cuda", index))
        own[:256].zero_()
        return own.data_ptr(), own.numel(), own
    kept = _stream_ws.get((index, handle))
    if kept is None or kept[1] < need:
        with _stream_ws_lock:
            kept = _stream_ws.get((index, handle))
            if kept is None or kept[1] < need:
                ws = Workspace(need if kept is None else max(need, 2 * kept[1]),
                               torch.device("cuda", index))
                kept = _stream_ws[(index, handle)] = (ws.ptr, ws.nbytes, ws, kept)
    return kept[:3]


def _refuse_grad(where: str, **tensors):
    """Says which tensor asks for a gradient: forward calls record nothing for autograd, and it
    would not get one."""
    for name, t in tensors.items():
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} requires grad, and {where} records no gradient: call it under "
                             f"torch.no_grad() or on detached tensors, and {where}_backward for "
                             "the gradients")


def _rope_spec(q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved):
    """The spec of a call and its views of q and k."""
    _cuda_device(q, "q")
    dev, shape, dtype = q.get_device(), q.shape, q.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"q and k must be float32 or bfloat16, got {dtype}")
    vq = _heads(q, "q", shape, dtype, dev)
    t, hq, d = shape
    k_shape = k.shape
    if len(k_shape) != 3:
        raise ValueError(f"k must be [tokens, heads, head_dim], got {tuple(k_shape)}")
    hk = k_shape[1]
    vk = _heads(k, "k", (t, hk, d), dtype, dev)
    table = cos.shape
    if len(table) != 2 or table != sin.shape:
        raise ValueError("cos and sin must be [length, rot_dim / 2] of one shape")
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights belong to the norm: norm=False takes none")
    f32 = torch.float32
    p_pos = p_qw = p_kw = None
    if positions is not None:
        p_pos = _ptr(positions, "positions", dev, torch.int32, (t,))
    if q_weight is not None:
        p_qw = _ptr(q_weight, "q_weight", dev, f32, (d,))
    if k_weight is not None:
        p_kw = _ptr(k_weight, "k_weight", dev, f32, (d,))
    return _NormRope(1 if dtype is torch.bfloat16 else 0, t, hq, hk, d, 2 * table[1],
                     1 if norm else 0, 1 if interleaved else 0, eps, table[0],
                     _ptr(cos, "cos", dev, f32), _ptr(sin, "sin", dev, f32),
                     p_pos, p_qw, p_kw), vq, vk


def qk_norm_rope(q, k, cos, sin, *, q_weight=None, k_weight=None, positions=None,
                 norm: bool = True, eps: float = ROPE_EPS, interleaved: bool = False,
                 q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [tokens, q_heads, head_dim] and k [tokens, k_heads, head_dim]
    (bf16 or fp32, strided along tokens and heads), times q_weight / k_weight ([head_dim] fp32),
    then the rotation of its first 2 * cos.shape[1] elements by rows `positions` (int32; the
    token's index when None) of the tables cos, sin (see rope_tables).  Pairs are (i, i + half),
    or (2i, 2i + 1) when interleaved.  Returns (q_out, k_out); they may be q and k themselves, and
    overlap nothing else.  Nothing is recorded for autograd: tensors that require grad are refused
    while it records, see qk_norm_rope_backward."""
    L = _lib or load_library()
    spec, vq, vk = _rope_spec(q, k, cos, sin, positions, q_weight, k_weight, norm, eps,
                              interleaved)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or (
            q_weight is not None and q_weight.requires_grad) or (
            k_weight is not None and k_weight.requires_grad)):
        _refuse_grad("qk_norm_rope", q=q, k=k, q_weight=q_weight, k_weight=k_weight)
    index = q.get_device()
    if stream is not None or index != _current_device():
        with _launch_on(q.device, stream):
            return qk_norm_rope(q, k, cos, sin, q_weight=q_weight, k_weight=k_weight,
                                positions=positions, norm=norm, eps=eps, interleaved=interleaved,
                                q_out=q_out, k_out=k_out)
    q_out, vqo = _out_heads(q_out, "q_out", q)
    k_out, vko = _out_heads(k_out, "k_out", k)
    _raise(L.muon_qk_norm_rope(spec, vq, vk, vqo, vko, _current_handle(index)),
           "muon_qk_norm_rope")
    return q_out, k_out


@functools.lru_cache(maxsize=256)
def norm_rope_workspace_bytes(head_dim: int) -> int:
    return int(load_library().muon_norm_rope_workspace_bytes(head_dim))


def qk_norm_rope_backward(dq_out, dk_out, q, k, cos, sin, *, q_weight=None, k_weight=None,
                          positions=None, norm: bool = True, eps: float = ROPE_EPS,
                          interleaved: bool = False, dq=None, dk=None,
                          workspace: Workspace | None = None, stream=None):
    """Gradients of qk_norm_rope: from those of its outputs, and its inputs, returns (dq, dk,
    dq_weight, dk_weight); the weights' are fp32, and None where no weight is given.  dq may be
    dq_out or q itself, dk likewise."""
    L = _lib or load_library()
    spec, vq, vk = _rope_spec(q, k, cos, sin, positions, q_weight, k_weight, norm, eps,
                              interleaved)
    index, dtype = q.get_device(), q.dtype
    if stream is not None or index != _current_device():
        with _launch_on(q.device, stream):
            return qk_norm_rope_backward(
                dq_out, dk_out, q, k, cos, sin, q_weight=q_weight, k_weight=k_weight,
                positions=positions, norm=norm, eps=eps, interleaved=interleaved, dq=dq, dk=dk,
                workspace=workspace)
    vdqo = _heads(dq_out, "dq_out", q.shape, dtype, index)
    vdko = _heads(dk_out, "dk_out", k.shape, dtype, index)
    dq, vdq = _out_heads(dq, "dq", q)
    dk, vdk = _out_heads(dk, "dk", k)
    dqw = torch.empty_like(q_weight) if q_weight is not None else None
    dkw = torch.empty_like(k_weight) if k_weight is not None else None
    handle = _current_handle(index)
    ws, ws_bytes, _owner = _stream_workspace(
        workspace, norm_rope_workspace_bytes(spec.head_dim), index, handle)
    _raise(L.muon_qk_norm_rope_backward(
        spec, vdqo, vdko, vq, vk, vdq, vdk, None if dqw is None else dqw.data_ptr(),
        None if dkw is None else dkw.data_ptr(), ws, ws_bytes, handle),
        "muon_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


@functools.lru_cache(maxsize=1024)
def attention_workspace_bytes(tokens: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(load_library().muon_attention_workspace_bytes(tokens, q_heads, kv_heads, head_dim))


def _attention_spec(q, k, v, cu_seqlens, scale):
    """The spec of a call and its views of q, k and v."""
    _cuda_device(q, "q")
    dev, shape, dtype = q.get_device(), q.shape, q.dtype
    if dtype is not torch.bfloat16:
        raise TypeError(f"q, k and v must be bfloat16, got {dtype}")
    vq = _heads(q, "q", shape, dtype, dev)
    t, hq, d = shape
    kv_shape = k.shape
    if len(kv_shape) != 3:
        raise ValueError(f"k must be [tokens, heads, head_dim], got {tuple(kv_shape)}")
    hk = kv_shape[1]
    if hk == 0 or hq == 0 or hq % hk:
        raise ValueError(f"q heads ({hq}) must be a multiple of k heads ({hk})")
    kv_shape = (t, hk, d)
    vk = _heads(k, "k", kv_shape, dtype, dev)
    vv = _heads(v, "v", kv_shape, dtype, dev)
    n_seqs, cu = 0, None
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [sequences + 1]")
        cu = _ptr(cu_seqlens, "cu_seqlens", dev, torch.int32)
        n_seqs = cu_seqlens.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0
    return _AttentionSpec(t, hq, hk, d, n_seqs, cu, scale), vq, vk, vv


def attention(q, k, v, cu_seqlens=None, *, scale: float | None = None, out=None, lse=None,
              workspace: Workspace | None = None, stream=None):
    """Causal attention of bf16 heads over sequences packed along the tokens: q [tokens, q_heads,
    head_dim], k and v [tokens, kv_heads, head_dim] (strided along tokens and heads), cu_seqlens
    int32 [sequences + 1] on the device (None: one sequence).  scale is 1 / sqrt(head_dim) when
    None.  Returns (out, lse): out like q, lse [q_heads, tokens] fp32.  Tokens past the last
    sequence get out 0 and lse -inf.  After a device-side wait that gave up, calls on the same
    workspace leave their outputs as they are (new ones undefined) until workspace_status(
    workspace, clear=True); None there is the stream's default, as here.  Nothing is recorded for
    autograd: tensors that require grad are refused while it records, see attention_backward."""
    L = _lib or load_library()
    spec, vq, vk, vv = _attention_spec(q, k, v, cu_seqlens, scale)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        _refuse_grad("attention", q=q, k=k, v=v)
    index = q.get_device()
    if stream is not None or index != _current_device():
        with _launch_on(q.device, stream):
            return attention(q, k, v, cu_seqlens, scale=scale, out=out, lse=lse,
                             workspace=workspace)
    t, hq, _ = q.shape
    out, vo = _out_heads(out, "out", q)
    if lse is None:
        lse = torch.empty((hq, t), dtype=torch.float32, device=q.device)
        p_lse = lse.data_ptr()
    else:
        p_lse = _ptr(lse, "lse", index, torch.float32, (hq, t))
    handle = _current_handle(index)
    ws, ws_bytes, _owner = _stream_workspace(
        workspace, attention_workspace_bytes(t, hq, spec.kv_heads, spec.head_dim), index, handle)
    _raise(L.muon_attention(spec, vq, vk, vv, vo, p_lse, ws, ws_bytes, handle),
           "muon_attention")
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_seqlens=None, *, scale: float | None = None,
                       dq=None, dk=None, dv=None, workspace: Workspace | None = None,
                       stream=None):
    """Gradients of attention's out: from dout, the inputs, and its out and lse, returns (dq, dk,
    dv) in bf16 (dk and dv summed over the query heads of a group).  They overlap no input."""
    L = _lib or load_library()
    spec, vq, vk, vv = _attention_spec(q, k, v, cu_seqlens, scale)
    index, dtype = q.get_device(), q.dtype
    if stream is not None or index != _current_device():
        with _launch_on(q.device, stream):
            return attention_backward(dout, q, k, v, out, lse, cu_seqlens, scale=scale, dq=dq,
                                      dk=dk, dv=dv, workspace=workspace)
    t, hq, _ = q.shape
    vg = _heads(dout, "dout", q.shape, dtype, index)
    vo = _heads(out, "out", q.shape, dtype, index)
    p_lse = _ptr(lse, "lse", index, torch.float32, (hq, t))
    dq, vdq = _out_heads(dq, "dq", q)
    dk, vdk = _out_heads(dk, "dk", k)
    dv, vdv = _out_heads(dv, "dv", k)
    handle = _current_handle(index)
    ws, ws_bytes, _owner = _stream_workspace(
        workspace, attention_workspace_bytes(t, hq, spec.kv_heads, spec.head_dim), index, handle)
    _raise(L.muon_attention_backward(spec, vg, vq, vk, vv, vo, p_lse, vdq, vdk, vdv, ws,
                                     ws_bytes, handle), "muon_attention_backward")
    return dq, dk, dv


def workspace_status(workspace: Workspace | None, clear: bool = False, stream=None) -> int:
    """Synchronise and read the workspace's sticky device error word (0 = ok, 4 = timeout).
    With None: that of the workspace which attention, its gradients and those of qk_norm_rope
    keep for the current device and `stream` when the caller passes none.  (The one that a call
    captured into a CUDA graph takes is cleared by each replay and cannot be read: pass a
    Workspace to a captured call whose failure should be seen.)"""
    handle = _stream_handle(stream)
    if workspace is not None:
        return int(load_library().muon_workspace_status(workspace.ptr, workspace.nbytes, handle,
                                                        int(clear)))
    status, kept = 0, _stream_ws.get((_current_device(), handle))
    while kept is not None:                   # the one in use, and those that it outgrew
        ptr, nbytes, _, kept = kept
        status = max(status, int(load_library().muon_workspace_status(ptr, nbytes, handle,
                                                                      int(clear))))
    return status


def noalloc_status(clear: bool = False, stream=None) -> int:
    """Synchronise and read the error word of step_noalloc()'s built-in scratch on the
    current device (0 = ok, 4 = a bounded wait gave up during the latest call)."""
    return int(load_library().muon_noalloc_status(_stream_handle(stream), int(clear)))


def selftest_wait_timeout(workspace: Workspace | None, limit_us: int = 1000, stream=None):
    """Run the device-side bounded-wait timeout path once (see the C header); with
    workspace None it records the timeout in step_noalloc()'s built-in scratch."""
    ptr, nbytes = (workspace.ptr, workspace.nbytes) if workspace is not None else (None, 0)
    _raise(load_library().muon_selftest_wait_timeout(ptr, nbytes, limit_us,
                                                     _stream_handle(stream)),
           "muon_selftest_wait_timeout")


def set_fused_ns(enable: bool) -> bool:
    """Run the NS rounds of 64 <= min(r, c) <= 256, max(r, c) <= 512 matrices in one fused
    kernel (True, the default) or in the staged GEMM launches (False); returns the previous
    value."""
    prev = int(load_library().muon_set_fused_ns(int(bool(enable))))
    if prev < 0:
        raise MuonError(1, "muon_set_fused_ns")
    return bool(prev)


def set_persistent_rounds(mode) -> int:
    """Launch structure of the tensor-core NS rounds: True/1 one persistent launch,
    False/0 one launch per stage and round, "auto"/2 (the default) persistent when
    a round is short; returns the previous mode (0, 1 or 2)."""
    m = 2 if mode == "auto" else int(mode)
    prev = int(load_library().muon_set_persistent_rounds(m))
    if prev < 0:
        raise MuonError(1, "muon_set_persistent_rounds")
    return prev


class persistent_rounds:
    """Context manager: `with persistent_rounds(True): ...` runs the block with the
    persistent rounds kernel."""

    def __init__(self, mode):
        self.mode = mode
        self.prev = None

    def __enter__(self):
        self.prev = set_persistent_rounds(self.mode)
        return self

    def __exit__(self, *exc):
        set_persistent_rounds(self.prev)
        return False


def set_streamed_apply(enable: bool) -> bool:
    """Run the parameter write beside the persistent rounds kernel's last round (True,
    the default, where the call allows it) or after it (False); returns the previous
    value."""
    return bool(load_library().muon_set_streamed_apply(int(bool(enable))))


class streamed_apply:
    """Context manager: `with streamed_apply(False): ...` runs the block with the
    parameter write after the rounds kernel."""

    def __init__(self, enable: bool):
        self.enable = enable
        self.prev = None

    def __enter__(self):
        self.prev = set_streamed_apply(self.enable)
        return self

    def __exit__(self, *exc):
        set_streamed_apply(self.prev)
        return False


class fused_ns:
    """Context manager: `with fused_ns(False): ...` runs the block on the staged path."""

    def __init__(self, enable: bool):
        self.enable = bool(enable)
        self.prev = None

    def __enter__(self):
        self.prev = set_fused_ns(self.enable)
        return self

    def __exit__(self, *exc):
        set_fused_ns(self.prev)
        return False


def kernel_launch_count() -> int:
    return int(load_library().muon_kernel_launch_count())


def trace_begin(max_launches: int = 4096):
    _raise(load_library().muon_trace_begin(max_launches), "muon_trace_begin")


def trace_end(max_records: int = 4096):
    """Stop tracing; list of {kind, round, ms, flops, bytes} in launch order."""
    recs = (_TraceRecord * max(1, max_records))()
    n = ctypes.c_int(0)
    _raise(load_library().muon_trace_end(recs, max_records, ctypes.byref(n)), "muon_trace_end")
    return [{"kind": KERNEL_KINDS.get(r.kind, str(r.kind)), "round": r.round, "ms": r.ms,
             "flops": r.flops, "bytes": r.bytes} for r in recs[: n.value]]
