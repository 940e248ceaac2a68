"""Dropless MoE SwiGLU layer, and the operators around it, on one GB300 -- Python binding.

Thin ctypes binding over the C ABI in ``include/moe.h`` (library
``libmoe_gb300.so`` built in-tree by ``build.py``).  Functions carry the C
names without the ``moe_`` prefix, take torch tensors (device memory only,
any stream), check dtypes/shapes/contiguity, and pass raw pointers plus the
current CUDA stream, or the one given as ``stream``.  What a call allocates is
safe on both: it belongs to the stream of the call, and its memory is not used
again before the current one has passed the tensor's end.  (Either waits for
the other, where it reads the other's results, by the caller's doing.)  Every
step of the layer runs in the library's kernels; there is no fallback: if the
library is missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch
from torch._C._dynamo.guards import TensorGuards as _Guards  # types, shapes, strides and devices in one comparison

from . import build as _build

__all__ = [
    "MoEError", "lib", "router_logits", "router_workspace_size", "route", "route_workspace_size", "permute",
    "grouped_mlp",
    "grouped_gemm1_swiglu", "grouped_gemm2", "unpermute", "forward", "forward_workspace_size",
    "forward_views", "forward_host", "device_status", "last_device_status", "launch_count", "MoELayer",
    "mxfp8_quantize", "mxfp8_scales_size", "mxfp8_act_scales_size", "permute_mxfp8",
    "grouped_gemm1_swiglu_mxfp8", "grouped_gemm2_mxfp8", "forward_mxfp8", "forward_mxfp8_views", "MoELayerMXFP8",
    "grouped_gemm2_combine", "grouped_gemm1_swiglu_gather", "last_device_status", "forward_fuses_permute",
    "RouteRule", "RouteBuffers", "route_scored", "route_scored_backward", "NormResidual", "NormResidualGrads",
    "norm_residual", "norm_residual_backward", "GradClipper", "MoEBlock", "gated_ffn", "gated_ffn_backward",
    "GatedFFN", "GatedFFNGrads",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
           4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_TIMEOUT"}


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = lib.moe_status_string(code).decode() if _LIB is not None else _STATUS.get(code, str(code))
        super().__init__(f"{where}: {msg}")


class _Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "logits", "topk_idx", "topk_w", "counts", "offsets", "row_of", "src_tok", "route_ws",
        "router_ws", "x_perm", "h", "y_perm", "x_dev", "y_dev", "total")]


class _RouteRule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("n_group", ctypes.c_int), ("topk_group", ctypes.c_int),
                ("group_top", ctypes.c_int), ("renorm", ctypes.c_int), ("scale", ctypes.c_float)]


class _LayoutBW(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "dw", "dl", "dl_row", "dy_perm", "dh", "a", "da", "dx_perm", "WrT", "rw_part", "tmaps", "total")]


class _LayoutMX(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "logits", "topk_idx", "topk_w", "counts", "offsets", "row_of", "src_tok", "route_ws", "router_ws",
        "xq_perm", "sfa", "hq", "sfh", "y_perm", "total")]


def _load():
    path = _build.lib_path()
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(path)
    P, I, S, U64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64, ctypes.c_float
    D = ctypes.c_double
    RULE = P  # moe_route_rule_t *
    sig = {
        "moe_status_string": (ctypes.c_char_p, [I]),
        "moe_abi_version": (I, []),
        "moe_launch_count": (U64, []),
        "moe_router_workspace_size": (S, [I, I]),
        "moe_router_logits": (I, [P, P, P, I, I, I, P, P, S, P]),
        "moe_route_workspace_size": (S, [I, I, I]),
        "moe_route": (I, [P, I, I, I, P, P, P, P, P, P, P, S, P]),
        "moe_permute": (I, [P, P, I, I, I, P, P]),
        "moe_grouped_mlp": (I, [P, P, I, I, I, I, P, P, P, P, P]),
        "moe_grouped_gemm1_swiglu": (I, [P, P, I, I, I, I, P, P, P]),
        "moe_grouped_gemm1_swiglu_preact": (I, [P, P, I, I, I, I, P, P, P, P]),
        "moe_grouped_gemm1_swiglu_gather": (I, [P, P, P, I, I, I, I, I, P, P, P]),
        "moe_grouped_gemm2": (I, [P, P, I, I, I, I, P, P, P]),
        "moe_unpermute": (I, [P, P, P, I, I, I, P, P]),
        "moe_forward_workspace_size": (S, [I, I, I, I, I]),
        "moe_forward_fuses_permute": (I, [I, I, I, I, I]),
        "moe_forward_views": (I, [I, I, I, I, I, ctypes.POINTER(_Layout)]),
        "moe_forward": (I, [P, P, P, P, P, I, I, I, I, I, P, P, S, P]),
        "moe_forward_train": (I, [P, P, P, P, P, I, I, I, I, I, P, P, S, P, P]),
        "moe_forward_host_pipelined_workspace_size": (S, [I, I, I, I, I]),
        "moe_forward_host_pipelined": (I, [P, P, I, P, P, P, P, I, I, I, I, I, P, S, P]),
        "moe_forward_mxfp8_host_pipelined_workspace_size": (S, [I, I, I, I, I]),
        "moe_forward_mxfp8_host_pipelined": (I, [P, P, I, P, P, P, P, P, P, I, I, I, I, I, P, S, P]),
        "moe_forward_host": (I, [P, P, P, P, P, I, I, I, I, I, P, P, S, P]),
        "moe_mxfp8_scales_size": (S, [I, I]),
        "moe_mxfp8_quantize": (I, [P, I, I, P, P, P]),
        "moe_mxfp8_act_scales_size": (S, [I, I, I]),
        "moe_permute_mxfp8": (I, [P, P, P, P, I, I, I, I, P, P, S, P]),
        "moe_grouped_gemm1_swiglu_mxfp8": (I, [P, P, S, P, I, I, I, I, P, P, P, P, S, P]),
        "moe_grouped_gemm2_mxfp8": (I, [P, P, S, P, I, I, I, I, P, P, P, P]),
        "moe_forward_mxfp8_workspace_size": (S, [I, I, I, I, I]),
        "moe_forward_mxfp8_views": (I, [I, I, I, I, I, ctypes.POINTER(_LayoutMX)]),
        "moe_forward_mxfp8": (I, [P, P, P, P, P, P, P, I, I, I, I, I, P, P, S, P]),
        "moe_backward_workspace_size": (S, [I, I, I, I, I]),
        "moe_backward_views": (I, [I, I, I, I, I, ctypes.POINTER(_LayoutBW)]),
        "moe_backward": (I, [P, P, P, P, P, I, I, I, I, I, P, P, S, P, P, P, P, P, P, P, S, P]),
        "moe_combine_counters_size": (S, [I, I]),
        "moe_grouped_gemm2_combine": (I, [P, P, I, I, I, I, P, P, P, P, I, I, P, P, S, P, P]),
        "moe_route_scored_workspace_size": (S, [I, I, I]),
        "moe_route_scored": (I, [P, P, I, I, I, RULE, P, P, P, P, P, P, P, S, P]),
        "moe_route_scored_backward": (I, [P, P, P, I, I, I, RULE, P, P]),
        "moe_forward_scored": (I, [P, P, P, P, RULE, P, P, I, I, I, I, I, P, P, S, P, P]),
        "moe_backward_scored": (I, [P, P, RULE, P, P, I, I, I, I, I, P, P, S, P, P, P, P, P, P, P, S, P]),
        "moe_norm_residual": (I, [P, I, P, P, P, I, F, P, F, I, I, P, P, P, P, P]),
        "moe_norm_residual_backward_workspace_size": (S, [I, I]),
        "moe_norm_residual_backward": (I, [P, I, P, P, P, I, F, P, P, P, P, P, I, I, P, P, P, P, P, P, S, P]),
        "moe_norm_residual_dropout": (I, [P, I, P, P, P, I, F, P, F, D, P, I, I, P, P, P, P, P, P]),
        "moe_norm_residual_dropout_backward": (I, [P, I, P, P, P, I, F, P, D, P, P, P, P, P, I, I, P, P, P, P, P, P, S,
                                                   P]),
        "moe_gated_ffn_workspace_size": (S, [I, I, I]),
        "moe_gated_ffn": (I, [P, P, P, P, I, I, I, I, P, P, P, S, P]),
        "moe_gated_ffn_backward_workspace_size": (S, [I, I, I]),
        "moe_gated_ffn_backward": (I, [P, P, P, P, P, P, I, I, I, I, P, P, P, I, P, S, P]),
        "moe_grad_norm_workspace_size": (S, [I]),
        "moe_grad_norm": (I, [P, P, P, I, P, P, S, P]),
        "moe_grad_norm_clip": (I, [P, P, P, P, I, F, P, P, S, P]),
        "moe_device_status": (I, [ctypes.POINTER(I)]),
        "moe_last_device_status": (I, [P, P]),
        "moe_check_bounded_wait": (I, [U64, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


_LIB = _load()
lib = _LIB


# ------------------------------------------------------------------ helpers
def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _stream_of(t, stream=None) -> int:
    """The given stream, or the current one of the tensor's device (asked for
    without building a torch.cuda.Stream: a microsecond per call)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream.cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _check(code: int, where: str):
    if code != 0:
        raise MoEError(code, where)


def _need(t, dtype, shape, name):
    if t is not None and t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _in(t, dtype, shape, name) -> int:
    """The address of a tensor that _need() accepts, in one step."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _need(t, dtype, shape, name).data_ptr()


def _here(*tensors) -> int:
    """The current device, on which the library works; tensors of another one are refused (None: not given)."""
    device = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor is on device {t.get_device()}, the current one is {device}")
    return device


class _Buffers:
    """Buffers that are checked once: tensors that are not the last check's in
    address, type, shape, order and device (replaced, resized, copied, another
    view of the same memory) are checked again.  The memory is held, so that
    another tensor cannot come to lie at an old address."""
    _checked = None   # (key, addresses, guards, what the call passes, memory)

    def _same(self, key, tensors):
        """What a call with these tensors passes, if the last check was of them as they are and for
        this key (which tells what each is for); else None.  (us a call of norm_residual by
        addresses alone, with guards, and with type, shape and order asked of each tensor from
        here: 6.5, 7.0, 7.6; of route_scored 5.1, 5.8, 6.9.)"""
        c = self._checked
        if c is None or c[0] != key or not c[2](*tensors) or [t.data_ptr() for t in tensors] != c[1]:
            return None
        return c[3]

    def _keep(self, key, tensors, passed):
        guards = _Guards(*tensors, dynamic_dims_sizes=[list(t.shape) for t in tensors],
                         dynamic_dims_strides=[list(t.stride()) for t in tensors])
        self._checked = (key, [t.data_ptr() for t in tensors], guards.check, passed,
                         [t.untyped_storage() for t in tensors])
        return passed

    def __getstate__(self):  # copies are checked by themselves
        return {k: v for k, v in self.__dict__.items() if k != "_checked"}


def _on(stream, make):
    """make()'s tensors for a call on ``stream`` (None: the current one): they
    belong to that stream, so that their memory is not given to work of another
    one while the call still uses it, nor back to that stream before the
    current one, which may read the results, has passed their end."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        made = make()
    reader = torch.cuda.current_stream()
    for t in [made] if isinstance(made, torch.Tensor) else _tensors_of(made):
        t.record_stream(reader)
    return made


def _tensors_of(buffers):
    for v in vars(buffers).values():
        if isinstance(v, torch.Tensor):
            yield v
        elif isinstance(v, Routing):
            yield from _tensors_of(v)


def _empty(shape, dtype, like, stream=None):
    return _on(stream, lambda: torch.empty(shape, dtype=dtype, device=like.device))


# ------------------------------------------------------------------ a0
def router_workspace_size(d, E) -> int:
    return int(lib.moe_router_workspace_size(d, E))


def router_logits(x, Wr, bias=None, out=None, workspace=None, stream=None):
    """logits[T,E] fp32 = x[t,:] . Wr[:,e] + bias[e]: exact products (Wr split
    into three bf16 pieces) summed in fp32 on the tensor cores."""
    T, d = x.shape
    E = Wr.shape[1]
    _need(x, torch.bfloat16, (T, d), "x")
    _need(Wr, torch.float32, (d, E), "Wr")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    out = _empty((T, E), torch.float32, x, stream) if out is None else _need(out, torch.float32, (T, E), "logits")
    nbytes = router_workspace_size(d, E)
    if nbytes == 0:
        raise MoEError(2, "moe_router_workspace_size")
    if workspace is None:
        workspace = _empty((nbytes,), torch.uint8, x, stream)
    _check(lib.moe_router_logits(_ptr(x), _ptr(Wr), _ptr(bias), T, d, E, _ptr(out), _ptr(workspace),
                                 workspace.numel(), _stream(stream)), "moe_router_logits")
    return out


# ------------------------------------------------------------------ a1 + a2
@dataclass
class Routing:
    topk_idx: torch.Tensor   # [T, K] int32
    topk_w: torch.Tensor     # [T, K] fp32
    counts: torch.Tensor     # [E] int32
    offsets: torch.Tensor    # [E+1] int32
    row_of: torch.Tensor     # [T, K] int32
    src_tok: torch.Tensor    # [TK] int32


def route_workspace_size(T: int, E: int, K: int) -> int:
    return int(lib.moe_route_workspace_size(T, E, K))


def route(logits, K: int, workspace=None, stream=None) -> Routing:
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    i32 = torch.int32
    r = Routing(_empty((T, K), i32, logits, stream), _empty((T, K), torch.float32, logits, stream),
                _empty((E,), i32, logits, stream), _empty((E + 1,), i32, logits, stream),
                _empty((T, K), i32, logits, stream), _empty((T * K,), i32, logits, stream))
    nbytes = route_workspace_size(T, E, K)
    if workspace is None:
        workspace = _empty((max(nbytes, 4),), torch.uint8, logits, stream)
    _check(lib.moe_route(_ptr(logits), T, E, K, _ptr(r.topk_idx), _ptr(r.topk_w), _ptr(r.counts),
                         _ptr(r.offsets), _ptr(r.row_of), _ptr(r.src_tok), _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _stream(stream)), "moe_route")
    return r


# ------------------------------------------------------------------ routing by scores
@dataclass(frozen=True)
class RouteRule:
    """How route_scored chooses and weighs: ``score`` "sigmoid" or "softmax";
    ``n_group`` runs of experts of which the ``topk_group`` best stay open, each
    scored by its ``group_top`` (1 or 2) best experts; weights divided by their
    sum (``renorm``) and times ``scale``."""
    score: str = "sigmoid"
    n_group: int = 1
    topk_group: int = 1
    group_top: int = 1
    renorm: bool = True
    scale: float = 1.0

    def __post_init__(self):
        if self.score not in ("sigmoid", "softmax"):
            raise ValueError(f"score must be 'sigmoid' or 'softmax', got {self.score!r}")
        object.__setattr__(self, "_struct", _RouteRule(int(self.score == "softmax"), self.n_group, self.topk_group,
                                                       self.group_top, int(self.renorm), self.scale))

    @property
    def _c(self) -> int:
        """The struct's address, asked for at each call: a copy of the rule has a struct of its own."""
        return ctypes.addressof(self._struct)


class RouteBuffers(_Buffers):
    """The outputs and the workspace of route_scored for one size, to be used
    again from call to call: a call overwrites what the last one returned, so
    calls on two streams need buffers of their own."""

    def __init__(self, T: int, E: int, K: int, device="cuda"):
        i32, n = torch.int32, int(lib.moe_route_scored_workspace_size(T, E, K))
        if n == 0:
            raise MoEError(2, "moe_route_scored_workspace_size")

        def make(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=device)

        self.size = (T, E, K)
        self.routing = Routing(make(i32, T, K), make(torch.float32, T, K), make(i32, E), make(i32, E + 1),
                               make(i32, T, K), make(i32, T * K))
        self.workspace = make(torch.uint8, n)

    def _pointers(self):
        """Addresses of the outputs and of the workspace, and its bytes."""
        r, ws = self.routing, self.workspace
        tensors = [r.topk_idx, r.topk_w, r.counts, r.offsets, r.row_of, r.src_tok, ws]
        at = self._same(self.size, tensors)
        if at is None:
            (T, E, K), i32 = self.size, torch.int32
            _need(r.topk_idx, i32, (T, K), "buffers.routing.topk_idx")
            _need(r.topk_w, torch.float32, (T, K), "buffers.routing.topk_w")
            _need(r.counts, i32, (E,), "buffers.routing.counts")
            _need(r.offsets, i32, (E + 1,), "buffers.routing.offsets")
            _need(r.row_of, i32, (T, K), "buffers.routing.row_of")
            _need(r.src_tok, i32, (T * K,), "buffers.routing.src_tok")
            _need(ws, torch.uint8, (ws.numel(),), "buffers.workspace")
            at = self._keep(self.size, tensors, (*[t.data_ptr() for t in tensors], ws.numel()))
        return at


def route_scored(logits, K: int, rule: RouteRule, sel_bias=None, buffers: RouteBuffers | None = None,
                 stream=None) -> Routing:
    """Routing by scores of all experts (see RouteRule); ``sel_bias`` [E] fp32
    is added to the scores for the choice only.  Ties go to the lower expert.
    ``buffers`` holds the outputs (then reused) and the workspace."""
    T, E = logits.shape
    lp = _in(logits, torch.float32, (T, E), "logits")
    bp = None if sel_bias is None else _in(sel_bias, torch.float32, (E,), "sel_bias")
    if buffers is None:
        buffers = _on(stream, lambda: RouteBuffers(T, E, K, logits.device))
    elif buffers.size != (T, E, K):
        raise ValueError(f"buffers are for (T, E, K) = {buffers.size}, not {(T, E, K)}")
    _check(lib.moe_route_scored(lp, bp, T, E, K, rule._c, *buffers._pointers(), _stream_of(logits, stream)),
           "moe_route_scored")
    return buffers.routing


def route_scored_backward(logits, topk_idx, dw, rule: RouteRule, out=None, stream=None):
    """dlogits [T, E] fp32 of sum(dw * topk_w) for the forward's choice."""
    T, E = logits.shape
    K = topk_idx.shape[1]
    args = (_in(logits, torch.float32, (T, E), "logits"), _in(topk_idx, torch.int32, (T, K), "topk_idx"),
            _in(dw, torch.float32, (T, K), "dw"))
    if out is None:
        out = _empty((T, E), torch.float32, logits, stream)
    _check(lib.moe_route_scored_backward(*args, T, E, K, rule._c, _in(out, torch.float32, (T, E), "dlogits"),
                                         _stream_of(logits, stream)), "moe_route_scored_backward")
    return out


# ------------------------------------------------------------------ norms, gate and residual
@dataclass
class NormResidual(_Buffers):
    r: torch.Tensor                      # [T, d], the residual stream
    n: torch.Tensor | None = None        # [T, d] bf16, what the next layer reads
    rstd_post: torch.Tensor | None = None   # [T] fp32
    rstd_pre: torch.Tensor | None = None    # [T] fp32
    rng: torch.Tensor | None = None         # [2] int64, what a call with dropout drew from
    _eps = None                             # that a call used

    @classmethod
    def empty(cls, T: int, d: int, dtype=torch.bfloat16, y=True, post=True, pre=True, device="cuda", rng=False):
        """Output buffers of norm_residual: ``dtype`` of the residual stream;
        with an output ``y`` to add, its norm (``post``), the next norm (``pre``)
        and dropout (``rng``)."""
        def make(on, dt, *shape):
            return torch.empty(shape, dtype=dt, device=device) if on else None

        return cls(make(y, dtype, T, d), make(pre, torch.bfloat16, T, d), make(post, torch.float32, T),
                   make(pre, torch.float32, T), make(rng, torch.int64, 2))

    def _addresses(self, key):
        """Of the buffers that the call (T, d, dtype, y, post, pre) writes."""
        _, _, _, y, post, pre = key
        return (_ptr(self.r) if y else None, _ptr(self.n) if pre else None, _ptr(self.rstd_post) if post else None,
                _ptr(self.rstd_pre) if pre else None)

    def _pointers(self, key, rng=None, stream=None, device=None):
        """The addresses, checked; with dropout (then on the current `device`) also of its state and of
        where a call leaves it."""
        T, d, dtype, y, post, pre = key
        tensors = [self.r] if y else []
        if pre:
            tensors += (self.n, self.rstd_pre)
        if post:
            tensors.append(self.rstd_post)
        if rng is not None:
            if self.rng is None:
                self.rng = _empty((2,), torch.int64, rng, stream)
            tensors += (rng, self.rng)
            key = (*key, device)
        at = self._same(key, tensors)
        if at is None:
            if rng is not None:
                _rng_in(rng)
                _need(self.rng, torch.int64, (2,), "out.rng")
                _here(*tensors)
            if y:
                _need(self.r, dtype, (T, d), "out.r")
            if pre:
                _need(self.n, torch.bfloat16, (T, d), "out.n")
                _need(self.rstd_pre, torch.float32, (T,), "out.rstd_pre")
            if post:
                _need(self.rstd_post, torch.float32, (T,), "out.rstd_post")
            at = self._addresses(key[:6])
            at = self._keep(key, tensors, at if rng is None else (*at, rng.data_ptr(), self.rng.data_ptr()))
        return at


@dataclass
class NormResidualGrads(_Buffers):
    dr: torch.Tensor                        # [T, d], the residual's type
    dy: torch.Tensor | None = None          # [T, d] bf16
    dgamma_pre: torch.Tensor | None = None  # [d] fp32
    dgamma_post: torch.Tensor | None = None
    dgate: torch.Tensor | None = None       # shaped like the gate
    workspace: torch.Tensor | None = None

    @classmethod
    def empty(cls, T: int, d: int, dtype=torch.bfloat16, y=True, post=True, pre=True, gate="none", device="cuda"):
        """Output buffers of norm_residual_backward; ``gate``: "none", "channel" or "token"."""
        def make(on, dt, *shape):
            return torch.empty(shape, dtype=dt, device=device) if on else None

        f32, n = torch.float32, int(lib.moe_norm_residual_backward_workspace_size(T, d))
        if n == 0:
            raise MoEError(2, "moe_norm_residual_backward_workspace_size")
        return cls(make(True, dtype, T, d), make(y, torch.bfloat16, T, d), make(pre, f32, d), make(post, f32, d),
                   make(gate != "none", f32, *((d,) if gate == "channel" else (T, 1))), make(True, torch.uint8, n))

    def _addresses(self, key):
        """Of the buffers that the call (T, d, dtype, y, post, pre, gate) writes, and the workspace's bytes."""
        _, _, _, y, post, pre, gate = key
        ws = self.workspace
        return (_ptr(self.dr), _ptr(self.dy) if y else None, _ptr(self.dgamma_pre) if pre else None,
                _ptr(self.dgamma_post) if post else None, _ptr(self.dgate) if gate != "none" else None, ws.data_ptr(),
                ws.numel())

    def _pointers(self, key, stream=None, rng=None, device=None):
        """The addresses, checked; with dropout (then on the current `device`) also of its state."""
        if self.workspace is None:
            n = int(lib.moe_norm_residual_backward_workspace_size(*key[:2]))
            self.workspace = _empty((n,), torch.uint8, _need(self.dr, key[2], key[:2], "out.dr"), stream)
        T, d, dtype, y, post, pre, gate = key
        ws = self.workspace
        tensors = [self.dr, ws]
        if y:
            tensors.append(self.dy)
        if pre:
            tensors.append(self.dgamma_pre)
        if post:
            tensors.append(self.dgamma_post)
        if gate != "none":
            tensors.append(self.dgate)
        if rng is not None:
            tensors.append(rng)
            key = (*key, device)
        at = self._same(key, tensors)
        if at is None:
            if rng is not None:
                _rng_in(rng)
                _here(*tensors)
            _need(self.dr, dtype, (T, d), "out.dr")
            if y:
                _need(self.dy, torch.bfloat16, (T, d), "out.dy")
            if pre:
                _need(self.dgamma_pre, torch.float32, (d,), "out.dgamma_pre")
            if post:
                _need(self.dgamma_post, torch.float32, (d,), "out.dgamma_post")
            if gate != "none":
                _need(self.dgate, torch.float32, (d,) if gate == "channel" else (T, 1), "out.dgate")
            _need(ws, torch.uint8, (ws.numel(),), "out.workspace")
            at = self._addresses(key[:7])
            at = self._keep(key, tensors, at if rng is None else (*at, rng.data_ptr()))
        return at


_GATES = ("none", "channel", "token")


def _norm_args(r, y, gamma_post, gate, gamma_pre):
    """T, d, the kind of gate, and the addresses of r, y, gamma_post, gate and gamma_pre; checked."""
    T, d = r.shape
    dtype = r.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"the residual stream must be bfloat16 or float32, got {dtype}")
    f32, cols = torch.float32, (d,)
    kind, gp = 0, None
    if gate is not None:
        kind = 1 if gate.dim() == 1 else 2
        gp = _in(gate, f32, cols if kind == 1 else (T, 1), "gate")
    return (T, d, kind, _in(r, dtype, (T, d), "r"), None if y is None else _in(y, torch.bfloat16, (T, d), "y"),
            None if gamma_post is None else _in(gamma_post, f32, cols, "gamma_post"), gp,
            None if gamma_pre is None else _in(gamma_pre, f32, cols, "gamma_pre"))


def _rng_in(rng) -> int:
    """The address of a dropout's state, checked."""
    if rng is None:
        raise ValueError("dropout needs rng, its seed and call number: an int64 CUDA tensor [2]")
    return _in(rng, torch.int64, (2,), "rng")


def norm_residual(r, y=None, *, gamma_post=None, gate=None, gamma_pre=None, res_scale: float = 1.0,
                  eps: float = 1e-6, dropout: float = 0.0, rng=None, out: NormResidual | None = None,
                  stream=None) -> NormResidual:
    """What stands between two layers, in one kernel: r' = res_scale * r +
    gate * norm(y) * gamma_post and n = norm(r') * gamma_pre (RMS norms; parts
    without their tensor are left out).  r [T, d] bf16 or fp32, y [T, d] bf16,
    gammas [d] fp32, gate fp32 [d] (per channel) or [T, 1] (per token).
    Without y: n = norm(r) * gamma_pre, and the result's r is r itself (``out``
    keeps its own).  ``out.r`` may be r (updated in place).

    ``dropout`` > 0 drops that share of what is added to res_scale * r (and
    scales the rest by 1 / (1 - dropout)), by draws from ``rng``, a seed and a
    call number [2] int64 on the device: another number in each call draws anew,
    the same one the same mask again.
    The result's ``rng`` is a copy of them for the backward; no mask is kept.
    0 drops nothing, and rng is not read."""
    T, d, kind, rp, yp, postp, gatep, prep = _norm_args(r, y, gamma_post, gate, gamma_pre)
    key = (T, d, r.dtype, yp is not None, postp is not None, prep is not None)
    device = None
    if dropout:
        device = _here(r, y, gamma_post, gate, gamma_pre)
        if rng is None or out is None:
            _rng_in(rng)
            _here(rng)
    else:
        rng = None
    if out is None:
        out = _on(stream, lambda: NormResidual.empty(*key, r.device, rng is not None))
        at = out._addresses(key)
        if dropout:
            at = (*at, rng.data_ptr(), out.rng.data_ptr())
    else:
        at = out._pointers(key, rng, stream, device)
    if dropout:
        _check(lib.moe_norm_residual_dropout(rp, int(r.dtype is torch.float32), yp, postp, gatep, kind, res_scale, prep,
                                             eps, dropout, at[4], T, d, at[0], at[1], at[2], at[3], at[5],
                                             _stream_of(r, stream)), "moe_norm_residual_dropout")
    else:
        _check(lib.moe_norm_residual(rp, int(r.dtype is torch.float32), yp, postp, gatep, kind, res_scale, prep, eps,
                                     T, d, *at, _stream_of(r, stream)), "moe_norm_residual")
    if y is None:
        out = NormResidual(r, out.n, None, out.rstd_pre)
    out._eps = eps
    return out


def norm_residual_backward(r, dr, dn=None, y=None, *, gamma_post=None, gate=None, gamma_pre=None,
                           res_scale: float = 1.0, rstd_post=None, rstd_pre=None, dropout: float = 0.0, rng=None,
                           out: NormResidualGrads | None = None, stream=None) -> NormResidualGrads:
    """Gradients of norm_residual for ``dr`` (of its output stream, the
    residual's type; None: zero, with gamma_pre) and ``dn`` (with gamma_pre),
    from its output stream ``r`` as stored, y and the factors it returned; with
    ``dropout`` its share and the ``rng`` it returned."""
    T, d, kind, rp, yp, postp, gatep, prep = _norm_args(r, y, gamma_post, gate, gamma_pre)
    drp = None if dr is None else _in(dr, r.dtype, (T, d), "dr")
    dnp = _in(dn, torch.bfloat16, (T, d), "dn") if prep is not None else None
    rqp = _in(rstd_pre, torch.float32, (T,), "rstd_pre") if prep is not None else None
    rpp = _in(rstd_post, torch.float32, (T,), "rstd_post") if postp is not None else None
    key = (T, d, r.dtype, yp is not None, postp is not None, prep is not None, _GATES[kind])
    device = None
    if dropout:
        device = _here(r, dr, dn, y, gamma_post, gate, gamma_pre, rstd_post, rstd_pre)
        if rng is None or out is None:
            _rng_in(rng)
            _here(rng)
    else:
        rng = None
    if out is None:
        out = _on(stream, lambda: NormResidualGrads.empty(*key, r.device))
        at = out._addresses(key)
    else:
        at = out._pointers(key, stream, rng, device)[:7]
    if dropout:
        _check(lib.moe_norm_residual_dropout_backward(
            rp, int(r.dtype is torch.float32), yp, postp, gatep, kind, res_scale, prep, dropout, rng.data_ptr(), rpp, rqp,
            drp, dnp, T, d, *at, _stream_of(r, stream)), "moe_norm_residual_dropout_backward")
    else:
        _check(lib.moe_norm_residual_backward(
            rp, int(r.dtype is torch.float32), yp, postp, gatep, kind, res_scale, prep, rpp, rqp, drp, dnp, T, d,
            *at, _stream_of(r, stream)), "moe_norm_residual_backward")
    return out


# ------------------------------------------------------------------ gated feed-forward of all tokens
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


def _act(name) -> int:
    if name not in _ACTS:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {name!r}")
    return _ACTS[name]


def _ffn_sizes(W1, W2):
    """d, f of a feed-forward's weights, and their addresses; checked."""
    d, f = W2.shape
    bf16 = torch.bfloat16
    return d, f, _in(W1, bf16, (2 * f, d), "W1"), _in(W2, bf16, (d, f), "W2")


def gated_ffn(x, W1, W2, act: str = "silu", *, add=None, out=None, preact=None, workspace=None, stream=None):
    """y = (act(x W1g^T) * (x W1u^T)) W2^T + add: x, add and y [T, d], W1 [2f, d]
    (gate rows, then up rows) and W2 [d, f], all bf16; ``act`` "silu", "gelu",
    "gelu_tanh" or "relu".  ``out`` may be ``add`` (y += ...).  ``preact``
    [T, 2f] bf16 receives what the activation and the product take, for
    gated_ffn_backward.  d and f are multiples of 8."""
    T = x.shape[0]
    d, f, w1, w2 = _ffn_sizes(W1, W2)
    bf16, shape = torch.bfloat16, (T, d)
    xp, ap = _in(x, bf16, shape, "x"), None if add is None else _in(add, bf16, shape, "add")
    pp = None if preact is None else _in(preact, bf16, (T, 2 * f), "preact")
    _here(x, W1, W2, add, out, preact, workspace)
    if out is None:
        out = _empty(shape, bf16, x, stream)
    yp = _in(out, bf16, shape, "y")
    if workspace is None:
        workspace = _empty((int(lib.moe_gated_ffn_workspace_size(T, d, f)),), torch.uint8, x, stream)
    n = workspace.numel()
    _check(lib.moe_gated_ffn(xp, w1, w2, ap, _act(act), T, d, f, yp, pp, _in(workspace, torch.uint8, (n,), "workspace"), n,
                             _stream_of(x, stream)), "moe_gated_ffn")
    return out


@dataclass
class GatedFFNGrads(_Buffers):
    """Outputs and workspace of gated_ffn_backward, written over by each call
    (so calls that may run at the same time need buffers of their own)."""
    dx: torch.Tensor | None = None    # [T, d] bf16
    dW1: torch.Tensor | None = None   # shaped like the weights, bf16 or fp32
    dW2: torch.Tensor | None = None
    workspace: torch.Tensor | None = None

    @classmethod
    def empty(cls, T: int, d: int, f: int, dtype=torch.bfloat16, dx=True, weights=True, device="cuda"):
        """Output buffers of gated_ffn_backward; ``dtype`` of the weights' gradients."""
        n = int(lib.moe_gated_ffn_backward_workspace_size(T, d, f))
        if n == 0:
            raise MoEError(2, "moe_gated_ffn_backward_workspace_size")

        def make(on, dt, *shape):
            return torch.empty(shape, dtype=dt, device=device) if on else None

        return cls(make(dx, torch.bfloat16, T, d), make(weights, dtype, 2 * f, d), make(weights, dtype, d, f),
                   make(True, torch.uint8, n))

    def _pointers(self, T, d, f, stream, device):
        """Addresses of dx, dW1, dW2, whether the weights' are fp32, the workspace and its bytes; checked
        (to be on the current `device`, too)."""
        if self.workspace is None:
            n = int(lib.moe_gated_ffn_backward_workspace_size(T, d, f))
            like = next((t for t in (self.dx, self.dW1, self.dW2) if t is not None), None)
            if like is None:
                raise ValueError("out has none of dx, dW1 and dW2")
            self.workspace = _empty((n,), torch.uint8, like, stream)
        dx, dW1, dW2, ws = self.dx, self.dW1, self.dW2, self.workspace
        key = (T, d, f, dx is None, dW1 is None, dW2 is None, device)
        tensors = [t for t in (dx, dW1, dW2, ws) if t is not None]
        at = self._same(key, tensors)
        if at is None:
            f32 = torch.float32
            wide = f32 if any(t is not None and t.dtype is f32 for t in (dW1, dW2)) else torch.bfloat16
            if dx is not None:
                _need(dx, torch.bfloat16, (T, d), "out.dx")
            if dW1 is not None:
                _need(dW1, wide, (2 * f, d), "out.dW1")
            if dW2 is not None:
                _need(dW2, wide, (d, f), "out.dW2")
            _need(ws, torch.uint8, (ws.numel(),), "out.workspace")
            _here(*tensors)
            at = self._keep(key, tensors, (_ptr(dx), _ptr(dW1), _ptr(dW2), int(wide is f32), ws.data_ptr(), ws.numel()))
        return at


def gated_ffn_backward(x, preact, dy, W1, W2, act: str = "silu", *, add=None, out: GatedFFNGrads | None = None,
                       stream=None) -> GatedFFNGrads:
    """Gradients of gated_ffn for ``dy``, from x and the ``preact`` it kept.
    ``add`` [T, d] bf16 is added to dx (``out.dx`` may be ``add``).  What ``out``
    has no tensor for is not computed; without ``out`` all are, the weights' in bf16."""
    T = x.shape[0]
    d, f, w1, w2 = _ffn_sizes(W1, W2)
    bf16, shape = torch.bfloat16, (T, d)
    xp, dyp, ap = _in(x, bf16, shape, "x"), _in(dy, bf16, shape, "dy"), None if add is None else _in(add, bf16, shape,
                                                                                                    "add")
    pp = _in(preact, bf16, (T, 2 * f), "preact")
    device = _here(x, preact, dy, W1, W2, add)
    if out is None:
        out = _on(stream, lambda: GatedFFNGrads.empty(T, d, f, device=x.device))
    _check(lib.moe_gated_ffn_backward(xp, pp, dyp, w1, w2, ap, _act(act), T, d, f, *out._pointers(T, d, f, stream, device),
                                      _stream_of(x, stream)), "moe_gated_ffn_backward")
    return out


# ------------------------------------------------------------------ gradient norm and clipping
class GradClipper:
    """The global norm of a fixed set of gradient tensors (contiguous CUDA
    tensors, fp32 or bf16, of any sizes) and clipping by it.  The tensors, or
    ``outs`` of the same shapes and types for the clipped ones (None: in
    place), are held and keep their sizes; their values are read at every call,
    where they lie then (a tensor that was given other memory is checked again).

    ``clipper(max_norm)`` clips and returns the norm [1] (fp32, on the device,
    reused: calls on two streams need clippers of their own); ``clipper()``
    only returns the norm."""

    def __init__(self, grads, outs=None):
        self._grads = tuple(grads)
        self._clipped = None if outs is None else tuple(outs)
        if self.outs is not None and len(self.outs) != len(self.grads):
            raise ValueError("outs must hold one tensor for each gradient")
        for i, g in enumerate(self.grads):
            if not isinstance(g, torch.Tensor) or g.dtype not in (torch.float32, torch.bfloat16):
                raise TypeError(f"grads[{i}] must be a float32 or bfloat16 tensor")
        self._kept = [(g.dtype, g.shape) for g in self.grads]
        self._check_tensors()
        n = len(self.grads)
        device = self.grads[0].device if n else "cuda"
        self._norm = torch.empty((1,), dtype=torch.float32, device=device)
        self._workspace = torch.empty((int(lib.moe_grad_norm_workspace_size(n)),), dtype=torch.uint8, device=device)
        self._sizes = (ctypes.c_int64 * n)(*[g.numel() for g in self.grads])
        self._kinds = (ctypes.c_int32 * n)(*[int(g.dtype == torch.bfloat16) for g in self.grads])
        self._tensors = [*self.grads, *(self.outs or ()), self._norm, self._workspace]
        self._index = list(range(len(self._tensors)))
        self._take_addresses()

    grads = property(lambda self: self._grads)
    outs = property(lambda self: self._clipped)
    norm = property(lambda self: self._norm)
    workspace = property(lambda self: self._workspace)

    def _check_tensors(self):
        for i, (dtype, shape) in enumerate(self._kept):
            _need(self.grads[i], dtype, shape, f"grads[{i}]")
            if self.outs is not None:
                _need(self.outs[i], dtype, shape, f"outs[{i}]")

    def _check_overlap(self, at):
        """No element is written that is read or written elsewhere too: it would be scaled twice, or when it is late."""
        n = len(self.grads)
        nbytes = [m * (2 if k else 4) for m, k in zip(self._sizes, self._kinds)]
        spans = [(a, a + m, True) for a, m in zip(at if self.outs is None else at[n:2 * n], nbytes) if m]
        if self.outs is not None:
            spans += [(a, a + m, False) for a, o, m in zip(at, at[n:], nbytes) if m and a != o]
        spans.sort()
        written = used = 0  # the ends of what lies before
        for first, end, write in spans:
            if first < (used if write else written):
                raise ValueError("the tensors to be written overlap each other or another gradient")
            used = max(used, end)
            if write:
                written = max(written, end)

    def _take_addresses(self):
        n, at = len(self.grads), [t.data_ptr() for t in self._tensors]
        self._check_overlap(at)
        # held, so that no other tensor comes to lie at one of these addresses
        self._held = [t.untyped_storage() for t in self._tensors]
        self._ptrs = (ctypes.c_void_p * n)(*at[:n])
        self._outs = None if self.outs is None else (ctypes.c_void_p * n)(*at[n:2 * n])
        self._ws = (at[-2], at[-1], self._workspace.numel())
        self._at = at

    def __reduce__(self):  # a copy takes its tensors' addresses itself
        return GradClipper, (self.grads, self.outs)

    def __call__(self, max_norm: float | None = None, stream=None):
        # all addresses in one call (20 us for 602 of them, 35 from a loop here)
        if not torch._C._tensors_data_ptrs_at_indices_equal(self._tensors, self._at, self._index):
            self._check_tensors()
            self._take_addresses()
        n, ws = len(self.grads), (*self._ws, _stream_of(self.norm, stream))
        if max_norm is None:
            _check(lib.moe_grad_norm(self._ptrs, self._sizes, self._kinds, n, *ws), "moe_grad_norm")
        else:
            _check(lib.moe_grad_norm_clip(self._ptrs, self._outs, self._sizes, self._kinds, n, max_norm, *ws),
                   "moe_grad_norm_clip")
        return self.norm


# ------------------------------------------------------------------ a3
def permute(x, row_of, out=None, stream=None):
    """x_perm[row_of[t,k]] = x[t]."""
    T, d = x.shape
    K = row_of.shape[1]
    _need(x, torch.bfloat16, (T, d), "x")
    _need(row_of, torch.int32, (T, K), "row_of")
    out = _empty((T * K, d), torch.bfloat16, x, stream) if out is None else \
        _need(out, torch.bfloat16, (T * K, d), "x_perm")
    _check(lib.moe_permute(_ptr(x), _ptr(row_of), T, K, d, _ptr(out), _stream(stream)), "moe_permute")
    return out


# ------------------------------------------------------------------ a4 + a5
def _mlp_shapes(x_perm, offsets, W1=None, W2=None):
    TK, d = x_perm.shape
    E = offsets.shape[0] - 1
    f = W1.shape[1] // 2 if W1 is not None else W2.shape[2]
    return TK, d, E, f


def grouped_gemm1_swiglu(x_perm, offsets, W1, h=None, preact=None, stream=None):
    """h [TK, f]; with ``preact`` ([TK, 2f] bf16) the pre-activations are stored too."""
    TK, d, E, f = _mlp_shapes(x_perm, offsets, W1=W1)
    _need(x_perm, torch.bfloat16, (TK, d), "x_perm")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(W1, torch.bfloat16, (E, 2 * f, d), "W1")
    h = _empty((TK, f), torch.bfloat16, x_perm, stream) if h is None else _need(h, torch.bfloat16, (TK, f), "h")
    if preact is None:
        _check(lib.moe_grouped_gemm1_swiglu(_ptr(x_perm), _ptr(offsets), E, TK, d, f, _ptr(W1), _ptr(h),
                                            _stream(stream)), "moe_grouped_gemm1_swiglu")
    else:
        _need(preact, torch.bfloat16, (TK, 2 * f), "preact")
        _check(lib.moe_grouped_gemm1_swiglu_preact(_ptr(x_perm), _ptr(offsets), E, TK, d, f, _ptr(W1), _ptr(h),
                                                   _ptr(preact), _stream(stream)), "moe_grouped_gemm1_swiglu_preact")
    return h


def grouped_gemm1_swiglu_gather(x, src_tok, offsets, W1, h=None, stream=None):
    """GEMM1 + SwiGLU with the permute fused into its operand load: row r of
    expert e's group is read as x[src_tok[r]]; h [TK, f] equals
    grouped_gemm1_swiglu(permute(x, row_of), offsets, W1) bit for bit."""
    T, d = x.shape
    TK = src_tok.shape[0]
    E = offsets.shape[0] - 1
    f = W1.shape[1] // 2
    _need(x, torch.bfloat16, (T, d), "x")
    _need(src_tok, torch.int32, (TK,), "src_tok")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(W1, torch.bfloat16, (E, 2 * f, d), "W1")
    h = _empty((TK, f), torch.bfloat16, x, stream) if h is None else _need(h, torch.bfloat16, (TK, f), "h")
    _check(lib.moe_grouped_gemm1_swiglu_gather(_ptr(x), _ptr(src_tok), _ptr(offsets), T, E, TK, d, f, _ptr(W1),
                                               _ptr(h), _stream(stream)), "moe_grouped_gemm1_swiglu_gather")
    return h


def grouped_gemm2(h, offsets, W2, y_perm=None, stream=None):
    TK, f = h.shape
    E = offsets.shape[0] - 1
    d = W2.shape[1]
    _need(h, torch.bfloat16, (TK, f), "h")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(W2, torch.bfloat16, (E, d, f), "W2")
    y_perm = _empty((TK, d), torch.bfloat16, h, stream) if y_perm is None else \
        _need(y_perm, torch.bfloat16, (TK, d), "y_perm")
    _check(lib.moe_grouped_gemm2(_ptr(h), _ptr(offsets), E, TK, d, f, _ptr(W2), _ptr(y_perm), _stream(stream)),
           "moe_grouped_gemm2")
    return y_perm


def grouped_mlp(x_perm, offsets, W1, W2, h=None, y_perm=None, stream=None):
    TK, d, E, f = _mlp_shapes(x_perm, offsets, W1=W1)
    _need(x_perm, torch.bfloat16, (TK, d), "x_perm")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(W1, torch.bfloat16, (E, 2 * f, d), "W1")
    _need(W2, torch.bfloat16, (E, d, f), "W2")
    h = _empty((TK, f), torch.bfloat16, x_perm, stream) if h is None else _need(h, torch.bfloat16, (TK, f), "h")
    y_perm = _empty((TK, d), torch.bfloat16, x_perm, stream) if y_perm is None else \
        _need(y_perm, torch.bfloat16, (TK, d), "y_perm")
    _check(lib.moe_grouped_mlp(_ptr(x_perm), _ptr(offsets), E, TK, d, f, _ptr(W1), _ptr(W2), _ptr(h), _ptr(y_perm),
                               _stream(stream)), "moe_grouped_mlp")
    return h, y_perm


# ------------------------------------------------------------------ a6
def unpermute(y_perm, row_of, topk_w, out=None, stream=None):
    """y[t] = bf16(sum_k topk_w[t,k] * y_perm[row_of[t,k]]), fp32 accumulate."""
    T, K = row_of.shape
    d = y_perm.shape[1]
    _need(y_perm, torch.bfloat16, (T * K, d), "y_perm")
    _need(row_of, torch.int32, (T, K), "row_of")
    _need(topk_w, torch.float32, (T, K), "topk_w")
    out = _empty((T, d), torch.bfloat16, y_perm, stream) if out is None else _need(out, torch.bfloat16, (T, d), "y")
    _check(lib.moe_unpermute(_ptr(y_perm), _ptr(row_of), _ptr(topk_w), T, K, d, _ptr(out), _stream(stream)),
           "moe_unpermute")
    return out


def grouped_gemm2_combine(h, r: "Routing", W2, out=None, y_perm=None, counters=None, stream=None):
    """GEMM2 with the combine fused into its epilogue: y [T, d] bf16, equal
    bit for bit to unpermute(grouped_gemm2(h)).  y_perm and counters are
    scratch (allocated when not given)."""
    TK, f = h.shape
    E, d, _ = W2.shape
    T, K = r.row_of.shape
    _need(h, torch.bfloat16, (TK, f), "h")
    _need(W2, torch.bfloat16, (E, d, f), "W2")
    if y_perm is None:
        y_perm = _empty((TK, d), torch.bfloat16, h, stream)
    if counters is None:
        counters = _empty((max(1, int(lib.moe_combine_counters_size(T, d)) // 4),), torch.int32, h, stream)
    out = _empty((T, d), torch.bfloat16, h, stream) if out is None else _need(out, torch.bfloat16, (T, d), "y")
    _check(lib.moe_grouped_gemm2_combine(_ptr(h), _ptr(r.offsets), E, TK, d, f, _ptr(W2), _ptr(r.src_tok),
                                         _ptr(r.row_of), _ptr(r.topk_w), T, K, _ptr(y_perm), _ptr(counters),
                                         counters.numel() * 4, _ptr(out), _stream(stream)),
           "moe_grouped_gemm2_combine")
    return out


# ------------------------------------------------------------------ whole layer
def forward_workspace_size(T, d, E, K, f) -> int:
    return int(lib.moe_forward_workspace_size(T, d, E, K, f))


def forward_views(T, d, E, K, f) -> dict:
    lay = _Layout()
    _check(lib.moe_forward_views(T, d, E, K, f, ctypes.byref(lay)), "moe_forward_views")
    return {n: getattr(lay, n) for n, _ in _Layout._fields_}


def _weights_check(x, Wr, bias, W1, W2, K):
    T, d = x.shape
    E = Wr.shape[1]
    f = W1.shape[1] // 2
    _need(Wr, torch.float32, (d, E), "Wr")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    _need(W1, torch.bfloat16, (E, 2 * f, d), "W1")
    _need(W2, torch.bfloat16, (E, d, f), "W2")
    return T, d, E, f


def forward(x, Wr, bias, W1, W2, K: int, out=None, workspace=None, stream=None, preact=None,
            rule: RouteRule | None = None, sel_bias=None):
    """The whole layer in one C-ABI call (9 kernel launches, no host sync).
    With ``preact`` ([T*K, 2f] bf16) GEMM1 also stores the pre-activations
    for a backward pass (moe_forward_train).  With ``rule`` the routing is
    route_scored's (moe_forward_scored)."""
    T, d, E, f = _weights_check(x, Wr, bias, W1, W2, K)
    _need(x, torch.bfloat16, (T, d), "x")
    nbytes = forward_workspace_size(T, d, E, K, f)
    if nbytes == 0:
        raise MoEError(2, "moe_forward_workspace_size")
    if workspace is None:
        workspace = _empty((nbytes,), torch.uint8, x, stream)
    out = _empty((T, d), torch.bfloat16, x, stream) if out is None else _need(out, torch.bfloat16, (T, d), "y")
    if preact is not None:
        _need(preact, torch.bfloat16, (T * K, 2 * f), "preact")
    if rule is not None:
        if sel_bias is not None:
            _need(sel_bias, torch.float32, (E,), "sel_bias")
        _check(lib.moe_forward_scored(_ptr(x), _ptr(Wr), _ptr(bias), _ptr(sel_bias), rule._c, _ptr(W1), _ptr(W2), T, d,
                                      E, K, f, _ptr(out), _ptr(workspace), workspace.numel(), _ptr(preact),
                                      _stream(stream)), "moe_forward_scored")
    elif sel_bias is not None:
        raise ValueError("sel_bias needs a rule")
    elif preact is None:
        _check(lib.moe_forward(_ptr(x), _ptr(Wr), _ptr(bias), _ptr(W1), _ptr(W2), T, d, E, K, f, _ptr(out),
                               _ptr(workspace), workspace.numel(), _stream(stream)), "moe_forward")
    else:
        _check(lib.moe_forward_train(_ptr(x), _ptr(Wr), _ptr(bias), _ptr(W1), _ptr(W2), T, d, E, K, f, _ptr(out),
                                     _ptr(workspace), workspace.numel(), _ptr(preact), _stream(stream)),
               "moe_forward_train")
    return out


def forward_host(x_host, Wr, bias, W1, W2, K: int, y_host=None, workspace=None, stream=None):
    """The layer with activations in host memory (pinned for async copies):
    x_host [T,d] bf16 (CPU) -> y_host [T,d] bf16 (CPU).  Copies happen on the
    stream inside the C call; synchronize the stream before reading y_host."""
    if x_host.is_cuda or x_host.dtype != torch.bfloat16 or not x_host.is_contiguous():
        raise ValueError("x_host must be a contiguous CPU bf16 tensor")
    T, d = x_host.shape
    _, _, E, f = _weights_check(x_host, Wr, bias, W1, W2, K)
    nbytes = forward_workspace_size(T, d, E, K, f)
    if workspace is None:
        workspace = _empty((nbytes,), torch.uint8, W1, stream)
    if y_host is None:
        y_host = torch.empty((T, d), dtype=torch.bfloat16, pin_memory=x_host.is_pinned())
    _check(lib.moe_forward_host(_ptr(x_host), _ptr(Wr), _ptr(bias), _ptr(W1), _ptr(W2), T, d, E, K, f,
                                _ptr(y_host), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_forward_host")
    return y_host


def _host_batches(x_hosts, y_hosts, T, d):
    """Pointer arrays of the host batches (checked: contiguous CPU bf16 [T, d])."""
    if len(x_hosts) != len(y_hosts) or not x_hosts:
        raise ValueError("x_hosts and y_hosts must be non-empty and of equal length")
    for t in list(x_hosts) + list(y_hosts):
        if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or tuple(t.shape) != (T, d):
            raise ValueError("host batches must be contiguous CPU bf16 [T, d] tensors")
    xp = (ctypes.c_void_p * len(x_hosts))(*[t.data_ptr() for t in x_hosts])
    yp = (ctypes.c_void_p * len(y_hosts))(*[t.data_ptr() for t in y_hosts])
    return xp, yp


def forward_host_pipelined(x_hosts, y_hosts, Wr, bias, W1, W2, K: int, workspace=None, stream=None):
    """The layer over a list of host batches (pinned [T,d] bf16 CPU tensors;
    entries may repeat), y_hosts[i] written from x_hosts[i]; host<->device
    copies overlap the compute of neighbouring batches.  Synchronize the
    stream before reading y_hosts."""
    T, d = x_hosts[0].shape
    _, _, E, f = _weights_check(x_hosts[0], Wr, bias, W1, W2, K)
    xp, yp = _host_batches(x_hosts, y_hosts, T, d)
    nbytes = int(lib.moe_forward_host_pipelined_workspace_size(T, d, E, K, f))
    if nbytes == 0:
        raise MoEError(2, "moe_forward_host_pipelined_workspace_size")
    if workspace is None:
        workspace = _empty((nbytes,), torch.uint8, W1, stream)
    _check(lib.moe_forward_host_pipelined(xp, yp, len(x_hosts), _ptr(Wr), _ptr(bias), _ptr(W1), _ptr(W2), T, d, E,
                                          K, f, _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_forward_host_pipelined")
    return y_hosts


def forward_mxfp8_host_pipelined(x_hosts, y_hosts, Wr, bias, W1q, W1s, W2q, W2s, K: int, workspace=None,
                                 stream=None):
    """forward_host_pipelined with the MXFP8 expert matmuls (weights quantised)."""
    T, d = x_hosts[0].shape
    E, two_f, _ = W1q.shape
    f = two_f // 2
    xp, yp = _host_batches(x_hosts, y_hosts, T, d)
    nbytes = int(lib.moe_forward_mxfp8_host_pipelined_workspace_size(T, d, E, K, f))
    if nbytes == 0:
        raise MoEError(2, "moe_forward_mxfp8_host_pipelined_workspace_size")
    if workspace is None:
        workspace = _empty((nbytes,), torch.uint8, W1q, stream)
    _check(lib.moe_forward_mxfp8_host_pipelined(xp, yp, len(x_hosts), _ptr(Wr), _ptr(bias), _ptr(W1q), _ptr(W1s),
                                                _ptr(W2q), _ptr(W2s), T, d, E, K, f, _ptr(workspace),
                                                workspace.numel(), _stream(stream)),
           "moe_forward_mxfp8_host_pipelined")
    return y_hosts


def device_status() -> int:
    v = ctypes.c_int(0)
    _check(lib.moe_device_status(ctypes.byref(v)), "moe_device_status")
    return v.value


def last_device_status(out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Queues a read-and-clear of the device status word on the stream into
    ``out`` (one int32 on the device, allocated when None), without
    synchronizing: capture-safe.  Read ``out`` after the stream has run."""
    if out is None:
        out = _on(stream, lambda: torch.empty((1,), dtype=torch.int32, device="cuda"))
    if out.dtype != torch.int32 or not out.is_cuda or out.numel() < 1:
        raise ValueError("out must be an int32 CUDA tensor with at least one element")
    _check(lib.moe_last_device_status(out.data_ptr(), _stream(stream)), "moe_last_device_status")
    return out


def check_bounded_wait(limit_ns: int = 2_000_000, stream=None) -> None:
    """Launches a kernel whose only wait never completes; it times out after
    limit_ns and records MOE_ERR_DEVICE_TIMEOUT (see device_status())."""
    _check(lib.moe_check_bounded_wait(limit_ns, _stream(stream)), "moe_check_bounded_wait")


def forward_fuses_permute(T: int, d: int, E: int, K: int, f: int) -> bool:
    """True when moe_forward fuses the permute into GEMM1 for these sizes
    (then its workspace region x_perm is left unwritten)."""
    return bool(lib.moe_forward_fuses_permute(T, d, E, K, f))


def launch_count() -> int:
    return int(lib.moe_launch_count())


class MoELayer:
    """Holds one layer's weights and a persistent workspace; ``__call__(x)``
    runs the forward with one C call.  Intermediates can be read back with
    ``views()`` after a call (they live in the workspace).  With ``rule`` (and
    ``sel_bias`` [E] fp32, which may be changed between calls) it routes by
    route_scored; backward() then takes every rule but softmax without renorm
    (route_scored_backward has that one's gradient)."""

    def __init__(self, Wr, bias, W1, W2, K: int, T_max: int, rule: RouteRule | None = None, sel_bias=None):
        if sel_bias is not None and rule is None:
            raise ValueError("sel_bias needs a rule")
        self.Wr, self.bias, self.W1, self.W2, self.K = Wr, bias, W1, W2, K
        self.rule, self.sel_bias = rule, sel_bias
        self.d = W1.shape[2]
        self.E = Wr.shape[1]
        self.f = W1.shape[1] // 2
        self.T_max = T_max
        n = forward_workspace_size(T_max, self.d, self.E, K, self.f)
        if n == 0:
            raise MoEError(2, "moe_forward_workspace_size")
        self.workspace = torch.empty((n,), dtype=torch.uint8, device=W1.device)
        self._preact_buf = None
        self.preact = None
        self.calls = 0   # whose intermediates the workspace holds

    def __call__(self, x, out=None, stream=None, save_preact=False):
        """y = layer(x).  ``save_preact``: also keep GEMM1's pre-activations
        ([T*K, 2f] bf16, held by the layer) for the next backward(), which
        then skips recomputing them."""
        if x.shape[0] > self.T_max:
            raise ValueError("more tokens than the workspace was sized for")
        self.calls += 1
        self.preact = pre = None   # until they are written: backward() takes nothing of a call that was refused
        if save_preact:
            n = x.shape[0] * self.K * 2 * self.f
            if self._preact_buf is None or self._preact_buf.numel() < n:
                self._preact_buf = _empty((self.T_max * self.K * 2 * self.f,), torch.bfloat16, x, stream)
            pre = self._preact_buf[:n].view(x.shape[0] * self.K, 2 * self.f)
        out = forward(x, self.Wr, self.bias, self.W1, self.W2, self.K, out=out, workspace=self.workspace,
                      stream=stream, preact=pre, rule=self.rule, sel_bias=self.sel_bias)
        self.preact = pre
        # moe_forward may fuse the permute into GEMM1 and leave x_perm
        # unwritten; the training forward (save_preact) always writes it
        self._x_perm_written = save_preact or not forward_fuses_permute(x.shape[0], self.d, self.E, self.K, self.f)
        return out

    def backward(self, x, dy, grads=None, workspace=None, stream=None):
        """Gradients of sum(dy * y) for the last call (same x): dict of dx
        [T,d] bf16 and dWr, dbias, dW1, dW2 (fp32, shaped like the weights).
        Uses the pre-activations the last call saved, if it did."""
        T, d = x.shape
        pre = self.preact if self.preact is not None and self.preact.shape[0] == T * self.K else None
        _need(x, torch.bfloat16, (T, d), "x")
        _need(dy, torch.bfloat16, (T, d), "dy")
        n = int(lib.moe_backward_workspace_size(T, d, self.E, self.K, self.f))
        if n == 0:
            raise MoEError(2, "moe_backward_workspace_size")
        if workspace is None:
            workspace = _empty((n,), torch.uint8, x, stream)
        if not getattr(self, "_x_perm_written", True):
            # the last forward fused the permute: write the grouped rows the
            # backward reads (one permute kernel)
            v = self.views(T)
            permute(x, v["row_of"], out=v["x_perm"], stream=stream)
            self._x_perm_written = True
        if grads is None:
            f32 = torch.float32
            grads = dict(dx=_empty((T, d), torch.bfloat16, x, stream), dWr=_empty(self.Wr.shape, f32, x, stream),
                         dbias=_empty((self.E,), f32, x, stream), dW1=_empty(self.W1.shape, f32, x, stream),
                         dW2=_empty(self.W2.shape, f32, x, stream))
        fn, name, route = (lib.moe_backward, "moe_backward", _ptr(self.bias)) if self.rule is None else \
            (lib.moe_backward_scored, "moe_backward_scored", self.rule._c)
        _check(fn(_ptr(x), _ptr(self.Wr), route, _ptr(self.W1), _ptr(self.W2), T, d, self.E,
                  self.K, self.f, _ptr(dy), _ptr(self.workspace), self.workspace.numel(),
                  _ptr(pre), _ptr(grads["dx"]), _ptr(grads["dWr"]), _ptr(grads["dbias"]), _ptr(grads["dW1"]),
                  _ptr(grads["dW2"]), _ptr(workspace), workspace.numel(), _stream(stream)), name)
        self.bw_workspace = workspace
        return grads

    def backward_views(self, T: int) -> dict:
        """Typed views of the backward's intermediates (after backward())."""
        lay = _LayoutBW()
        _check(lib.moe_backward_views(T, self.d, self.E, self.K, self.f, ctypes.byref(lay)), "moe_backward_views")
        ws = self.bw_workspace
        TK = T * self.K

        def v(name, n, dtype, shape):
            off = getattr(lay, name)
            return ws[off:off + n * torch.tensor([], dtype=dtype).element_size()].view(dtype).view(shape)

        return dict(dw=v("dw", TK, torch.float32, (T, self.K)), dl=v("dl", TK, torch.float32, (T, self.K)),
                    dy_perm=v("dy_perm", TK * self.d, torch.bfloat16, (TK, self.d)),
                    dh=v("dh", TK * self.f, torch.bfloat16, (TK, self.f)),
                    a=v("a", TK * 2 * self.f, torch.bfloat16, (TK, 2 * self.f)),
                    da=v("da", TK * 2 * self.f, torch.bfloat16, (TK, 2 * self.f)),
                    dx_perm=v("dx_perm", TK * self.d, torch.bfloat16, (TK, self.d)))

    def views(self, T: int) -> dict:
        """Typed tensor views of the intermediates of the last call with T tokens."""
        lay = forward_views(T, self.d, self.E, self.K, self.f)
        ws = self.workspace
        K, E, d, f = self.K, self.E, self.d, self.f
        TK = T * K

        def v(name, n, dtype, shape):
            return ws[lay[name]:lay[name] + n * torch.tensor([], dtype=dtype).element_size()].view(dtype).view(shape)

        return dict(
            logits=v("logits", T * E, torch.float32, (T, E)),
            topk_idx=v("topk_idx", TK, torch.int32, (T, K)),
            topk_w=v("topk_w", TK, torch.float32, (T, K)),
            counts=v("counts", E, torch.int32, (E,)),
            offsets=v("offsets", E + 1, torch.int32, (E + 1,)),
            row_of=v("row_of", TK, torch.int32, (T, K)),
            src_tok=v("src_tok", TK, torch.int32, (TK,)),
            x_perm=v("x_perm", TK * d, torch.bfloat16, (TK, d)),
            h=v("h", TK * f, torch.bfloat16, (TK, f)),
            y_perm=v("y_perm", TK * d, torch.bfloat16, (TK, d)),
        )


class GatedFFN(_Buffers):
    """A gated feed-forward's weights (see gated_ffn) and a persistent workspace
    for up to T_max tokens: a dense layer, or the ``shared`` expert of a MoEBlock.
    ``__call__(x)`` runs the forward; with ``save_preact`` it keeps what
    backward() needs of it (its last call's), as MoELayer does.  The weights
    may be replaced between calls by others of their shapes.  Calls (and
    captured graphs) that may run at the same time need objects of their own."""
    rule = None

    def __init__(self, W1, W2, act: str = "silu", T_max: int = 1):
        self.W1, self.W2, self.act, self.T_max = W1, W2, act, T_max
        self.d, self.f, _, _ = _ffn_sizes(W1, W2)
        _act(act)
        n = int(lib.moe_gated_ffn_workspace_size(T_max, self.d, self.f))
        if n == 0:
            raise MoEError(2, "moe_gated_ffn_workspace_size")
        self.workspace = torch.empty((n,), dtype=torch.uint8, device=W1.device)
        self._preact_buf = None
        self.preact = None
        self.calls = 0   # whose pre-activations are kept

    def __call__(self, x, out=None, stream=None, save_preact=False, add=None):
        T = x.shape[0]
        if T > self.T_max:
            raise ValueError("more tokens than the workspace was sized for")
        self.calls += 1
        self.preact = None   # until they are written: backward() takes nothing of a call that was refused
        bf16, shape = torch.bfloat16, (T, self.d)
        xp, ap = _in(x, bf16, shape, "x"), None if add is None else _in(add, bf16, shape, "add")
        pre = None
        if save_preact:
            if self._preact_buf is None:
                self._preact_buf = _empty((self.T_max, 2 * self.f), bf16, x, stream)
            pre = self._preact_buf[:T]
        device = _here(x, add, out, pre)
        if out is None:
            out = _empty(shape, bf16, x, stream)
        w1, w2, ws, n = self._pointers(device)
        _check(lib.moe_gated_ffn(xp, w1, w2, ap, _act(self.act), T, self.d, self.f, _in(out, bf16, shape, "y"), _ptr(pre),
                                 ws, n, _stream_of(x, stream)), "moe_gated_ffn")
        self.preact = pre
        return out

    def _pointers(self, device):
        """Addresses of the weights and of the workspace, and its bytes; checked where they are new."""
        tensors = [self.W1, self.W2, self.workspace]
        at = self._same(device, tensors)
        if at is None:
            W1, W2, ws = tensors
            at = (_in(W1, torch.bfloat16, (2 * self.f, self.d), "W1"), _in(W2, torch.bfloat16, (self.d, self.f), "W2"),
                  _in(ws, torch.uint8, (ws.numel(),), "workspace"), ws.numel())
            _here(*tensors)
            self._keep(device, tensors, at)
        return at

    def backward(self, x, dy, grads=None, workspace=None, stream=None, add=None):
        """Gradients of sum(dy * y) for the last call (same x, with
        save_preact): dict of dx [T, d] bf16 (plus ``add``) and dW1, dW2 (fp32
        like MoELayer's, or of the type of those in ``grads``)."""
        if self.preact is None or self.preact.shape[0] != x.shape[0]:
            raise RuntimeError("backward() needs the last call to be of these tokens, with save_preact=True")
        if grads is None:
            f32 = torch.float32
            grads = dict(dx=_empty(x.shape, torch.bfloat16, x, stream), dW1=_empty(self.W1.shape, f32, x, stream),
                         dW2=_empty(self.W2.shape, f32, x, stream))
        gated_ffn_backward(x, self.preact, dy, self.W1, self.W2, self.act, add=add, stream=stream,
                           out=GatedFFNGrads(grads.get("dx"), grads.get("dW1"), grads.get("dW2"), workspace))
        return grads


class MoEBlock:
    """A layer inside a residual stream, as a model trains it:

        n  = norm(r) * gamma_pre
        y  = layer(n) + shared(n)
        r' = res_scale * r + drop(gate * norm(y) * gamma_post)

    ``layer``: a MoELayer, or a GatedFFN (a dense block); ``shared``: a GatedFFN
    that every token passes beside the routed experts, or None; ``gamma_post``
    and ``gate`` may be None; ``dropout``: the share that drop() drops.  Blocks
    that follow one another share a kernel: ``block(r, pre)`` takes what the
    block before it returned for ``next_gamma=block.gamma_pre`` (that norm is
    taken with the eps of the block before, so theirs must agree).  The layer
    keeps the routing and activations of its last call only, so blocks that
    share one run forward and backward one after the other."""

    def __init__(self, layer: MoELayer | GatedFFN, gamma_pre, gamma_post=None, gate=None, res_scale: float = 1.0,
                 eps: float = 1e-6, shared: GatedFFN | None = None, dropout: float = 0.0):
        if shared is not None and shared is layer:
            raise ValueError("shared must be another feed-forward than the layer")
        self.layer, self.gamma_pre, self.gamma_post, self.gate = layer, gamma_pre, gamma_post, gate
        self.res_scale, self.eps, self.shared, self.dropout = res_scale, eps, shared, dropout
        self._saved = None

    def __call__(self, r, pre: NormResidual | None = None, next_gamma=None, save: bool = False,
                 stream=None, rng=None) -> NormResidual:
        """The stream after the block, and with ``next_gamma`` its norm for the
        next block.  ``pre``: what the block before returned for this block's
        gamma_pre (else the norm is taken here).  ``save`` keeps what backward()
        needs.  ``rng`` (see norm_residual) turns the dropout on: without it
        nothing is dropped, as when a model answers.  It is neither advanced nor
        told apart by block: give each block of each step a call number of its
        own (``rng[1] += 1`` between them will do, the backward goes by a copy),
        as blocks with the same one drop the same elements."""
        rule = self.layer.rule
        if save and rule is not None and rule.score == "softmax" and not rule.renorm:
            raise ValueError("raw softmax scores have no backward in the layer: save=True needs a rule with renorm")
        own_pre = pre is None
        if own_pre:
            pre = norm_residual(r, gamma_pre=self.gamma_pre, eps=self.eps, stream=stream)
        elif pre._eps not in (None, self.eps):
            raise ValueError(f"pre was taken with eps {pre._eps}, this block's is {self.eps}")
        y = self.layer(pre.n, stream=stream, save_preact=save)
        if self.shared is not None:
            y = self.shared(pre.n, out=y, add=y, stream=stream, save_preact=save)
        drop = self.dropout if rng is not None else 0.0
        out = norm_residual(r, y, gamma_post=self.gamma_post, gate=self.gate, gamma_pre=next_gamma,
                            res_scale=self.res_scale, eps=self.eps, dropout=drop, rng=rng, stream=stream)
        self._saved = (pre, y, out, next_gamma, own_pre, self._calls(), drop) if save else None
        return out

    def _calls(self):
        return self.layer.calls, None if self.shared is None else self.shared.calls

    def backward(self, dr, dn=None, stream=None) -> dict:
        """Gradients for ``dr`` of the stream after the block and ``dn`` of its
        norm (with next_gamma): dr [T, d] of the stream before it, dn of its
        own norm's output (None when the norm was taken here: then it is in
        dr), the layer's gradients, those of the shared expert (shared_dW1,
        shared_dW2), dgamma_pre, dgamma_post, dgate, dnext_gamma."""
        if self._saved is None:
            raise RuntimeError("backward() needs a forward with save=True")
        pre, y, out, next_gamma, own_pre, calls, drop = self._saved
        if self._calls() != calls:
            raise RuntimeError("the layer has run since this block's forward: what backward() needs is no longer there")
        g = norm_residual_backward(out.r, dr, dn, y, gamma_post=self.gamma_post, gate=self.gate,
                                   gamma_pre=next_gamma, res_scale=self.res_scale, rstd_post=out.rstd_post,
                                   rstd_pre=out.rstd_pre, dropout=drop, rng=out.rng, stream=stream)
        grads = self.layer.backward(pre.n, g.dy, stream=stream)
        if self.shared is not None:
            f32 = torch.float32
            both = dict(dx=grads["dx"], dW1=_empty(self.shared.W1.shape, f32, pre.n, stream),
                        dW2=_empty(self.shared.W2.shape, f32, pre.n, stream))
            self.shared.backward(pre.n, g.dy, both, stream=stream, add=both["dx"])
            grads.update(shared_dW1=both["dW1"], shared_dW2=both["dW2"])
        grads.update(dgamma_post=g.dgamma_post, dgate=g.dgate, dnext_gamma=g.dgamma_pre, dr=g.dr, dn=grads.pop("dx"))
        if own_pre:
            # the stream before the block feeds the sum and the norm
            h = norm_residual_backward(pre.r, g.dr, grads["dn"], gamma_pre=self.gamma_pre, rstd_pre=pre.rstd_pre,
                                       stream=stream)
            grads.update(dr=h.dr, dn=None, dgamma_pre=h.dgamma_pre)
        return grads


# ------------------------------------------------------------------ MXFP8 path
def mxfp8_scales_size(rows: int, K: int) -> int:
    return int(lib.moe_mxfp8_scales_size(rows, K))


def mxfp8_act_scales_size(TK: int, E: int, K: int) -> int:
    return int(lib.moe_mxfp8_act_scales_size(TK, E, K))


def mxfp8_quantize(src, stream=None):
    """bf16 [..., K] (K a multiple of 128) -> (codes uint8 [..., K], scale
    atoms uint8 [moe_mxfp8_scales_size(rows, K)]), rows = src.numel() / K."""
    if not src.is_cuda or src.dtype != torch.bfloat16 or not src.is_contiguous():
        raise ValueError("src must be a contiguous CUDA bf16 tensor")
    K = src.shape[-1]
    rows = src.numel() // K
    n = mxfp8_scales_size(rows, K)
    if n == 0:
        raise MoEError(2, "moe_mxfp8_scales_size")
    codes = _empty(src.shape, torch.uint8, src, stream)
    scales = _empty((n,), torch.uint8, src, stream)
    _check(lib.moe_mxfp8_quantize(_ptr(src), rows, K, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_mxfp8_quantize")
    return codes, scales


def permute_mxfp8(x, r: "Routing", stream=None):
    """(xq_perm uint8 [TK, d], sfa scale atoms) of the routed tokens."""
    T, d = x.shape
    K = r.topk_idx.shape[1]
    E = r.counts.shape[0]
    _need(x, torch.bfloat16, (T, d), "x")
    n = mxfp8_act_scales_size(T * K, E, d)
    if n == 0:
        raise MoEError(2, "moe_mxfp8_act_scales_size")
    xq = _empty((T * K, d), torch.uint8, x, stream)
    sfa = _empty((n,), torch.uint8, x, stream)
    _check(lib.moe_permute_mxfp8(_ptr(x), _ptr(r.topk_idx), _ptr(r.row_of), _ptr(r.offsets), T, K, d, E, _ptr(xq),
                                 _ptr(sfa), sfa.numel(), _stream(stream)), "moe_permute_mxfp8")
    return xq, sfa


def grouped_gemm1_swiglu_mxfp8(xq, sfa, offsets, W1q, W1s, stream=None):
    """(hq uint8 [TK, f], sfh scale atoms)."""
    TK, d = xq.shape
    E, two_f, _ = W1q.shape
    f = two_f // 2
    n = mxfp8_act_scales_size(TK, E, f)
    hq = _empty((TK, f), torch.uint8, xq, stream)
    sfh = _empty((n,), torch.uint8, xq, stream)
    _check(lib.moe_grouped_gemm1_swiglu_mxfp8(_ptr(xq), _ptr(sfa), sfa.numel(), _ptr(offsets), E, TK, d, f,
                                              _ptr(W1q), _ptr(W1s), _ptr(hq), _ptr(sfh), sfh.numel(),
                                              _stream(stream)), "moe_grouped_gemm1_swiglu_mxfp8")
    return hq, sfh


def grouped_gemm2_mxfp8(hq, sfh, offsets, W2q, W2s, out=None, stream=None):
    """y_perm bf16 [TK, d]."""
    TK, f = hq.shape
    E, d, _ = W2q.shape
    out = _empty((TK, d), torch.bfloat16, hq, stream) if out is None else _need(out, torch.bfloat16, (TK, d), "y_perm")
    _check(lib.moe_grouped_gemm2_mxfp8(_ptr(hq), _ptr(sfh), sfh.numel(), _ptr(offsets), E, TK, d, f, _ptr(W2q),
                                       _ptr(W2s), _ptr(out), _stream(stream)), "moe_grouped_gemm2_mxfp8")
    return out


def forward_mxfp8_views(T, d, E, K, f) -> dict:
    lay = _LayoutMX()
    _check(lib.moe_forward_mxfp8_views(T, d, E, K, f, ctypes.byref(lay)), "moe_forward_mxfp8_views")
    return {n: getattr(lay, n) for n, _ in _LayoutMX._fields_}


def forward_mxfp8(x, Wr, bias, W1q, W1s, W2q, W2s, K: int, out=None, workspace=None, stream=None):
    """The whole layer with MXFP8 expert matmuls in one C-ABI call."""
    T, d = x.shape
    E, two_f, _ = W1q.shape
    f = two_f // 2
    _need(x, torch.bfloat16, (T, d), "x")
    _need(Wr, torch.float32, (d, E), "Wr")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    _need(W1q, torch.uint8, (E, 2 * f, d), "W1q")
    _need(W2q, torch.uint8, (E, d, f), "W2q")
    nbytes = int(lib.moe_forward_mxfp8_workspace_size(T, d, E, K, f))
    if nbytes == 0:
        raise MoEError(2, "moe_forward_mxfp8_workspace_size")
    if workspace is None:
        workspace = _empty((nbytes,), torch.uint8, x, stream)
    out = _empty((T, d), torch.bfloat16, x, stream) if out is None else _need(out, torch.bfloat16, (T, d), "y")
    _check(lib.moe_forward_mxfp8(_ptr(x), _ptr(Wr), _ptr(bias), _ptr(W1q), _ptr(W1s), _ptr(W2q), _ptr(W2s), T, d,
                                 E, K, f, _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_forward_mxfp8")
    return out


class MoELayerMXFP8:
    """A layer whose expert weights are quantised to MXFP8 once at
    construction; ``__call__(x)`` runs the MXFP8 forward with one C call."""

    def __init__(self, Wr, bias, W1, W2, K: int, T_max: int):
        self.Wr, self.bias, self.K = Wr, bias, K
        self.E, two_f, self.d = W1.shape
        self.f = two_f // 2
        self.W1q, self.W1s = mxfp8_quantize(W1)
        self.W2q, self.W2s = mxfp8_quantize(W2)
        self.T_max = T_max
        n = int(lib.moe_forward_mxfp8_workspace_size(T_max, self.d, self.E, K, self.f))
        if n == 0:
            raise MoEError(2, "moe_forward_mxfp8_workspace_size")
        self.workspace = torch.empty((n,), dtype=torch.uint8, device=W1.device)

    def __call__(self, x, out=None, stream=None):
        if x.shape[0] > self.T_max:
            raise ValueError("more tokens than the workspace was sized for")
        return forward_mxfp8(x, self.Wr, self.bias, self.W1q, self.W1s, self.W2q, self.W2s, self.K, out=out,
                             workspace=self.workspace, stream=stream)

    def views(self, T: int) -> dict:
        """Typed views of the intermediates of the last call with T tokens."""
        lay = forward_mxfp8_views(T, self.d, self.E, self.K, self.f)
        ws = self.workspace
        K, E, d, f = self.K, self.E, self.d, self.f
        TK = T * K

        def v(name, n, dtype, shape):
            return ws[lay[name]:lay[name] + n * torch.tensor([], dtype=dtype).element_size()].view(dtype).view(shape)

        return dict(
            logits=v("logits", T * E, torch.float32, (T, E)),
            topk_idx=v("topk_idx", TK, torch.int32, (T, K)),
            topk_w=v("topk_w", TK, torch.float32, (T, K)),
            counts=v("counts", E, torch.int32, (E,)),
            offsets=v("offsets", E + 1, torch.int32, (E + 1,)),
            row_of=v("row_of", TK, torch.int32, (T, K)),
            src_tok=v("src_tok", TK, torch.int32, (TK,)),
            xq_perm=v("xq_perm", TK * d, torch.uint8, (TK, d)),
            sfa=ws[lay["sfa"]:lay["hq"]],
            hq=v("hq", TK * f, torch.uint8, (TK, f)),
            sfh=ws[lay["sfh"]:lay["y_perm"]],
            y_perm=v("y_perm", TK * d, torch.bfloat16, (TK, d)),
        )
