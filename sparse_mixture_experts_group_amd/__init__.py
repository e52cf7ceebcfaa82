"""Beam Mixture-of-Experts layer for MI355X (gfx950): Python binding of libbeam_moe.so.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Tensors passed here must already live on the GPU (torch is used for
device memory and streams); the binding checks dtypes and shapes, hands raw
pointers to the C ABI declared in include/beam_moe.h, and raises on any nonzero
status.  There is no CPU path: if the library is missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbeam_moe.so")

BEAM_OK, BEAM_ERR_INVALID_ARG, BEAM_ERR_UNSUPPORTED, BEAM_ERR_WORKSPACE, BEAM_ERR_HIP = range(5)
BEAM_DTYPE_F32, BEAM_DTYPE_BF16, BEAM_DTYPE_FP8_E4M3, BEAM_DTYPE_MXFP4 = range(4)
BEAM_FP8_SCALES_FP32, BEAM_FP8_SCALES_POW2 = range(2)

C_FUNCTIONS = ("beam_moe_status_string", "beam_moe_abi_version", "beam_moe_workspace_size",
               "beam_moe_workspace_map", "beam_moe_route", "beam_moe_forward",
               "beam_moe_sublayer_forward", "beam_moe_time_kernel", "beam_dense_workspace_size",
               "beam_dense_forward", "beam_dense_sublayer_forward", "beam_moe_forward_noalloc",
               "beam_moe_sort_workspace_size", "beam_moe_sort", "beam_moe_dispatch", "beam_moe_dispatch_backward",
               "beam_moe_combine", "beam_moe_combine_backward", "beam_moe_swiglu_workspace_size", "beam_moe_swiglu", "beam_moe_swiglu_backward",
               "beam_moe_route_backward_workspace_size", "beam_moe_route_backward")
BEAM_KERNEL_NONE, BEAM_KERNEL_ROUTER_LOGITS, BEAM_KERNEL_GATE_UP, BEAM_KERNEL_DOWN, BEAM_KERNEL_COMBINE = range(5)


class beam_moe_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("routed_scale", ctypes.c_float), ("act_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("fp8_block", ctypes.c_int32),
                ("norm_eps", ctypes.c_float), ("fp8_scale_kind", ctypes.c_int32)]


ABI_VERSION = 5          # BEAM_MOE_ABI_VERSION of the structures below


class beam_moe_ws_map(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("logits", "expert_count", "expert_off", "row_of_pair",
                                               "pair_of_row", "hidden", "expert_out", "scores", "xhat",
                                               "x_q", "x_q_scale", "h_q", "h_q_scale", "total")]


class BeamMoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def make_config(hidden=5120, inter=2560, n_experts=256, n_groups=8, topk_groups=4, topk=8,
                routed_scale=2.5, act_dtype=BEAM_DTYPE_BF16, weight_dtype=BEAM_DTYPE_BF16,
                fp8_block=128, norm_eps=1e-6, fp8_scale_kind=BEAM_FP8_SCALES_FP32) -> beam_moe_config:
    """Layer configuration; the defaults are Beam's (hidden 5120, 256 experts in 8 groups
    of 32, top-4 groups, top-8 experts, intermediate 2560, scale 2.5).  fp8_scale_kind:
    BEAM_FP8_SCALES_POW2 only when every FP8 block scale is a power of two."""
    return beam_moe_config(hidden, inter, n_experts, n_groups, topk_groups, topk, routed_scale,
                           act_dtype, weight_dtype, fp8_block, norm_eps, fp8_scale_kind)


_lib = None


def lib() -> ctypes.CDLL:
    """Load libbeam_moe.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_mixture_experts_group_amd.build` (no fallback path exists)")
    L = ctypes.CDLL(LIB_PATH)
    L.beam_moe_abi_version.restype = ctypes.c_int
    if L.beam_moe_abi_version() != ABI_VERSION:
        raise ImportError(f"{LIB_PATH} has ABI {L.beam_moe_abi_version()}, this binding expects {ABI_VERSION}: "
                          "rebuild it with `python -m sparse_mixture_experts_group_amd.build`")
    vp, cfgp = ctypes.c_void_p, ctypes.POINTER(beam_moe_config)
    i64, sz = ctypes.c_int64, ctypes.c_size_t
    L.beam_moe_status_string.restype = ctypes.c_char_p
    L.beam_moe_status_string.argtypes = [ctypes.c_int]
    L.beam_moe_abi_version.restype = ctypes.c_int
    L.beam_moe_workspace_size.restype = sz
    L.beam_moe_workspace_size.argtypes = [cfgp, i64]
    L.beam_moe_workspace_map.restype = ctypes.c_int
    L.beam_moe_workspace_map.argtypes = [cfgp, i64, ctypes.POINTER(beam_moe_ws_map)]
    L.beam_moe_route.restype = ctypes.c_int
    L.beam_moe_route.argtypes = [cfgp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.beam_moe_forward.restype = ctypes.c_int
    L.beam_moe_forward.argtypes = [cfgp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.beam_moe_sublayer_forward.restype = ctypes.c_int
    L.beam_moe_sublayer_forward.argtypes = [cfgp, i64, vp, vp, vp, ctypes.c_int32, vp, vp, vp, vp, vp,
                                            vp, vp, vp, vp, vp, vp, sz, vp]
    L.beam_moe_time_kernel.restype = ctypes.c_int
    L.beam_moe_time_kernel.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
    L.beam_dense_workspace_size.restype = sz
    L.beam_dense_workspace_size.argtypes = [cfgp, i64]
    L.beam_dense_forward.restype = ctypes.c_int
    L.beam_dense_forward.argtypes = [cfgp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.beam_moe_forward_noalloc.restype = ctypes.c_int
    L.beam_moe_forward_noalloc.argtypes = [cfgp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.beam_dense_sublayer_forward.restype = ctypes.c_int
    L.beam_dense_sublayer_forward.argtypes = [cfgp, i64, vp, vp, vp, ctypes.c_int32, vp, vp, vp, vp, vp, vp, sz,
                                              vp]
    L.beam_moe_sort_workspace_size.restype = sz
    L.beam_moe_sort_workspace_size.argtypes = [cfgp, i64]
    L.beam_moe_sort.restype = ctypes.c_int
    L.beam_moe_sort.argtypes = [cfgp, i64, vp, vp, vp, vp, vp, sz, vp]
    L.beam_moe_dispatch.restype = ctypes.c_int
    L.beam_moe_dispatch.argtypes = [cfgp, i64, vp, vp, vp, i64, vp, vp, vp, vp]
    L.beam_moe_dispatch_backward.restype = ctypes.c_int
    L.beam_moe_dispatch_backward.argtypes = [cfgp, i64, vp, vp, i64, vp, vp]
    L.beam_moe_combine.restype = ctypes.c_int
    L.beam_moe_combine.argtypes = [cfgp, i64, vp, vp, i64, vp, vp, vp]
    L.beam_moe_combine_backward.restype = ctypes.c_int
    L.beam_moe_combine_backward.argtypes = [cfgp, i64, vp, vp, vp, i64, vp, vp, vp, vp]
    L.beam_moe_swiglu.restype = ctypes.c_int
    L.beam_moe_swiglu.argtypes = [cfgp, i64, vp, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    L.beam_moe_swiglu_workspace_size.restype = sz
    L.beam_moe_swiglu_workspace_size.argtypes = [cfgp, i64, i64]
    L.beam_moe_swiglu_backward.restype = ctypes.c_int
    L.beam_moe_swiglu_backward.argtypes = [cfgp, i64, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    L.beam_moe_route_backward_workspace_size.restype = sz
    L.beam_moe_route_backward_workspace_size.argtypes = [cfgp, i64]
    L.beam_moe_route_backward.restype = ctypes.c_int
    L.beam_moe_route_backward.argtypes = [cfgp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().beam_moe_status_string(int(status)).decode()


def abi_version() -> int:
    return int(lib().beam_moe_abi_version())


def beam_moe_workspace_size(cfg: beam_moe_config, T: int) -> int:
    return int(lib().beam_moe_workspace_size(ctypes.byref(cfg), int(T)))


def beam_moe_workspace_map(cfg: beam_moe_config, T: int) -> dict:
    m = beam_moe_ws_map()
    st = lib().beam_moe_workspace_map(ctypes.byref(cfg), int(T), ctypes.byref(m))
    if st != BEAM_OK:
        raise BeamMoEError(st, "beam_moe_workspace_map")
    return {n: int(getattr(m, n)) for n, _ in beam_moe_ws_map._fields_}


# ---------------------------------------------------------------------------
# tensor marshalling
# ---------------------------------------------------------------------------
def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(st: int, where: str):
    if st != BEAM_OK:
        raise BeamMoEError(st, where)


def alloc_workspace(cfg: beam_moe_config, T: int, device="cuda"):
    """Device workspace (uint8 tensor) sized by beam_moe_workspace_size."""
    import torch
    n = beam_moe_workspace_size(cfg, T)
    if n == 0 and T > 0:
        raise BeamMoEError(BEAM_ERR_INVALID_ARG, "beam_moe_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def beam_moe_route(cfg, x, w_router, logit_bias=None, ids=None, weights=None, ws=None, stream=None,
                   select_bias=None):
    """Router: returns (ids [T,K] int32, weights [T,K] float32) on the GPU."""
    import torch
    T = x.shape[0]
    K = cfg.topk
    ids = torch.empty((T, K), dtype=torch.int32, device=x.device) if ids is None else ids
    weights = torch.empty((T, K), dtype=torch.float32, device=x.device) if weights is None else weights
    ws = alloc_workspace(cfg, T, x.device) if ws is None else ws
    st = lib().beam_moe_route(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias),
                              _ptr(ids), _ptr(weights), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "beam_moe_route")
    return ids, weights


def beam_moe_forward(cfg, x, w_router, w13, w2, logit_bias=None, w13_scale=None, w2_scale=None, y=None,
                     ids=None, weights=None, ws=None, stream=None, select_bias=None):
    """One MoE layer: returns y [T,H] (same dtype as x) on the GPU."""
    import torch
    T = x.shape[0]
    y = torch.empty_like(x) if y is None else y
    ws = alloc_workspace(cfg, T, x.device) if ws is None else ws
    st = lib().beam_moe_forward(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(logit_bias),
                                _ptr(select_bias), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(y), _ptr(ids), _ptr(weights),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "beam_moe_forward")
    return y


NOALLOC_SCRATCH_BYTES = 64 << 20       # BEAM_MOE_NOALLOC_SCRATCH_BYTES


def beam_moe_forward_noalloc(cfg, x, w_router, w13, w2, logit_bias=None, w13_scale=None, w2_scale=None, y=None,
                             ids=None, weights=None, stream=None, select_bias=None):
    """beam_moe_forward on the library's static per-device scratch array (no workspace;
    the library allocates nothing).  y must be given by callers that cannot allocate."""
    import torch
    T = x.shape[0]
    y = torch.empty_like(x) if y is None else y
    st = lib().beam_moe_forward_noalloc(ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(logit_bias),
                                        _ptr(select_bias), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale),
                                        _ptr(y), _ptr(ids), _ptr(weights), _stream(stream))
    _check(st, "beam_moe_forward_noalloc")
    return y


class KernelTimer:
    """Brackets the next `n` launches of one library kernel with torch CUDA events
    (recorded by the library on the launch stream).  Use as a context manager; after
    synchronising, `times_ms()` gives each bracketed launch's duration."""

    def __init__(self, kernel: int, n: int):
        import torch
        self.kernel, self.n = kernel, n
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * n)]
        for e in self.events:          # torch creates the HIP event on its first record
            e.record()
        torch.cuda.synchronize()
        self._arr = (ctypes.c_void_p * (2 * n))(*[e.cuda_event for e in self.events])

    def __enter__(self):
        _check(lib().beam_moe_time_kernel(self.kernel, self._arr, self.n), "beam_moe_time_kernel")
        return self

    def __exit__(self, *exc):
        lib().beam_moe_time_kernel(BEAM_KERNEL_NONE, None, 0)
        return False

    def times_ms(self):
        return [self.events[2 * i].elapsed_time(self.events[2 * i + 1]) for i in range(self.n)]


def beam_moe_sublayer_forward(cfg, h, step_k, w_router, w13, w2, pre_gain=None, post_gain=None,
                              logit_bias=None, w13_scale=None, w2_scale=None, moe_out=None, ids=None,
                              weights=None, ws=None, stream=None, select_bias=None):
    """pre-RMSNorm -> MoE -> post-RMSNorm -> constant-scale residual, updating h in place."""
    T = h.shape[0]
    ws = alloc_workspace(cfg, T, h.device) if ws is None else ws
    st = lib().beam_moe_sublayer_forward(ctypes.byref(cfg), T, _ptr(h), _ptr(pre_gain), _ptr(post_gain),
                                         int(step_k), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias),
                                         _ptr(w13),
                                         _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(moe_out), _ptr(ids),
                                         _ptr(weights), _ptr(ws), ws.numel() * ws.element_size(),
                                         _stream(stream))
    _check(st, "beam_moe_sublayer_forward")
    return h


# ---------------------------------------------------------------------------
# dense SwiGLU MLP (the first decoder layers)
# ---------------------------------------------------------------------------
def make_dense_config(hidden=5120, inter=20480, act_dtype=BEAM_DTYPE_BF16, weight_dtype=BEAM_DTYPE_BF16,
                      fp8_block=128, norm_eps=1e-6, fp8_scale_kind=BEAM_FP8_SCALES_FP32) -> beam_moe_config:
    """Configuration of the dense MLP (only these fields are read; the router fields are
    left at their defaults).  The default width 20480 is a reading (8 x 2560), not a
    number on the pages."""
    return make_config(hidden=hidden, inter=inter, act_dtype=act_dtype, weight_dtype=weight_dtype,
                       fp8_block=fp8_block, norm_eps=norm_eps, fp8_scale_kind=fp8_scale_kind)


def beam_dense_workspace_size(cfg: beam_moe_config, T: int) -> int:
    return int(lib().beam_dense_workspace_size(ctypes.byref(cfg), int(T)))


def alloc_dense_workspace(cfg: beam_moe_config, T: int, device="cuda"):
    """Device workspace (uint8 tensor) sized by beam_dense_workspace_size."""
    import torch
    n = beam_dense_workspace_size(cfg, T)
    if n == 0 and T > 0:
        raise BeamMoEError(BEAM_ERR_INVALID_ARG, "beam_dense_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def beam_dense_forward(cfg, x, w13, w2, w13_scale=None, w2_scale=None, y=None, ws=None, stream=None):
    """Dense SwiGLU MLP: returns y [T,H] (same dtype as x) on the GPU."""
    import torch
    T = x.shape[0]
    y = torch.empty_like(x) if y is None else y
    ws = alloc_dense_workspace(cfg, T, x.device) if ws is None else ws
    st = lib().beam_dense_forward(ctypes.byref(cfg), T, _ptr(x), _ptr(w13), _ptr(w13_scale), _ptr(w2),
                                  _ptr(w2_scale), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream))
    _check(st, "beam_dense_forward")
    return y


def beam_dense_sublayer_forward(cfg, h, step_k, w13, w2, pre_gain=None, post_gain=None, w13_scale=None,
                                w2_scale=None, mlp_out=None, ws=None, stream=None):
    """pre-RMSNorm -> dense MLP -> post-RMSNorm -> constant-scale residual, updating h in place."""
    T = h.shape[0]
    ws = alloc_dense_workspace(cfg, T, h.device) if ws is None else ws
    st = lib().beam_dense_sublayer_forward(ctypes.byref(cfg), T, _ptr(h), _ptr(pre_gain), _ptr(post_gain),
                                           int(step_k), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale),
                                           _ptr(mlp_out), _ptr(ws), ws.numel() * ws.element_size(),
                                           _stream(stream))
    _check(st, "beam_dense_sublayer_forward")
    return h


# ---------------------------------------------------------------------------
# training operators
# ---------------------------------------------------------------------------
KEEP_BLOCK = 32          # columns that share one exponent of the 8-bit copy


def keep_blocks(cols: int) -> int:
    """Exponent bytes of one row of `cols` columns."""
    return -(-cols // KEEP_BLOCK)


def _act_torch(cfg):
    import torch
    if cfg.act_dtype == BEAM_DTYPE_BF16:
        return torch.bfloat16
    if cfg.act_dtype == BEAM_DTYPE_F32:
        return torch.float32
    raise BeamMoEError(BEAM_ERR_UNSUPPORTED, "act_dtype")


# Where a training operator runs: on the device of its tensors (all on one GPU), on the
# caller's stream or that device's current one.  _elsewhere names the stream to switch to
# when that is not where the caller stands: the operator then calls itself inside it, so
# that its device is current and its outputs and temporaries belong to its stream (a
# temporary is not handed out again before the stream is done with it).  The calls of a
# decode step cost as much on the host as on the GPU, hence the short paths.
def _elsewhere(stream, t):
    import torch
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensor must be on the GPU")
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"stream of {stream.device} for tensors on {t.device}")
        return None if dev == torch.cuda.current_device() and stream == torch.cuda.current_stream(dev) else stream
    return None if dev == torch.cuda.current_device() else torch.cuda.current_stream(dev)


def _handle(t):
    """The raw current stream of t's device."""
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _arg(name, t, dev, shape, dtype, other=None):
    """Checks one tensor's device, dtype (`dtype` or `other`) and shape and that it is dense;
    returns its address (None for None; an empty tensor has none)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on GPU {dev}, got one on {t.device}")
    if (t.dtype != dtype and t.dtype != other) or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype}{f' or {other}' if other else ''} of shape {tuple(shape)}, "
                         f"got {t.dtype} of shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr() or None


def _temporary(ws, need, like):
    """(workspace to keep alive, address, bytes): the caller's, or `need` bytes."""
    import torch
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = like.new_empty(need, dtype=torch.uint8)
    elif ws.get_device() != like.get_device() or not ws.is_contiguous():
        raise ValueError("ws: must be contiguous and on the GPU of the other tensors")
    return ws, ws.data_ptr() or None, ws.numel() * ws.element_size()


def _rows_by(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected two dimensions, got shape {tuple(t.shape)}")
    return t.shape[0]


def route_logits(cfg, T, ws):
    """The logits [T, E] that the last beam_moe_route or forward call left in its workspace
    (a view, which beam_moe_route_backward reads; the next call with ws overwrites it)."""
    import torch
    at = beam_moe_workspace_map(cfg, T)["logits"]
    return ws[at:at + 4 * T * cfg.n_experts].view(torch.float32).view(T, cfg.n_experts)


def _call(fn, args, ws, need, like):
    """fn(*args, workspace, its bytes, stream).  Without a workspace of the caller's the call
    is first made with none, which small ones do not need; only if it asks for one are its
    need() bytes allocated."""
    keep, p_ws, n_ws = _temporary(ws, 0, like)
    st = fn(*args, p_ws, n_ws, _handle(like))
    if st == BEAM_ERR_WORKSPACE and ws is None:
        keep, p_ws, n_ws = _temporary(None, need(), like)
        st = fn(*args, p_ws, n_ws, _handle(like))
    _check(st, fn.__name__)


def beam_moe_sort_workspace_size(cfg: beam_moe_config, T: int) -> int:
    return int(lib().beam_moe_sort_workspace_size(ctypes.byref(cfg), int(T)))


def beam_moe_sort(cfg, ids, expert_off=None, row_of_pair=None, pair_of_row=None, ws=None, stream=None):
    """Rows for the picks `ids` [T, K] int32, by expert: (expert_off [E+1], row_of_pair
    [T, K], pair_of_row [T*K]), all int32.  Ids outside [0, E) are dropped (row -1)."""
    import torch
    T, K, E, i32 = _rows_by(ids, "ids"), cfg.topk, cfg.n_experts, torch.int32
    on = _elsewhere(stream, ids)
    if on is not None:
        with torch.cuda.stream(on):
            return beam_moe_sort(cfg, ids, expert_off, row_of_pair, pair_of_row, ws)
    dev = ids.get_device()
    p_ids = _arg("ids", ids, dev, (T, K), i32)
    expert_off = ids.new_empty(E + 1) if expert_off is None else expert_off
    row_of_pair = ids.new_empty((T, K)) if row_of_pair is None else row_of_pair
    pair_of_row = ids.new_empty(T * K) if pair_of_row is None else pair_of_row
    _call(lib().beam_moe_sort, (ctypes.byref(cfg), T, p_ids, _arg("expert_off", expert_off, dev, (E + 1,), i32),
                                _arg("row_of_pair", row_of_pair, dev, (T, K), i32),
                                _arg("pair_of_row", pair_of_row, dev, (T * K,), i32)),
          ws, lambda: beam_moe_sort_workspace_size(cfg, T), ids)
    return expert_off, row_of_pair, pair_of_row


def beam_moe_dispatch(cfg, x, row_of_pair, xs=None, rows=None, x_scale=None, keep8=False, keep_q=None,
                      keep_scale=None, stream=None):
    """xs[row_of_pair[t, i]] = x[t]: returns xs [rows, H] (rows: T*K by default; those of no
    pair are left as they were).  x_scale: x holds the codes of an 8-bit copy.  keep8 (or
    keep_q and keep_scale): returns (xs, keep_q, keep_scale) with the 8-bit copy of x;
    rows=0 makes the copy alone (xs is None).  row_of_pair None: row t for token t."""
    import torch
    T, K, H, act = _rows_by(x, "x"), cfg.topk, cfg.hidden, _act_torch(cfg)
    on = _elsewhere(stream, x)
    if on is not None:
        with torch.cuda.stream(on):
            return beam_moe_dispatch(cfg, x, row_of_pair, xs, rows, x_scale, keep8, keep_q, keep_scale)
    u8, f8 = torch.uint8, torch.float8_e4m3fn
    dev = x.get_device()
    p_x = _arg("x", x, dev, (T, H), act) if x_scale is None else _arg("x", x, dev, (T, H), f8, u8)
    copy_alone = xs is None and rows == 0
    if xs is not None:
        rows = _rows_by(xs, "xs")
    rows = T * K if rows is None else int(rows)
    if xs is None and not copy_alone:
        xs = x.new_empty((rows, H), dtype=act)
    nb = keep_blocks(H)
    if keep8 and keep_q is None:
        keep_q = x.new_empty((T, H), dtype=f8)
    if keep8 and keep_scale is None:
        keep_scale = x.new_empty((T, nb), dtype=u8)
    st = lib().beam_moe_dispatch(ctypes.byref(cfg), T, p_x, _arg("x_scale", x_scale, dev, (T, nb), u8),
                                 _arg("row_of_pair", row_of_pair, dev, (T, K), torch.int32), rows,
                                 _arg("xs", xs, dev, (rows, H), act), _arg("keep_q", keep_q, dev, (T, H), f8, u8),
                                 _arg("keep_scale", keep_scale, dev, (T, nb), u8), _handle(x))
    _check(st, "beam_moe_dispatch")
    return xs if keep_q is None else (xs, keep_q, keep_scale)


def beam_moe_dispatch_backward(cfg, dxs, row_of_pair, dx=None, stream=None):
    """dx[t] = sum of the gradients dxs [rows, H] of token t's rows: returns dx [T, H]."""
    import torch
    rows, T, K, H = _rows_by(dxs, "dxs"), _rows_by(row_of_pair, "row_of_pair"), cfg.topk, cfg.hidden
    act = _act_torch(cfg)
    on = _elsewhere(stream, dxs)
    if on is not None:
        with torch.cuda.stream(on):
            return beam_moe_dispatch_backward(cfg, dxs, row_of_pair, dx)
    dev = dxs.get_device()
    dx = dxs.new_empty((T, H)) if dx is None else dx
    st = lib().beam_moe_dispatch_backward(ctypes.byref(cfg), T, _arg("dxs", dxs, dev, (rows, H), act),
                                          _arg("row_of_pair", row_of_pair, dev, (T, K), torch.int32), rows,
                                          _arg("dx", dx, dev, (T, H), act), _handle(dxs))
    _check(st, "beam_moe_dispatch_backward")
    return dx


def beam_moe_combine(cfg, expert_out, row_of_pair, weights, y=None, stream=None):
    """y[t] = sum_i weights[t, i] * expert_out[row_of_pair[t, i]]: returns y [T, H]."""
    import torch
    rows, T, K, H = _rows_by(expert_out, "expert_out"), _rows_by(row_of_pair, "row_of_pair"), cfg.topk, cfg.hidden
    act = _act_torch(cfg)
    on = _elsewhere(stream, expert_out)
    if on is not None:
        with torch.cuda.stream(on):
            return beam_moe_combine(cfg, expert_out, row_of_pair, weights, y)
    dev = expert_out.get_device()
    y = expert_out.new_empty((T, H)) if y is None else y
    st = lib().beam_moe_combine(ctypes.byref(cfg), T, _arg("expert_out", expert_out, dev, (rows, H), act),
                                _arg("row_of_pair", row_of_pair, dev, (T, K), torch.int32), rows,
                                _arg("weights", weights, dev, (T, K), torch.float32), _arg("y", y, dev, (T, H), act),
                                _handle(expert_out))
    _check(st, "beam_moe_combine")
    return y


def beam_moe_combine_backward(cfg, dy, expert_out, row_of_pair, weights, deo=None, dweights=None, rows=None,
                              stream=None):
    """Gradients of combine: (deo [rows, H], dweights [T, K]).  expert_out None: (deo, None),
    with `rows` rows (T*K by default).  deo may be expert_out itself."""
    import torch
    T, K, H, act = _rows_by(dy, "dy"), cfg.topk, cfg.hidden, _act_torch(cfg)
    on = _elsewhere(stream, dy)
    if on is not None:
        with torch.cuda.stream(on):
            return beam_moe_combine_backward(cfg, dy, expert_out, row_of_pair, weights, deo, dweights, rows)
    dev = dy.get_device()
    for t in (deo, expert_out):
        rows = _rows_by(t, "rows") if t is not None else rows
    rows = T * K if rows is None else int(rows)
    deo = dy.new_empty((rows, H)) if deo is None else deo
    if expert_out is not None and dweights is None:
        dweights = dy.new_empty((T, K), dtype=torch.float32)
    p_eo = _arg("expert_out", expert_out, dev, (rows, H), act)
    p_dw = _arg("dweights", dweights, dev, (T, K), torch.float32)
    if expert_out is not None and rows == 0:               # no row to read: every pair is dropped
        dweights.zero_()
        p_eo = p_dw = None
    st = lib().beam_moe_combine_backward(ctypes.byref(cfg), T, _arg("dy", dy, dev, (T, H), act), p_eo,
                                         _arg("row_of_pair", row_of_pair, dev, (T, K), torch.int32), rows,
                                         _arg("weights", weights, dev, (T, K), torch.float32),
                                         _arg("deo", deo, dev, (rows, H), act), p_dw, _handle(dy))
    _check(st, "beam_moe_combine_backward")
    return deo, dweights


def beam_moe_swiglu_workspace_size(cfg: beam_moe_config, T: int, rows: int) -> int:
    return int(lib().beam_moe_swiglu_workspace_size(ctypes.byref(cfg), int(T), int(rows)))


def beam_moe_swiglu(cfg, gu, weights=None, row_of_pair=None, h=None, keep8=False, keep_q=None, keep_scale=None,
                    ws=None, stream=None):
    """h[r] = weights[p] * SiLU(g) * u for the rows r of the pairs p, (g, u) the halves of gu
    [rows, 2I]: returns h [rows, I], with keep8 (or keep_q and keep_scale) (h, keep_q,
    keep_scale) with the 8-bit copy of gu.  row_of_pair None: row t for token t (K = 1)."""
    import torch
    rows, K, I, act = _rows_by(gu, "gu"), cfg.topk, cfg.inter, _act_torch(cfg)
    T = rows if row_of_pair is None else _rows_by(row_of_pair, "row_of_pair")
    on = _elsewhere(stream, gu)
    if on is not None:
        with torch.cuda.stream(on):
            return beam_moe_swiglu(cfg, gu, weights, row_of_pair, h, keep8, keep_q, keep_scale, ws)
    u8, f8 = torch.uint8, torch.float8_e4m3fn
    dev, nb = gu.get_device(), keep_blocks(I)
    h = gu.new_empty((rows, I)) if h is None else h
    if keep8 and keep_q is None:
        keep_q = gu.new_empty((rows, 2 * I), dtype=f8)
    if keep8 and keep_scale is None:
        keep_scale = gu.new_empty((rows, 2, nb), dtype=u8)
    _call(lib().beam_moe_swiglu, (ctypes.byref(cfg), T, _arg("gu", gu, dev, (rows, 2 * I), act),
                                  _arg("row_of_pair", row_of_pair, dev, (T, K), torch.int32), rows,
                                  _arg("weights", weights, dev, (T, K), torch.float32),
                                  _arg("h", h, dev, (rows, I), act), _arg("keep_q", keep_q, dev, (rows, 2 * I), f8, u8),
                                  _arg("keep_scale", keep_scale, dev, (rows, 2, nb), u8)),
          ws, lambda: beam_moe_swiglu_workspace_size(cfg, T, rows), gu)
    return h if keep_q is None else (h, keep_q, keep_scale)


def beam_moe_swiglu_backward(cfg, dh, gu, gu_scale=None, weights=None, row_of_pair=None, dgu=None, h=None,
                             dweights=None, again=True, ws=None, stream=None):
    """Gradients of swiglu from gu, or from its 8-bit copy with gu_scale: (dgu [rows, 2I],
    h [rows, I] computed again, or None with again=False, dweights [T, K], or None without
    weights).  dgu may be gu itself (not a copy), h may be dh itself."""
    import torch
    rows, K, I, act = _rows_by(gu, "gu"), cfg.topk, cfg.inter, _act_torch(cfg)
    T = rows if row_of_pair is None else _rows_by(row_of_pair, "row_of_pair")
    on = _elsewhere(stream, dh)
    if on is not None:
        with torch.cuda.stream(on):
            return beam_moe_swiglu_backward(cfg, dh, gu, gu_scale, weights, row_of_pair, dgu, h, dweights, again, ws)
    u8, f32, dev = torch.uint8, torch.float32, dh.get_device()
    dgu = dh.new_empty((rows, 2 * I)) if dgu is None else dgu
    if again and h is None:
        h = dh.new_empty((rows, I))
    if weights is not None and dweights is None:
        dweights = dh.new_empty((T, K), dtype=f32)
    p_gu = _arg("gu", gu, dev, (rows, 2 * I), act) if gu_scale is None else \
        _arg("gu", gu, dev, (rows, 2 * I), torch.float8_e4m3fn, u8)
    _call(lib().beam_moe_swiglu_backward, (ctypes.byref(cfg), T, _arg("dh", dh, dev, (rows, I), act), p_gu,
                                           _arg("gu_scale", gu_scale, dev, (rows, 2, keep_blocks(I)), u8),
                                           _arg("row_of_pair", row_of_pair, dev, (T, K), torch.int32), rows,
                                           _arg("weights", weights, dev, (T, K), f32),
                                           _arg("dgu", dgu, dev, (rows, 2 * I), act), _arg("h", h, dev, (rows, I), act),
                                           _arg("dweights", dweights, dev, (T, K), f32)),
          ws, lambda: beam_moe_swiglu_workspace_size(cfg, T, rows), dh)
    return dgu, h, dweights


def beam_moe_route_backward_workspace_size(cfg: beam_moe_config, T: int) -> int:
    return int(lib().beam_moe_route_backward_workspace_size(ctypes.byref(cfg), int(T)))


def beam_moe_route_backward(cfg, x, w_router, logits, ids, dweights, dx_add=None, dx=None, dw_router=None,
                            dlogit_bias=None, ws=None, stream=None):
    """Gradients of the router's weights: (dx [T, H] = dx_add + the router's part, dw_router
    [H, E], dlogit_bias [E]).  logits [T, E]: `route_logits` of the forward call's
    workspace.  dx may be dx_add itself."""
    import torch
    T, K, H, E, act = _rows_by(x, "x"), cfg.topk, cfg.hidden, cfg.n_experts, _act_torch(cfg)
    on = _elsewhere(stream, x)
    if on is not None:
        with torch.cuda.stream(on):
            return beam_moe_route_backward(cfg, x, w_router, logits, ids, dweights, dx_add, dx, dw_router, dlogit_bias, ws)
    f32, dev = torch.float32, x.get_device()
    dx = x.new_empty((T, H)) if dx is None else dx
    dw_router = x.new_empty((H, E), dtype=f32) if dw_router is None else dw_router
    dlogit_bias = x.new_empty(E, dtype=f32) if dlogit_bias is None else dlogit_bias
    ws, p_ws, n_ws = _temporary(ws, beam_moe_route_backward_workspace_size(cfg, T) if ws is None else 0, x)
    st = lib().beam_moe_route_backward(ctypes.byref(cfg), T, _arg("x", x, dev, (T, H), act),
                                       _arg("w_router", w_router, dev, (H, E), f32),
                                       _arg("logits", logits, dev, (T, E), f32),
                                       _arg("ids", ids, dev, (T, K), torch.int32),
                                       _arg("dweights", dweights, dev, (T, K), f32),
                                       _arg("dx_add", dx_add, dev, (T, H), act), _arg("dx", dx, dev, (T, H), act),
                                       _arg("dw_router", dw_router, dev, (H, E), f32),
                                       _arg("dlogit_bias", dlogit_bias, dev, (E,), f32), p_ws, n_ws, _handle(x))
    _check(st, "beam_moe_route_backward")
    return dx, dw_router, dlogit_bias
