"""Python binding of libgdn.so (the C ABI in include/gdn.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels.  PyTorch provides device memory and streams.  The names mirror the
C entry points:

    step(q, k, v, beta, gate, state, out)        -> gdn_step
    step(..., cached=True)                       -> gdn_step_ex(GDN_STATE_CACHED)
    bind_step(q, k, v, beta, gate, state, out)   -> a prepared gdn_step call
    seq(q, k, v, beta, gate, state, out)         -> gdn_seq
    seq(..., exact=True)                         -> gdn_seq_exact
    pair(q, k, v, beta, gate, state, state_next, out) -> gdn_pair
    layer_tail(x, conv_w, conv_state, beta, gate, state, z, norm_w, y, ...)
                                                 -> gdn_layer_tail
    layer_tail_workspace_bytes(B)                -> gdn_layer_tail_workspace_bytes
    layer_tail_noalloc(x, conv_w, conv_state, beta, gate, state, z, norm_w, y, ...)
                                                 -> gdn_layer_tail_noalloc
    layer_tail_pair(x, conv_w, conv_state, conv_state_next, beta, gate, state,
                    state_next, z, norm_w, y)    -> gdn_layer_tail_pair
    gate_transform(ba, a_log, dt_bias, beta, gate) -> gdn_gate_transform
    layer_tail_ba(x, conv_w, conv_state, ba, a_log, dt_bias, state, z, norm_w, y, ...)
                                                 -> gdn_layer_tail_ba
    layer_tail_ba_workspace_bytes(B)             -> gdn_layer_tail_ba_workspace_bytes
    add_rmsnorm_q8(x, residual, residual_out, norm_w, q, scale) -> gdn_add_rmsnorm_q8
    quantize_q8(x, q, scale)                     -> gdn_quantize_q8
    linear_q8(a, a_scale, w, w_scale, outs)      -> gdn_linear_q8
    verify(target, draft, draft_tokens, u_accept, u_sample, accepted, tokens, ...)
                                                 -> gdn_verify
    verify_workspace_bytes(B, V)                 -> gdn_verify_workspace_bytes
    pair_commit(accepted, state, state_next, conv_state, conv_state_next)
                                                 -> gdn_pair_commit
    last_error(), version()

If the library has not been built, importing this package raises: there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import os

from ._build import LIBRARY

__all__ = ["GdnError", "Dims", "TailParams", "GateInputs", "lib", "step", "bind_step", "seq",
           "pair",
           "layer_tail", "layer_tail_workspace_bytes", "layer_tail_noalloc", "layer_tail_pair",
           "gate_transform",
           "layer_tail_ba",
           "layer_tail_ba_workspace_bytes", "add_rmsnorm_q8", "quantize_q8", "linear_q8",
           "verify", "verify_workspace_bytes", "pair_commit", "last_error", "version", "PAGE_DIMS",
           "PAGE_TAIL", "ERRORS"]

if not os.path.exists(LIBRARY):
    raise ImportError(f"{LIBRARY} is not built; run __graft_entry__.build() "
                      "(hipcc --offload-arch=gfx950) first")


class Dims(ctypes.Structure):
    """gdn_dims"""
    _fields_ = [("n_v_heads", ctypes.c_int32), ("n_k_heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32)]


class TailParams(ctypes.Structure):
    """gdn_tail_params"""
    _fields_ = [("conv_kernel", ctypes.c_int32), ("norm_group", ctypes.c_int32),
                ("norm_eps", ctypes.c_float), ("force_unfused", ctypes.c_int32)]


class GateInputs(ctypes.Structure):
    """gdn_gate_inputs (device pointers)"""
    _fields_ = [("ba", ctypes.c_void_p), ("a_log", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p)]


PAGE_DIMS = Dims(32, 16, 128, 128)
PAGE_TAIL = TailParams(4, 128, 1e-6, 0)

ERRORS = {0: "GDN_OK", -1: "GDN_ERR_NULL", -2: "GDN_ERR_SHAPE", -3: "GDN_ERR_ALIGN",
          -4: "GDN_ERR_ALIAS", -5: "GDN_ERR_WORKSPACE", -6: "GDN_ERR_HIP"}

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_DP = ctypes.POINTER(Dims)
_TP = ctypes.POINTER(TailParams)
_GP = ctypes.POINTER(GateInputs)

lib = ctypes.CDLL(LIBRARY)
lib.gdn_version.restype = ctypes.c_int
lib.gdn_version.argtypes = []
lib.gdn_last_error.restype = ctypes.c_char_p
lib.gdn_last_error.argtypes = []
lib.gdn_step.restype = ctypes.c_int
lib.gdn_step.argtypes = [_DP, _i32] + [_vp] * 7 + [_vp]
lib.gdn_step_ex.restype = ctypes.c_int
lib.gdn_step_ex.argtypes = [_DP, _i32] + [_vp] * 7 + [ctypes.c_uint32, _vp]
STATE_CACHED = 1
lib.gdn_seq.restype = ctypes.c_int
lib.gdn_seq.argtypes = [_DP, _i32, _i32] + [_vp] * 7 + [_vp]
lib.gdn_seq_exact.restype = ctypes.c_int
lib.gdn_seq_exact.argtypes = [_DP, _i32, _i32] + [_vp] * 7 + [_vp]
lib.gdn_pair.restype = ctypes.c_int
lib.gdn_pair.argtypes = [_DP, _i32] + [_vp] * 8 + [_vp]
lib.gdn_layer_tail.restype = ctypes.c_int
lib.gdn_layer_tail.argtypes = [_DP, _TP, _i32] + [_vp] * 11 + [_vp, ctypes.c_size_t, _vp]
lib.gdn_layer_tail_pair.restype = ctypes.c_int
lib.gdn_layer_tail_pair.argtypes = [_DP, _TP, _i32] + [_vp] * 11 + [_vp]
lib.gdn_layer_tail_noalloc.restype = ctypes.c_int
lib.gdn_layer_tail_noalloc.argtypes = [_DP, _TP, _i32] + [_vp] * 11 + [_vp]
lib.gdn_layer_tail_workspace_bytes.restype = ctypes.c_size_t
lib.gdn_layer_tail_workspace_bytes.argtypes = [_DP, _i32]
lib.gdn_gate_transform.restype = ctypes.c_int
lib.gdn_gate_transform.argtypes = [_DP, _i32, _GP, _vp, _vp, _vp]
lib.gdn_layer_tail_ba.restype = ctypes.c_int
lib.gdn_layer_tail_ba.argtypes = [_DP, _TP, _i32] + [_vp] * 3 + [_GP] + [_vp] * 6 + \
    [_vp, ctypes.c_size_t, _vp]
lib.gdn_layer_tail_ba_workspace_bytes.restype = ctypes.c_size_t
lib.gdn_layer_tail_ba_workspace_bytes.argtypes = [_DP, _i32]


class LinearOut(ctypes.Structure):
    """gdn_linear_out"""
    _fields_ = [("out", ctypes.c_void_p), ("n", ctypes.c_int32)]


LINEAR_MAX_OUTS = 4
_GROUPS = [LinearOut * n for n in range(LINEAR_MAX_OUTS + 1)]
_OUTS = [f"outs[{i}]" for i in range(LINEAR_MAX_OUTS)]

lib.gdn_add_rmsnorm_q8.restype = ctypes.c_int
lib.gdn_add_rmsnorm_q8.argtypes = [_i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, ctypes.c_float,
                                   _vp, _vp, _vp]
lib.gdn_quantize_q8.restype = ctypes.c_int
lib.gdn_quantize_q8.argtypes = [_i32, _i32, _i32, _vp, _vp, _vp, _vp]
lib.gdn_linear_q8.restype = ctypes.c_int
lib.gdn_linear_q8.argtypes = [_i32, _i32] + [_vp] * 5 + [_i32, ctypes.POINTER(LinearOut), _i32,
                                                         _vp]
lib.gdn_verify.restype = ctypes.c_int
lib.gdn_verify.argtypes = [_i32] * 4 + [_vp] * 8 + [_vp, ctypes.c_size_t, _vp]
lib.gdn_verify_workspace_bytes.restype = ctypes.c_size_t
lib.gdn_verify_workspace_bytes.argtypes = [_i32, _i32]
lib.gdn_pair_commit.restype = ctypes.c_int
lib.gdn_pair_commit.argtypes = [_DP, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp]


class GdnError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{ERRORS.get(code, code)}: {message}")
        self.code = code


def version() -> int:
    return lib.gdn_version()


def last_error() -> str:
    return lib.gdn_last_error().decode()


def _check(rc: int) -> None:
    if rc != 0:
        raise GdnError(rc, last_error())


try:
    import torch as _torch
    _F32 = _torch.float32
except ImportError:       # the checks below then raise the import error
    _F32 = None


def _ptr(t, name, shape=None, optional=False):
    """Device address of a contiguous float32 GPU tensor of the given shape.
    The common case is tested in one expression; anything else goes through
    the checks one by one, which name what is wrong."""
    try:
        if (t.dtype is _F32 and t.is_cuda and t.is_contiguous()
                and (shape is None or t.shape == shape)):
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr_checked(t, name, shape, optional)


def _ptr_checked(t, name, shape, optional):
    import torch
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dims_of(q, v):
    Hk, dk = q.shape[-2], q.shape[-1]
    Hv, dv = v.shape[-2], v.shape[-1]
    return Dims(Hv, Hk, dk, dv)


def step(q, k, v, beta, gate, state, out, stream=None, cached=False) -> None:
    """gdn_step: q,k [B][Hk][dk], v [B][Hv][dv], beta/gate [B][Hv],
    state [B][Hv][dv][dk] (updated in place), out [B][Hv][dv].  cached=True
    calls gdn_step_ex with GDN_STATE_CACHED (states resident in the Infinity
    Cache across calls)."""
    B = q.shape[0]
    d = _dims_of(q, v)
    args = (ctypes.byref(d), B,
            _ptr(q, "q", (B, d.n_k_heads, d.d_k)), _ptr(k, "k", (B, d.n_k_heads, d.d_k)),
            _ptr(v, "v", (B, d.n_v_heads, d.d_v)),
            _ptr(beta, "beta", (B, d.n_v_heads)), _ptr(gate, "gate", (B, d.n_v_heads)),
            _ptr(state, "state", (B, d.n_v_heads, d.d_v, d.d_k)),
            _ptr(out, "out", (B, d.n_v_heads, d.d_v)))
    if cached:
        _check(lib.gdn_step_ex(*args, STATE_CACHED, _stream(stream)))
    else:
        _check(lib.gdn_step(*args, _stream(stream)))


def bind_step(q, k, v, beta, gate, state, out, stream=None, cached=False):
    """A prepared gdn_step call for latency-bound decode loops that step the
    same buffers again and again (new token values written into q, k, v,
    beta and gate between calls): the tensors are checked once here and the
    returned function only re-issues the C call with the converted
    arguments.  The tensors must stay alive and in place while it is used.
    The library still validates every call."""
    B = q.shape[0]
    d = _dims_of(q, v)
    ptrs = (_ptr(q, "q", (B, d.n_k_heads, d.d_k)), _ptr(k, "k", (B, d.n_k_heads, d.d_k)),
            _ptr(v, "v", (B, d.n_v_heads, d.d_v)),
            _ptr(beta, "beta", (B, d.n_v_heads)), _ptr(gate, "gate", (B, d.n_v_heads)),
            _ptr(state, "state", (B, d.n_v_heads, d.d_v, d.d_k)),
            _ptr(out, "out", (B, d.n_v_heads, d.d_v)))
    args = [ctypes.byref(d), ctypes.c_int32(B), *(ctypes.c_void_p(p) for p in ptrs)]
    if cached:
        fn = lib.gdn_step_ex
        args.append(ctypes.c_uint32(STATE_CACHED))
    else:
        fn = lib.gdn_step
    args.append(ctypes.c_void_p(_stream(stream)))
    args = tuple(args)
    keep = (d, q, k, v, beta, gate, state, out)

    def call() -> None:
        rc = fn(*args)
        if rc != 0:
            raise GdnError(rc, last_error())
    call.tensors = keep
    return call


def seq(q, k, v, beta, gate, state, out, stream=None, exact=False) -> None:
    """gdn_seq (gdn_seq_exact with exact=True): q,k [B][T][Hk][dk],
    v [B][T][Hv][dv], beta/gate [B][T][Hv], state [B][Hv][dv][dk] (in/out),
    out [B][T][Hv][dv]."""
    B, T = q.shape[0], q.shape[1]
    d = _dims_of(q, v)
    _check((lib.gdn_seq_exact if exact else lib.gdn_seq)(
        ctypes.byref(d), B, T,
        _ptr(q, "q", (B, T, d.n_k_heads, d.d_k)), _ptr(k, "k", (B, T, d.n_k_heads, d.d_k)),
        _ptr(v, "v", (B, T, d.n_v_heads, d.d_v)),
        _ptr(beta, "beta", (B, T, d.n_v_heads)), _ptr(gate, "gate", (B, T, d.n_v_heads)),
        _ptr(state, "state", (B, d.n_v_heads, d.d_v, d.d_k)),
        _ptr(out, "out", (B, T, d.n_v_heads, d.d_v)), _stream(stream)))


def pair(q, k, v, beta, gate, state, state_next, out, stream=None) -> None:
    """gdn_pair: q,k [B][2][Hk][dk], v [B][2][Hv][dv], beta/gate [B][2][Hv];
    state [B][Hv][dv][dk] is committed with position 1 in place;
    state_next (same shape) receives the tentative state after position 2;
    out [B][2][Hv][dv]."""
    B = q.shape[0]
    d = _dims_of(q, v)
    _check(lib.gdn_pair(
        ctypes.byref(d), B,
        _ptr(q, "q", (B, 2, d.n_k_heads, d.d_k)), _ptr(k, "k", (B, 2, d.n_k_heads, d.d_k)),
        _ptr(v, "v", (B, 2, d.n_v_heads, d.d_v)),
        _ptr(beta, "beta", (B, 2, d.n_v_heads)), _ptr(gate, "gate", (B, 2, d.n_v_heads)),
        _ptr(state, "state", (B, d.n_v_heads, d.d_v, d.d_k)),
        _ptr(state_next, "state_next", (B, d.n_v_heads, d.d_v, d.d_k)),
        _ptr(out, "out", (B, 2, d.n_v_heads, d.d_v)), _stream(stream)))


def layer_tail_workspace_bytes(B: int, dims: Dims = PAGE_DIMS) -> int:
    return int(lib.gdn_layer_tail_workspace_bytes(ctypes.byref(dims), B))


def _workspace(workspace):
    import torch
    if workspace is None:
        return None, 0
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous GPU tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def layer_tail(x, conv_w, conv_state, beta, gate, state, z, norm_w, y,
               dbg_qkv=None, dbg_core=None, workspace=None,
               dims: Dims = PAGE_DIMS, params: TailParams = PAGE_TAIL, stream=None) -> None:
    """gdn_layer_tail.  workspace: a GPU tensor of at least
    layer_tail_workspace_bytes(B) bytes (any dtype), or None when both dbg
    buffers are given."""
    B, C = x.shape
    K = params.conv_kernel
    nv = dims.n_v_heads * dims.d_v
    ws_ptr, ws_bytes = _workspace(workspace)
    _check(lib.gdn_layer_tail(
        ctypes.byref(dims), ctypes.byref(params), B,
        _ptr(x, "x", (B, C)), _ptr(conv_w, "conv_w", (C, K)),
        _ptr(conv_state, "conv_state", (B, K - 1, C)),
        _ptr(beta, "beta", (B, dims.n_v_heads)), _ptr(gate, "gate", (B, dims.n_v_heads)),
        _ptr(state, "state", (B, dims.n_v_heads, dims.d_v, dims.d_k)),
        _ptr(z, "z", (B, nv)), _ptr(norm_w, "norm_w", (params.norm_group,)),
        _ptr(y, "y", (B, nv)),
        _ptr(dbg_qkv, "dbg_qkv", (B, C), optional=True),
        _ptr(dbg_core, "dbg_core", (B, dims.n_v_heads, dims.d_v), optional=True),
        ws_ptr, ws_bytes, _stream(stream)))


def layer_tail_noalloc(x, conv_w, conv_state, beta, gate, state, z, norm_w, y,
                       dbg_qkv=None, dbg_core=None,
                       dims: Dims = PAGE_DIMS, params: TailParams = PAGE_TAIL,
                       stream=None) -> None:
    """gdn_layer_tail_noalloc: layer_tail with the library's static per-GPU
    scratch in place of a workspace (allocates nothing)."""
    B, C = x.shape
    K = params.conv_kernel
    nv = dims.n_v_heads * dims.d_v
    _check(lib.gdn_layer_tail_noalloc(
        ctypes.byref(dims), ctypes.byref(params), B,
        _ptr(x, "x", (B, C)), _ptr(conv_w, "conv_w", (C, K)),
        _ptr(conv_state, "conv_state", (B, K - 1, C)),
        _ptr(beta, "beta", (B, dims.n_v_heads)), _ptr(gate, "gate", (B, dims.n_v_heads)),
        _ptr(state, "state", (B, dims.n_v_heads, dims.d_v, dims.d_k)),
        _ptr(z, "z", (B, nv)), _ptr(norm_w, "norm_w", (params.norm_group,)),
        _ptr(y, "y", (B, nv)),
        _ptr(dbg_qkv, "dbg_qkv", (B, C), optional=True),
        _ptr(dbg_core, "dbg_core", (B, dims.n_v_heads, dims.d_v), optional=True),
        _stream(stream)))


def layer_tail_pair(x, conv_w, conv_state, conv_state_next, beta, gate, state, state_next,
                    z, norm_w, y, dims: Dims = PAGE_DIMS, params: TailParams = PAGE_TAIL,
                    stream=None) -> None:
    """gdn_layer_tail_pair: x [B][2][C], beta/gate [B][2][Hv], z/y [B][2][Hv*dv].
    conv_state and state are committed with position 1 in place;
    conv_state_next and state_next receive the tentative ring and state after
    position 2."""
    B, _, C = x.shape
    K = params.conv_kernel
    nv = dims.n_v_heads * dims.d_v
    st = (B, dims.n_v_heads, dims.d_v, dims.d_k)
    _check(lib.gdn_layer_tail_pair(
        ctypes.byref(dims), ctypes.byref(params), B,
        _ptr(x, "x", (B, 2, C)), _ptr(conv_w, "conv_w", (C, K)),
        _ptr(conv_state, "conv_state", (B, K - 1, C)),
        _ptr(conv_state_next, "conv_state_next", (B, K - 1, C)),
        _ptr(beta, "beta", (B, 2, dims.n_v_heads)), _ptr(gate, "gate", (B, 2, dims.n_v_heads)),
        _ptr(state, "state", st), _ptr(state_next, "state_next", st),
        _ptr(z, "z", (B, 2, nv)), _ptr(norm_w, "norm_w", (params.norm_group,)),
        _ptr(y, "y", (B, 2, nv)), _stream(stream)))


def _gate_inputs(ba, a_log, dt_bias, B, Hv):
    return GateInputs(_ptr(ba, "ba", (B, 2 * Hv)), _ptr(a_log, "a_log", (Hv,)),
                      _ptr(dt_bias, "dt_bias", (Hv,)))


def gate_transform(ba, a_log, dt_bias, beta, gate, dims: Dims = PAGE_DIMS, stream=None) -> None:
    """gdn_gate_transform: ba [B][2*Hv] (beta logits | alpha logits), a_log and
    dt_bias [Hv] -> beta, gate [B][Hv]."""
    B = ba.shape[0]
    Hv = dims.n_v_heads
    gi = _gate_inputs(ba, a_log, dt_bias, B, Hv)
    _check(lib.gdn_gate_transform(ctypes.byref(dims), B, ctypes.byref(gi),
                                  _ptr(beta, "beta", (B, Hv)), _ptr(gate, "gate", (B, Hv)),
                                  _stream(stream)))


def layer_tail_ba_workspace_bytes(B: int, dims: Dims = PAGE_DIMS) -> int:
    return int(lib.gdn_layer_tail_ba_workspace_bytes(ctypes.byref(dims), B))


def layer_tail_ba(x, conv_w, conv_state, ba, a_log, dt_bias, state, z, norm_w, y,
                  dbg_qkv=None, dbg_core=None, workspace=None,
                  dims: Dims = PAGE_DIMS, params: TailParams = PAGE_TAIL, stream=None) -> None:
    """gdn_layer_tail_ba: layer_tail with beta and gate made from the raw gate
    inputs.  workspace: at least layer_tail_ba_workspace_bytes(B) bytes."""
    B, C = x.shape
    K = params.conv_kernel
    nv = dims.n_v_heads * dims.d_v
    gi = _gate_inputs(ba, a_log, dt_bias, B, dims.n_v_heads)
    ws_ptr, ws_bytes = _workspace(workspace)
    _check(lib.gdn_layer_tail_ba(
        ctypes.byref(dims), ctypes.byref(params), B,
        _ptr(x, "x", (B, C)), _ptr(conv_w, "conv_w", (C, K)),
        _ptr(conv_state, "conv_state", (B, K - 1, C)), ctypes.byref(gi),
        _ptr(state, "state", (B, dims.n_v_heads, dims.d_v, dims.d_k)),
        _ptr(z, "z", (B, nv)), _ptr(norm_w, "norm_w", (params.norm_group,)),
        _ptr(y, "y", (B, nv)),
        _ptr(dbg_qkv, "dbg_qkv", (B, C), optional=True),
        _ptr(dbg_core, "dbg_core", (B, dims.n_v_heads, dims.d_v), optional=True),
        ws_ptr, ws_bytes, _stream(stream)))


# ---------------------------------------------------------------------------
# The layer around the recurrent branch, in 8 bits, and the verification of a
# speculative pair.  These take several element types; all tensors of a call
# must be on one GPU, and the call is made on that GPU's current stream (or
# the stream given, which must be that GPU's) whichever GPU is current.
try:
    _TYPES = {_torch.float32: 0, _torch.bfloat16: 1, _torch.float16: 2}
    _I8, _I32 = _torch.int8, _torch.int32
except NameError:
    _TYPES, _I8, _I32 = {}, None, None
_NO_TYPE = -1
_INT32_MAX = 2 ** 31 - 1


def _addr(t, name, dtype, shape, device):
    """Device address of a contiguous tensor of the given type and shape on
    GPU `device`."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == device
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _typed(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype)[6:]}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on GPU {t.get_device()}, expected GPU {device}")
    raise ValueError(f"{name} must be contiguous")


def _typed(t, name, types=None):
    import torch
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if types is not None and t.dtype not in types:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def _lead(t, name, ndim, types=None):
    """The GPU of the tensor that a call's sizes are read from."""
    if t.__class__ is not _torch.Tensor or not t.is_cuda or (types and t.dtype not in types):
        _typed(t, name, types)
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if t.numel() > _INT32_MAX and max(t.shape) > _INT32_MAX:    # the C arguments are int32
        raise ValueError(f"{name} has shape {tuple(t.shape)}, no dimension may pass {_INT32_MAX}")
    return t.get_device()


def _issue(fn, args, device, stream) -> None:
    """fn(*args, stream) with GPU `device` current."""
    if stream is None:
        raw = _torch._C._cuda_getCurrentRawStream(device)
    else:
        on = getattr(stream, "device_index", device)
        if on != device:
            raise ValueError(f"stream is on GPU {on}, the tensors are on GPU {device}")
        raw = _stream(stream)
    if device == _torch._C._cuda_getDevice():
        rc = fn(*args, raw)
    else:
        with _torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc != 0:
        raise GdnError(rc, last_error())


def add_rmsnorm_q8(x, residual, residual_out, norm_w, q, scale, eps=1e-6, stream=None) -> None:
    """gdn_add_rmsnorm_q8: x [rows][n] and residual (None: no residual) of
    float32, bfloat16 or float16, residual_out like residual (the same tensor:
    in place), norm_w [n] float32 -> codes q [rows][n] int8 and scale [rows]
    float32; q * scale is the normed row times norm_w."""
    dev = _lead(x, "x", 2, _TYPES)
    rows, n = shape = x.shape
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out is given without a residual")
        rtype, rp, ro = _NO_TYPE, None, None
    else:
        if getattr(residual, "dtype", None) not in _TYPES:
            _typed(residual, "residual", _TYPES)
        rtype = _TYPES[residual.dtype]
        rp = _addr(residual, "residual", residual.dtype, shape, dev)
        ro = _addr(residual_out, "residual_out", residual.dtype, shape, dev)
    _issue(lib.gdn_add_rmsnorm_q8,
           (rows, n, _TYPES[x.dtype], _addr(x, "x", x.dtype, shape, dev), rtype, rp, ro,
            _addr(norm_w, "norm_w", _F32, (n,), dev), eps, _addr(q, "q", _I8, shape, dev),
            _addr(scale, "scale", _F32, (rows,), dev)), dev, stream)


def quantize_q8(x, q, scale, stream=None) -> None:
    """gdn_quantize_q8: x [rows][n] of float32, bfloat16 or float16 -> codes
    q [rows][n] int8 and scale [rows] float32."""
    dev = _lead(x, "x", 2, _TYPES)
    rows, n = shape = x.shape
    _issue(lib.gdn_quantize_q8,
           (rows, n, _TYPES[x.dtype], _addr(x, "x", x.dtype, shape, dev),
            _addr(q, "q", _I8, shape, dev), _addr(scale, "scale", _F32, (rows,), dev)),
           dev, stream)


def linear_q8(a, a_scale, w, w_scale, outs, bias=None, stream=None) -> None:
    """gdn_linear_q8: a [M][K] int8 with a_scale [M], w [N][K] int8 with w_scale
    [N] (bias [N] float32 or None) -> outs: a tensor [M][N], or up to four
    [M][n_i] that take the N channels in order; float32, bfloat16 or float16,
    all of one type."""
    dev = _lead(a, "a", 2)
    M, K = a.shape
    if not isinstance(outs, (list, tuple)):
        outs = (outs,)
    if not 1 <= len(outs) <= LINEAR_MAX_OUTS:
        raise ValueError(f"outs must be 1 to {LINEAR_MAX_OUTS} tensors, got {len(outs)}")
    _lead(outs[0], "outs[0]", 2, _TYPES)
    dtype = outs[0].dtype
    addrs = []
    N = 0
    for i, o in enumerate(outs):
        name = _OUTS[i]
        if i:
            _lead(o, name, 2, _TYPES)
        n = o.shape[1]
        addrs.append((_addr(o, name, dtype, (M, n), dev), n))
        N += n
    groups = _GROUPS[len(outs)](*addrs)
    _issue(lib.gdn_linear_q8,
           (M, K, _addr(a, "a", _I8, (M, K), dev), _addr(a_scale, "a_scale", _F32, (M,), dev),
            _addr(w, "w", _I8, (N, K), dev), _addr(w_scale, "w_scale", _F32, (N,), dev),
            None if bias is None else _addr(bias, "bias", _F32, (N,), dev),
            _TYPES[dtype], groups, len(outs)), dev, stream)


def verify_workspace_bytes(B: int, V: int) -> int:
    if not (0 < B <= _INT32_MAX and 0 < V <= _INT32_MAX):     # the C arguments are int32
        return 0
    return int(lib.gdn_verify_workspace_bytes(B, V))


def verify(target, draft, draft_tokens, u_accept, u_sample, accepted, tokens, n_draft=None,
           workspace=None, stream=None) -> None:
    """gdn_verify: target [B][K+1][V] and draft [B][K][V] (None: greedy drafts)
    probabilities of one type (float32, bfloat16 or float16), draft_tokens
    [B][K] int32, n_draft [B] int32 or None, u_accept [B][K] and u_sample [B]
    float32 -> accepted [B] and tokens [B][K+1] int32.  workspace: a GPU tensor
    of at least verify_workspace_bytes(B, V) bytes (any dtype)."""
    dev = _lead(target, "target", 3, _TYPES)
    B, K1, V = target.shape
    K = K1 - 1
    ws_ptr, ws_bytes = _workspace(workspace)
    if ws_ptr is not None and workspace.get_device() != dev:
        raise ValueError(f"workspace is on GPU {workspace.get_device()}, expected GPU {dev}")
    _issue(lib.gdn_verify,
           (B, K, V, _TYPES[target.dtype],
            _addr(target, "target", target.dtype, (B, K1, V), dev),
            None if draft is None else _addr(draft, "draft", target.dtype, (B, K, V), dev),
            _addr(draft_tokens, "draft_tokens", _I32, (B, K), dev),
            None if n_draft is None else _addr(n_draft, "n_draft", _I32, (B,), dev),
            _addr(u_accept, "u_accept", _F32, (B, K), dev),
            _addr(u_sample, "u_sample", _F32, (B,), dev),
            _addr(accepted, "accepted", _I32, (B,), dev),
            _addr(tokens, "tokens", _I32, (B, K1), dev), ws_ptr, ws_bytes), dev, stream)


def pair_commit(accepted, state, state_next, conv_state=None, conv_state_next=None,
                stream=None) -> None:
    """gdn_pair_commit: accepted [B] int32; state and state_next [B][Hv][dv][dk]
    (or [layers][B][Hv][dv][dk]) and, optionally, conv_state and
    conv_state_next [B][K-1][C] (or [layers][B][K-1][C]): the tentative
    buffers of the sequences with accepted >= 1 replace the committed ones.  A
    pair holds one drafted position: accepted is that of a verify of one draft
    a sequence."""
    if getattr(state, "ndim", 5) == 4:
        dev, layers, sh = _lead(state, "state", 4), 1, tuple(state.shape)
        lead = sh[:1]
    else:
        dev = _lead(state, "state", 5)
        sh = tuple(state.shape)
        layers, lead = sh[0], sh[:2]
    B, Hv, dv, dk = sh[-4:]
    rs, ring = None, 0
    if conv_state is not None or conv_state_next is not None:
        _lead(conv_state, "conv_state", len(lead) + 2)
        rs = lead + tuple(conv_state.shape[len(lead):])
        ring = rs[-1] * rs[-2]
        if ring > _INT32_MAX:
            raise ValueError(f"conv_state holds {ring} floats a sequence, at most {_INT32_MAX}")
    d = Dims(Hv, Hv, dk, dv)           # the copy does not depend on the key heads
    _issue(lib.gdn_pair_commit,
           (ctypes.byref(d), layers, B, _addr(accepted, "accepted", _I32, (B,), dev),
            _addr(state, "state", _F32, sh, dev),
            _addr(state_next, "state_next", _F32, sh, dev), ring,
            None if rs is None else _addr(conv_state, "conv_state", _F32, rs, dev),
            None if rs is None else _addr(conv_state_next, "conv_state_next", _F32, rs, dev)),
           dev, stream)
