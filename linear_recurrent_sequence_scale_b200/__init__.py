"""Multi-scale retention on B200: thin Python binding over libretention.so.

Every function here only checks and marshals arguments: it takes torch CUDA
tensors (PyTorch supplies device memory and the current stream) and calls the
C ABI declared in include/retention.h.  All arithmetic runs in the library's
CUDA kernels; there is no CPU or PyTorch fallback.  If the library is missing
or cannot be loaded the calls raise.

Layouts (row-major, contiguous): q, k [B,H,N,dk]; v, o [B,H,N,dv];
state [B,H,dk,dv] float32; gammas [H] float32.  q, k, v share one dtype,
torch.float32 or torch.bfloat16.
"""
from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libretention.so")

RET_F32, RET_BF16 = 0, 1
RET_OK, RET_EINVAL, RET_EUNSUPPORTED, RET_ECUDA, RET_EWORKSPACE = 0, -1, -2, -3, -4
SCAN_CHUNK = 64                                    # RET_SCAN_CHUNK
SCAN_FORMS = {"logit": 0, "log": 1}                # ret_scan_form
NORMS = {None: -1, "layer": 0, "rms": 1}           # ret_norm_kind
ROW_NORMS = {"layer": 0, "rms": 1}

# name -> (restype, argtypes) of every symbol include/retention.h declares
_P, _I, _F, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_L = ctypes.c_longlong
SIGNATURES = {
    "ret_parallel": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "ret_chunkwise_workspace": (_S, [_I, _I, _I, _I, _I, _I, _I]),
    "ret_chunkwise": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _S, _P]),
    "ret_chunkwise_noalloc": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F,
                                   _P]),
    "ret_chunkwise_states": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _P, _S, _P]),
    "ret_chunkwise_output": (_I, [_P, _P, _P, _P, _I, _I, _P, _I, _I, _I, _I, _I, _I, _F, _P, _S,
                                  _P]),
    "ret_step": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "ret_parallel_gated": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "ret_chunkwise_gated": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F,
                                 _P, _S, _P]),
    "ret_chunkwise_output_gated": (_I, [_P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _I,
                                        _F, _P, _S, _P]),
    "ret_step_gated": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "ret_step_rotated": (_I, [_P, _P, _P, _P, _P, ctypes.c_longlong, _P, _P, _P, _I, _I, _I, _I,
                              _I, _F, _P]),
    "ret_state_combine": (_I, [_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P]),
    "ret_chunkwise_backward_workspace": (_S, [_I, _I, _I, _I, _I, _I, _I]),
    "ret_chunkwise_backward": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I,
                                    _I, _I, _I, _P, _S, _P]),
    "ret_rotate": (_I, [_P, _P, _P, ctypes.c_longlong, _I, _I, _I, _I, _I, _P]),
    "ret_scan_workspace": (_S, [_I, _I, _I, _I]),
    "ret_scan": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _S, _P]),
    "ret_scan_step": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "ret_scan_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P,
                               _S, _P]),
    "ret_norm_gate": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _L, _L, _I, _P]),
    "ret_norm_gate_backward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _L, _L, _L,
                                    _I, _P]),
    "ret_add_norm": (_I, [_P, _P, _P, _P, _P, _P, _L, _I, _I, _I, _F, _F, _F, _I, _P]),
    "ret_add_norm_backward_workspace": (_S, [_L, _I]),
    "ret_add_norm_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _L, _I, _I, _I, _F, _F,
                                   _F, _I, _P, _S, _P]),
    "ret_status_string": (ctypes.c_char_p, [_I]),
    "ret_last_cuda_error": (_I, []),
    "ret_version": (ctypes.c_char_p, []),
    "ret_device_error": (_I, []),
    "ret_selftest_bounded_wait": (_I, [_I, _P]),
    "ret_selftest_scan_wait": (_I, [_I, _P, _S, _P]),
}

_lib = None


class RetentionError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status}){detail}")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libretention.so (once) and bind every exported symbol."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m linear_recurrent_sequence_scale_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().ret_status_string(status).decode()


def device_error() -> int:
    """Read and clear the kernels' timed-out-wait flag (0 = none).  What was written
    since the last reading is not valid where this returns another code."""
    return int(load_library().ret_device_error())


def version() -> str:
    return load_library().ret_version().decode()


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return RET_F32
    if t.dtype == torch.bfloat16:
        return RET_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _check(t, name, dtype=None, shape=None, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _raise(fn, status):
    lib = load_library()
    detail = f", cudaError {lib.ret_last_cuda_error()}" if status == RET_ECUDA else ""
    raise RetentionError(fn, status, detail)


def _seq_args(q, k, v, gammas):
    torch = _torch()
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B,H,N,d]")
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    _check(q, "q", device=dev)
    _check(k, "k", dtype=q.dtype, shape=(B, H, N, dk), device=dev)
    _check(v, "v", dtype=q.dtype, shape=(B, H, N, dv), device=dev)
    _check(gammas, "gammas", dtype=torch.float32, shape=(H,), device=dev)
    return B, H, N, dk, dv, dev


def _gate(gate, like, shape, dev):
    if gate is not None:
        _check(gate, "gate", dtype=like.dtype, shape=shape, device=dev)
    return gate


def parallel(q, k, v, gammas, gn_eps=None, out=None, gate=None):
    """Parallel form O = (Q K^T (.) D) V (ret_parallel); returns o.  With a
    gate (same shape as o): o = swish(gate) * O (ret_parallel_gated)."""
    torch = _torch()
    B, H, N, dk, dv, dev = _seq_args(q, k, v, gammas)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=q.dtype, device=dev)
    _check(out, "out", dtype=q.dtype, shape=(B, H, N, dv), device=dev)
    gate = _gate(gate, q, (B, H, N, dv), dev)
    eps = -1.0 if gn_eps is None else float(gn_eps)
    lib = load_library()
    if gate is None:
        s = lib.ret_parallel(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), _ptr(out),
                             B, H, N, dk, dv, _dtype_code(q), eps, _stream(dev))
    else:
        s = lib.ret_parallel_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), _ptr(gate), _ptr(out),
                                   B, H, N, dk, dv, _dtype_code(q), eps, _stream(dev))
    if s != RET_OK:
        _raise("ret_parallel", s)
    return out


def chunkwise_workspace_bytes(B, H, N, dk, dv, chunk, dtype) -> int:
    torch = _torch()
    code = RET_BF16 if dtype == torch.bfloat16 else RET_F32
    return int(load_library().ret_chunkwise_workspace(B, H, N, dk, dv, chunk, code))


def chunkwise(q, k, v, gammas, chunk, state_in=None, state_out=None, return_state=False,
              gn_eps=None, out=None, workspace=None, gate=None):
    """Chunkwise-recurrent form (ret_chunkwise; ret_chunkwise_gated with a gate).

    Returns o, or (o, state) when return_state is True or state_out is given.
    state_out may be the same tensor as state_in (updated in place).
    workspace: optional uint8 CUDA tensor of at least chunkwise_workspace_bytes().
    gate: optional tensor shaped like o; o is then multiplied by swish(gate).
    """
    torch = _torch()
    B, H, N, dk, dv, dev = _seq_args(q, k, v, gammas)
    sshape = (B, H, dk, dv)
    if state_in is not None:
        _check(state_in, "state_in", dtype=torch.float32, shape=sshape, device=dev)
    if state_out is None and return_state:
        state_out = torch.empty(sshape, dtype=torch.float32, device=dev)
    if state_out is not None:
        _check(state_out, "state_out", dtype=torch.float32, shape=sshape, device=dev)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=q.dtype, device=dev)
    _check(out, "out", dtype=q.dtype, shape=(B, H, N, dv), device=dev)
    gate = _gate(gate, q, (B, H, N, dv), dev)
    workspace, ws_bytes = _workspace(workspace, B, H, N, dk, dv, chunk, q.dtype, dev)
    eps = -1.0 if gn_eps is None else float(gn_eps)
    lib = load_library()
    if gate is None:
        s = lib.ret_chunkwise(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), int(chunk),
                              _ptr(state_in), _ptr(state_out), _ptr(out),
                              B, H, N, dk, dv, _dtype_code(q), eps,
                              _ptr(workspace), ws_bytes, _stream(dev))
    else:
        s = lib.ret_chunkwise_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), int(chunk),
                                    _ptr(state_in), _ptr(state_out), _ptr(gate), _ptr(out),
                                    B, H, N, dk, dv, _dtype_code(q), eps,
                                    _ptr(workspace), ws_bytes, _stream(dev))
    if s != RET_OK:
        _raise("ret_chunkwise", s)
    if state_out is not None:
        return out, state_out
    return out


def _workspace(workspace, B, H, N, dk, dv, chunk, dtype, dev):
    torch = _torch()
    need = chunkwise_workspace_bytes(B, H, N, dk, dv, chunk, dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0
    if workspace is not None:
        _check(workspace, "workspace", device=dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    return workspace, ws_bytes


def chunkwise_states(k, v, gammas, chunk, workspace, state_in=None, state_out=None):
    """First phase of the chunkwise form (ret_chunkwise_states): the state
    entering every chunk into `workspace` (uint8 CUDA tensor of at least
    chunkwise_workspace_bytes()), and the final state into state_out if given."""
    torch = _torch()
    B, H, N, dk, dv, dev = _seq_args(k, k, v, gammas)
    sshape = (B, H, dk, dv)
    if state_in is not None:
        _check(state_in, "state_in", dtype=torch.float32, shape=sshape, device=dev)
    if state_out is not None:
        _check(state_out, "state_out", dtype=torch.float32, shape=sshape, device=dev)
    workspace, ws_bytes = _workspace(workspace, B, H, N, dk, dv, chunk, k.dtype, dev)
    s = load_library().ret_chunkwise_states(_ptr(k), _ptr(v), _ptr(gammas), int(chunk),
                                            _ptr(state_in), _ptr(state_out), B, H, N, dk, dv,
                                            _dtype_code(k), _ptr(workspace), ws_bytes,
                                            _stream(dev))
    if s != RET_OK:
        _raise("ret_chunkwise_states", s)
    return workspace


def chunkwise_output(q, k, v, gammas, chunk, workspace, has_state_in=False, gn_eps=None,
                     out=None, gate=None):
    """Second phase of the chunkwise form (ret_chunkwise_output, or
    ret_chunkwise_output_gated with a gate): o from the workspace that
    chunkwise_states wrote for the same sizes; returns o."""
    torch = _torch()
    B, H, N, dk, dv, dev = _seq_args(q, k, v, gammas)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=q.dtype, device=dev)
    _check(out, "out", dtype=q.dtype, shape=(B, H, N, dv), device=dev)
    gate = _gate(gate, q, (B, H, N, dv), dev)
    workspace, ws_bytes = _workspace(workspace, B, H, N, dk, dv, chunk, q.dtype, dev)
    eps = -1.0 if gn_eps is None else float(gn_eps)
    lib = load_library()
    if gate is None:
        s = lib.ret_chunkwise_output(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), int(chunk),
                                     1 if has_state_in else 0, _ptr(out), B, H, N, dk, dv,
                                     _dtype_code(q), eps, _ptr(workspace), ws_bytes,
                                     _stream(dev))
    else:
        s = lib.ret_chunkwise_output_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), int(chunk),
                                           1 if has_state_in else 0, _ptr(gate), _ptr(out),
                                           B, H, N, dk, dv, _dtype_code(q), eps,
                                           _ptr(workspace), ws_bytes, _stream(dev))
    if s != RET_OK:
        _raise("ret_chunkwise_output", s)
    return out


def chunkwise_backward(q, k, v, gammas, chunk, d_o, state_in=None, d_state_out=None,
                       workspace=None):
    """Gradients of ret_chunkwise (no GroupNorm, no gate): returns
    (dq, dk, dv, d_state_in) for the output gradient d_o [B,H,N,dv] and the
    optional final-state gradient d_state_out (ret_chunkwise_backward)."""
    torch = _torch()
    B, H, N, dk, dv, dev = _seq_args(q, k, v, gammas)
    _check(d_o, "d_o", dtype=q.dtype, shape=(B, H, N, dv), device=dev)
    sshape = (B, H, dk, dv)
    for t, name in ((state_in, "state_in"), (d_state_out, "d_state_out")):
        if t is not None:
            _check(t, name, dtype=torch.float32, shape=sshape, device=dev)
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ds = torch.empty(sshape, dtype=torch.float32, device=dev)
    lib = load_library()
    need = int(lib.ret_chunkwise_backward_workspace(B, H, N, dk, dv, int(chunk), _dtype_code(q)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    s = lib.ret_chunkwise_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), int(chunk),
                                   _ptr(state_in), _ptr(d_o), _ptr(d_state_out), _ptr(dq),
                                   _ptr(dk_), _ptr(dv_), _ptr(ds), B, H, N, dk, dv,
                                   _dtype_code(q), _ptr(workspace), wsb, _stream(dev))
    if s != RET_OK:
        _raise("ret_chunkwise_backward", s)
    return dq, dk_, dv_, ds


def state_combine(locals_, spans, r, gammas, state0=None, out=None):
    """State entering span r of a sequence split into spans (ret_state_combine).
    locals_: [R,B,H,dk,dv] float32 end states of the spans computed from a zero
    state; spans: R span lengths (host ints); state0: state entering span 0 or
    None.  r = R gives the end state of the whole sequence."""
    torch = _torch()
    R, B, H, dk, dv = locals_.shape
    dev = locals_.device
    _check(locals_, "locals", dtype=torch.float32, device=dev)
    if not 0 <= r <= R or len(spans) != R:
        raise ValueError("need 0 <= r <= number of spans and one length per span")
    _check(gammas, "gammas", dtype=torch.float32, shape=(H,), device=dev)
    if state0 is not None:
        _check(state0, "state0", dtype=torch.float32, shape=(B, H, dk, dv), device=dev)
    if out is None:
        out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    _check(out, "out", dtype=torch.float32, shape=(B, H, dk, dv), device=dev)
    sp = (ctypes.c_int * max(R, 1))(*[int(n) for n in spans])
    s = load_library().ret_state_combine(_ptr(locals_), sp, int(r), _ptr(gammas), _ptr(state0),
                                         _ptr(out), B, H, dk, dv, _stream(dev))
    if s != RET_OK:
        _raise("ret_state_combine", s)
    return out


def rotate(x, theta, pos0=0, out=None):
    """xPos-style rotation of q or k rows (ret_rotate): channel pair c of the
    row at position pos0 + j turns by (pos0 + j) * theta[c].
    x [B,H,N,d] or [B,H,d] (one position, e.g. a decode step); theta [d/2]
    float32; out may be x itself (in place).  Returns out."""
    torch = _torch()
    if x.dim() not in (3, 4):
        raise ValueError("x must be [B,H,N,d] or [B,H,d]")
    B, H = x.shape[0], x.shape[1]
    N = x.shape[2] if x.dim() == 4 else 1
    d = x.shape[-1]
    dev = x.device
    _check(x, "x", device=dev)
    code = _dtype_code(x)
    _check(theta, "theta", dtype=torch.float32, shape=(d // 2,), device=dev)
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", dtype=x.dtype, shape=tuple(x.shape), device=dev)
    s = load_library().ret_rotate(_ptr(x), _ptr(out), _ptr(theta), int(pos0), B, H, N, d, code,
                                  _stream(dev))
    if s != RET_OK:
        _raise("ret_rotate", s)
    return out


def step(q, k, v, gammas, state, gn_eps=None, out=None, gate=None, theta=None, pos=0):
    """One recurrent decode step (ret_step; ret_step_gated with a gate [B,H,dv];
    ret_step_rotated with theta [dk/2], q and k then rotated by pos * theta as
    they are read): state is updated in place; returns o.
    q, k [B,H,dk]; v [B,H,dv]; state [B,H,dk,dv] float32."""
    torch = _torch()
    if q.dim() != 3:
        raise ValueError("q, k, v must be [B,H,d] for a decode step")
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    _check(q, "q", device=dev)
    _check(k, "k", dtype=q.dtype, shape=(B, H, dk), device=dev)
    _check(v, "v", dtype=q.dtype, shape=(B, H, dv), device=dev)
    _check(gammas, "gammas", dtype=torch.float32, shape=(H,), device=dev)
    _check(state, "state", dtype=torch.float32, shape=(B, H, dk, dv), device=dev)
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=dev)
    _check(out, "out", dtype=q.dtype, shape=(B, H, dv), device=dev)
    gate = _gate(gate, q, (B, H, dv), dev)
    eps = -1.0 if gn_eps is None else float(gn_eps)
    lib = load_library()
    if theta is not None:
        _check(theta, "theta", dtype=torch.float32, shape=(dk // 2,), device=dev)
        s = lib.ret_step_rotated(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), _ptr(theta), int(pos),
                                 _ptr(state), _ptr(gate), _ptr(out), B, H, dk, dv,
                                 _dtype_code(q), eps, _stream(dev))
    elif gate is None:
        s = lib.ret_step(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), _ptr(state), _ptr(out),
                         B, H, dk, dv, _dtype_code(q), eps, _stream(dev))
    else:
        s = lib.ret_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gammas), _ptr(state), _ptr(gate),
                               _ptr(out), B, H, dk, dv, _dtype_code(q), eps, _stream(dev))
    if s != RET_OK:
        _raise("ret_step", s)
    return out


def _code(names, name, what):
    try:
        return names[name]
    except (KeyError, TypeError):
        raise ValueError(f"unknown {what} {name!r}; use one of {list(names)}") from None


# The calls below serve single tokens as well, where the host's time counts:
# checks pass on one comparison each and explain themselves only on failure.

def _same(t, name, dtype, shape, device):
    if t.dtype is dtype and t.device == device and t.shape == shape and t.is_cuda:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _dense(t, name, dtype, shape, device):
    _same(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _like(x):
    """A new dense tensor of x's shape and type."""
    return _torch().empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _pitches(x, names, *operands):
    """Pitches (elements) of x and the other [..., D] operands (None: absent), in
    order: a host array for the library with one entry per leading axis of
    each, or None when all are dense.  Channels must be adjacent; the library
    checks the rest."""
    shape, dtype, device = x.shape, x.dtype, x.device
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dense = x.is_contiguous()
    for t, name in zip(operands, names):
        if t is not None:
            _same(t, name, dtype, shape, device)
            dense = dense and t.is_contiguous()
    if dense:
        return None
    lead = len(shape) - 1
    got = []
    for t, name in zip((x,) + operands, ("x",) + names):
        if t is None:
            got += [0] * lead
            continue
        st = t.stride()
        if st[-1] != 1 and shape[-1] > 1:
            raise ValueError(f"{name}: channels must be adjacent, got strides {st}")
        got += st[:-1]
    return (_L * len(got))(*got)


def _call(name, device, *args):
    """Runs a library call on the current stream of `device`, with that device
    current; raises on a status other than RET_OK."""
    torch = _torch()
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(name, device, *args)
    # the raw handle: a Stream object costs as much as the library call itself
    s = getattr(_lib or load_library(), name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if s != RET_OK:
        _raise(name, s)


def _addr(t):
    return None if t is None else t.data_ptr()


def _own_workspace(workspace, need, device):
    torch = _torch()
    if workspace is None:
        if need == 0:
            return None, 0
        return torch.empty(need, dtype=torch.uint8, device=device), need
    _check(workspace, "workspace", device=device)
    return workspace, workspace.numel() * workspace.element_size()


def _state(t, name, shape, device):
    if t is not None:
        _dense(t, name, _torch().float32, shape, device)


def scan_workspace_bytes(B, N, D, dtype) -> int:
    code = RET_BF16 if dtype == _torch().bfloat16 else RET_F32
    return int(load_library().ret_scan_workspace(B, N, D, code))


def scan(x, f, form="logit", gate=None, state_in=None, state_out=None, return_state=False,
         chunk_states=None, return_chunk_states=False, out=None, workspace=None):
    """Gated linear recurrence over [B,N,D] (ret_scan): h_t = a_t h_(t-1) + u_t
    per channel, with a = sigmoid(f), u = (1 - a) x (form "logit") or
    a = exp(f), u = x (form "log"); returns y = h, or swish(gate) * h.

    x, f, gate and out: [B,N,D] of one dtype (gate may be None), dense, slices
    of a projection's output, a span of a longer sequence, or a time-major
    tensor seen as [B,N,D]; channels must be adjacent.
    state_in, state_out: [B,D] float32 before the first and after the last
    token; state_out may be state_in.  chunk_states:
    [B, ceil(N / SCAN_CHUNK), D] float32, kept for scan_backward.
    Long sequences are dealt over blocks that wait for one another, each wait
    with a limit: device_error() tells whether one ran out.
    Returns y, or the tuple (y[, state][, chunk_states]) with what
    return_state / state_out and return_chunk_states / chunk_states ask for.
    """
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [B,N,D]")
    dev = x.device
    code, kind = _dtype_code(x), _code(SCAN_FORMS, form, "form")
    B, N, D = x.shape
    _state(state_in, "state_in", (B, D), dev)
    if state_out is None and return_state:
        state_out = x.new_empty((B, D), dtype=torch.float32)
    else:
        _state(state_out, "state_out", (B, D), dev)
    if chunk_states is None and return_chunk_states:
        chunk_states = x.new_empty((B, -(-N // SCAN_CHUNK), D), dtype=torch.float32)
    else:
        _state(chunk_states, "chunk_states", (B, -(-N // SCAN_CHUNK), D), dev)
    out = _like(x) if out is None else out
    pitches = _pitches(x, ("f", "gate", "out"), f, gate, out)
    workspace, wsb = _own_workspace(workspace, load_library().ret_scan_workspace(B, N, D, code),
                                    dev)
    _call("ret_scan", dev, _addr(x), _addr(f), _addr(gate), _addr(state_in), _addr(state_out),
          _addr(chunk_states), _addr(out), pitches, B, N, D, kind, code, _addr(workspace), wsb)
    got = tuple(t for t in (state_out, chunk_states) if t is not None)
    return (out,) + got if got else out


def scan_step(x, f, state, form="logit", gate=None, out=None, state_out=None):
    """One token of the gated linear recurrence (ret_scan_step): x, f, gate
    [B,D]; state [B,D] float32 is updated in place, or left alone with the new
    state written to state_out.  Returns y."""
    if x.dim() != 2:
        raise ValueError("x must be [B,D] for a single token")
    shape, dev = x.shape, x.device
    code, kind = _dtype_code(x), _code(SCAN_FORMS, form, "form")
    B, D = shape
    _state(state, "state", shape, dev)
    _state(state_out, "state_out", shape, dev)
    out = _like(x) if out is None else out
    pitches = _pitches(x, ("f", "gate", "out"), f, gate, out)
    _call("ret_scan_step", dev, _addr(x), _addr(f), _addr(gate), _addr(state),
          _addr(state if state_out is None else state_out), _addr(out), pitches, B, D, kind, code)
    return out


def scan_backward(x, f, chunk_states, d_y, form="logit", gate=None, d_state_out=None,
                  grad_x=None, grad_f=None, grad_gate=None, workspace=None):
    """Backward of scan (ret_scan_backward): returns (grad_x, grad_f, grad_gate
    or None, d_state_in) for the gradient d_y of y and, optionally, d_state_out
    of the final state.  chunk_states comes from the forward call with the same
    x, f and state_in.  grad_x, grad_f and grad_gate may be given as slices of
    one buffer."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [B,N,D]")
    dev = x.device
    code, kind = _dtype_code(x), _code(SCAN_FORMS, form, "form")
    B, N, D = x.shape
    _state(chunk_states, "chunk_states", (B, -(-N // SCAN_CHUNK), D), dev)
    _state(d_state_out, "d_state_out", (B, D), dev)
    if gate is None and grad_gate is not None:
        raise ValueError("grad_gate given without a gate")
    grad_x = _like(x) if grad_x is None else grad_x
    grad_f = _like(x) if grad_f is None else grad_f
    if gate is not None and grad_gate is None:
        grad_gate = _like(x)
    pitches = _pitches(x, ("f", "gate", "d_y", "grad_x", "grad_f", "grad_gate"), f, gate, d_y,
                       grad_x, grad_f, grad_gate)
    d_state_in = x.new_empty((B, D), dtype=torch.float32)
    workspace, wsb = _own_workspace(workspace, load_library().ret_scan_workspace(B, N, D, code),
                                    dev)
    _call("ret_scan_backward", dev, _addr(x), _addr(f), _addr(gate), _addr(chunk_states),
          _addr(d_y), _addr(d_state_out), _addr(grad_x), _addr(grad_f), _addr(grad_gate),
          _addr(d_state_in), pitches, B, N, D, kind, code, _addr(workspace), wsb)
    return grad_x, grad_f, grad_gate, d_state_in


def _head_args(y, token_major):
    if y.dim() != 4:
        raise ValueError("y must be [B,H,N,dv]")
    if not y.is_cuda:
        raise ValueError("y must be a CUDA tensor")
    if not y.is_contiguous():
        raise ValueError("y must be contiguous")
    B, H, N, dv = y.shape
    return B, H, N, dv, (B, N, H, dv) if token_major else (B, H, N, dv)


def _head_pitch(t, name, dt, shape, dev, token_major):
    """Elements between tokens of a [B,N,H,dv] tensor whose heads are adjacent and
    whose tokens are evenly spaced (0 for the head-major layout, which must be
    dense)."""
    if not token_major:
        _dense(t, name, dt, shape, dev)
        return 0
    _same(t, name, dt, shape, dev)
    if t.is_contiguous():
        return 0
    B, N, H, dv = shape
    sb, sn, sh, sd = t.stride()
    ld = sn if N > 1 else (sb if B > 1 else H * dv)
    if sd != 1 or (H > 1 and sh != dv) or (B > 1 and N > 1 and sb != N * sn):
        raise ValueError(f"{name}: heads must be adjacent and tokens evenly spaced, "
                         f"got strides {t.stride()}")
    return ld


def norm_gate(y, gate=None, norm="layer", eps=1e-5, token_major=False, out=None):
    """Per-head norm and output gate of retention outputs (ret_norm_gate):
    o = swish(gate) * z, z each row of y [B,H,N,dv] normalised ("layer": the
    GroupNorm of gn_eps; "rms").  With token_major, gate and o are [B,N,H,dv]
    (dense, or the gate a slice of a projection's output viewed as such);
    otherwise [B,H,N,dv].  gate None: o = z.  dv: a multiple of 8 up to 1024;
    B H up to 65535.  Returns o."""
    B, H, N, dv, shape = _head_args(y, token_major)
    dev, dt, code = y.device, y.dtype, _dtype_code(y)
    kind = _code(ROW_NORMS, norm, "norm")
    ldg = 0 if gate is None else _head_pitch(gate, "gate", dt, shape, dev, token_major)
    if out is None:
        out, ldo = y.new_empty(shape) if token_major else _torch().empty_like(y), 0
    else:
        ldo = _head_pitch(out, "out", dt, shape, dev, token_major)
    _call("ret_norm_gate", dev, _addr(y), _addr(gate), _addr(out), B, H, N, dv, kind, float(eps),
          int(token_major), ldg, ldo, code)
    return out


def norm_gate_backward(y, gate, d_o, norm="layer", eps=1e-5, token_major=False, grad_y=None,
                       grad_gate=None):
    """Backward of norm_gate (ret_norm_gate_backward): returns (grad_y,
    grad_gate or None).  d_o and grad_gate are laid out like o and gate."""
    B, H, N, dv, shape = _head_args(y, token_major)
    dev, dt, code = y.device, y.dtype, _dtype_code(y)
    kind = _code(ROW_NORMS, norm, "norm")
    ldg = 0 if gate is None else _head_pitch(gate, "gate", dt, shape, dev, token_major)
    lddo = _head_pitch(d_o, "d_o", dt, shape, dev, token_major)
    if grad_y is None:
        grad_y = _torch().empty_like(y)
    else:
        _dense(grad_y, "grad_y", dt, y.shape, dev)
    ldgg = 0
    if gate is None:
        if grad_gate is not None:
            raise ValueError("grad_gate given without a gate")
    elif grad_gate is None:
        grad_gate = y.new_empty(shape)
    else:
        ldgg = _head_pitch(grad_gate, "grad_gate", dt, shape, dev, token_major)
    _call("ret_norm_gate_backward", dev, _addr(y), _addr(gate), _addr(d_o), _addr(grad_y),
          _addr(grad_gate), B, H, N, dv, kind, float(eps), int(token_major), ldg, lddo, ldgg, code)
    return grad_y, grad_gate


def _weight(w, name, d, dev):
    if w is not None:
        _dense(w, name, _torch().float32, (d,), dev)


def add_norm(x, residual, w=None, w_post=None, post_norm=None, norm="rms", alpha=1.0, beta=1.0,
             eps=1e-5, res_out=None, out=None):
    """Residual sum with the norms around it (ret_add_norm), over the last
    axis of x [..., d]: u = w_post * N_post(x), r = alpha * residual + beta * u,
    y = w * N(r); returns (r, y).  norm and post_norm: "rms" or "layer"
    (post_norm None: no norm); w, w_post: [d] float32 or None; residual may be
    None.  res_out may be residual (in place)."""
    torch = _torch()
    dev, dt, code, shape = x.device, x.dtype, _dtype_code(x), x.shape
    if x.dim() < 1:
        raise ValueError("x must have a feature axis")
    _dense(x, "x", dt, shape, dev)
    d = shape[-1]
    if residual is not None:
        _dense(residual, "residual", dt, shape, dev)
    _weight(w, "w", d, dev)
    _weight(w_post, "w_post", d, dev)
    if res_out is None:
        res_out = torch.empty_like(x)
    else:
        _dense(res_out, "res_out", dt, shape, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _dense(out, "out", dt, shape, dev)
    _call("ret_add_norm", dev, _addr(x), _addr(residual), _addr(w_post), _addr(w), _addr(res_out),
          _addr(out), x.numel() // d if d else 0, d, _code(NORMS, post_norm, "post_norm"),
          _code(ROW_NORMS, norm, "norm"), float(alpha), float(beta), float(eps), code)
    return res_out, out


def add_norm_backward(x, res_out, w, d_y, d_res_out=None, w_post=None, post_norm=None, norm="rms",
                      alpha=1.0, beta=1.0, eps=1e-5, grad_x=None, grad_residual=None,
                      workspace=None):
    """Backward of add_norm (ret_add_norm_backward) from the stored sum res_out:
    returns (grad_x, grad_residual, grad_w or None, grad_w_post or None); a
    weight that is None has no gradient.  x may be None where neither post_norm
    nor w_post is given."""
    torch = _torch()
    dev, dt, code, shape = res_out.device, res_out.dtype, _dtype_code(res_out), res_out.shape
    if res_out.dim() < 1:
        raise ValueError("res_out must have a feature axis")
    _dense(res_out, "res_out", dt, shape, dev)
    d = shape[-1]
    for t, name in ((x, "x"), (d_y, "d_y"), (d_res_out, "d_res_out"), (grad_x, "grad_x"),
                    (grad_residual, "grad_residual")):
        if t is not None:
            _dense(t, name, dt, shape, dev)
    _weight(w, "w", d, dev)
    _weight(w_post, "w_post", d, dev)
    grad_x = torch.empty_like(res_out) if grad_x is None else grad_x
    grad_residual = torch.empty_like(res_out) if grad_residual is None else grad_residual
    grad_w = None if w is None else torch.empty_like(w)
    grad_w_post = None if w_post is None else torch.empty_like(w_post)
    rows = res_out.numel() // d if d else 0
    need = 0
    if grad_w is not None or grad_w_post is not None:
        need = load_library().ret_add_norm_backward_workspace(rows, d)
    workspace, wsb = _own_workspace(workspace, need, dev)
    _call("ret_add_norm_backward", dev, _addr(x), _addr(res_out), _addr(w_post), _addr(w),
          _addr(d_y), _addr(d_res_out), _addr(grad_x), _addr(grad_residual), _addr(grad_w),
          _addr(grad_w_post), rows, d, _code(NORMS, post_norm, "post_norm"),
          _code(ROW_NORMS, norm, "norm"), float(alpha), float(beta), float(eps), code,
          _addr(workspace), wsb)
    return grad_x, grad_residual, grad_w, grad_w_post
