"""ctypes binding of the C ABI in ``include/mhla.h`` — argument marshalling only.

Every function here has the name of the C entry point it calls, takes torch
CUDA tensors, passes their device pointers, sizes and the current CUDA stream
to the library, and raises :class:`MhlaError` on a non-OK status.  All work
runs in the library's CUDA kernels; there is no fallback: if the library is
missing or CUDA is unavailable the call fails.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

from .build import LIB_PATH

MHLA_OK, MHLA_ERR_INVALID_ARG, MHLA_ERR_UNSUPPORTED, MHLA_ERR_CUDA, MHLA_ERR_TIMEOUT = range(5)
MHLA_F32, MHLA_BF16 = 0, 1
PATH_NAMES = {0: "none", 1: "simt", 2: "tcgen05", 3: "tcgen05_stream"}

_lib = None

_vp, _sz, _i, _f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float

_SIGNATURES = {
    "mhla_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "mhla_forward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "mhla_forward_causal": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "linattn_decode_step": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp]),
    "linattn_decode_steps": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _vp]),
    "mhla_causal_stream": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _vp]),
    "mhla_forward_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _sz, _vp]),
    "mhla_forward_ex_path": (_i, [_i, _i, _i, _i, _i, _i, _i, _i, _vp]),
    "mhla_forward_grid": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "mhla_forward_grid_path": (_i, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "mhla_locality_mixing": (_i, [_vp, _i, _i]),
    "rala_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "rala_forward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "mhla_forward_path": (_i, [_i, _i, _i, _i, _i, _i, _i]),
    "rala_forward_path": (_i, [_i, _i, _i, _i, _i, _i]),
    "mhla_query_status": (_i, [_vp, _vp]),
    "mhla_status_string": (ctypes.c_char_p, [_i]),
    "mhla_launch_count": (ctypes.c_ulonglong, []),
    "mhla_forward_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp]),
    "mhla_debug_set_wait_limit_ns": (None, [ctypes.c_ulonglong]),
    "mhla_backward_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "mhla_backward_path": (_i, [_i, _i, _i, _i, _i, _i]),
    "retention_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "retention_forward": (_i, [_vp] * 9 + [_i] * 4 + [_vp, _vp, _vp, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "retention_backward": (_i, [_vp] * 15 + [_i] * 4 + [_vp, _i, _vp, _vp, _sz, _vp]),
    "retention_step": (_i, [_vp] * 9 + [_i, _vp, _vp, _i, _i, _i, _i, _vp, _vp]),
    "retention_copy_states": (_i, [_vp, _i, _i, _i, _vp, _vp, _i, _vp]),
    "mhla_backward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
}

EXPORTED = tuple(_SIGNATURES)


class MhlaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def load(path: str = LIB_PATH):
    """Loads the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"MHLA CUDA library not built at {path}; call __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().mhla_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != MHLA_OK:
        raise MhlaError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MHLA_F32
    if t.dtype == torch.bfloat16:
        return MHLA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _stream(stream, device=None):
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _expect(t, name, shape, dtype):
    """Raises ValueError unless tensor ``t`` has this shape and dtype (checked before any device use)."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _same_device(q, *ts):
    """All tensors contiguous on q's CUDA device; returns that device."""
    _need_cuda(q, *ts)
    for t in ts:
        if t is not None and t.device != q.device:
            raise ValueError(f"tensor on {t.device}, expected {q.device} (the device of q)")
    return q.device


def _mhla_args(q, k, v, mixing, y, den_out, block, mixing_required=True):
    if q.dim() != 4:
        raise ValueError(f"q: expected [B, H, N, d], got shape {tuple(q.shape)}")
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("y", y)):
        _expect(t, name, q.shape, q.dtype)
    _expect(den_out, "den_out", (B, H, N), torch.float32)
    if mixing is None:
        if mixing_required:
            raise ValueError("mixing: required")
    elif block > 0 and N % block == 0:
        _expect(mixing, "mixing", (H, N // block, N // block), torch.float32)
    return B, H, N, d


def mhla_workspace_bytes(B: int, H: int, N: int, d: int, block_size: int, causal: int = 0) -> int:
    return int(load().mhla_workspace_bytes(B, H, N, d, block_size, causal))


def mhla_backward_workspace_bytes(B: int, H: int, N: int, d: int, block_size: int) -> int:
    return int(load().mhla_backward_workspace_bytes(B, H, N, d, block_size))


def rala_workspace_bytes(B: int, H: int, N: int, d: int, cx: int) -> int:
    return int(load().rala_workspace_bytes(B, H, N, d, cx))


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """Zero-filled uint8 device buffer of ``nbytes`` (the library needs it zeroed before first use)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def mhla_forward_path(B, H, N, d, block_size, causal, dtype) -> str:
    dt = MHLA_BF16 if dtype == torch.bfloat16 else MHLA_F32
    return PATH_NAMES[int(load().mhla_forward_path(B, H, N, d, block_size, causal, dt))]


def mhla_forward_grid_path(B, H, grid_h, grid_w, tile_h, tile_w, d, dtype) -> str:
    dt = MHLA_BF16 if dtype == torch.bfloat16 else MHLA_F32
    return PATH_NAMES[int(load().mhla_forward_grid_path(B, H, grid_h, grid_w, tile_h, tile_w, d, dt))]


def locality_mixing(blocks_h, blocks_w) -> torch.Tensor:
    """The locality-based initial mixing matrix [M, M] (fp32, CPU) for blocks on a grid."""
    M = blocks_h * blocks_w
    m = torch.empty(max(M, 0), max(M, 0), dtype=torch.float32)
    _check("mhla_locality_mixing", load().mhla_locality_mixing(_ptr(m), blocks_h, blocks_w))
    return m


def rala_forward_path(B, H, N, d, cx, dtype) -> str:
    dt = MHLA_BF16 if dtype == torch.bfloat16 else MHLA_F32
    return PATH_NAMES[int(load().rala_forward_path(B, H, N, d, cx, dt))]


# Every wrapper checks shapes and dtypes against q, then that every tensor is a
# contiguous CUDA tensor on q's device, and runs the call with q's device
# current (the library takes its device from the current device).

def mhla_forward(q, k, v, mixing, y, block_size, *, causal=0, eps=1e-6, den_out=None,
                 workspace=None, stream=None):
    """Non-causal (or, with causal=1, causal) MHLA forward; q/k/v/y [B, H, N, d], mixing [H, M, M] fp32."""
    B, H, N, d = _mhla_args(q, k, v, mixing, y, den_out, block_size, mixing_required=not causal)
    dev = _same_device(q, k, v, mixing, y, den_out, workspace)
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(mhla_workspace_bytes(B, H, N, d, block_size, causal), dev)
        st = load().mhla_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(mixing), _ptr(y), _ptr(den_out),
                                 B, H, N, d, block_size, causal, _dtype(q), eps, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream, dev))
    _check("mhla_forward", st)
    return y


FEATURES = {"elu1": 0, "relu": 1, "exp": 2}


class MhlaOptions(ctypes.Structure):
    """The C struct mhla_options: feature map, normaliser on / off, causal decay."""
    _fields_ = [("feature", ctypes.c_int), ("normalise", ctypes.c_int), ("gamma", ctypes.c_float)]


def _options(feature, normalise, gamma):
    if feature not in FEATURES:
        raise ValueError(f"feature: one of {sorted(FEATURES)}, got {feature!r}")
    return MhlaOptions(FEATURES[feature], 1 if normalise else 0, float(gamma))


def mhla_forward_ex_path(B, H, N, d, block_size, causal, with_mixing, dtype, *, feature="elu1", normalise=True,
                         gamma=1.0) -> str:
    dt = MHLA_BF16 if dtype == torch.bfloat16 else MHLA_F32
    opt = _options(feature, normalise, gamma)
    return PATH_NAMES[int(load().mhla_forward_ex_path(B, H, N, d, block_size, causal, int(bool(with_mixing)), dt,
                                                      ctypes.byref(opt)))]


def mhla_forward_ex(q, k, v, mixing, y, block_size, *, causal=0, feature="elu1", normalise=True, gamma=1.0,
                    eps=1e-6, den_out=None, workspace=None, stream=None):
    """mhla_forward with variants: feature map ("elu1", "relu", "exp"), normalise (False: the
    numerator alone), gamma (decay; plain causal linear attention, mixing None, only)."""
    opt = _options(feature, normalise, gamma)
    B, H, N, d = _mhla_args(q, k, v, mixing, y, den_out, block_size, mixing_required=not causal)
    dev = _same_device(q, k, v, mixing, y, den_out, workspace)
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(mhla_workspace_bytes(B, H, N, d, block_size, causal), dev)
        st = load().mhla_forward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(mixing), _ptr(y), _ptr(den_out),
                                    B, H, N, d, block_size, causal, _dtype(q), eps, ctypes.byref(opt),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream, dev))
    _check("mhla_forward_ex", st)
    return y


def mhla_forward_grid(q, k, v, mixing, y, grid_hw, tile_hw, *, eps=1e-6, den_out=None, workspace=None,
                      stream=None):
    """Non-causal MHLA with 2-D blocks: the N tokens are a grid_hw = (grid_h, grid_w) grid in
    row-major order, the blocks its tile_hw = (tile_h, tile_w) tiles; mixing [H, M, M] fp32."""
    (gh, gw), (th, tw) = grid_hw, tile_hw
    if q.dim() != 4:
        raise ValueError(f"q: expected [B, H, N, d], got shape {tuple(q.shape)}")
    if q.shape[2] != gh * gw:
        raise ValueError(f"q: N = {q.shape[2]}, expected grid_h * grid_w = {gh * gw}")
    if th <= 0 or tw <= 0 or gh % th or gw % tw:
        raise ValueError(f"tiles {tile_hw} do not cover the grid {grid_hw}")
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("y", y)):
        _expect(t, name, q.shape, q.dtype)
    _expect(den_out, "den_out", (B, H, N), torch.float32)
    M = (gh // th) * (gw // tw)
    _expect(mixing, "mixing", (H, M, M), torch.float32)
    dev = _same_device(q, k, v, mixing, y, den_out, workspace)
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(mhla_workspace_bytes(B, H, N, d, th * tw, 0), dev)
        st = load().mhla_forward_grid(_ptr(q), _ptr(k), _ptr(v), _ptr(mixing), _ptr(y), _ptr(den_out),
                                      B, H, gh, gw, th, tw, d, _dtype(q), eps, _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream, dev))
    _check("mhla_forward_grid", st)
    return y


def mhla_causal_stream(q, k, v, mixing, S, z, out, t0, block, *, eps=1e-6, den_out=None, stream=None):
    """Causal MHLA inference for tokens t0 .. t0 + T - 1: q/k/v/out [T, B, H, d], mixing [H, M, M]
    fp32, S [B, H, M, d, d] and z [B, H, M, d] fp32 block summaries (updated)."""
    if q.dim() != 4 or S.dim() != 5:
        raise ValueError("q: expected [T, B, H, d]; S: expected [B, H, M, d, d]")
    T, B, H, d = q.shape
    M = S.shape[2]
    for name, t in (("k", k), ("v", v), ("out", out)):
        _expect(t, name, q.shape, q.dtype)
    _expect(mixing, "mixing", (H, M, M), torch.float32)
    _expect(S, "S", (B, H, M, d, d), torch.float32)
    _expect(z, "z", (B, H, M, d), torch.float32)
    _expect(den_out, "den_out", (T, B, H), torch.float32)
    dev = _same_device(q, k, v, mixing, S, z, out, den_out)
    with torch.cuda.device(dev):
        st = load().mhla_causal_stream(_ptr(q), _ptr(k), _ptr(v), _ptr(mixing), _ptr(S), _ptr(z), _ptr(out),
                                       _ptr(den_out), t0, T, B, H, d, block, M, _dtype(q), eps,
                                       _stream(stream, dev))
    _check("mhla_causal_stream", st)
    return out


def mhla_forward_causal(q, k, v, mixing, y, chunk, *, eps=1e-6, den_out=None, workspace=None,
                        stream=None):
    """Causal chunked forward; mixing None = plain causal linear attention."""
    B, H, N, d = _mhla_args(q, k, v, mixing, y, den_out, chunk, mixing_required=False)
    dev = _same_device(q, k, v, mixing, y, den_out, workspace)
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(mhla_workspace_bytes(B, H, N, d, chunk, 1), dev)
        st = load().mhla_forward_causal(_ptr(q), _ptr(k), _ptr(v), _ptr(mixing), _ptr(y), _ptr(den_out),
                                        B, H, N, d, chunk, _dtype(q), eps, _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream, dev))
    _check("mhla_forward_causal", st)
    return y


def mhla_backward_path(B, H, N, d, block_size, dtype) -> str:
    dt = MHLA_BF16 if dtype == torch.bfloat16 else MHLA_F32
    return PATH_NAMES[int(load().mhla_backward_path(B, H, N, d, block_size, dt))]


def mhla_backward(q, k, v, mixing, dy, dq, dk, dv, dmixing, block_size, *, eps=1e-6, workspace=None, stream=None):
    """Gradients of the non-causal MHLA forward: dq, dk, dv [B, H, N, d] (q's dtype) and dmixing
    [H, M, M] fp32 from dy = dL/dY; all four are written."""
    B, H, N, d = _mhla_args(q, k, v, mixing, dy, None, block_size)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _expect(t, name, q.shape, q.dtype)
    _expect(dmixing, "dmixing", mixing.shape, torch.float32)
    dev = _same_device(q, k, v, mixing, dy, dq, dk, dv, dmixing, workspace)
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(mhla_backward_workspace_bytes(B, H, N, d, block_size), dev)
        st = load().mhla_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(mixing), _ptr(dy), _ptr(dq), _ptr(dk), _ptr(dv),
                                  _ptr(dmixing), B, H, N, d, block_size, _dtype(q), eps, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream, dev))
    _check("mhla_backward", st)
    return dq, dk, dv, dmixing


def linattn_decode_step(q, k, v, S, z, out, *, eps=1e-6, den_out=None, stream=None):
    """One recurrent decode step; q/k/v/out [B, H, d], S [B, H, d, d] fp32, z [B, H, d] fp32 (updated)."""
    if q.dim() != 3:
        raise ValueError(f"q: expected [B, H, d], got shape {tuple(q.shape)}")
    B, H, d = q.shape
    for name, t in (("k", k), ("v", v), ("out", out)):
        _expect(t, name, q.shape, q.dtype)
    _expect(S, "S", (B, H, d, d), torch.float32)
    _expect(z, "z", (B, H, d), torch.float32)
    _expect(den_out, "den_out", (B, H), torch.float32)
    dev = _same_device(q, k, v, S, z, out, den_out)
    with torch.cuda.device(dev):
        st = load().linattn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(S), _ptr(z), _ptr(out),
                                        _ptr(den_out), B, H, d, _dtype(q), eps, _stream(stream, dev))
    _check("linattn_decode_step", st)
    return out


def linattn_decode_steps(q, k, v, S, z, out, *, eps=1e-6, gamma=1.0, den_out=None, stream=None):
    """T recurrent decode steps in one call; q/k/v/out [T, B, H, d], S [B, H, d, d] fp32,
    z [B, H, d] fp32 (updated), den_out [T, B, H] fp32; ``gamma`` the decay in [0, 1]."""
    if q.dim() != 4:
        raise ValueError(f"q: expected [T, B, H, d], got shape {tuple(q.shape)}")
    T, B, H, d = q.shape
    for name, t in (("k", k), ("v", v), ("out", out)):
        _expect(t, name, q.shape, q.dtype)
    _expect(S, "S", (B, H, d, d), torch.float32)
    _expect(z, "z", (B, H, d), torch.float32)
    _expect(den_out, "den_out", (T, B, H), torch.float32)
    dev = _same_device(q, k, v, S, z, out, den_out)
    with torch.cuda.device(dev):
        st = load().linattn_decode_steps(_ptr(q), _ptr(k), _ptr(v), _ptr(S), _ptr(z), _ptr(out),
                                         _ptr(den_out), T, B, H, d, _dtype(q), eps, gamma,
                                         _stream(stream, dev))
    _check("linattn_decode_steps", st)
    return out


class _Strides(ctypes.Structure):
    """The C struct mhla_strides: element strides of b, h and n."""
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("n", ctypes.c_longlong)]


class _RetentionOptions(ctypes.Structure):
    """The C struct retention_options."""
    _fields_ = [("feature", ctypes.c_int), ("scale", ctypes.c_float)]


_RETENTION_FEATURES = {**FEATURES, "identity": 3}


# The retention entries are called for single tokens, where the host's time counts: the small C structs
# (plain values, never written) are kept for the values seen last, pointers go as integers.
@functools.lru_cache(maxsize=256)
def _retention_options(feature, scale):
    if feature not in _RETENTION_FEATURES:
        raise ValueError(f"feature: one of {sorted(_RETENTION_FEATURES)}, got {feature!r}")
    return ctypes.byref(_RetentionOptions(_RETENTION_FEATURES[feature], scale))


@functools.lru_cache(maxsize=1024)
def _c_strides(st):
    return ctypes.byref(_Strides(st[0], st[1], st[2] if len(st) == 4 else 0))


def _strided(t, name):
    """(pointer, strides) of a token tensor [B, H, N, d] or [B, H, d] with contiguous rows."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous, its stride is {st[-1]}")
    return t.data_ptr(), _c_strides(st)


def _address(t):
    return None if t is None else t.data_ptr()


def _expect_like(q, *named):
    """Every (name, tensor) of q's shape and dtype."""
    shape, dtype = q.shape, q.dtype
    for name, t in named:
        if t.shape != shape or t.dtype != dtype:
            _expect(t, name, shape, dtype)


def _retention_device(tokens, others):
    """The one CUDA device of all tensors; ``others`` (not the token tensors) must be contiguous."""
    index = tokens[0].get_device()  # -1: not a CUDA tensor
    for t in tokens:
        if t.get_device() != index or index < 0:
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA tensors")
            raise ValueError(f"tensor on {t.device}, expected {tokens[0].device} (the device of q)")
    for t in others:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("tensors must be contiguous CUDA tensors")
            raise ValueError(f"tensor on {t.device}, expected {tokens[0].device} (the device of q)")
    return tokens[0].device


# the current stream's handle without a Stream object around it, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _retention_call(name, dev, args, stream):
    """Calls entry ``name`` with ``dev`` current and the stream last."""
    if stream is not None:
        handle = stream.cuda_stream
    else:
        handle = _raw_stream(dev.index) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    fn = getattr(_lib or load(), name)
    if _current_device() == dev.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != MHLA_OK:
        raise MhlaError(name, st)


def _expect_fast(t, name, shape, dtype):
    """_expect, quicker where it holds."""
    if t is not None and (t.dtype != dtype or t.shape != shape):
        _expect(t, name, shape, dtype)


def _fits_int(**sizes):
    """ctypes would cut a size that the C entry's int does not hold."""
    for name, n in sizes.items():
        if n > 0x7fffffff:
            raise ValueError(f"{name}: {n}, at most {0x7fffffff}")


def _retention_sizes(q, cu_seqlens):
    """B (sequences), H, N (packed: all tokens), d of q [B, H, N, d]; packed: q [1, H, tokens, d]."""
    if q.dim() != 4:
        raise ValueError(f"q: expected [B, H, N, d], got shape {tuple(q.shape)}")
    B, H, N, d = q.shape
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError(f"q: expected [1, H, tokens, d] with cu_seqlens, got shape {tuple(q.shape)}")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError(f"cu_seqlens: expected [sequences + 1], got shape {tuple(cu_seqlens.shape)}")
        _expect_fast(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32)
        B = cu_seqlens.numel() - 1
    if B > 0x7fffffff or H > 0x7fffffff or N > 0x7fffffff or d > 0x7fffffff:
        _fits_int(B=B, H=H, N=N, d=d)
    return B, H, N, d


def _retention_states(states, slots, B, H, d):
    if states is None:
        if slots is not None:
            raise ValueError("slots: given without states")
        return 0
    shape = states.shape
    if len(shape) != 4:
        raise ValueError(f"states: expected [slots, H, d, d], got shape {tuple(shape)}")
    _expect_fast(states, "states", (shape[0], H, d, d), torch.float32)
    _expect_fast(slots, "slots", (B,), torch.int32)
    if shape[0] > 0x7fffffff:
        _fits_int(slots=shape[0])
    return shape[0]


def retention_workspace_bytes(B: int, H: int, tokens: int, d: int, backward: bool = False) -> int:
    if max(B, H, tokens, d) > 0x7fffffff:
        return 0
    return int(load().retention_workspace_bytes(B, H, tokens, d, 1 if backward else 0))


def _retention_workspace(workspace, B, H, N, d, packed, backward, dev, stream):
    """The caller's workspace or, where there is none, a new one: zeroed on the call's stream and of that
    stream's memory, so that neither the zeros nor a later owner of the memory can meet the call's kernels."""
    if workspace is None:
        nbytes = retention_workspace_bytes(B, H, N if packed else B * N, d, backward)
        with torch.cuda.stream(stream):
            workspace = new_workspace(nbytes, dev)
    return workspace


def retention_forward(q, k, v, gamma, y, *, cu_seqlens=None, states=None, slots=None, load_state=False, scale=1.0,
                      feature="identity", workspace=None, stream=None):
    """Linear attention with a decay for each head, y_t = scale phi(q_t) S_t, S_t = gamma S_{t-1} +
    phi(k_t) v_t^T, over whole prompts.  q/k/v/y [B, H, N, d] with any strides (rows contiguous),
    gamma [H] fp32; packed sequences: q/k/v/y [1, H, tokens, d] and int32 ``cu_seqlens``
    [sequences + 1].  ``states`` [slots, H, d, d] fp32 receives the final states (``slots``: the slot
    of each sequence, int32); with ``load_state`` the sequences start from them.  d is 16, 32, 64 or 128.
    ``workspace``: of ``retention_workspace_bytes``; without one the call makes its own, and whether a device-side
    wait gave up cannot be asked afterwards (``mhla_query_status`` reads the workspace)."""
    B, H, N, d = _retention_sizes(q, cu_seqlens)
    _expect_like(q, ("k", k), ("v", v), ("y", y))
    _expect_fast(gamma, "gamma", (H,), torch.float32)
    if load_state and states is None:
        raise ValueError("load_state: needs states")
    n_slots = _retention_states(states, slots, B, H, d)
    opt = _retention_options(feature, float(scale))
    dev = _retention_device((q, k, v, y), (gamma, cu_seqlens, states, slots, workspace))
    ws = _retention_workspace(workspace, B, H, N, d, cu_seqlens is not None, False, dev, stream)
    _retention_call("retention_forward", dev,
                    (*_strided(q, "q"), *_strided(k, "k"), *_strided(v, "v"), gamma.data_ptr(), *_strided(y, "y"),
                     B, H, N, d, _address(cu_seqlens), _address(states), _address(slots), n_slots,
                     1 if load_state else 0, _dtype(q), opt, ws.data_ptr(), ws.nbytes), stream)
    return y


def retention_backward(q, k, v, gamma, dy, dq, dk, dv, *, cu_seqlens=None, scale=1.0, feature="identity",
                       workspace=None, stream=None):
    """Gradients of retention_forward (without states) from dy = dL/dY; dq, dk and dv are written.
    Shapes and workspace as there; every tensor may have its own strides."""
    B, H, N, d = _retention_sizes(q, cu_seqlens)
    _expect_like(q, ("k", k), ("v", v), ("dy", dy), ("dq", dq), ("dk", dk), ("dv", dv))
    _expect_fast(gamma, "gamma", (H,), torch.float32)
    opt = _retention_options(feature, float(scale))
    dev = _retention_device((q, k, v, dy, dq, dk, dv), (gamma, cu_seqlens, workspace))
    ws = _retention_workspace(workspace, B, H, N, d, cu_seqlens is not None, True, dev, stream)
    _retention_call("retention_backward", dev,
                    (*_strided(q, "q"), *_strided(k, "k"), *_strided(v, "v"), gamma.data_ptr(), *_strided(dy, "dy"),
                     *_strided(dq, "dq"), *_strided(dk, "dk"), *_strided(dv, "dv"), B, H, N, d, _address(cu_seqlens),
                     _dtype(q), opt, ws.data_ptr(), ws.nbytes), stream)
    return dq, dk, dv


def retention_step(q, k, v, gamma, states, out, *, slots=None, scale=1.0, feature="identity", stream=None):
    """One token for every row: q/k/v/out [B, H, d] with any strides (rows contiguous), gamma [H] fp32,
    states [slots, H, d, d] fp32 (updated); ``slots`` int32 [B], an entry outside the pool leaves its
    row out."""
    if q.dim() != 3:
        raise ValueError(f"q: expected [B, H, d], got shape {tuple(q.shape)}")
    B, H, d = q.shape
    if B > 0x7fffffff or H > 0x7fffffff or d > 0x7fffffff:
        _fits_int(B=B, H=H, d=d)
    _expect_like(q, ("k", k), ("v", v), ("out", out))
    _expect_fast(gamma, "gamma", (H,), torch.float32)
    if states is None:
        raise ValueError("states: required")
    n_slots = _retention_states(states, slots, B, H, d)
    opt = _retention_options(feature, float(scale))
    dev = _retention_device((q, k, v, out), (gamma, states, slots))
    _retention_call("retention_step", dev,
                    (*_strided(q, "q"), *_strided(k, "k"), *_strided(v, "v"), gamma.data_ptr(), states.data_ptr(),
                     _address(slots), n_slots, *_strided(out, "out"), B, H, d, _dtype(q), opt), stream)
    return out


def retention_copy_states(states, src, dst, *, stream=None):
    """states[dst[i]] = states[src[i]] for all pairs at once (src < 0: zeros); states [slots, H, d, d]
    fp32, src and dst int32 [n], n <= 1024."""
    if states.dim() != 4 or states.shape[2] != states.shape[3]:
        raise ValueError(f"states: expected [slots, H, d, d], got shape {tuple(states.shape)}")
    _expect_fast(states, "states", states.shape, torch.float32)
    if src.dim() != 1:
        raise ValueError(f"src: expected [n], got shape {tuple(src.shape)}")
    for name, t in (("src", src), ("dst", dst)):
        _expect_fast(t, name, src.shape, torch.int32)
    slots, H, d, _ = states.shape
    n = src.shape[0]
    if slots > 0x7fffffff or H > 0x7fffffff or d > 0x7fffffff or n > 0x7fffffff:
        _fits_int(slots=slots, H=H, d=d, n=n)
    dev = _retention_device((states,), (states, src, dst))
    _retention_call("retention_copy_states", dev,
                    (states.data_ptr(), slots, H, d, src.data_ptr(), dst.data_ptr(), n), stream)
    return states


def rala_forward(q, k, v, x, w, y, *, workspace=None, stream=None):
    """Rank-augmented linear attention; q/k/v/y [B, H, N, d], x [B, N, cx], w [cx, d]."""
    if q.dim() != 4 or x.dim() != 3:
        raise ValueError("q: expected [B, H, N, d]; x: expected [B, N, cx]")
    B, H, N, d = q.shape
    cx = x.shape[-1]
    for name, t in (("k", k), ("v", v), ("y", y)):
        _expect(t, name, q.shape, q.dtype)
    _expect(x, "x", (B, N, cx), q.dtype)
    _expect(w, "w", (cx, d), q.dtype)
    dev = _same_device(q, k, v, x, w, y, workspace)
    with torch.cuda.device(dev):
        if workspace is None:
            workspace = new_workspace(rala_workspace_bytes(B, H, N, d, cx), dev)
        st = load().rala_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(w), _ptr(y), B, H, N, d, cx,
                                 _dtype(q), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream, dev))
    _check("rala_forward", st)
    return y


def mhla_forward_noalloc(q, k, v, mixing, y, block_size, *, eps=1e-6, den_out=None, stream=None):
    """Non-causal MHLA forward with no workspace: for callers that cannot allocate device memory.

    The library keeps a fixed 32 MiB scratch array per GPU for it; calls that
    overlap on the GPU share that array and must not run concurrently.
    """
    B, H, N, d = _mhla_args(q, k, v, mixing, y, den_out, block_size)
    dev = _same_device(q, k, v, mixing, y, den_out)
    with torch.cuda.device(dev):
        st = load().mhla_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(mixing), _ptr(y), _ptr(den_out),
                                         B, H, N, d, block_size, _dtype(q), eps, _stream(stream, dev))
    _check("mhla_forward_noalloc", st)
    return y


def mhla_query_status(workspace, stream=None) -> int:
    with torch.cuda.device(workspace.device):
        return int(load().mhla_query_status(_ptr(workspace), _stream(stream, workspace.device)))


def mhla_launch_count() -> int:
    return int(load().mhla_launch_count())


def mhla_debug_set_wait_limit_ns(ns: int) -> None:
    """Diagnostic: limit of the device-side waits of the bf16 tensor-core forward (0 = default)."""
    load().mhla_debug_set_wait_limit_ns(int(ns))
