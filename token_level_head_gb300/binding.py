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
    "gated_scan_checkpoint_rows": (ctypes.c_longlong, [_i, _i]),
    "gated_scan_forward": (_i, [_vp] * 6 + [_i] * 3 + [_vp, _vp, _vp, _i, _i, _vp, _i, _i, _vp]),
    "gated_scan_backward": (_i, [_vp] * 11 + [_i] * 3 + [_vp] * 4 + [_i, _i, _vp]),
    "gated_scan_step": (_i, [_vp] * 6 + [_i, _vp, _vp, _i, _i, _i, _i, _vp]),
    "linattn_cross_workspace_bytes": (_sz, [_i] * 7),
    "linattn_cross_states": (_i, [_vp] * 6 + [_i] * 4 + [_vp, _vp, _vp, _i, _i, _vp, _vp, _sz, _vp]),
    "linattn_cross_read": (_i, [_vp] * 6 + [_i] * 5 + [_vp, _vp, _i, _i, _vp, _f, _vp, _sz, _vp]),
    "linattn_cross_backward": (_i, [_vp] * 16 + [_i] * 6 + [_vp, _vp, _vp, _i, _vp, _f, _vp, _sz, _vp]),
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


# The gated scan and the cross attention are called for single tokens too: what follows from shapes, strides, types and
# options alone (their checks, and the C arguments) is kept for the values seen last.
def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _is_meta(m, name, shape, dtype):
    """The same checks as _expect on (shape, stride, dtype), and contiguity."""
    if m is None:
        return
    if tuple(m[0]) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(m[0])}, expected {tuple(shape)}")
    if m[2] != dtype:
        raise ValueError(f"{name}: dtype {m[2]}, expected {dtype}")
    dense = 1
    for n, s in zip(reversed(m[0]), reversed(m[1])):
        if n > 1 and s != dense:
            raise ValueError(f"{name}: must be contiguous, its strides are {tuple(m[1])}")
        dense *= max(n, 1)


def _token_metas(first, *named):
    """Token tensors (name, meta) of the first one's shape and dtype with contiguous rows; their C dtype."""
    name, m = first
    if m[2] not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported dtype {m[2]}; use float32 or bfloat16")
    for other, o in (first, *named):
        if o[0] != m[0]:
            raise ValueError(f"{other}: shape {tuple(o[0])}, expected {tuple(m[0])}")
        if o[2] != m[2]:
            raise ValueError(f"{other}: dtype {o[2]}, expected {m[2]}")
        if o[1][-1] != 1 and o[0][-1] > 1:
            raise ValueError(f"{other}: the last dimension must be contiguous, its stride is {o[1][-1]}")
    return MHLA_BF16 if m[2] == torch.bfloat16 else MHLA_F32


def _sequences(shape, cu, name, what, cu_name="cu_seqlens"):
    """The sequences of tokens [B, ..]: B, or packed those of the offsets."""
    _fits_int(**{f"{name}.shape[{i}]": n for i, n in enumerate(shape)})
    if cu is None:
        return shape[0]
    if shape[0] != 1:
        raise ValueError(f"{name}: expected [1, {what}] with {cu_name}, got shape {tuple(shape)}")
    if len(cu[0]) != 1 or cu[0][0] < 1:
        raise ValueError(f"{cu_name}: expected [sequences + 1], got shape {tuple(cu[0])}")
    _is_meta(cu, cu_name, cu[0], torch.int32)
    _fits_int(sequences=cu[0][0] - 1)
    return cu[0][0] - 1


def _one_device(*ts):
    """The index of the one CUDA device of all tensors."""
    index = ts[0].get_device()  # -1: not a CUDA tensor
    for t in ts:
        if t is not None and (t.get_device() != index or index < 0):
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA tensors")
            raise ValueError(f"tensor on {t.device}, expected {ts[0].device}")
    return index


def _call_on(name, index, stream, *args):
    """Calls entry ``name`` with device ``index`` current and the stream last."""
    if stream is not None:
        handle = stream.cuda_stream
    else:
        handle = _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream
    fn = getattr(_lib or load(), name)
    if _current_device() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st != MHLA_OK:
        raise MhlaError(name, st)


GATES = {"sigmoid": 0, "log": 1, "decay": 2}


def _gate(gate):
    if gate not in GATES:
        raise ValueError(f"gate: {gate!r}, one of {', '.join(GATES)}")
    return GATES[gate]


def _scan_strides(m):
    st = m[1]
    return ctypes.byref(_Strides(st[0], 0, st[1] if len(st) == 3 else 0))


def _scan_pool(states, slots, B, D):
    """The slots of a pool [slots, D]."""
    if states is None:
        if slots is not None:
            raise ValueError("slots: given without states")
        return 0
    if len(states[0]) != 2:
        raise ValueError(f"states: expected [slots, D], got shape {tuple(states[0])}")
    _is_meta(states, "states", (states[0][0], D), torch.float32)
    _is_meta(slots, "slots", (B,), torch.int32)
    _fits_int(slots=states[0][0])
    return states[0][0]


def gated_scan_checkpoint_rows(B: int, N: int) -> int:
    """Rows of the fp32 [rows, D] tensor that gated_scan_forward keeps for gated_scan_backward; B, N: the first two
    sizes of x."""
    return 0 if max(B, N) > 0x7fffffff else int(load().gated_scan_checkpoint_rows(B, N))


def _scan_sizes(x, cu, kept):
    if len(x[0]) != 3:
        raise ValueError(f"x: expected [B, N, D], got shape {tuple(x[0])}")
    B = _sequences(x[0], cu, "x", "tokens, D")
    if kept is not None:
        _is_meta(kept, "checkpoints", (gated_scan_checkpoint_rows(x[0][0], x[0][1]), x[0][2]), torch.float32)
    return B, x[0][1], x[0][2]


@functools.lru_cache(maxsize=256)
def _scan_forward_plan(x, g, y, cu, states, slots, load_state, kept, gate):
    B, N, D = _scan_sizes(x, cu, kept)
    dt = _token_metas(("x", x), ("g", g), ("y", y))
    if load_state and states is None:
        raise ValueError("load_state: needs states")
    n_slots = _scan_pool(states, slots, B, D)
    return B, N, D, dt, n_slots, _gate(gate), _scan_strides(x), _scan_strides(g), _scan_strides(y)


def gated_scan_forward(x, g, y, *, gate="sigmoid", cu_seqlens=None, states=None, slots=None, load_state=False,
                       checkpoints=None, stream=None):
    """h_t = a_t h_{t-1} + b_t, y_t = h_t over whole prompts, with a gate of its own for every token and channel:
    "sigmoid" a = sigmoid(g), b = (1 - a) x; "log" a = exp(g), b = x; "decay" a = g, b = x.  x/g/y [B, N, D] with any
    strides (rows contiguous); packed sequences: [1, tokens, D] and int32 ``cu_seqlens`` [sequences + 1].  ``states``
    [slots, D] fp32 receives the final states (``slots``: the slot of each sequence, int32); with ``load_state`` the
    sequences start from them.  ``checkpoints`` (``gated_scan_checkpoint_rows``) is written for the backward pass."""
    load_state = bool(load_state)
    B, N, D, dt, n_slots, code, sx, sg, sy = _scan_forward_plan(
        _meta(x), _meta(g), _meta(y), _meta(cu_seqlens), _meta(states), _meta(slots), load_state, _meta(checkpoints), gate)
    _call_on("gated_scan_forward", _one_device(x, g, y, cu_seqlens, states, slots, checkpoints), stream,
             x.data_ptr(), sx, g.data_ptr(), sg, y.data_ptr(), sy, B, N, D, _address(cu_seqlens), _address(states),
             _address(slots), n_slots, 1 if load_state else 0, _address(checkpoints), dt, code)
    return y


@functools.lru_cache(maxsize=256)
def _scan_backward_plan(x, g, dy, kept, dx, dg, cu, h0, dh_last, dh0, gate):
    if kept is None:
        raise ValueError("checkpoints: required")
    B, N, D = _scan_sizes(x, cu, kept)
    dt = _token_metas(("x", x), ("g", g), ("dy", dy), ("dx", dx), ("dg", dg))
    for name, m in (("h0", h0), ("dh_last", dh_last), ("dh0", dh0)):
        _is_meta(m, name, (B, D), torch.float32)
    return B, N, D, dt, _gate(gate), *(_scan_strides(m) for m in (x, g, dy, dx, dg))


def gated_scan_backward(x, g, dy, checkpoints, dx, dg, *, gate="sigmoid", cu_seqlens=None, h0=None, dh_last=None,
                        dh0=None, stream=None):
    """Gradients of gated_scan_forward from dy = dL/dy and, where given, ``dh_last`` = dL/d(last states): dx and dg are
    written, and ``dh0`` = dL/d(starts).  ``checkpoints``: of the forward call; ``h0``: the states that it started from
    (load_state; None: zero).  h0, dh_last, dh0: fp32 [sequences, D]."""
    B, N, D, dt, code, sx, sg, sd, sdx, sdg = _scan_backward_plan(
        _meta(x), _meta(g), _meta(dy), _meta(checkpoints), _meta(dx), _meta(dg), _meta(cu_seqlens), _meta(h0),
        _meta(dh_last), _meta(dh0), gate)
    _call_on("gated_scan_backward", _one_device(x, g, dy, checkpoints, dx, dg, cu_seqlens, h0, dh_last, dh0), stream,
             x.data_ptr(), sx, g.data_ptr(), sg, dy.data_ptr(), sd, checkpoints.data_ptr(), dx.data_ptr(), sdx,
             dg.data_ptr(), sdg, B, N, D, _address(cu_seqlens), _address(h0), _address(dh_last), _address(dh0), dt, code)
    return dx, dg


@functools.lru_cache(maxsize=256)
def _scan_step_plan(x, g, states, out, slots, gate):
    if len(x[0]) != 2:
        raise ValueError(f"x: expected [B, D], got shape {tuple(x[0])}")
    B, D = x[0]
    _fits_int(B=B, D=D)
    dt = _token_metas(("x", x), ("g", g), ("out", out))
    if states is None:
        raise ValueError("states: required")
    return B, D, dt, _scan_pool(states, slots, B, D), _gate(gate), _scan_strides(x), _scan_strides(g), _scan_strides(out)


def gated_scan_step(x, g, states, out, *, gate="sigmoid", slots=None, stream=None):
    """One token for every row: x/g/out [B, D] with any strides (rows contiguous), states [slots, D] fp32 (updated);
    ``slots`` int32 [B], an entry outside the pool leaves its row out."""
    B, D, dt, n_slots, code, sx, sg, so = _scan_step_plan(_meta(x), _meta(g), _meta(states), _meta(out), _meta(slots), gate)
    _call_on("gated_scan_step", _one_device(x, g, states, out, slots), stream, x.data_ptr(), sx, g.data_ptr(), sg,
             states.data_ptr(), _address(slots), n_slots, out.data_ptr(), so, B, D, dt, code)
    return out


def _cross_options(feature, normalise):
    if feature not in _RETENTION_FEATURES:
        raise ValueError(f"feature: one of {sorted(_RETENTION_FEATURES)}, got {feature!r}")
    return ctypes.byref(MhlaOptions(_RETENTION_FEATURES[feature], 1 if normalise else 0, 1.0))


def _cross_strides(m):
    return ctypes.byref(_Strides(*m[1][:3]))


def _cross_side(m, cu, name, cu_name="cu_seqlens"):
    """B (sequences), heads, N (packed: all tokens), d of [B, heads, N, d]."""
    if len(m[0]) != 4:
        raise ValueError(f"{name}: expected [B, heads, N, d], got shape {tuple(m[0])}")
    return _sequences(m[0], cu, name, "heads, tokens, d", cu_name), *m[0][1:]


def _cross_sums(S, z, H, d):
    """The slots and heads of S [slots, Hk, d, d] and z [slots, Hk, d], H a multiple of Hk."""
    if S is None or z is None:
        raise ValueError("S, z: required")
    if len(S[0]) != 4:
        raise ValueError(f"S: expected [slots, Hk, d, d], got shape {tuple(S[0])}")
    n, Hk = S[0][:2]
    if Hk == 0 or H % Hk != 0:
        raise ValueError(f"S: {Hk} heads, {H} query heads are no multiple of them")
    _is_meta(S, "S", (n, Hk, d, d), torch.float32)
    _is_meta(z, "z", (n, Hk, d), torch.float32)
    _fits_int(slots=n)
    return n, Hk


def linattn_cross_workspace_bytes(B: int, H: int, Hk: int, tokens_q: int, tokens_k: int, d: int,
                                  backward: bool = False) -> int:
    if max(B, H, Hk, tokens_q, tokens_k, d) > 0x7fffffff:
        return 0
    return int(load().linattn_cross_workspace_bytes(B, H, Hk, tokens_q, tokens_k, d, 1 if backward else 0))


def _cross_workspace(workspace, sizes, backward, device, stream):
    if workspace is None:  # of the call's stream, as in _retention_workspace
        with torch.cuda.stream(stream):
            workspace = new_workspace(linattn_cross_workspace_bytes(*sizes, backward), device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace


@functools.lru_cache(maxsize=256)
def _cross_states_plan(k, v, S, z, cu, lens, slots, feature, normalise):
    B, Hk, N, d = _cross_side(k, cu, "k")
    dt = _token_metas(("k", k), ("v", v))
    n_slots, heads = _cross_sums(S, z, Hk, d)
    if heads != Hk:
        raise ValueError(f"S: {heads} heads, k has {Hk}")
    _is_meta(lens, "lens", (B,), torch.int32)
    _is_meta(slots, "slots", (B,), torch.int32)
    return B, Hk, N, d, n_slots, dt, _cross_options(feature, normalise), _cross_strides(k), _cross_strides(v)


def linattn_cross_states(k, v, S, z, *, cu_seqlens=None, lens=None, slots=None, feature="elu1", normalise=True,
                         workspace=None, stream=None):
    """The sums S = sum phi(k_j) v_j^T, z = sum phi(k_j) of encoder sequences: k/v [B, Hk, N, d] with any strides (rows
    contiguous), S [slots, Hk, d, d] and z [slots, Hk, d] fp32, written.  Packed sequences: k/v [1, Hk, tokens, d] and
    int32 ``cu_seqlens`` [sequences + 1]; a padded batch: int32 ``lens`` [B], the tokens of each row.  ``slots`` int32:
    the slot of each sequence."""
    B, Hk, N, d, n_slots, dt, opt, sk, sv = _cross_states_plan(
        _meta(k), _meta(v), _meta(S), _meta(z), _meta(cu_seqlens), _meta(lens), _meta(slots), feature, bool(normalise))
    index = _one_device(k, v, S, z, cu_seqlens, lens, slots, workspace)
    ws = _cross_workspace(workspace, (B, Hk, Hk, 0, N if cu_seqlens is not None else B * N, d), False, k.device, stream)
    _call_on("linattn_cross_states", index, stream, k.data_ptr(), sk, v.data_ptr(), sv, S.data_ptr(), z.data_ptr(), B, Hk, N,
             d, _address(cu_seqlens), _address(lens), _address(slots), n_slots, dt, opt, ws.data_ptr(), ws.nbytes)
    return S, z


@functools.lru_cache(maxsize=256)
def _cross_read_plan(q, S, z, y, cu, slots, feature, normalise):
    B, H, N, d = _cross_side(q, cu, "q")
    dt = _token_metas(("q", q), ("y", y))
    n_slots, Hk = _cross_sums(S, z, H, d)
    _is_meta(slots, "slots", (B,), torch.int32)
    return B, H, Hk, N, d, n_slots, dt, _cross_options(feature, normalise), _cross_strides(q), _cross_strides(y)


def linattn_cross_read(q, S, z, y, *, cu_seqlens=None, slots=None, feature="elu1", normalise=True, eps=1e-6,
                       workspace=None, stream=None):
    """y_t = phi(q_t) S / (phi(q_t) . z + eps) from the sums of linattn_cross_states: q/y [B, H, N, d] with any strides
    (rows contiguous), H a multiple of S's heads; packed queries: [1, H, tokens, d] and int32 ``cu_seqlens``.  ``slots``
    int32: the slot that each sequence reads, an entry outside the pool leaves its rows out.  N = 1: a decoder's step."""
    B, H, Hk, N, d, n_slots, dt, opt, sq, sy = _cross_read_plan(
        _meta(q), _meta(S), _meta(z), _meta(y), _meta(cu_seqlens), _meta(slots), feature, bool(normalise))
    index = _one_device(q, y, S, z, cu_seqlens, slots, workspace)
    if workspace is not None or N != 1 or cu_seqlens is not None:
        workspace = _cross_workspace(workspace, (B, H, Hk, N if cu_seqlens is not None else B * N, 0, d), False, q.device, stream)
    _call_on("linattn_cross_read", index, stream, q.data_ptr(), sq, S.data_ptr(), z.data_ptr(), y.data_ptr(), sy, B, H, Hk, N,
             d, _address(cu_seqlens), _address(slots), n_slots, dt, opt, eps, _address(workspace),
             0 if workspace is None else workspace.nbytes)
    return y


@functools.lru_cache(maxsize=256)
def _cross_backward_plan(q, k, v, S, z, dy, dq, dk, dv, cu_q, cu_k, lens, feature, normalise):
    B, H, Nq, d = _cross_side(q, cu_q, "q", "cu_seqlens_q")
    Bk, Hk, Nk, d_k = _cross_side(k, cu_k, "k", "cu_seqlens_k")
    if Bk != B or d_k != d or k[2] != q[2]:
        raise ValueError(f"k: {Bk} sequences of width {d_k}, {k[2]}; expected {B} of width {d}, {q[2]}")
    dt = _token_metas(("q", q), ("dy", dy), ("dq", dq))
    _token_metas(("k", k), ("v", v), ("dk", dk), ("dv", dv))
    slots, heads = _cross_sums(S, z, H, d)
    if heads != Hk:
        raise ValueError(f"S: {heads} heads, k has {Hk}")
    if slots != B:
        raise ValueError(f"S: {slots} slots, expected one for each of {B} sequences")
    _is_meta(lens, "lens", (B,), torch.int32)
    return B, H, Hk, Nq, Nk, d, dt, _cross_options(feature, normalise), *(_cross_strides(m) for m in (q, k, v, dy, dq, dk, dv))


def linattn_cross_backward(q, k, v, S, z, dy, dq, dk, dv, *, cu_seqlens_q=None, cu_seqlens_k=None, lens=None,
                           feature="elu1", normalise=True, eps=1e-6, workspace=None, stream=None):
    """Gradients of linattn_cross_read of linattn_cross_states (slot i is sequence i) from dy = dL/dY; dq, dk and dv are
    written, rows of a padded encoder batch behind ``lens`` as zeros.  Shapes as there."""
    B, H, Hk, Nq, Nk, d, dt, opt, sq, sk, sv, sdy, sdq, sdk, sdv = _cross_backward_plan(
        _meta(q), _meta(k), _meta(v), _meta(S), _meta(z), _meta(dy), _meta(dq), _meta(dk), _meta(dv), _meta(cu_seqlens_q),
        _meta(cu_seqlens_k), _meta(lens), feature, bool(normalise))
    index = _one_device(q, k, v, S, z, dy, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, lens, workspace)
    ws = _cross_workspace(workspace, (B, H, Hk, Nq if cu_seqlens_q is not None else B * Nq,
                                      Nk if cu_seqlens_k is not None else B * Nk, d), True, q.device, stream)
    _call_on("linattn_cross_backward", index, stream, q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, S.data_ptr(),
             z.data_ptr(), dy.data_ptr(), sdy, dq.data_ptr(), sdq, dk.data_ptr(), sdk, dv.data_ptr(), sdv, B, H, Hk, Nq, Nk, d,
             _address(cu_seqlens_q), _address(cu_seqlens_k), _address(lens), dt, opt, eps, ws.data_ptr(), ws.nbytes)
    return dq, dk, dv


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
