"""Refusals of the retention entry points (CPU: every call fails validation, or is an empty no-op,
before the library touches CUDA)."""

import ctypes

import pytest
import torch

from token_level_head_gb300 import binding
from token_level_head_gb300.build import build_library

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
P = 1 << 24  # fake, aligned "device" addresses 16 MB apart; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build_library()
    return binding.load()


def strides(*s):
    return ctypes.byref(binding._Strides(*s))


def opt(feature=3, scale=1.0):
    return ctypes.byref(binding._RetentionOptions(feature, scale))


def fwd(lib, q=P, k=2 * P, v=3 * P, gamma=4 * P, y=5 * P, qs=None, ks=None, vs=None, ys=None, B=2, H=3, N=200, d=64,
        cu=None, states=6 * P, slots=None, n_slots=2, load=0, dt=BF16, o=None, ws=8 * P, wsb=1 << 30):
    return lib.retention_forward(q, qs, k, ks, v, vs, gamma, y, ys, B, H, N, d, cu, states, slots, n_slots, load, dt,
                                 o, ws, wsb, None)


def bwd(lib, q=P, k=2 * P, v=3 * P, gamma=4 * P, dy=5 * P, dq=6 * P, dk=7 * P, dv=8 * P, B=2, H=3, N=200, d=64,
        cu=None, dt=BF16, o=None, ws=9 * P, wsb=1 << 30, dqs=None, dks=None, dvs=None, ks=None):
    return lib.retention_backward(q, None, k, ks, v, None, gamma, dy, None, dq, dqs, dk, dks, dv, dvs, B, H, N, d, cu,
                                  dt, o, ws, wsb, None)


def step(lib, q=P, k=2 * P, v=3 * P, gamma=4 * P, states=5 * P, slots=None, n_slots=4, out=9 * P, B=4, H=3, d=64,
         dt=BF16, o=None, os=None):
    return lib.retention_step(q, None, k, None, v, None, gamma, states, slots, n_slots, out, os, B, H, d, dt, o, None)


def copy(lib, states=P, n_slots=8, H=4, d=64, src=4 * P, dst=5 * P, n=3):
    return lib.retention_copy_states(states, n_slots, H, d, src, dst, n, None)


def test_forward_refusals(lib):
    assert fwd(lib, d=48) == INVALID
    assert fwd(lib, B=-1) == INVALID
    assert fwd(lib, dt=5) == INVALID
    assert fwd(lib, o=opt(4)) == INVALID
    assert fwd(lib, o=opt(-1)) == INVALID
    assert fwd(lib, o=opt(3, float("nan"))) == INVALID
    assert fwd(lib, load=2) == INVALID
    assert fwd(lib, states=None, load=1) == INVALID             # nothing to load from
    assert fwd(lib, states=None, slots=7 * P) == INVALID
    assert fwd(lib, n_slots=-1) == INVALID
    for name in ("q", "k", "v", "y", "gamma"):
        assert fwd(lib, **{name: None}) == INVALID
        assert fwd(lib, **{name: P * 7 + 2}) == INVALID          # misaligned
    assert fwd(lib, states=6 * P + 4) == INVALID
    assert fwd(lib, slots=7 * P + 2) == INVALID
    assert fwd(lib, cu=7 * P + 2) == INVALID
    assert fwd(lib, ws=None) == INVALID
    assert fwd(lib, ws=8 * P + 16) == INVALID
    assert fwd(lib, wsb=64) == INVALID
    assert fwd(lib, y=P) == INVALID
    assert fwd(lib, y=2 * P + 2 * 3 * 200 * 64 * 2 - 16) == INVALID  # y starts in k's last row
    assert fwd(lib, y=6 * P + 128) == INVALID                    # in the states
    assert fwd(lib, y=4 * P) == INVALID                          # over gamma
    assert fwd(lib, ws=6 * P) == INVALID                         # over the states
    assert fwd(lib, cu=5 * P, B=2) == INVALID                    # over y
    assert fwd(lib, slots=6 * P) == INVALID                      # over the states
    assert fwd(lib, B=1 << 15, N=1 << 17) == UNSUPPORTED         # more than 2^31 tokens


def test_strides_refusals(lib):
    assert fwd(lib, qs=strides(3 * 200 * 64, 200 * 64, 68)) == INVALID     # not a multiple of 16 bytes
    assert fwd(lib, ks=strides(3 * 200 * 64, 200 * 64, -64)) == INVALID
    assert fwd(lib, vs=strides(1 << 40, 200 * 64, 64)) == INVALID
    assert fwd(lib, ys=strides(3 * 200 * 64, 0, 64)) == INVALID            # an output over itself
    assert fwd(lib, ys=strides(3 * 200 * 64, 64, 64)) == INVALID
    assert fwd(lib, ys=strides(200 * 64, 200 * 64, 64)) == INVALID
    # y as the fourth slice of a [B, N, 4, H, d] tensor that q, k and v are slices of: wrong only where it meets one
    s = strides(200 * 4 * 3 * 64, 64, 4 * 3 * 64)
    at = lambda i: P + i * 3 * 64 * 2
    kw = dict(q=at(0), k=at(1), v=at(2), qs=s, ks=s, vs=s, ys=s, wsb=0)
    assert fwd(lib, y=at(1), **kw) == INVALID
    assert fwd(lib, y=at(1) + 64 * 2, **kw) == INVALID                     # head 1 of the slice k
    # dense outputs inside a strided input's range are refused, whether they meet a row or not
    assert fwd(lib, y=at(0) + 64, **{**kw, "ys": None}) == INVALID


def test_interleaved_outputs_are_found_apart_or_not(lib):
    """dq, dk, dv as slices of one [B, N, 3, H, d] tensor, shifted so that rows meet (apart they are taken:
    the GPU tests run that call)."""
    s = strides(200 * 3 * 3 * 64, 64, 3 * 3 * 64)
    at = lambda i: 6 * P + i * 3 * 64 * 2
    good = dict(dq=at(0), dk=at(1), dv=at(2), dqs=s, dks=s, dvs=s)
    assert bwd(lib, **{**good, "dv": at(1)}) == INVALID
    assert bwd(lib, **{**good, "dk": at(0) + 64 * 2 * 2}) == INVALID      # overlaps slices 0 and 1
    assert bwd(lib, **{**good, "dk": at(0) + 9 * 64 * 2}) == INVALID      # dq, a token later: all rows but one meet


def test_backward_refusals(lib):
    assert bwd(lib, d=24) == INVALID
    assert bwd(lib, N=-1) == INVALID
    assert bwd(lib, dt=-1) == INVALID
    assert bwd(lib, o=opt(9)) == INVALID
    for name in ("q", "k", "v", "dy", "dq", "dk", "dv", "gamma", "ws"):
        assert bwd(lib, **{name: None}) == INVALID
    for name in ("dq", "dk", "dv"):
        for other in (P, 2 * P, 3 * P, 5 * P, 4 * P, 9 * P):               # q, k, v, dy, gamma, the workspace
            assert bwd(lib, **{name: other}) == INVALID
    assert bwd(lib, dq=7 * P) == INVALID and bwd(lib, dk=8 * P) == INVALID and bwd(lib, dv=6 * P) == INVALID
    assert bwd(lib, dks=strides(3 * 200 * 64, 0, 64)) == INVALID
    assert bwd(lib, q=9 * P) == INVALID                                    # an input in the workspace
    assert bwd(lib, cu=9 * P) == INVALID
    assert bwd(lib, wsb=0) == INVALID


def test_step_refusals(lib):
    assert step(lib, d=0) == INVALID
    assert step(lib, H=-1) == INVALID
    assert step(lib, dt=2) == INVALID
    assert step(lib, n_slots=-1) == INVALID
    assert step(lib, o=opt(7)) == INVALID
    for name in ("q", "k", "v", "gamma", "states", "out"):
        assert step(lib, **{name: None}) == INVALID
        assert step(lib, **{name: 10 * P + 2}) == INVALID
    assert step(lib, slots=7 * P + 1) == INVALID
    assert step(lib, out=P) == INVALID
    assert step(lib, out=5 * P) == INVALID                                 # in the states
    assert step(lib, q=5 * P + 256) == INVALID
    assert step(lib, gamma=5 * P) == INVALID
    assert step(lib, slots=5 * P) == INVALID
    assert step(lib, os=strides(3 * 64, 0, 0)) == INVALID
    assert step(lib, B=1 << 20, H=1 << 12) == UNSUPPORTED


def test_copy_refusals(lib):
    assert copy(lib, d=65) == INVALID
    assert copy(lib, n=-1) == INVALID
    assert copy(lib, n_slots=-1) == INVALID
    for name in ("states", "src", "dst"):
        assert copy(lib, **{name: None}) == INVALID
        assert copy(lib, **{name: 9 * P + 2}) == INVALID
    assert copy(lib, src=P + 64) == INVALID
    assert copy(lib, dst=P + 64) == INVALID
    assert copy(lib, n=1025) == UNSUPPORTED


def test_empty_calls_do_nothing(lib):
    assert fwd(lib, B=0, q=None, ws=None) == OK
    assert fwd(lib, N=0, q=None, k=None, v=None, y=None) == OK
    assert fwd(lib, H=0) == OK
    assert bwd(lib, N=0, dq=None) == OK
    assert step(lib, B=0, out=None) == OK
    assert copy(lib, n=0, src=None) == OK
    assert copy(lib, n_slots=0) == OK


def test_workspace_query(lib):
    w = binding.retention_workspace_bytes
    assert w(1, 8, 65536, 128) > w(1, 8, 100, 128) > 0
    assert w(1, 8, 65536, 128, backward=True) > w(1, 8, 100, 128, backward=True) > 0
    assert w(4, 16, 100, 63) == 0 and w(-1, 16, 100, 64) == 0
    assert lib.retention_workspace_bytes(1, 1, 1, 64, 2) == 0
    # the query covers the dense and the packed reading of its sizes
    for B, H, N, d in [(3, 5, 1000, 64), (1, 1, 129, 16), (7, 2, 4096, 128), (600, 1, 1, 64)]:
        assert fwd(lib, B=B, H=H, N=N, d=d, wsb=w(B, H, B * N, d), q=None) == INVALID


def test_binding_refusals():
    """Shapes, dtypes, devices: ValueError before any device use."""
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    g, st = t(3, dt=torch.float32), t(4, 3, 64, 64, dt=torch.float32)
    f = binding.retention_forward
    x = t(2, 3, 10, 64)
    for bad in [dict(gamma=t(4, dt=torch.float32)), dict(k=t(2, 3, 11, 64)), dict(v=x.float()), dict(q=x[0]),
                dict(load_state=True), dict(slots=t(2, dt=torch.int32)), dict(feature="silu"),
                dict(states=st, slots=t(3, dt=torch.int32)), dict(states=st, slots=t(2, dt=torch.int64)),
                dict(states=st[:, :2]), dict(states=st.half()), dict(cu_seqlens=t(3, dt=torch.int32)),
                dict(cu_seqlens=t(3, dt=torch.int64)), dict()]:
        a = dict(q=x, k=x, v=x, gamma=g, y=x.clone())
        a.update(bad)
        with pytest.raises(ValueError):   # the last: CPU tensors
            f(**a)
    with pytest.raises(ValueError):
        binding.retention_backward(x, x, x, g, x, x, x, t(2, 3, 10, 32))
    with pytest.raises(ValueError):
        binding.retention_step(x, x, x, g, st, x)
    with pytest.raises(ValueError):
        binding.retention_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g, None, x[:, :, 0])
    with pytest.raises(ValueError):
        binding.retention_copy_states(st, t(2, dt=torch.int32), t(3, dt=torch.int32))
    with pytest.raises(ValueError):
        binding.retention_copy_states(st, t(2, dt=torch.int64), t(2, dt=torch.int64))
