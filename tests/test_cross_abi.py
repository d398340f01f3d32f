"""Refusals of the cross attention's entry points (CPU: every call fails validation, or is an empty no-op, before the
library touches CUDA)."""

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


def opt(feature=0, normalise=1, gamma=1.0):
    return ctypes.byref(binding.MhlaOptions(feature, normalise, gamma))


def states(lib, k=P, v=2 * P, S=3 * P, z=4 * P, ks=None, B=2, Hk=3, N=200, d=64, cu=None, lens=None, slots=None, n_slots=2, dt=BF16,
           o=None, ws=8 * P, wsb=1 << 30):
    return lib.linattn_cross_states(k, ks, v, None, S, z, B, Hk, N, d, cu, lens, slots, n_slots, dt, o, ws, wsb, None)


def read(lib, q=P, S=2 * P, z=3 * P, y=4 * P, qs=None, ys=None, B=2, H=6, Hk=3, N=200, d=64, cu=None, slots=None, n_slots=2, dt=BF16,
         o=None, eps=1e-6, ws=8 * P, wsb=1 << 30):
    return lib.linattn_cross_read(q, qs, S, z, y, ys, B, H, Hk, N, d, cu, slots, n_slots, dt, o, eps, ws, wsb, None)


def bwd(lib, q=P, k=2 * P, v=3 * P, S=4 * P, z=5 * P, dy=6 * P, dq=7 * P, dk=8 * P, dv=9 * P, dqs=None, dks=None, B=2, H=6, Hk=3,
        Nq=200, Nk=100, d=64, cq=None, ck=None, lens=None, dt=BF16, o=None, eps=1e-6, ws=1 << 40, wsb=1 << 36):
    return lib.linattn_cross_backward(q, None, k, None, v, None, S, z, dy, None, dq, dqs, dk, dks, dv, None, B, H, Hk, Nq, Nk, d,
                                      cq, ck, lens, dt, o, eps, ws, wsb, None)


def test_states_refusals(lib):
    for bad in [dict(d=48), dict(B=-1), dict(Hk=-1), dict(N=-1), dict(dt=4), dict(o=opt(4)), dict(o=opt(-1)), dict(o=opt(0, 2)),
                dict(o=opt(0, 1, 0.5)), dict(o=opt(3, 1)), dict(n_slots=-1), dict(cu=5 * P, lens=6 * P), dict(cu=5 * P + 2),
                dict(lens=5 * P + 2), dict(slots=5 * P + 2), dict(ws=None), dict(ws=8 * P + 16), dict(wsb=64),
                dict(ks=strides(3 * 200 * 64, 200 * 64, 68))]:
        assert states(lib, **bad) == INVALID, bad
    for name in ("k", "v", "S", "z"):
        assert states(lib, **{name: None}) == INVALID
        assert states(lib, **{name: 7 * P + 8}) == INVALID
    for bad in [dict(S=P), dict(z=2 * P), dict(z=3 * P), dict(S=8 * P), dict(k=8 * P), dict(cu=3 * P), dict(lens=4 * P),
                dict(slots=3 * P), dict(slots=8 * P)]:
        assert states(lib, **bad) == INVALID, bad
    assert states(lib, B=1 << 15, N=1 << 17) == UNSUPPORTED                # more than 2^31 tokens
    assert states(lib, N=100000, wsb=1 << 19) == INVALID                   # parts need more


def test_read_refusals(lib):
    for bad in [dict(d=24), dict(H=7), dict(Hk=0), dict(H=-6), dict(N=-1), dict(dt=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(o=opt(3, 1)), dict(o=opt(5, 0)), dict(n_slots=-1), dict(cu=5 * P + 1), dict(slots=5 * P + 2),
                dict(ws=None), dict(wsb=0), dict(ws=8 * P + 128)]:
        assert read(lib, **bad) == INVALID, bad
    for name in ("q", "S", "z", "y"):
        assert read(lib, **{name: None}) == INVALID
        assert read(lib, **{name: 7 * P + 8}) == INVALID
    for bad in [dict(y=P), dict(y=2 * P), dict(y=3 * P), dict(cu=4 * P), dict(slots=4 * P), dict(ws=P), dict(ws=2 * P),
                dict(ys=strides(6 * 200 * 64, 0, 64)), dict(qs=strides(6 * 200 * 64, 200 * 64, 60))]:
        assert read(lib, **bad) == INVALID, bad
    assert read(lib, N=1, ws=None, y=P) == INVALID                         # a step without a workspace is checked all the same
    assert read(lib, N=1, ws=P) == INVALID
    assert read(lib, B=1 << 15, N=1 << 17) == UNSUPPORTED


def test_backward_refusals(lib):
    for bad in [dict(d=8), dict(H=4), dict(Nk=-1), dict(Nq=-1), dict(dt=7), dict(eps=-1e-3), dict(o=opt(3, 1)), dict(ck=20 * P, lens=21 * P),
                dict(cq=20 * P + 2), dict(lens=20 * P + 1), dict(ws=None), dict(wsb=1 << 19), dict(ws=(1 << 40) + 8)]:
        assert bwd(lib, **bad) == INVALID, bad
    for name in ("q", "k", "v", "S", "z", "dy", "dq", "dk", "dv"):
        assert bwd(lib, **{name: None}) == INVALID, name
        assert bwd(lib, **{name: 30 * P + 8}) == INVALID, name
    for name in ("dq", "dk", "dv"):
        for other in (P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 1 << 40):      # q, k, v, S, z, dy, the workspace
            assert bwd(lib, **{name: other}) == INVALID, (name, other)
    assert bwd(lib, dq=8 * P) == INVALID and bwd(lib, dk=9 * P) == INVALID and bwd(lib, dv=7 * P) == INVALID
    assert bwd(lib, lens=8 * P) == INVALID and bwd(lib, cq=7 * P) == INVALID and bwd(lib, ck=9 * P) == INVALID
    assert bwd(lib, dks=strides(3 * 100 * 64, 0, 64)) == INVALID
    assert bwd(lib, B=1 << 15, Nk=1 << 17) == UNSUPPORTED and bwd(lib, B=1 << 15, Nq=1 << 17) == UNSUPPORTED


def test_empty_calls_do_nothing(lib):
    assert states(lib, B=0, k=None, ws=None) == OK and states(lib, Hk=0, S=None) == OK
    assert read(lib, B=0, q=None) == OK and read(lib, N=0, q=None, y=None) == OK and read(lib, H=0, Hk=0) == OK
    assert bwd(lib, B=0, q=None) == OK and bwd(lib, Nq=0, Nk=0, q=None, k=None) == OK


def test_workspace_query(lib):
    w = binding.linattn_cross_workspace_bytes
    assert w(1, 8, 8, 100, 65536, 128) > w(1, 8, 8, 100, 100, 128) > 0
    assert w(1, 8, 8, 65536, 100, 64, backward=True) > w(1, 8, 8, 65536, 100, 64)
    assert w(4, 16, 3, 100, 100, 64) == 0 and w(4, 16, 4, 100, 100, 63) == 0 and w(-1, 16, 4, 1, 1, 64) == 0
    assert w(1, 1, 1, 1 << 40, 1, 64) == 0 and lib.linattn_cross_workspace_bytes(1, 1, 1, 1, 1, 64, 2) == 0
    # the query covers both types, dense and packed: what it says is enough (one byte less or a null tensor is refused)
    for B, H, Hk, nq, nk, d in [(3, 6, 2, 1000, 70, 64), (1, 4, 4, 129, 9000, 16), (7, 2, 1, 4096, 33, 128), (600, 1, 1, 1, 1, 32)]:
        for dt in (F32, BF16):
            n = w(B, H, Hk, B * nq, B * nk, d, backward=True)
            assert bwd(lib, B=B, H=H, Hk=Hk, Nq=nq, Nk=nk, d=d, dt=dt, wsb=n, dv=None) == INVALID


def test_binding_refusals():
    """Shapes, dtypes, devices: ValueError before any device use."""
    build_library()
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    k, S, z, q = t(2, 3, 10, 64), t(2, 3, 64, 64, dt=f32), t(2, 3, 64, dt=f32), t(2, 6, 7, 64)
    for bad in [dict(v=t(2, 3, 11, 64)), dict(v=k.float()), dict(k=k[0]), dict(S=None), dict(z=None), dict(S=S.half()), dict(S=S[:, :2]),
                dict(z=z[:1]), dict(S=S[0]), dict(lens=t(3, dt=i32)), dict(lens=t(2, dt=torch.int64)), dict(slots=t(1, dt=i32)),
                dict(cu_seqlens=t(3, dt=i32)), dict(feature="silu"), dict(S=S.transpose(2, 3)), dict()]:
        a = dict(k=k, v=k, S=S, z=z)
        a.update(bad)
        with pytest.raises(ValueError):   # the last: CPU tensors
            binding.linattn_cross_states(**a)
    for bad in [dict(y=t(2, 6, 7, 32)), dict(q=t(2, 5, 7, 64), y=t(2, 5, 7, 64)), dict(S=S[:, :, :32]), dict(slots=t(3, dt=i32)),
                dict(q=q[0]), dict(cu_seqlens=t(2, dt=i32)), dict(z=None), dict()]:
        a = dict(q=q, S=S, z=z, y=q.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            binding.linattn_cross_read(**a)
    for bad in [dict(dq=q[:1]), dict(dk=t(2, 3, 10, 32)), dict(S=t(3, 3, 64, 64, dt=f32), z=t(3, 3, 64, dt=f32)), dict(k=k[:1], v=k[:1]),
                dict(S=t(2, 2, 64, 64, dt=f32), z=t(2, 2, 64, dt=f32)), dict(lens=t(1, dt=i32)), dict(dy=q.float()), dict()]:
        a = dict(q=q, k=k, v=k, S=S, z=z, dy=q, dq=q.clone(), dk=k.clone(), dv=k.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            binding.linattn_cross_backward(**a)
