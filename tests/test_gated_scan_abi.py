"""Refusals of the gated scan's entry points (CPU: every call fails validation, or is an empty no-op, before the
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


def strides(b, n):
    return ctypes.byref(binding._Strides(b, 0, n))


def fwd(lib, x=P, g=2 * P, y=3 * P, xs=None, gs=None, ys=None, B=2, N=200, D=64, cu=None, states=4 * P, slots=None,
        n_slots=2, load=0, kept=5 * P, dt=BF16, gate=0):
    return lib.gated_scan_forward(x, xs, g, gs, y, ys, B, N, D, cu, states, slots, n_slots, load, kept, dt, gate, None)


def bwd(lib, x=P, g=2 * P, dy=3 * P, kept=4 * P, dx=5 * P, dg=6 * P, xs=None, dxs=None, dgs=None, B=2, N=200, D=64, cu=None,
        h0=7 * P, dl=8 * P, dh0=9 * P, dt=BF16, gate=0):
    return lib.gated_scan_backward(x, xs, g, None, dy, None, kept, dx, dxs, dg, dgs, B, N, D, cu, h0, dl, dh0, dt, gate, None)


def step(lib, x=P, g=2 * P, states=3 * P, slots=None, n_slots=4, out=4 * P, os=None, B=4, D=64, dt=BF16, gate=0):
    return lib.gated_scan_step(x, None, g, None, states, slots, n_slots, out, os, B, D, dt, gate, None)


def test_forward_refusals(lib):
    for bad in [dict(B=-1), dict(N=-1), dict(D=-8), dict(dt=2), dict(gate=3), dict(gate=-1), dict(load=2), dict(D=60),
                dict(D=66, dt=F32), dict(n_slots=-1), dict(states=None, load=1), dict(states=None, slots=6 * P)]:
        assert fwd(lib, **bad) == INVALID, bad
    for name in ("x", "g", "y"):
        assert fwd(lib, **{name: None}) == INVALID
        assert fwd(lib, **{name: 7 * P + 8}) == INVALID            # misaligned
    for name in ("states", "kept"):
        assert fwd(lib, **{name: 7 * P + 8}) == INVALID
    for name in ("cu", "slots"):
        assert fwd(lib, **{name: 7 * P + 2}) == INVALID
    assert fwd(lib, y=P) == INVALID and fwd(lib, y=2 * P + 2 * 200 * 64 * 2 - 16) == INVALID   # over x, in g's last row
    assert fwd(lib, y=4 * P) == INVALID and fwd(lib, kept=4 * P) == INVALID and fwd(lib, kept=3 * P) == INVALID
    assert fwd(lib, kept=P) == INVALID                             # over an input
    assert fwd(lib, cu=3 * P) == INVALID and fwd(lib, slots=4 * P) == INVALID and fwd(lib, slots=5 * P) == INVALID
    assert fwd(lib, N=(1 << 31) - 1) == UNSUPPORTED
    assert fwd(lib, n_slots=(1 << 31) - 1, D=1 << 30) == INVALID   # a pool of no memory's size


def test_strides_refusals(lib):
    assert fwd(lib, xs=strides(200 * 64, 68)) == INVALID           # not a multiple of 16 bytes
    assert fwd(lib, gs=strides(200 * 64, -64)) == INVALID
    assert fwd(lib, xs=strides(1 << 40, 64)) == INVALID
    assert fwd(lib, xs=strides(200 * 64, 0)) == INVALID            # rows of their own
    assert fwd(lib, ys=strides(0, 64)) == INVALID                  # an output over itself
    assert fwd(lib, ys=strides(200 * 64, 32)) == INVALID
    s = strides(200 * 3 * 64, 3 * 64)                              # slices of one [B, N, 3, D] tensor
    assert fwd(lib, x=P, g=P + 128, y=P + 128, xs=s, gs=s, ys=s) == INVALID
    assert fwd(lib, x=P, g=P + 128, y=P + 64, xs=s, gs=s, ys=s) == INVALID


def test_backward_refusals(lib):
    for bad in [dict(B=-1), dict(dt=-1), dict(gate=9), dict(D=4), dict(kept=None), dict(kept=P + 8), dict(h0=P + 4),
                dict(dl=P + 4), dict(dh0=P + 4), dict(cu=P + 1), dict(N=(1 << 31) - 100, D=8)]:
        assert bwd(lib, **bad) in (INVALID, UNSUPPORTED), bad
    for name in ("x", "g", "dy", "dx", "dg"):
        assert bwd(lib, **{name: None}) == INVALID
    for name in ("dx", "dg"):
        for other in (P, 2 * P, 3 * P, 4 * P, 7 * P, 8 * P):       # x, g, dy, kept states, h0, dh_last
            assert bwd(lib, **{name: other}) == INVALID
    assert bwd(lib, dx=6 * P) == INVALID and bwd(lib, dh0=5 * P) == INVALID and bwd(lib, dh0=7 * P) == INVALID
    assert bwd(lib, dh0=8 * P) == INVALID and bwd(lib, dh0=4 * P) == INVALID and bwd(lib, cu=9 * P) == INVALID
    assert bwd(lib, dxs=strides(0, 64)) == INVALID


def test_step_refusals(lib):
    for bad in [dict(B=-1), dict(D=12), dict(dt=3), dict(gate=5), dict(n_slots=-1), dict(states=None), dict(out=None),
                dict(states=3 * P + 8), dict(slots=5 * P + 2), dict(out=P), dict(out=2 * P), dict(out=3 * P), dict(x=3 * P),
                dict(slots=3 * P), dict(slots=4 * P), dict(os=strides(0, 0))]:
        assert step(lib, **bad) == INVALID, bad


def test_empty_calls_do_nothing(lib):
    assert fwd(lib, B=0, x=None) == OK and fwd(lib, N=0, y=None) == OK and fwd(lib, D=0) == OK
    assert bwd(lib, B=0, dx=None) == OK and bwd(lib, D=0) == OK and bwd(lib, N=0, dh0=None) == OK
    assert step(lib, B=0, out=None) == OK


def test_checkpoint_rows():
    w = binding.gated_scan_checkpoint_rows
    build_library()
    assert (w(1, 0), w(1, 1), w(1, 64), w(1, 65), w(3, 129)) == (0, 1, 1, 2, 9)
    assert w(-1, 5) == 0 and w(1, -5) == 0 and w(1, 1 << 40) == 0 and w(1, (1 << 31) - 1) == 0


def test_binding_refusals():
    """Shapes, dtypes, devices: ValueError before any device use."""
    build_library()
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    x, st, ck = t(2, 100, 16), t(4, 16, dt=f32), t(4, 16, dt=f32)
    for bad in [dict(g=t(2, 100, 8)), dict(y=x.float()), dict(x=x[0]), dict(load_state=True), dict(slots=t(2, dt=i32)),
                dict(gate="tanh"), dict(states=st, slots=t(3, dt=i32)), dict(states=st, slots=t(2, dt=torch.int64)),
                dict(states=st.half()), dict(states=t(4, 8, dt=f32)), dict(states=t(16, 4, dt=f32).t()), dict(checkpoints=ck[:3]),
                dict(cu_seqlens=t(3, dt=i32)), dict(g=t(16, 100, 2).permute(2, 1, 0)), dict()]:
        a = dict(x=x, g=x, y=x.clone())
        a.update(bad)
        with pytest.raises(ValueError):   # the last: CPU tensors
            binding.gated_scan_forward(**a)
    with pytest.raises(TypeError):
        binding.gated_scan_forward(x.half(), x.half(), x.half())
    for bad in [dict(checkpoints=None), dict(checkpoints=ck[:2]), dict(dx=x[:1]), dict(h0=t(3, 16, dt=f32)), dict(dh0=t(2, 16)), dict()]:
        a = dict(x=x, g=x, dy=x, checkpoints=ck, dx=x.clone(), dg=x.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            binding.gated_scan_backward(**a)
    for bad in [dict(states=None), dict(x=x), dict(out=t(2, 8)), dict(slots=t(3, dt=i32)), dict()]:
        a = dict(x=x[:, 0], g=x[:, 0], states=st, out=x[:, 0].clone())
        a.update(bad)
        with pytest.raises(ValueError):
            binding.gated_scan_step(**a)


def test_a_call_runs_on_its_tensors_device(monkeypatch):
    """With another device current the binding makes that of the tensors current around the call, takes its stream,
    and goes back also when the call fails."""
    log = []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            log.append(("enter", self.index))

        def __exit__(self, *_):
            log.append(("exit", self.index))

    class Entries:
        status = OK

        def gated_scan_step(self, *args):
            log.append(("call", args))
            return self.status

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(binding, "_lib", Entries())
    binding._call_on("gated_scan_step", 1, None, 7)
    assert log == [("enter", 1), ("call", (7, 1001)), ("exit", 1)]
    log.clear()
    binding._call_on("gated_scan_step", 0, Stream(), 7)
    assert log == [("call", (7, 77))]
    log.clear()
    monkeypatch.setattr(binding, "status_string", lambda status: "refused")
    binding._lib.status = INVALID
    with pytest.raises(binding.MhlaError):
        binding._call_on("gated_scan_step", 1, None, 7)
    assert [e[0] for e in log] == ["enter", "call", "exit"]


def test_tensors_of_two_devices_are_refused():
    class Tensor:
        def __init__(self, index):
            self.index, self.is_cuda, self.device = index, index >= 0, f"cuda:{index}" if index >= 0 else "cpu"

        def get_device(self):
            return self.index

    assert binding._one_device(Tensor(1), None, Tensor(1)) == 1
    for other in (0, -1):
        with pytest.raises(ValueError):
            binding._one_device(Tensor(1), Tensor(other))
