"""Host side of the retention entries on the CPU: the calls that are accepted.

``tests/retention_host_check.cu`` compiles ``csrc/retention_api.cu`` with launches that only note their arguments, so
that addresses of no memory can be passed.  Checked are the overlap test of outputs against the sets of bytes that the
tensors take, the workspace query against the plan of every kind of call, the plan's counts against the segments of
random packed sequences, and the binding's switch to the tensors' device.
"""

import ctypes
import itertools
import os
import random
import subprocess

import pytest
import torch

from token_level_head_gb300 import binding
from token_level_head_gb300 import build as builder

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
P = 1 << 24
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """The entries with noted launches."""
    so = str(tmp_path_factory.mktemp("host") / "libretention_host.so")
    subprocess.run([builder.nvcc(), *builder.ARCH, *builder.NVCC_FLAGS, "-shared", os.path.join(HERE, "retention_host_check.cu"),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    for name, (res, args) in binding._SIGNATURES.items():
        if name.startswith("retention_"):
            getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    lib.check_calls.restype = ctypes.c_longlong
    lib.check_plan.argtypes = [ctypes.POINTER(ctypes.c_longlong)]
    return lib


def strides(s):
    return None if s is None else ctypes.byref(binding._Strides(*s))


def forward(host, B, H, N, d, dt=BF16, cu=None, states=None, load=0, q=P, k=P, v=P, y=32 * P, s=None, ys=None,
            wsb=1 << 40, ws=1 << 50):
    return host.retention_forward(q, strides(s), k, strides(s), v, strides(s), 1 << 48, y, strides(ys), B, H, N, d, cu,
                                  states, None, B if states else 0, load, dt, None, ws, wsb, None)


def backward(host, B, H, N, d, dt=BF16, cu=None, q=P, dy=2 * P, out=(32 * P, 64 * P, 96 * P), s=None, os_=None,
             wsb=1 << 40, ws=1 << 50):
    o = list(itertools.chain(*[(p, strides(os_)) for p in out]))
    return host.retention_backward(*[q, strides(s)] * 3, 1 << 48, dy, strides(s), *o, B, H, N, d, cu, dt, None, ws, wsb, None)


def plan(host):
    v = (ctypes.c_longlong * 7)()
    host.check_plan(v)
    return dict(zip(("L", "G", "inner", "split", "W", "nsum", "bytes"), v))


def rows(p, s, B, H, N, d, es):
    """The 16-byte pieces of a tensor's rows."""
    return {(p + (b * s[0] + h * s[1] + n * s[2] + c) * es) // 16 for b in range(B) for h in range(H) for n in range(N)
            for c in range(0, d, 16 // es)}


def test_slices_of_a_fused_tensor_are_taken(host):
    """y as the fourth slice of a [B, N, 4, H, d] tensor that q, k and v are slices of; dq, dk, dv as those of another."""
    B, H, N, d = 2, 3, 200, 64
    s = (N * 4 * H * d, d, 4 * H * d)
    at = lambda i, base=P: base + i * H * d * 2
    n = host.check_calls()
    assert forward(host, B, H, N, d, q=at(0), k=at(1), v=at(2), y=at(3), s=s, ys=s) == OK
    assert host.check_calls() == n + 1
    kw = dict(q=at(0), k=at(1), v=at(2), s=s, ys=s)
    assert forward(host, B, H, N, d, **{**kw, "y": at(1)}) == INVALID
    assert forward(host, B, H, N, d, **{**kw, "y": at(1) + d * 2}) == INVALID      # head 1 of the slice k
    assert forward(host, B, H, N, d, **{**kw, "y": at(0) + 64, "ys": None}) == INVALID
    assert backward(host, B, H, N, d, s=s, os_=s, q=at(0), dy=at(1), out=[at(i, 32 * P) for i in range(3)]) == OK
    assert backward(host, B, H, N, d, s=s, os_=s, q=at(0), dy=at(1), out=[at(i, 32 * P) for i in (0, 1, 1)]) == INVALID
    assert host.check_calls() == n + 2


def test_overlaps_are_those_of_the_bytes(host):
    """Random strides, orders and offsets: an output that is accepted shares no byte with an input and none with
    itself, and one of an input's own strides that shares none is accepted."""
    rng = random.Random(5)
    taken = refused = 0
    for _ in range(4000):
        B, H, N, d = rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 4), 16
        dt = rng.choice([F32, BF16])
        es, q = (4, 4) if dt == F32 else (2, 8)
        order, inner, s = rng.sample(range(3), 3), d * rng.choice([1, 1, 2, 4]), [0, 0, 0]
        for i in order:  # from the innermost out, with gaps
            s[i] = inner
            inner *= (B, H, N)[i]
            inner += q * rng.choice([0, 0, 0, 1, 4])
        ys = s if rng.random() < 0.7 else [x + q * rng.choice([0, 0, 1]) for x in s]
        if rng.random() < 0.1:
            ys = [x if rng.random() < 0.7 else rng.choice(s) for x in ys]
        y = P + 16 * rng.randint(-inner * es // 16 - 2, inner * es // 16 + 2)
        mine, theirs = rows(y, ys, B, H, N, d, es), rows(P, s, B, H, N, d, es)
        itself = len(mine) < B * H * N * (d * es // 16)
        got = forward(host, B, H, N, d, dt=dt, y=y, s=s, ys=ys)
        if got == OK:
            assert not (mine & theirs) and not itself, (B, H, N, dt, s, ys, y - P)
            taken += 1
        else:
            assert got == INVALID
            refused += 1
            if ys == s:
                assert mine & theirs or itself, (B, H, N, dt, s, y - P)
    assert taken > 500 and refused > 500


def test_the_workspace_query_covers_every_call(host):
    """Both types, dense and packed, with and without states, both directions: what the query says is enough, one
    byte less than the plan's own size is not, and the plan's states end inside."""
    rng = random.Random(6)
    for _ in range(1500):
        B, H, d = rng.choice([1, 1, 2, 7, 33, 600]), rng.choice([1, 3, 16, 40]), rng.choice([16, 32, 64, 128])
        N = int(2 ** rng.uniform(0, 20))
        dt, packed, back, states = rng.choice([F32, BF16]), rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5
        tokens = N if packed else B * N
        kw = dict(dt=dt, cu=1 << 47 if packed else None)
        far = dict(out=[1 << 51, 1 << 52, 1 << 53]) if back else dict(y=1 << 51, states=1 << 54 if states else None)
        call = backward if back else forward
        size = host.retention_workspace_bytes(B, H, tokens, d, 1 if back else 0)
        if call(host, B, H, N, d, **kw, **far) == UNSUPPORTED:
            continue
        p = plan(host)
        assert p["bytes"] <= size
        assert call(host, B, H, N, d, wsb=size, **kw, **far) == OK
        assert call(host, B, H, N, d, wsb=p["bytes"], **kw, **far) == OK
        assert call(host, B, H, N, d, wsb=p["bytes"] - 1, **kw, **far) == INVALID


def test_the_plan_holds_the_segments_of_any_lengths(host):
    """Blocks for every segment, for every one that enters another, for every split sequence, and states for the split
    ones', whatever the lengths."""
    rng = random.Random(7)
    for _ in range(400):
        B, H, T = rng.choice([1, 2, 5, 40, 300]), rng.choice([1, 4, 16]), int(2 ** rng.uniform(0, 21))
        back = rng.random() < 0.5
        d, dt = rng.choice([16, 64, 128]), rng.choice([F32, BF16])
        far = dict(out=[1 << 51, 1 << 52, 1 << 53]) if back else dict(y=1 << 51)
        assert (backward if back else forward)(host, B, H, T, d, dt=dt, cu=1 << 47, **far) == OK
        p = plan(host)
        assert p["L"] % (64 if dt == F32 else 128) == 0
        for _ in range(20):
            if rng.random() < 0.3:  # as many as can be just over a segment's length
                lens = [min(p["L"] + 1, T)] * B
            else:
                lens = [int(T * rng.random() ** 4) for _ in range(B)]
            left, cut = T, []
            for n in lens:
                cut.append(min(n, left))
                left -= cut[-1]
            segs = [-(-n // p["L"]) for n in cut]
            assert sum(segs) <= p["G"]
            if T > p["L"]:
                assert sum(n - 1 for n in segs if n) <= p["inner"]
                assert sum(n >= 2 for n in segs) <= p["split"]
                assert sum(n for n in segs if n >= 2) <= p["W"]


def test_a_call_runs_on_its_tensors_device(monkeypatch):
    """With another device current the binding makes that of the tensors current around the call, takes its stream,
    and goes back also when the call fails."""
    log = []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            log.append(("enter", self.dev.index))

        def __exit__(self, *_):
            log.append(("exit", self.dev.index))

    class Entries:
        def __init__(self, status):
            self.status = status

        def retention_step(self, *args):
            log.append(("call", args))
            return self.status

    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(binding, "_lib", Entries(OK))
    binding._retention_call("retention_step", torch.device("cuda", 1), (7,), None)
    assert log == [("enter", 1), ("call", (7, 1001)), ("exit", 1)]
    log.clear()
    binding._retention_call("retention_step", torch.device("cuda", 0), (7,), None)
    assert log == [("call", (7, 1000))]
    log.clear()
    monkeypatch.setattr(binding, "status_string", lambda status: "refused")
    binding._lib.status = INVALID
    with pytest.raises(binding.MhlaError):
        binding._retention_call("retention_step", torch.device("cuda", 1), (7,), None)
    assert [e[0] for e in log] == ["enter", "call", "exit"]
