"""Host side of the cross attention's entries on the CPU: the calls that are accepted.

``tests/cross_host_check.cu`` compiles ``csrc/cross_api.cu`` with launches that only note their arguments, so that addresses
of no memory can be passed.  Checked are sides without a token or a head, the workspace query against what calls need, and
the denominators that eps allows.
"""

import ctypes
import os
import subprocess

import pytest

from token_level_head_gb300 import binding
from token_level_head_gb300 import build as builder

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
P = 1 << 32  # apart in no memory
HERE = os.path.dirname(os.path.abspath(__file__))
WIDTHS = [(16, F32), (16, BF16), (64, F32), (64, BF16), (128, F32), (128, BF16)]


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("host") / "libcross_host.so")
    subprocess.run([builder.nvcc(), *builder.ARCH, *builder.NVCC_FLAGS, "-shared", os.path.join(HERE, "cross_host_check.cu"),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    for name, (res, args) in binding._SIGNATURES.items():
        if name.startswith("linattn_cross_"):
            getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


def calls(host):
    v = (ctypes.c_longlong * 4)()
    host.check_calls(v)
    return list(v)   # states, read, backward, join


def plan(host, backward):
    v = (ctypes.c_longlong * 3)()
    host.check_plan(v, int(backward))
    return list(v)   # segments of the queries, of the keys, bytes of the workspace


def states(host, B=2, Hk=2, N=300, d=64, dt=BF16, cu=None, lens=None, k=P, wsb=1 << 40, ws=1 << 50):
    return host.linattn_cross_states(k, None, 2 * k if k else None, None, 3 * P, 4 * P, B, Hk, N, d, cu, lens, None, B, dt, None, ws,
                                     wsb, None)


def read(host, B=2, H=4, Hk=2, N=300, d=64, dt=BF16, cu=None, eps=1e-6, q=P, wsb=1 << 40, ws=1 << 50):
    return host.linattn_cross_read(q, None, 3 * P, 4 * P, 5 * P, None, B, H, Hk, N, d, cu, None, B, dt, None, eps, ws, wsb, None)


def backward(host, B=2, H=4, Hk=2, Nq=300, Nk=200, d=64, dt=BF16, cq=None, ck=None, lens=None, eps=1e-6, wsb=1 << 40, ws=1 << 50):
    q = [None] * 3 if Nq == 0 or H == 0 else [P, 6 * P, 7 * P]
    k = [None] * 4 if Nk == 0 else [2 * P, 3 * P, 8 * P, 9 * P]
    return host.linattn_cross_backward(q[0], None, k[0], None, k[1], None, 10 * P, 11 * P, q[1], None, q[2], None, k[2], None, k[3],
                                       None, B, H, Hk, Nq, Nk, d, cq, ck, lens, dt, None, eps, ws, wsb, None)


@pytest.mark.parametrize("d,dt", WIDTHS)
@pytest.mark.parametrize("packed", [False, True])
def test_an_encoder_without_a_token_has_no_segments(host, packed, d, dt):
    """S and z are zeroed by the join of no parts alone."""
    calls(host)
    assert states(host, N=0, k=None, d=d, dt=dt, cu=20 * P if packed else None) == OK
    assert calls(host) == [0, 0, 0, 1] and plan(host, False)[1] == 0


@pytest.mark.parametrize("d,dt", WIDTHS)
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_of_a_side_without_a_token_have_no_segments_there(host, packed, d, dt):
    cu = dict(cq=20 * P, ck=21 * P) if packed else {}
    calls(host)
    assert backward(host, Nk=0, d=d, dt=dt, **cu) == OK
    assert plan(host, True)[1] == 0 and plan(host, True)[0] > 0
    assert backward(host, Nq=0, d=d, dt=dt, **cu) == OK
    assert plan(host, True)[0] == 0 and plan(host, True)[1] > 0
    assert calls(host) == [0, 0, 2, 0]
    assert backward(host, Nq=0, Nk=0, d=d, dt=dt, **cu) == OK
    assert calls(host) == [0, 0, 0, 0]


@pytest.mark.parametrize("d,dt", WIDTHS)
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_without_a_query_head(host, packed, d, dt):
    """No query head on two of keys: no segments of queries, dk and dv are zeros."""
    cu = dict(cq=20 * P, ck=21 * P) if packed else {}
    calls(host)
    assert backward(host, H=0, d=d, dt=dt, **cu) == OK
    assert plan(host, True)[0] == 0 and plan(host, True)[1] > 0
    assert backward(host, H=0, Nk=0, d=d, dt=dt, **cu) == OK
    assert calls(host) == [0, 0, 1, 0]


@pytest.mark.parametrize("d,dt", WIDTHS)
@pytest.mark.parametrize("B,H,Hk,nq,nk", [(3, 6, 2, 1000, 70), (1, 4, 4, 129, 9000), (7, 2, 1, 4096, 33), (600, 1, 1, 1, 1),
                                          (1, 16, 4, 777, 65536), (2, 2, 2, 0, 500), (2, 2, 2, 500, 0)])
def test_the_workspace_query_is_enough_and_less_than_a_calls_need_is_refused(host, B, H, Hk, nq, nk, d, dt):
    """Dense, packed and mixed; calls on exactly the queried bytes, and on one less than what the call itself uses."""
    n = binding.linattn_cross_workspace_bytes
    builder.build_library()
    cu = 20 * P
    forward, back = n(B, H, Hk, B * nq, B * nk, d), n(B, H, Hk, B * nq, B * nk, d, backward=True)
    assert back >= forward > 0
    for ck in (None, cu):
        for w in (forward, back):
            assert states(host, B, Hk, B * nk if ck else nk, d, dt, ck, k=P if nk else None, wsb=w) == OK
        need = plan(host, False)[2]
        joined = calls(host)[3] > 0
        assert need <= forward or not joined
        if joined:
            assert states(host, B, Hk, B * nk if ck else nk, d, dt, ck, k=P if nk else None, wsb=need - 1) == INVALID
        for cq in (None, cu + P):
            assert read(host, B, H, Hk, B * nq if cq else nq, d, dt, cq, wsb=forward) == OK
            args = dict(B=B, H=H, Hk=Hk, Nq=B * nq if cq else nq, Nk=B * nk if ck else nk, d=d, dt=dt, cq=cq, ck=ck)
            assert backward(host, wsb=back, **args) == OK
            need = plan(host, True)[2]
            assert need <= back
            assert backward(host, wsb=need, **args) == OK and backward(host, wsb=need - 1, **args) == INVALID
        calls(host)
