"""Cross attention and gated scan on the GPU where offsets pass 2^31 elements, and waits that give up."""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import gated_scan_oracle as go
from test_cross_gpu import Call
from token_level_head_gb300 import binding
from token_level_head_gb300.build import build_library

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def room(nbytes):
    if torch.cuda.mem_get_info()[0] < nbytes:
        pytest.skip("needs more free device memory")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_states_past_2_31_elements_of_a_pool(dtype):
    """The last slots of a pool of 2.2 x 10^9 elements: written, read by prompts and by single queries."""
    room(12 << 30)
    H, d = 16, 64
    n = (1 << 31) // (H * d * d) + 40
    c = Call(2, H, H, 130, 200, d, dtype).run(backward=False).check(backward=False)
    S, z = torch.empty(n, H, d, d, device="cuda"), torch.empty(n, H, d, device="cuda")
    slots = torch.tensor([n - 1, n - 3], dtype=torch.int32, device="cuda")
    lib.linattn_cross_states(c.k, c.v, S, z, slots=slots)
    assert torch.equal(S[slots.long()], c.S) and torch.equal(z[slots.long()], c.z)
    y = torch.empty_like(c.y)
    lib.linattn_cross_read(c.q, S, z, y, slots=slots)
    assert torch.equal(y, c.y)
    one, same = torch.empty_like(c.y[:, :, :1]), torch.empty_like(c.y[:, :, :1])
    lib.linattn_cross_read(c.q[:, :, :1], S, z, one, slots=slots)
    lib.linattn_cross_read(c.q[:, :, :1], c.S, c.z, same)
    assert torch.equal(one, same)


@pytest.mark.parametrize("d", [16, 64])
def test_tokens_past_2_31_elements(d):
    """Encoder tokens and queries behind 2^31 elements of one packed tensor: the last sequences as if alone."""
    T = (1 << 31) // d + 1000
    room(20 << 30)
    x, out = (torch.zeros(1, 1, T, d, dtype=BF, device="cuda") for _ in range(2))
    cu = [T - 700, T - 400, T - 100]
    x[:, :, T - 700:] = torch.randn(1, 1, 700, d, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    S, z = torch.empty(2, 1, d, d, device="cuda"), torch.empty(2, 1, d, device="cuda")
    lib.linattn_cross_states(x, x, S, z, cu_seqlens=c)
    lib.linattn_cross_read(x, S, z, out, cu_seqlens=c)
    assert not out[:, :, :T - 700].any() and not out[:, :, T - 100:].any()
    alone, So, zo = torch.empty(1, 1, 600, d, dtype=BF, device="cuda"), torch.empty_like(S), torch.empty_like(z)
    part = x[:, :, T - 700:T - 100].contiguous()
    small = torch.tensor([0, 300, 600], dtype=torch.int32, device="cuda")
    lib.linattn_cross_states(part, part, So, zo, cu_seqlens=small)
    lib.linattn_cross_read(part, So, zo, alone, cu_seqlens=small)
    # the sequences may be cut differently: fp32 sums in another order, 300 terms
    assert (S - So).abs().max() <= 300 * 2.0 ** -23 * So.abs().max() * 16
    assert (out[:, :, T - 700:T - 100].float() - alone.float()).abs().max() <= 2.0 ** -7 * alone.float().abs().max()


def test_scan_past_2_31_elements():
    """A sequence of 2^22 + 3000 tokens of 512 channels, and the last slot of a large pool."""
    N, D = (1 << 22) + 3000, 512
    room(30 << 30)
    x, g, y = (torch.zeros(1, N, D, dtype=BF, device="cuda") for _ in range(3))
    n = 2000
    x[:, N - n:] = torch.randn(1, n, D, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    g[:, N - n:] = torch.randn(1, n, D, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    rows = (1 << 31) // D + 5
    pool = torch.zeros(rows, D, device="cuda")
    slots = torch.tensor([rows - 1], dtype=torch.int32, device="cuda")
    ck = torch.empty(lib.gated_scan_checkpoint_rows(1, N), D, device="cuda")
    lib.gated_scan_forward(x, g, y, states=pool, slots=slots, load_state=True, checkpoints=ck)
    s = slice(0, 16)
    ref, e = go.scan(to_f64(x[0, N - n:, s]), to_f64(g[0, N - n:, s]), "sigmoid", None, 2.0 ** -19)
    assert not y[:, :N - n].any()
    assert (np.abs(to_f64(y[0, N - n:, s]) - ref) <= 2.0 ** -8 * np.abs(ref) + e + 1e-30).all()
    assert (np.abs(to_f64(pool[-1, s]) - ref[-1]) <= 2.0 ** -24 * np.abs(ref[-1]) + e[-1] + 1e-30).all()
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    lib.gated_scan_backward(x, g, y, ck, dx, dg)
    (rx, rg, _), (ex, eg, _) = go.scan_backward(to_f64(x[0, N - n:, s]), to_f64(g[0, N - n:, s]), to_f64(y[0, N - n:, s]), "sigmoid",
                                                delta=2.0 ** -19)
    assert (np.abs(to_f64(dx[0, N - n:, s]) - rx) <= 2.0 ** -8 * np.abs(rx) + ex + 1e-30).all()
    assert (np.abs(to_f64(dg[0, N - n:, s]) - rg) <= 2.0 ** -8 * np.abs(rg) + eg + 1e-30).all()
    lib.gated_scan_step(x[:, -1], g[:, -1], pool, y[:, 0], slots=slots)
    h = ref[-1:]
    a = 1 / (1 + np.exp(-to_f64(g[0, -1:, s])))
    now = a * h + (1 - a) * to_f64(x[0, -1:, s])
    assert np.abs(to_f64(pool[-1:, s]) - now).max() <= 2.0 ** -16


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["states", "read", "backward"])
def test_wait_limit_gives_up_then_next_call_is_correct(which, d):
    """With every wait at its shortest a call on the tensor cores gives up, MHLA_ERR_TIMEOUT is latched in its workspace,
    and the next call on the same workspace is right."""
    c = Call(2, 4, 2, 1500, 2000, d, BF)
    ws = lib.new_workspace(lib.linattn_cross_workspace_bytes(2, 4, 2, 3000, 4000, d, backward=True), "cuda")
    c.run(workspace=ws)
    assert binding.mhla_query_status(ws) == binding.MHLA_OK
    binding.mhla_debug_set_wait_limit_ns(1)
    try:
        if which == "states":
            lib.linattn_cross_states(c.k, c.v, c.S, c.z, workspace=ws)
        elif which == "read":
            lib.linattn_cross_read(c.q, c.S, c.z, c.y, workspace=ws)
        else:
            lib.linattn_cross_backward(c.q, c.k, c.v, c.S, c.z, c.dy, c.dq, c.dk, c.dv, workspace=ws)
        torch.cuda.synchronize()
    finally:
        binding.mhla_debug_set_wait_limit_ns(0)
    assert binding.mhla_query_status(ws) == binding.MHLA_ERR_TIMEOUT
    assert binding.mhla_query_status(ws) == binding.MHLA_OK
    c.run(workspace=ws).check()
    assert binding.mhla_query_status(ws) == binding.MHLA_OK


def test_calls_on_two_streams_at_once():
    """Two problems with their own workspaces on two streams, many times in turn, against one after the other."""
    calls = [Call(2, 4, 2, 900, 1100, d, BF) for d in (64, 128)]
    spaces = [lib.new_workspace(lib.linattn_cross_workspace_bytes(2, 4, 2, 1800, 2200, c.d, backward=True), "cuda") for c in calls]
    for c, ws in zip(calls, spaces):
        c.run(workspace=ws)
    torch.cuda.synchronize()
    want = [[t.clone() for t in (c.S, c.z, c.y, c.dq, c.dk, c.dv)] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for c, ws, s in zip(calls, spaces, streams):
            with torch.cuda.stream(s):
                c.run(workspace=ws)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        for t, r in zip((c.S, c.z, c.y, c.dq, c.dk, c.dv), w):
            assert torch.equal(t, r)
