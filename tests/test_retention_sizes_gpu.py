"""The retention operators on the GPU at the largest sizes and with offsets that claim more than there is."""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import retention_oracle as ro
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


@pytest.mark.parametrize("packed", [False, True])
def test_the_longest_sequence(packed):
    """2^31 - 128 tokens of one head: zeros but for the last 300, which are as if they stood alone.  q, k and v are
    one tensor.  Tolerance: scores and the state's copy in bf16, 2^-8 each of a term, and the result's rounding."""
    T, d, n = (1 << 31) - 128, 16, 300
    if torch.cuda.mem_get_info()[0] < 5 * T * d:
        pytest.skip("needs 160 GiB of free device memory")
    x, y = (torch.empty(1, 1, T, d, dtype=BF, device="cuda") for _ in range(2))
    x.zero_()
    y.fill_(7.0)
    tail = torch.randn(1, 1, n, d, generator=torch.Generator().manual_seed(1)).to(BF)
    x[:, :, T - n:] = tail.cuda()
    g = torch.tensor([0.9], device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if packed else None
    lib.retention_forward(x, x, x, g, y, cu_seqlens=cu)
    assert (y[:, :, :T - n:9973] == 0).all()
    assert (y[:, :, T - n - 200000:T - n] == 0).all()
    args = [to_f64(tail[0])] * 3 + [to_f64(g)]
    ref, mag = ro.retention(*args)[0], ro.retention(*args, magnitude=True)[0]
    assert (np.abs(to_f64(y[0, :, T - n:]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.05 * 2.0 ** -8 * mag).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_offsets_that_claim_more_segments_than_an_int_holds(dtype):
    """200,000 offsets 0, T, 0, T, ..: 100,000 sequences of all T tokens, 5 x 10^9 segments.  The first one has its
    place in the workspace and comes out right; nothing around the workspace, and no row behind T, is written."""
    T, d, n, pad = 200_000_001, 16, 300, 1 << 26
    es = torch.finfo(dtype).bits // 8
    if torch.cuda.mem_get_info()[0] < 3 * T * d * es:
        pytest.skip("needs 40 GB of free device memory")
    x, y = (torch.zeros(1, 1, T + 1, d, dtype=dtype, device="cuda") for _ in range(2))
    y.fill_(7.0)
    tail = torch.randn(1, 1, n, d, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[:, :, T - n:T] = tail.cuda()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda").repeat(100_000)
    size = lib.retention_workspace_bytes(cu.numel() - 1, 1, T + 1, d)
    buf = torch.zeros(pad + size + pad, dtype=torch.uint8, device="cuda")
    buf[:pad] = 77
    buf[pad + size:] = 77
    lib.retention_forward(x, x, x, torch.tensor([0.9], device="cuda"), y, cu_seqlens=cu, workspace=buf[pad:pad + size])
    assert (buf[:pad] == 77).all() and (buf[pad + size:] == 77).all() and (y[:, :, T:] == 7).all()
    assert (y[:, :, :T - n:997] == 0).all()
    args = [to_f64(tail[0])] * 3 + [np.array([np.float64(np.float32(0.9))])]
    ref, mag = ro.retention(*args)[0], ro.retention(*args, magnitude=True)[0]
    u, more = (2.0 ** -8, 2.05 * 2.0 ** -8) if dtype == BF else (2.0 ** -24, 300 * 2.0 ** -24 + 2.0 ** -18)
    assert (np.abs(to_f64(y[0, :, T - n:T]) - ref) <= u * np.abs(ref) + more * mag).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_states_past_32_bits(dtype):
    """A pool of 2^31 elements and more: prompts, tokens and copies on its first and its last slots, against the same
    calls on a small pool, bit for bit."""
    H, d, n, N = 16, 128, 8200, 150
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB of free device memory")
    far = torch.empty(n, H, d, d, device="cuda")
    assert far.numel() > (1 << 31)
    at = [n - 1, 0, 8192, n - 3]
    near = torch.randn(4, H, d, d, generator=torch.Generator().manual_seed(1)).cuda()
    for i, s in enumerate(at):
        far[s] = near[i]
    far[n - 2] = 7.0
    q, k, v = (torch.randn(3, H, N, d, generator=torch.Generator().manual_seed(i)).to(dtype).cuda() for i in range(3))
    g = (1 - 2.0 ** -torch.linspace(5, 9, H)).cuda()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = []
    for pool, slots in ((far, at), (near, range(4))):
        y, o, s = torch.empty_like(q), torch.empty(3, H, d, dtype=dtype, device="cuda"), list(slots)
        lib.retention_forward(q, k, v, g, y, states=pool, slots=ints(*s[:3]), load_state=True, scale=0.1)
        lib.retention_copy_states(pool, ints(s[0], s[1]), ints(s[3], s[0]))
        lib.retention_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, pool, o, slots=ints(s[2], s[3], s[0]), scale=0.1)
        out.append([y, o] + [pool[i].clone() for i in s])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert (far[n - 2] == 7).all()
