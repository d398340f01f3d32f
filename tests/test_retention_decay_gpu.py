"""Decays below 1/2 of the retention operators on the GPU against the float64 oracle.

Every token but one is zero, so each value is one power of gamma times terms that have it too: an error of the
decay is not hidden behind larger terms.  Tolerances, relative to the oracle's sum of absolute values:
  * a power gamma^n = 2^(n log2 gamma) in fp32: log2 within a step (2^-23), its product with n and the one with
    log2 e rounded (2^-24 each), so the exponent is off by less than 2.25 x 2^-23 n |log2 gamma| and the power,
    times ln 2, by less than n |log2 gamma| 2^-22; the exponential itself adds less than 2^-21;
  * sums of at most d = 64 products in fp32: 64 x 2^-24;
  * bf16 calls: the result's rounding and that of a score or of the state, 2^-8 each; a returned state is fp32.
Powers below the smallest normal fp32 number (1.2e-38) may be flushed.
"""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import retention_oracle as ro
from token_level_head_gb300.build import build_library

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
GAMMAS = [0.499, 0.4, 0.1, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 1e-7, 2e-8, 1e-12, 1e-30, 0.0]
H, D = len(GAMMAS), 64


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()


def rand(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def check(got, ref, mag, dtype, n, what):
    g = np.maximum(to_f64(torch.tensor(GAMMAS)), 1e-300)[:, None, None]
    tol = n * np.abs(np.log2(g)) * 2.0 ** -22 + 2.0 ** -21 + D * 2.0 ** -24 + (2 * 2.0 ** -8 if dtype == BF else 2.0 ** -24)
    err = np.abs(to_f64(got) - ref)
    bad = ~(err <= tol * mag + 1.3e-38 * np.maximum(mag, 1) * D * D)
    heads = sorted({GAMMAS[i] for i in np.nonzero(bad)[0]})
    assert not bad.any(), f"{what}: {bad.sum()} values off, decays {heads}"


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [1, 2, 3, 70])
def test_a_loaded_state_fades_as_gamma_says(N, dtype):
    """Keys are zero: y_t = gamma^(t+1) phi(q_t) S, the state after the call gamma^N S, and the same token by token."""
    g = torch.tensor(GAMMAS, device="cuda")
    q, v = rand((1, H, N, D), dtype, 1), rand((1, H, N, D), dtype, 2)
    k, y = torch.zeros_like(q), torch.empty_like(q)
    start = rand((1, H, D, D), F32, 3)
    st = start.clone()
    lib.retention_forward(q, k, v, g, y, states=st, load_state=True, scale=0.5)
    args = [to_f64(t[0]) for t in (q, k, v)] + [to_f64(g), 0.5, "identity", to_f64(start[0])]
    (ry, rs), (my, ms) = ro.retention(*args), ro.retention(*args, magnitude=True)
    check(y[0], ry, my, dtype, N, "y")
    check(st[0], rs, ms, F32, N, "state")
    steps, out = start.clone(), torch.empty(1, H, D, dtype=dtype, device="cuda")
    for t in range(N):
        lib.retention_step(q[:, :, t], k[:, :, t], v[:, :, t], g, steps, out, scale=0.5)
    check(steps[0], to_f64(st[0]), ms, F32, N, "state of the steps against the prompt's")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_one_key_fades_as_gamma_says(dtype):
    """Only the first key is not zero: y_t and the state are gamma^t and gamma^(N-1) of its product."""
    N, g = 4, torch.tensor(GAMMAS, device="cuda")
    q, k, v = (rand((1, H, N, D), dtype, i) for i in range(3))
    k[:, :, 1:] = 0
    y, st = torch.empty_like(q), torch.empty(1, H, D, D, device="cuda")
    lib.retention_forward(q, k, v, g, y, states=st, scale=0.5)
    args = [to_f64(t[0]) for t in (q, k, v)] + [to_f64(g), 0.5]
    (ry, rs), (my, ms) = ro.retention(*args), ro.retention(*args, magnitude=True)
    check(y[0], ry, my, dtype, N, "y")
    check(st[0], rs, ms, F32, N, "state")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gradients_fade_as_gamma_says(dtype):
    """Only the last token has a gradient, only the first a key: the sums of earlier and of later tokens are single powers."""
    N, g = 4, torch.tensor(GAMMAS, device="cuda")
    q, k, v, dy = (rand((1, H, N, D), dtype, i) for i in range(4))
    dy[:, :, :-1] = 0
    k[:, :, 1:] = 0
    grads = [torch.empty_like(q) for _ in range(3)]
    lib.retention_backward(q, k, v, g, dy, *grads, scale=0.5)
    args = [to_f64(t[0]) for t in (q, k, v)] + [to_f64(g), to_f64(dy[0]), 0.5]
    ref, mag = ro.retention_backward(*args), ro.retention_backward(*args, magnitude=True)
    for name, got, r, m in zip(("dq", "dk", "dv"), grads, ref, mag):
        check(got[0], r, m, dtype, N, name)
