"""Feature maps of the retention operators together with packed sequences, split sequences and returned states, and
norms of bf16 errors, on the GPU against the float64 oracle.

Elementwise tolerances, relative to the oracle's sum of the terms' absolute values (mag):
  * fp32 sums: at most d + 128 products and one term for each chunk and segment: (400 + N / 64) 2^-24; decays 2^-18;
    the feature maps' exponentials 2^-21 each;
  * bf16 calls: the result 2^-8 of itself; of a term 2^-8 for its score or its state and 2^-8 for every operand with a
    feature map (two at most), 2^-16 for the decayed key;
  * returned states of bf16 calls: three bf16 parts, or two where the decay leaves at most 2^-2.75: 2^-16 of a term.
Norms: a rounding to bf16 is off by at most 2^-8, evenly spread, so 2^-8 / sqrt(3) in the mean square; a term of y or
of a gradient meets that of its score or state, of the result and of its mapped operands, all independent: n of them
give 2^-8 sqrt(n / 3) of the norm, and a tenth more is allowed for chance.  (One token lost of 1500 is 0.026.)
"""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import retention_oracle as ro
from token_level_head_gb300 import binding
from token_level_head_gb300.build import build_library

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SLOW = [1 - 2.0 ** -5, 1 - 2.0 ** -7, 1 - 2.0 ** -9, 1.0]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()


def rand(shape, dtype, seed):
    """[B, H, N, d] of N(0, 1) / 2 in token-major storage."""
    B, H, N, d = shape
    g = torch.Generator().manual_seed(seed)
    return (0.5 * torch.randn(B, N, H, d, generator=g)).to(dtype).cuda().transpose(1, 2)


def check(got, ref, mag, dtype, N, operands, what):
    u = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    term = (400 + N / 64) * 2.0 ** -24 + 2.0 ** -18 + 3 * 2.0 ** -21 + operands
    err, tol = np.abs(to_f64(got) - ref), u * np.abs(ref) + term * mag + 1e-37
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.2f} x"


def operands(dtype, n):
    return 0.0 if dtype == F32 else (1 + n) * 2.0 ** -8 * 1.02 + 2.0 ** -16


def launches(call):
    n = binding.load().mhla_launch_count()
    call()
    return binding.load().mhla_launch_count() - n


CUTS = [[2, 2, 3, 70, 70, 198, 460, 467, 467], [4, 132, 260], [0, 2603, 2604, 4500]]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("feature", ["elu1", "relu", "exp"])
@pytest.mark.parametrize("cu", CUTS)
def test_packed_sequences_with_a_feature_map(cu, feature, d, dtype):
    """Tiles that reach into the next sequence are mapped, cleared and, where states are returned, read again; rows of
    no sequence are NaN and stay as they were in the outputs."""
    H, n, T = 4, len(cu) - 1, cu[-1] + 9
    q, k, v, dy = (rand((1, H, T, d), dtype, i) for i in range(4))
    for t in (q, k, v, dy):
        t[:, :, :cu[0]] = float("nan")
        t[:, :, cu[-1]:] = float("nan")
    g = torch.tensor([SLOW[2], 1.0, 0.0, 0.5], device="cuda")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    pool = 0.5 * torch.randn(n + 1, H, d, d, generator=torch.Generator().manual_seed(9)).cuda()
    start, slots = pool.clone(), torch.arange(n, 0, -1, dtype=torch.int32, device="cuda")
    y = torch.full_like(q, 7.0)
    call = lambda: lib.retention_forward(q, k, v, g, y, cu_seqlens=c, states=pool, slots=slots, load_state=True,
                                         scale=0.25, feature=feature)
    assert launches(call) == 3 or cu[-1] < 4000  # (the last is cut into segments)
    grads = [torch.full_like(q, 7.0) for _ in range(3)]
    lib.retention_backward(q, k, v, g, dy, *grads, cu_seqlens=c, scale=0.25, feature=feature)
    for t in [y] + grads:
        assert (t[:, :, :cu[0]] == 7).all() and (t[:, :, cu[-1]:] == 7).all()
    assert torch.equal(pool[0], start[0])
    for i in range(n):
        lo, hi, s = cu[i], cu[i + 1], n - i
        if lo == hi:
            assert torch.equal(pool[s], start[s])
            continue
        x = [to_f64(t[0, :, lo:hi]) for t in (q, k, v)]
        args = (*x, to_f64(g), 0.25, feature, to_f64(start[s]))
        (ry, rs), (my, ms) = ro.retention(*args), ro.retention(*args, magnitude=True)
        check(y[0, :, lo:hi], ry, my, dtype, hi - lo, operands(dtype, 2), f"y of sequence {i}")
        check(pool[s], rs, ms, F32, hi - lo, 2.0 ** -16 if dtype == BF else 0.0, f"state of sequence {i}")
        args = (*x, to_f64(g), to_f64(dy[0, :, lo:hi]), 0.25, feature)
        for name, got, r, m in zip(("dq", "dk", "dv"), grads, ro.retention_backward(*args),
                                   ro.retention_backward(*args, magnitude=True)):
            check(got[0, :, lo:hi], r, m, dtype, hi - lo, operands(dtype, 2), f"{name} of sequence {i}")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("feature", ["elu1", "exp"])
def test_a_sequence_of_nan_beside_mapped_ones(feature, dtype):
    """NaN and infinities of one sequence reach no row and no state of its neighbours, mapped or not."""
    H, T, d, cu = 2, 430, 64, [0, 70, 200, 430]
    q, k, v, dy = (rand((1, H, T, d), dtype, i) for i in range(4))
    for t, x in zip((q, k, v, dy), (float("nan"), float("inf"), float("-inf"), float("nan"))):
        t[:, :, 70:200] = x
    g, c = torch.tensor([0.99, 1.0], device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")

    def run(clean):
        x = [t.clone() for t in (q, k, v, dy)]
        if clean:
            for t in x:
                t[:, :, 70:200] = 0
        y, st = torch.zeros_like(q), torch.zeros(3, H, d, d, device="cuda")
        grads = [torch.zeros_like(q) for _ in range(3)]
        lib.retention_forward(*x[:3], g, y, cu_seqlens=c, states=st, feature=feature)
        lib.retention_backward(*x[:3], g, x[3], *grads, cu_seqlens=c, feature=feature)
        return [t[:, :, lo:hi] for t in [y] + grads for lo, hi in ((0, 70), (200, 430))] + [st[0], st[2]]

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("feature", ["elu1", "relu", "exp"])
def test_gradients_of_split_sequences_with_a_feature_map(feature, d, dtype):
    """Long enough to be cut: the segments' sums of mapped operands, their transposes, and phi' at once."""
    H, N = 2, 2700
    q, k, v, dy = (rand((1, H, N, d), dtype, 20 + i) for i in range(4))
    g = torch.tensor([SLOW[2], 0.9], device="cuda")
    grads = [torch.full_like(q, 7.0) for _ in range(3)]
    call = lambda: lib.retention_backward(q, k, v, g, dy, *grads, scale=-0.25, feature=feature)
    assert launches(call) == 3
    args = [to_f64(t[0]) for t in (q, k, v)] + [to_f64(g), to_f64(dy[0]), -0.25, feature]
    for name, got, r, m in zip(("dq", "dk", "dv"), grads, ro.retention_backward(*args),
                               ro.retention_backward(*args, magnitude=True)):
        check(got[0], r, m, dtype, N, operands(dtype, 2), name)


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("feature", ["identity", "elu1", "exp"])
def test_norms_of_bf16_errors(feature, d):
    """Every head's outputs and gradients over slow decays, in the norm."""
    H, N = len(SLOW), 1500
    q, k, v, dy = (rand((1, H, N, d), BF, 40 + i) for i in range(4))
    g = torch.tensor(SLOW, device="cuda")
    y, grads = torch.empty_like(q), [torch.empty_like(q) for _ in range(3)]
    lib.retention_forward(q, k, v, g, y, scale=0.25, feature=feature)
    lib.retention_backward(q, k, v, g, dy, *grads, scale=0.25, feature=feature)
    x = [to_f64(t[0]) for t in (q, k, v)]
    refs = [ro.retention(*x, to_f64(g), 0.25, feature)[0]] + list(
        ro.retention_backward(*x, to_f64(g), to_f64(dy[0]), 0.25, feature))
    mapped = [0, 0, 0, 0] if feature == "identity" else [2, 1, 1, 2]
    for name, got, ref, n in zip(("y", "dq", "dk", "dv"), [y] + grads, refs, mapped):
        got = to_f64(got[0])
        for h in range(H):
            rel = np.linalg.norm(got[h] - ref[h]) / np.linalg.norm(ref[h])
            assert rel <= 1.1 * 2.0 ** -8 * np.sqrt((2 + n) / 3), f"{name}, decay {SLOW[h]}: {rel:.5f}"
