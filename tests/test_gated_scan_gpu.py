"""The gated scan on the GPU against the float64 oracle.

Tolerance: the oracle's rounding bound, in which every gate, product and sum is off by ``DELTA`` of its terms, plus half a
step of the output's type (bf16 2^-8, fp32 2^-24, relative).  DELTA: the exponential is within 2 steps of 2^-23, the
quotient of the sigmoid within 2 more, its sum 1 + e and the products and sums of a token's way through a thread's rows, a
warp, a block and a cluster (at most 2 of each for a token, and one of each where runs are joined: their count per
token is below 4) within half a step each: (2 + 2 + 0.5 + 8 x 0.5) 2^-23 < 2^-19.
"""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import gated_scan_oracle as go
from token_level_head_gb300.build import build_library

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DELTA = 2.0 ** -19
GATES = ["sigmoid", "log", "decay"]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()


def rand(*shape, seed, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def gate_values(shape, gate, dtype, seed):
    """Long and short memories: logits around 3."""
    t = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * 2 + 3
    t = {"sigmoid": t, "log": -torch.exp(-t), "decay": torch.exp(-torch.exp(-t))}[gate]
    return t.to(dtype).cuda()


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def check(got, ref, bound, dtype, what):
    got = to_f64(got)
    tol = (half_step(dtype) * np.abs(ref) + bound) * 1.001 + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / tol):.2f} x"


def spans(cu, B, N):
    return [(b, 0, N) for b in range(B)] if cu is None else [(0, lo, hi) for lo, hi in zip(cu, cu[1:])]


def check_forward(x, g, y, gate, cu=None, start=None, final=None, channels=None):
    """y (and the final states) against the oracle, on the first ``channels``."""
    for i, (b, lo, hi) in enumerate(spans(cu, x.shape[0], x.shape[1])):
        if lo == hi:
            continue
        s = slice(channels)
        ry, e = go.scan(to_f64(x[b, lo:hi, s]), to_f64(g[b, lo:hi, s]), gate, None if start is None else to_f64(start[i, s]), DELTA)
        check(y[b, lo:hi, s], ry, e, x.dtype, f"y of sequence {i}")
        if final is not None:
            check(final[i, s], ry[-1], e[-1], F32, f"state of sequence {i}")


def check_backward(x, g, dy, dx, dg, gate, cu=None, h0=None, dl=None, dh0=None, channels=None):
    for i, (b, lo, hi) in enumerate(spans(cu, x.shape[0], x.shape[1])):
        if lo == hi:
            if dh0 is not None:
                assert torch.equal(dh0[i], torch.zeros_like(dh0[i]) if dl is None else dl[i])
            continue
        s = slice(channels)
        ref, e = go.scan_backward(to_f64(x[b, lo:hi, s]), to_f64(g[b, lo:hi, s]), to_f64(dy[b, lo:hi, s]), gate,
                                  None if h0 is None else to_f64(h0[i, s]), None if dl is None else to_f64(dl[i, s]), DELTA)
        check(dx[b, lo:hi, s], ref[0], e[0], x.dtype, f"dx of sequence {i}")
        check(dg[b, lo:hi, s], ref[1], e[1], x.dtype, f"dg of sequence {i}")
        if dh0 is not None:
            check(dh0[i, s], ref[2], e[2], F32, f"dh0 of sequence {i}")


def kept(x):
    return torch.full((lib.gated_scan_checkpoint_rows(*x.shape[:2]), x.shape[2]), float("nan"), device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("N", [1, 2, 3, 7, 8, 63, 64, 65, 127, 128, 129, 257, 1000])
def test_lengths(N, gate, dtype):
    """Forward with states and the gradients, dense; 72 channels: one group of a block and a part of another."""
    B, D = 3, 72
    x, dy = rand(B, N, D, seed=1, dtype=dtype), rand(B, N, D, seed=2, dtype=dtype)
    g = gate_values((B, N, D), gate, dtype, 3)
    h0, dl = rand(B, D, seed=4), rand(B, D, seed=5)
    y, dx, dg = (torch.full_like(x, 7.0) for _ in range(3))
    st, ck, dh0 = h0.clone(), kept(x), torch.full_like(h0, 7.0)
    lib.gated_scan_forward(x, g, y, gate=gate, states=st, load_state=True, checkpoints=ck)
    check_forward(x, g, y, gate, start=h0, final=st)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg, gate=gate, h0=h0, dh_last=dl, dh0=dh0)
    check_backward(x, g, dy, dx, dg, gate, h0=h0, dl=dl, dh0=dh0)
    # and without states
    lib.gated_scan_forward(x, g, y, gate=gate, checkpoints=ck)
    check_forward(x, g, y, gate)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg, gate=gate)
    check_backward(x, g, dy, dx, dg, gate)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("cu", [[0, 1], [0, 1, 2, 3], [0, 0, 5, 5, 5, 200, 201, 201], [3, 60, 64, 128, 129, 400],
                                [0, 700, 1500, 1503, 3000], [10, 10]], ids=str)
def test_packed(cu, gate, dtype):
    """Packed sequences, empty ones, rows before the first and behind the last."""
    T, D, B = cu[-1] + 5, 136, len(cu) - 1
    x, dy = rand(1, T, D, seed=1, dtype=dtype), rand(1, T, D, seed=2, dtype=dtype)
    g = gate_values((1, T, D), gate, dtype, 3)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h0, dl = rand(B, D, seed=4), rand(B, D, seed=5)
    y, dx, dg = (torch.full_like(x, 7.0) for _ in range(3))
    slots = torch.randperm(B + 2, generator=torch.Generator().manual_seed(6))[:B].int().cuda()
    pool = torch.full((B + 2, D), 5.0, device="cuda")
    pool[slots.long()] = h0
    before = pool.clone()
    ck, dh0 = kept(x), torch.full_like(h0, 7.0)
    lib.gated_scan_forward(x, g, y, gate=gate, cu_seqlens=c, states=pool, slots=slots, load_state=True, checkpoints=ck)
    check_forward(x, g, y, gate, cu, start=h0, final=pool[slots.long()])
    for i in range(B):
        if cu[i] == cu[i + 1]:
            assert torch.equal(pool[slots[i].long()], h0[i])
    rest = torch.ones(B + 2, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert torch.equal(pool[rest], before[rest])
    lib.gated_scan_backward(x, g, dy, ck, dx, dg, gate=gate, cu_seqlens=c, h0=h0, dh_last=dl, dh0=dh0)
    check_backward(x, g, dy, dx, dg, gate, cu, h0, dl, dh0)
    for t in (y, dx, dg):
        assert (t[0, :cu[0]] == 7).all() and (t[0, cu[-1]:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,N,D", [(1, 9000, 64), (1, 5000, 1024), (2, 2500, 640), (40, 300, 256), (1, 20000, 8)])
def test_clusters(B, N, D, dtype):
    """One block a chain to sixteen, several rounds of tiles; a part of the channels against the oracle, all of them
    against the same channels computed alone."""
    x, dy = rand(B, N, D, seed=1, dtype=dtype), rand(B, N, D, seed=2, dtype=dtype)
    g = gate_values((B, N, D), "sigmoid", dtype, 3)
    y, dx, dg = (torch.empty_like(x) for _ in range(3))
    ck = kept(x)
    lib.gated_scan_forward(x, g, y, checkpoints=ck)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg)
    check_forward(x[:2], g[:2], y[:2], "sigmoid", channels=16)
    check_backward(x[:2], g[:2], dy[:2], dx[:2], dg[:2], "sigmoid", channels=16)
    for c in range(0, D, 128):
        s = slice(c, c + 8)
        y1, dx1, dg1 = (torch.empty(B, N, 8, dtype=dtype, device="cuda") for _ in range(3))
        ck1 = kept(y1)
        lib.gated_scan_forward(x[..., s], g[..., s], y1, checkpoints=ck1)
        lib.gated_scan_backward(x[..., s], g[..., s], dy[..., s], ck1, dx1, dg1)
        tol = 2 * half_step(dtype) + 64 * DELTA
        for a, b in ((y, y1), (dx, dx1), (dg, dg1)):
            a, b = a[..., s].float(), b.float()
            assert (a - b).abs().max() <= tol * b.abs().max()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B", [1, 5, 8, 10, 14, 15, 16, 19, 23, 29, 37, 48, 80])
def test_clusters_of_every_size(B, packed):
    """64 channels of B rows of 4500 tokens (packed: 64 B channels): chains whose clusters have from sixteen blocks down to
    one, powers of two or not, the last round of tiles short."""
    N, D = 4500, 64
    gate = GATES[B % 3]
    shape = (1, N, 64 * B) if packed else (B, N, D)
    cu = [0, 1000, 1001, 4099, N] if packed else None
    x, dy, g = rand(*shape, seed=1, dtype=BF), rand(*shape, seed=2, dtype=BF), gate_values(shape, gate, BF, 3)
    y, dx, dg = (torch.empty_like(x) for _ in range(3))
    ck, kw = kept(x), dict(gate=gate, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None)
    lib.gated_scan_forward(x, g, y, checkpoints=ck, **kw)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg, **kw)
    for s in (slice(0, 8), slice(shape[2] - 8, shape[2])):
        part = [t[-1:, :, s] for t in (x, g, y, dy, dx, dg)]
        check_forward(*part[:3], gate, cu)
        check_backward(part[0], part[1], *part[3:], gate, cu)


def test_equal_calls_give_equal_bits():
    x, g, dy = rand(1, 7000, 512, seed=1, dtype=BF), gate_values((1, 7000, 512), "sigmoid", BF, 2), rand(1, 7000, 512, seed=3, dtype=BF)
    out = []
    for _ in range(3):
        y, dx, dg = (torch.empty_like(x) for _ in range(3))
        ck = kept(x)
        lib.gated_scan_forward(x, g, y, checkpoints=ck)
        lib.gated_scan_backward(x, g, dy, ck, dx, dg)
        out.append((y, dx, dg, ck))
    for a, b in zip(out[0], out[1]):
        assert torch.equal(a, b)
    for a, b in zip(out[0], out[2]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(dtype):
    """Slices of one fused projection as inputs and outputs, a gate shared by the batch (stride 0)."""
    B, N, D = 3, 200, 64
    f = rand(B, N, 4, D, seed=1, dtype=dtype)
    g1 = gate_values((1, N, D), "sigmoid", dtype, 2)
    x, dy, g = f[:, :, 0], f[:, :, 2], g1.expand(B, N, D)
    o = torch.full((B, N, 5, D), 7.0, dtype=dtype, device="cuda")
    y, dx, dg = o[:, :, 1], o[:, :, 2], o[:, :, 4]
    ck = kept(x)
    lib.gated_scan_forward(x, g, y, checkpoints=ck)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg)
    check_forward(x, g, y, "sigmoid")
    check_backward(x, g, dy, dx, dg, "sigmoid")
    assert (o[:, :, 0] == 7).all() and (o[:, :, 3] == 7).all()
    f2 = f.clone()
    lib.gated_scan_forward(f2[:, :, 0], g, f2[:, :, 1])     # an output beside its input in one tensor
    assert torch.equal(f2[:, :, 1], y)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", GATES)
def test_steps_are_the_prompt(gate, dtype):
    """Tokens one by one on a pool of states against the oracle's recurrence from the same start."""
    B, N, D = 5, 9, 520
    x, g = rand(B, N, D, seed=1, dtype=dtype), gate_values((B, N, D), gate, dtype, 2)
    pool = rand(8, D, seed=3)
    slots = torch.tensor([6, 2, 0, 7, 3], dtype=torch.int32, device="cuda")
    h0, other = pool[slots.long()].clone(), pool[[1, 4, 5]].clone()
    y = torch.empty_like(x)
    for t in range(N):
        lib.gated_scan_step(x[:, t], g[:, t], pool, y[:, t], gate=gate, slots=slots)
    check_forward(x, g, y, gate, start=h0, final=pool[slots.long()])
    assert torch.equal(pool[[1, 4, 5]], other)
    st = h0.clone()
    lib.gated_scan_step(x[:, 0], g[:, 0], st, y[:, 0], gate=gate)          # sequence i uses slot i
    check_forward(x[:, :1], g[:, :1], y[:, :1], gate, start=h0, final=st)


def test_slots_that_are_none():
    """Out of the pool, or taken by a sequence before: from zero, no state kept; the step leaves the row out."""
    B, N, D = 5, 70, 64
    x, g = rand(B, N, D, seed=1), gate_values((B, N, D), "sigmoid", F32, 2)
    slots = torch.tensor([1, -1, 1, 3, 9], dtype=torch.int32, device="cuda")
    for cu in (None, [0, 70, 140, 210, 280, 350]):
        pool = rand(4, D, seed=3)
        was = pool.clone()
        y = torch.full_like(x, 7.0)
        if cu is None:
            lib.gated_scan_forward(x, g, y, states=pool, slots=slots, load_state=True)
        else:
            lib.gated_scan_forward(x.view(1, -1, D), g.view(1, -1, D), y.view(1, -1, D), states=pool, slots=slots, load_state=True,
                                   cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        start = torch.zeros(B, D, device="cuda")
        start[0], start[3] = was[1], was[3]
        check_forward(x, g, y, "sigmoid", start=start)
        check_forward(x[[0, 3]], g[[0, 3]], y[[0, 3]], "sigmoid", start=start[[0, 3]], final=pool[[1, 3]])
        assert torch.equal(pool[[0, 2]], was[[0, 2]])
    pool, out = was.clone(), torch.full((B, D), 7.0, device="cuda")
    lib.gated_scan_step(x[:, 0], g[:, 0], pool, out, slots=slots)
    check_forward(x[[0, 3], :1], g[[0, 3], :1], out[[0, 3]][:, None], "sigmoid", start=was[[1, 3]], final=pool[[1, 3]])
    assert (out[[1, 2, 4]] == 7).all() and torch.equal(pool[[0, 2]], was[[0, 2]])


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_a_number_stays_in_its_sequence_and_channel(gate, bad):
    """In x, g and dy of one token, and in the rows of no sequence."""
    cu, T, D = [4, 150, 300, 301, 800], 810, 72
    x, g, dy = rand(1, T, D, seed=1), gate_values((1, T, D), gate, F32, 2), rand(1, T, D, seed=3)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def run(x, g, dy):
        y, dx, dg = (torch.full_like(x, 7.0) for _ in range(3))
        ck, dh0 = kept(x), torch.empty(4, D, device="cuda")
        lib.gated_scan_forward(x, g, y, gate=gate, cu_seqlens=c, checkpoints=ck)
        lib.gated_scan_backward(x, g, dy, ck, dx, dg, gate=gate, cu_seqlens=c, dh0=dh0)
        return y, dx, dg, dh0

    clean = run(x, g, dy)
    for where in ("x", "g", "dy"):
        t = {"x": x.clone(), "g": g.clone(), "dy": dy.clone()}
        for n in t:
            t[n][0, :4] = t[n][0, 800:] = float("nan")
        t[where][0, 200, 5] = bad if where != "g" or bad != bad or gate == "sigmoid" else float("nan")
        y, dx, dg, dh0 = run(**t)
        for got, ref in zip((y, dx, dg), clean):
            ok = torch.ones(T, D, dtype=torch.bool, device="cuda")
            ok[150:300, 5] = False
            assert torch.equal(got[0][ok], ref[0][ok])
            assert not ok.all()
        ok = torch.ones(4, D, dtype=torch.bool, device="cuda")
        ok[1, 5] = False
        assert torch.equal(dh0[ok], clean[3][ok])
        assert torch.equal(y[0, 150:200, 5], clean[0][0, 150:200, 5])       # tokens before it
        if where == "x":
            assert not torch.isfinite(y[0, 200:300, 5]).any() if gate != "sigmoid" else not torch.isfinite(y[0, 200, 5])


def test_gates_at_their_ends():
    """sigmoid of -inf, -200, 200, inf and log of -inf, 0: nothing overflows to not-a-number."""
    v = torch.tensor([float("-inf"), -200.0, -50.0, 50.0, 200.0, float("inf")], device="cuda")
    x = rand(1, 6, 8, seed=1)
    y, dx, dg, dy = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), rand(1, 6, 8, seed=2)
    g, ck, h0 = v[None, :, None].expand(1, 6, 8).contiguous(), kept(x), rand(1, 8, seed=3)
    lib.gated_scan_forward(x, g, y, states=h0.clone(), load_state=True, checkpoints=ck)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg, h0=h0)
    assert torch.isfinite(torch.stack([y, dx, dg])).all()
    check_forward(x, g, y, "sigmoid", start=h0)
    check_backward(x, g, dy, dx, dg, "sigmoid", h0=h0)
    g = torch.tensor([float("-inf"), 0.0, -100.0, -1e-3, 0.0, float("-inf")], device="cuda")[None, :, None].expand(1, 6, 8).contiguous()
    lib.gated_scan_forward(x, g, y, gate="log", states=h0.clone(), load_state=True, checkpoints=ck)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg, gate="log", h0=h0)
    assert torch.isfinite(torch.stack([y, dx, dg])).all()
    check_forward(x, g, y, "log", start=h0)


def test_offsets_that_break_their_contract():
    """Out of range and out of order: no row outside the tensors is touched (guard rows stay)."""
    T, D = 300, 64
    big = torch.full((T + 200, D), 7.0, device="cuda")
    x, g, dy = rand(1, T, D, seed=1), gate_values((1, T, D), "sigmoid", F32, 2), rand(1, T, D, seed=3)
    for cu in ([-5, 100, 900, 250, 10 ** 9], [200, 100, 50], [10 ** 9, 10 ** 9 + 5], [-(10 ** 9), -5, 5]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        pool, ck = rand(len(cu) - 1, D, seed=4), kept(x)
        y = big[100:100 + T][None]
        lib.gated_scan_forward(x, g, y, cu_seqlens=c, states=pool, load_state=True, checkpoints=ck)
        assert (big[:100] == 7).all() and (big[100 + T:] == 7).all()
        lib.gated_scan_backward(x, g, dy, ck.zero_(), y, torch.empty_like(x), cu_seqlens=c, dh0=torch.empty_like(pool))
        assert (big[:100] == 7).all() and (big[100 + T:] == 7).all()
        big.fill_(7.0)


def test_captured_training_steps_and_two_streams():
    """Forward and backward captured on a side stream, replayed on new inputs, while another stream runs the same."""
    B, N, D = 2, 3000, 256
    x, g, dy = rand(B, N, D, seed=1, dtype=BF), gate_values((B, N, D), "sigmoid", BF, 2), rand(B, N, D, seed=3, dtype=BF)
    y, dx, dg = (torch.empty_like(x) for _ in range(3))
    ck = kept(x)

    def both():
        lib.gated_scan_forward(x, g, y, checkpoints=ck)
        lib.gated_scan_backward(x, g, dy, ck, dx, dg)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        both()
        with torch.cuda.graph(graph, stream=side):
            both()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (5, 6):
        x.copy_(rand(B, N, D, seed=seed, dtype=BF))
        torch.cuda.synchronize()
        y2, dx2, dg2 = (torch.empty_like(x) for _ in range(3))
        ck2 = kept(x)
        with torch.cuda.stream(side):
            graph.replay()
        lib.gated_scan_forward(x, g, y2, checkpoints=ck2)
        lib.gated_scan_backward(x, g, dy, ck2, dx2, dg2)
        torch.cuda.synchronize()
        for a, b in ((y, y2), (dx, dx2), (dg, dg2)):
            assert torch.equal(a, b)
    check_forward(x, g, y, "sigmoid", channels=8)


def test_gradients_are_the_differences():
    """fp32 calls against central differences of the calls themselves: sum(dy y) for small moves of x, g and h0."""
    B, N, D = 1, 40, 8
    x, g, dy = rand(B, N, D, seed=1), gate_values((B, N, D), "sigmoid", F32, 2), rand(B, N, D, seed=3)
    h0, dl = rand(B, D, seed=4), rand(B, D, seed=5)
    y, dx, dg, ck, dh0 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), kept(x), torch.empty_like(h0)

    def value(x, g, h0):
        st = h0.clone()
        lib.gated_scan_forward(x, g, y, states=st, load_state=True, checkpoints=ck)
        return (dy.double() * y.double()).sum() + (dl.double() * st.double()).sum()

    value(x, g, h0)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg, h0=h0, dh_last=dl, dh0=dh0)
    for k, grad in enumerate((dx, dg, dh0)):
        for seed in range(3):
            d = rand(*grad.shape, seed=10 + seed)
            lo, hi = [x, g, h0], [x, g, h0]
            step = 1e-2
            lo[k], hi[k] = lo[k] - step * d, hi[k] + step * d
            diff = (value(*hi) - value(*lo)) / (2 * step)
            # third derivatives of a sigmoid's scan: at most step^2 of the terms; fp32 values: 2^-20 of the sum / step
            terms = (grad.double() * d.double()).abs().sum()
            assert abs(diff - (grad.double() * d.double()).sum()) <= terms * (step ** 2 * 10 + 2.0 ** -20 / step)
