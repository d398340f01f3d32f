"""The gated scan on the GPU at its edges, against the float64 oracle; tolerances as in ``test_gated_scan_gpu`` where no
other is derived."""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import gated_scan_oracle as go
from test_gated_scan_gpu import BF, F32, GATES, check, check_backward, check_forward, gate_values, kept, rand
from token_level_head_gb300.build import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()


def gates_by_the_step(g, gate):
    """The gates a that the library takes for g [n]: the state of a step on h = 1, x = 0."""
    n = -(-g.numel() // 8) * 8
    wide = torch.zeros(1, n, dtype=g.dtype, device="cuda")
    wide[0, :g.numel()] = g
    states, out = torch.ones(1, n, device="cuda"), torch.empty_like(wide)
    lib.gated_scan_step(torch.zeros_like(wide), wide, states, out, gate=gate)
    return to_f64(states[0, :g.numel()])


def all_bf16(lo, hi):
    """Every bf16 number of [lo, hi]."""
    v = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(BF)
    v = v[torch.isfinite(v.float())]
    return v[(v.float() >= lo) & (v.float() <= hi)].cuda()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_small_sigmoid_gates_keep_their_digits(dtype):
    """e / (1 + e), e = exp(g), relative to itself: e is within 2 steps of 2^-23 (fp32: expf), or within 2^-22, half a step of
    |g| log2 e and the rounding of log2 e, 2^-26 of itself (bf16); 1 + e half a step and the share of e's; its reciprocal and the product 1.5 steps more;
    the product with h none (h = 1).  Gates below 2^-126 may be zero."""
    g = torch.linspace(-87.0, 20.0, 60000, device="cuda") if dtype == F32 else all_bf16(-87.0, 20.0)
    a, ref = gates_by_the_step(g, "sigmoid"), 1 / (1 + np.exp(-to_f64(g)))
    exp_off = 2 * 2.0 ** -23 if dtype == F32 else 2.0 ** -22 + np.abs(to_f64(g)) * (2.0 ** -24 + 2.0 ** -26)
    assert (np.abs(a - ref) <= ref * (2 * exp_off + 2 * 2.0 ** -23) * 1.001 + 2.0 ** -126).all(), np.max(np.abs(a - ref) / ref)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("packed", [False, True])
def test_states_through_small_sigmoid_gates(packed, dtype):
    """Tokens without an input (x = 0, padding) and gates from 1/4 to e^-30 (bf16: e^-12): y and the state are the start times the
    gates, with their digits.  bf16: a gate is off by |g| 2^-24 + 2^-22 + 4 2^-23 < 2^-19 for |g| <= 12."""
    B, N, D = 3, 6, 64
    x = torch.zeros(B, N, D, dtype=dtype, device="cuda")
    g = -(1 + torch.rand(B, N, D, generator=torch.Generator().manual_seed(1)) * (29 if dtype == F32 else 11)).to(dtype).cuda()
    g[:, 3:] = 8.0                                     # and then kept
    h0, dl, dy = rand(B, D, seed=2), rand(B, D, seed=3), torch.zeros_like(x)
    y, dx, dg, st, dh0, kw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), h0.clone(), torch.empty_like(h0), {}
    t = [x, g, y, dy, dx, dg]
    if packed:
        t, kw = [a.view(1, -1, D) for a in t], dict(cu_seqlens=torch.arange(B + 1, dtype=torch.int32, device="cuda") * N)
    ck = kept(t[0])
    lib.gated_scan_forward(*t[:3], states=st, load_state=True, checkpoints=ck, **kw)
    check_forward(x, g, y, "sigmoid", start=h0, final=st)
    lib.gated_scan_backward(t[0], t[1], t[3], ck, *t[4:], h0=h0, dh_last=dl, dh0=dh0, **kw)
    check_backward(x, g, dy, dx, dg, "sigmoid", h0=h0, dl=dl, dh0=dh0)


def test_bf16_log_gates():
    """exp(g), relative to itself: the hardware's base-2 exponential is within 2^-22; half a step of |g| log2 e, and the rounding of
    log2 e (1.44269502 for 1.44269504, 0.9 2^-26 of itself).  Half a bf16 step of g is |g| 2^-9."""
    g = all_bf16(-87.0, 0.0)
    a, ref, size = gates_by_the_step(g, "log"), np.exp(to_f64(g)), np.abs(to_f64(g))
    tol = 2.0 ** -22 + size * (2.0 ** -24 + 2.0 ** -26)
    off = np.abs(a - ref) / ref
    assert (off <= tol * 1.001 + 2.0 ** -126 / ref).all(), (off / tol).max()


@pytest.mark.parametrize("rate", [-2.0 ** -10, -1e-4, -1e-5])
def test_long_memories_of_constant_log_gates(rate):
    """65,536 tokens of one bf16 gate near 1: the last state in 32 bits.  A token costs the state the gate's rounding (2^-25) and a
    product's or sum's (2^-24), and an eighth of those where runs of sixteen tokens are joined: below the oracle's 2 x 2^-24."""
    N, D = 65536, 64
    g = torch.full((1, N, D), rate, device="cuda").to(BF)
    x, y, st = rand(1, N, D, seed=1, dtype=BF) + 1, torch.empty(1, N, D, dtype=BF, device="cuda"), torch.empty(1, D, device="cuda")
    lib.gated_scan_forward(x, g, y, gate="log", states=st)
    s = slice(0, 64, 9)
    ref, e = go.scan(to_f64(x[0, :, s]), to_f64(g[0, :, s]), "log", None, 2.0 ** -24)
    check(st[0, s], ref[-1], e[-1], F32, "last state")


def test_no_gate_undoes_the_cut_between_sequences():
    """Decays of 0 and -0 behind a sequence's first token; not-a-number in the sequence before stays there."""
    T, D, cu = 300, 16, [0, 100, 300]
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for zeros in ([0.0], [-0.0], [-0.0, -0.0], [-0.0, 0.0, -0.0], [-0.0] * 3 + [0.5]):
        for dtype in (F32, BF):
            x, dy = rand(1, T, D, seed=1, dtype=dtype), rand(1, T, D, seed=2, dtype=dtype)
            g = gate_values((1, T, D), "decay", dtype, 3)
            g[0, 101:101 + len(zeros)] = torch.tensor(zeros, device="cuda")[:, None].to(dtype)
            g[0, 199:199 + len(zeros)] = torch.tensor(zeros, device="cuda")[:, None].to(dtype)
            x[0, 5], dy[0, 295] = float("nan"), 0.0
            y, dx, dg, ck = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), kept(x)
            lib.gated_scan_forward(x, g, y, gate="decay", cu_seqlens=c, checkpoints=ck)
            lib.gated_scan_backward(x, g, dy, ck, dx, dg, gate="decay", cu_seqlens=c)
            assert torch.isnan(y[0, 5:100]).all() and torch.isfinite(y[0, 100:]).all() and torch.isfinite(dg[0, 100:]).all()
            check_forward(x[:, 100:], g[:, 100:], y[:, 100:], "decay")
            check_backward(x[:, 100:], g[:, 100:], dy[:, 100:], dx[:, 100:], dg[:, 100:], "decay")
            # and backwards: not-a-number in the later sequence's gradients
            x[0, 5], dy[0, 200] = 0.0, float("nan")
            g[0, 95:95 + len(zeros)] = torch.tensor(zeros, device="cuda")[:, None].to(dtype)[:5]
            lib.gated_scan_forward(x, g, y, gate="decay", cu_seqlens=c, checkpoints=ck)
            lib.gated_scan_backward(x, g, dy, ck, dx, dg, gate="decay", cu_seqlens=c)
            check_backward(x[:, :100], g[:, :100], dy[:, :100], dx[:, :100], dg[:, :100], "decay")


def long_gates(shape, gate, dtype, seed):
    """Memories of some thousands of tokens: logits from 8 to 11, and every eighth channel 20 (a sequence's start stays to its end)."""
    t = 8 + 3 * torch.rand(*shape, generator=torch.Generator().manual_seed(seed))
    t[..., ::8] = 20.0
    t = {"sigmoid": t, "log": -torch.exp(-t), "decay": torch.exp(-torch.exp(-t))}[gate]
    return t.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("B,D,cu", [(1, 64, None), (2, 640, None), (15, 64, None), (23, 64, None), (80, 64, None),
                                    (1, 64, [0, 2000, 9001]), (1, 1024, [0, 1, 4500, 9001]), (1, 2048, [3, 8000, 8000, 9001])], ids=str)
def test_long_memories_across_tiles_and_clusters(B, D, cu, gate, dtype):
    """States and gradients that reach over tiles, warps, the blocks of a cluster and its rounds, from starts and ends that are not
    zero: they make up a visible part of the last state, of dh0 and of every row between."""
    N = 9001 if cu else 4500
    n = len(cu) - 1 if cu else B
    x, dy, g = rand(B, N, D, seed=1, dtype=dtype), rand(B, N, D, seed=2, dtype=dtype), long_gates((B, N, D), gate, dtype, 3)
    h0, dl = 100 * rand(n, D, seed=4), 100 * rand(n, D, seed=5)
    if gate == "sigmoid":
        x = x * 3 + 2
    y, dx, dg, st, dh0, ck = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), h0.clone(), torch.empty_like(h0), kept(x)
    kw = dict(gate=gate, cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"))
    lib.gated_scan_forward(x, g, y, states=st, load_state=True, checkpoints=ck, **kw)
    lib.gated_scan_backward(x, g, dy, ck, dx, dg, h0=h0, dh_last=dl, dh0=dh0, **kw)
    for s in (slice(0, 10), slice(D - 6, D)):
        rows = slice(max(0, B - 2), B)
        part = [t[rows, :, s] for t in (x, g, y, dy, dx, dg)]
        ends = [t[slice(max(0, n - 2), n) if cu is None else slice(None), s] for t in (h0, st, dl, dh0)]
        check_forward(*part[:3], gate, cu, start=ends[0], final=ends[1])
        check_backward(part[0], part[1], *part[3:], gate, cu, ends[0], ends[2], ends[3])


def owners(slots, n):
    """For each sequence its slot, -1 where that is out of the pool or a sequence before it has it."""
    seen, out = set(), []
    for s in slots:
        out.append(s if 0 <= s < n and s not in seen else -1)
        seen.add(s)
    return out


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("length,D", [(1, 64), (5, 192), (16, 1024), (1, 16)])
def test_thousands_of_packed_sequences_on_a_pool(length, D, dtype):
    """Slots of 3000 short sequences, some twice, some out of the pool, some with no token: states in and out."""
    B, pool_rows = 3000, 3500
    gen = torch.Generator().manual_seed(1)
    slots = torch.randperm(pool_rows + 200, generator=gen)[:B] - 100
    again = torch.randint(0, B, (300,), generator=gen)
    slots[again] = slots[torch.randint(0, B, (300,), generator=gen)]
    lens = torch.full((B,), length)
    lens[::7] = torch.randint(0, 2 * length + 1, (len(lens[::7]),), generator=gen)
    cu = torch.nn.functional.pad(torch.cumsum(lens, 0), (1, 0))
    T = int(cu[-1])
    x, g = rand(1, T, D, seed=1, dtype=dtype), gate_values((1, T, D), "sigmoid", dtype, 2)
    pool = rand(pool_rows, D, seed=3)
    was, y = pool.clone(), torch.empty_like(x)
    lib.gated_scan_forward(x, g, y, cu_seqlens=cu.int().cuda(), states=pool, slots=slots.int().cuda(), load_state=True)
    own = owners(slots.tolist(), pool_rows)
    start = torch.zeros(B, D, device="cuda")
    has = torch.tensor([s >= 0 for s in own]).cuda()
    start[has] = was[torch.tensor([s for s in own if s >= 0]).cuda()]
    alone, y2 = start.clone(), torch.empty_like(x)
    lib.gated_scan_forward(x, g, y2, cu_seqlens=cu.int().cuda(), states=alone, load_state=True)   # sequence i on slot i
    assert torch.equal(y, y2)
    want = was.clone()
    want[torch.tensor([s for s in own if s >= 0]).cuda()] = alone[has]
    assert torch.equal(pool, want)
    some = slice(0, 200)
    check_forward(x[:, :int(cu[200])], g[:, :int(cu[200])], y[:, :int(cu[200])], "sigmoid", cu[:201].tolist(), start=start[some],
                  final=alone[some], channels=8)


def us(fn, n=20):
    for _ in range(3):
        fn()
    best = 1e9
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            fn()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / n)
    return best


@pytest.mark.parametrize("packed", [True, False])
def test_the_search_for_slots_costs_little(packed):
    """Slots given or not: 4096 packed sequences of 16 tokens, and a dense batch of 1024 rows."""
    B, N, D = (1, 65536, 256) if packed else (1024, 64, 256)
    n = 4096 if packed else B
    x, g = rand(B, N, D, seed=1, dtype=BF), gate_values((B, N, D), "sigmoid", BF, 2)
    y, pool = torch.empty_like(x), rand(n, D, seed=3)
    kw = dict(cu_seqlens=torch.arange(0, N + 1, 16, dtype=torch.int32, device="cuda")) if packed else {}
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(4)).int().cuda()
    without = us(lambda: lib.gated_scan_forward(x, g, y, states=pool, load_state=True, **kw))
    given = us(lambda: lib.gated_scan_forward(x, g, y, states=pool, slots=slots, load_state=True, **kw))
    print(f"{'packed' if packed else 'dense'}: {without:.1f} us without slots, {given:.1f} with")
    assert given <= 2 * without + 10, (given, without)


def test_offsets_that_break_their_contract_on_a_pool():
    """Out of range and out of order, with slots, some twice and some out of the pool: nothing beside the tensors and the pool is touched."""
    T, D = 600, 64
    big, pools = torch.full((T + 200, D), 7.0, device="cuda"), torch.full((20, D), 5.0, device="cuda")
    x, g = rand(1, T, D, seed=1), gate_values((1, T, D), "sigmoid", F32, 2)
    for cu in ([-5, 100, 900, 250, 10 ** 9], [500, 200, 100, 50, 400, 0], [10 ** 9, 10 ** 9 + 5, 3], [-(10 ** 9), -5, 5, 4, 3, 599]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        slots = torch.tensor([2, 3, 2, -(1 << 31), (1 << 31) - 1][:len(cu) - 1], dtype=torch.int32, device="cuda")
        lib.gated_scan_forward(x, g, big[100:100 + T][None], cu_seqlens=c, states=pools[8:12], slots=slots, load_state=True)
        assert (big[:100] == 7).all() and (big[100 + T:] == 7).all() and (pools[:8] == 5).all() and (pools[12:] == 5).all()
        big.fill_(7.0)
        pools.fill_(5.0)
