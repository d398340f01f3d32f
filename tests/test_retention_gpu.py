"""The retention operators on the GPU against the float64 oracle.

Tolerances, with u = half a step of the output's type (bf16 2^-8, fp32 2^-24), elementwise, relative
to ``mag``, the oracle's sum of the terms' absolute values:
  * sums in 32 bits: n 2^-24 mag for a sum of n rounded terms; a sum here runs over d products, at most
    64 tokens of a chunk at a time and one term a chunk: n <= 128 + 128 + N / 64 + 16.
  * decays: gamma^n from a base-2 exponential, relative error at most 2^-18 where it is above 2^-32.
  * bf16 calls round the result (u |ref|) and, on the tensor cores, operands: the decayed scores or the
    state (2^-8 of a term), the decayed key where no fp32 state is asked for (2^-8), phi of each operand
    that has a feature map (2^-8 each, at most three).
  * fp32 states of bf16 calls carry the decayed key as the sum of two bf16 numbers: 2^-16 of a term.
The feature maps' exponentials add at most 2^-21 of a term each.
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
GAMMAS = [1.0, 1 - 2.0 ** -9, 0.0, 0.5, 1 - 2.0 ** -5]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()


def gammas(H):
    return torch.tensor([GAMMAS[i % len(GAMMAS)] for i in range(H)], dtype=F32, device="cuda")


def rand(shape, dtype, seed, layout="bhnd"):
    """[B, H, N, d] of N(0, 1) in the layout's storage."""
    B, H, N, d = shape
    g = torch.Generator().manual_seed(seed)
    if layout == "bhnd":
        return torch.randn(B, H, N, d, generator=g).to(dtype).cuda()
    if layout == "bnhd":
        return torch.randn(B, N, H, d, generator=g).to(dtype).cuda().transpose(1, 2)
    assert layout == "slice"  # of a fused [B, N, 3, H, d] projection
    return torch.randn(B, N, 3, H, d, generator=g).to(dtype).cuda()[:, :, 1].transpose(1, 2)


def tol_sum(N):
    return (128 + 128 + N / 64 + 16) * 2.0 ** -24 + 2.0 ** -18


def rounded(dtype, feature, roles):
    """Rounded operands of a term, in units of 2^-8: `roles` counts those that have a feature map."""
    if dtype == F32:
        return 0.0
    return (2.0 + (0 if feature == "identity" else roles)) * 2.0 ** -8 * 1.02


def check(got, ref, mag, dtype, N, extra, what):
    got = to_f64(got)
    u = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    tol = u * np.abs(ref) + (tol_sum(N) + extra) * mag + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / tol):.2f} x"


def ranges(cu, B, N):
    return [(b, 0, N) for b in range(B)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def check_forward(q, k, v, g, y, scale, feature, cu=None, start=None, final=None):
    """y (and `final` states, in the order of the sequences) against the oracle; `start` likewise."""
    dt, N = q.dtype, q.shape[2]
    for i, (b, lo, hi) in enumerate(ranges(cu, q.shape[0], N)):
        if lo == hi:
            continue
        x = [to_f64(t[b, :, lo:hi]) for t in (q, k, v)]
        s0 = None if start is None else to_f64(start[i])
        gn = to_f64(g)
        ry, rs = ro.retention(*x, gn, scale, feature, s0)
        my, ms = ro.retention(*x, gn, scale, feature, s0, magnitude=True)
        check(y[b, :, lo:hi], ry, my, dt, hi - lo, rounded(dt, feature, 2), f"y of sequence {i}")
        if final is not None:
            check(final[i], rs, ms, F32, hi - lo, 2.0 ** -16 * 1.02 if dt == BF else 0.0, f"state of sequence {i}")


LENGTHS = [1, 2, 63, 64, 65, 127, 128, 129, 300, 777]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("N", LENGTHS)
def test_forward_lengths(N, d, dtype):
    B, H = 2, 5
    q, k, v = (rand((B, H, N, d), dtype, 10 * N + i) for i in range(3))
    g, y = gammas(H), torch.full((B, H, N, d), 7.0, dtype=dtype, device="cuda")
    st = rand((B, H, d, d), F32, 9)
    start = st.clone()
    lib.retention_forward(q, k, v, g, y, states=st, load_state=True, scale=d ** -0.5)
    check_forward(q, k, v, g, y, d ** -0.5, "identity", start=start, final=st)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("feature", ["identity", "elu1", "relu", "exp"])
@pytest.mark.parametrize("states", [False, True])
def test_forward_features(feature, states, dtype):
    B, H, N, d = 1, 5, 260, 64
    q, k, v = (0.5 * rand((B, H, N, d), dtype, i) for i in range(3))
    g, y = gammas(H), torch.empty(B, H, N, d, dtype=dtype, device="cuda")
    st = torch.full((B, H, d, d), 3.0, device="cuda") if states else None   # not loaded, so overwritten
    lib.retention_forward(q, k, v, g, y, states=st, feature=feature, scale=-0.25)
    check_forward(q, k, v, g, y, -0.25, feature, final=st)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd", "slice"])
def test_forward_layouts(layout, d, dtype):
    B, H, N = 2, 3, 190
    q, k, v, y = (rand((B, H, N, d), dtype, i, layout) for i in range(4))
    lib.retention_forward(q, k, v, gammas(H), y)
    check_forward(q, k, v, gammas(H), y, 1.0, "identity")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_inputs_shared_by_heads_and_batch(dtype):
    """Keys of one head for all (stride 0), values of one batch entry for all."""
    B, H, N, d = 3, 4, 150, 64
    q, y = rand((B, H, N, d), dtype, 1), torch.empty(B, H, N, d, dtype=dtype, device="cuda")
    k = rand((B, 1, N, d), dtype, 2).expand(B, H, N, d)
    v = rand((1, H, N, d), dtype, 3).expand(B, H, N, d)
    lib.retention_forward(q, k, v, gammas(H), y)
    check_forward(q, k, v, gammas(H), y, 1.0, "identity")
    dy = rand((B, H, N, d), dtype, 4)
    grads = [torch.empty_like(q) for _ in range(3)]
    lib.retention_backward(q, k, v, gammas(H), dy, *grads)
    check_backward(q, k, v, gammas(H), dy, grads, 1.0, "identity")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,N,d", [(1, 9000, 64), (2, 5000, 128), (3, 2600, 16)])
def test_forward_long_sequences_are_split(H, N, d, dtype):
    q, k, v = (rand((1, H, N, d), dtype, i) for i in range(3))
    g = torch.tensor([1 - 2.0 ** -11, 1.0, 0.9], device="cuda")[:H].contiguous()
    y, st = torch.empty_like(q), rand((1, H, d, d), F32, 5)
    start = st.clone()
    lib.retention_forward(q, k, v, g, y, states=st, load_state=True, scale=0.1)
    check_forward(q, k, v, g, y, 0.1, "identity", start=start, final=st)
    again = torch.empty_like(y)
    st2 = start.clone()
    lib.retention_forward(q, k, v, g, again, states=st2, load_state=True, scale=0.1)
    assert torch.equal(y, again) and torch.equal(st, st2)


PACKED = [[0, 0, 1, 130, 130, 258, 700, 701, 701], [5, 5, 6, 600], [0, 1], [3, 200, 328, 333]]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cu", PACKED)
def test_packed_sequences(cu, d, dtype):
    """Empty sequences, rows before the first and behind the last sequence (NaN there) left as they were,
    a pool larger than the batch."""
    H, T, n = 5, 720, len(cu) - 1
    q, k, v, y = (rand((1, H, T, d), dtype, i, "bnhd") for i in range(4))
    for t in (q, k, v):
        t[:, :, :cu[0]] = float("nan")
        t[:, :, cu[-1]:] = float("nan")
    before = y.clone()
    pool = rand((n + 3, H, d, d), F32, 6)
    start = pool.clone()
    slots = torch.arange(n + 3)[torch.randperm(n + 3, generator=torch.Generator().manual_seed(n))][:n].int().cuda()
    lib.retention_forward(q, k, v, gammas(H), y, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                          states=pool, slots=slots, load_state=True, scale=0.3)
    ids = slots.long()
    check_forward(q, k, v, gammas(H), y, 0.3, "identity", cu, start[ids], pool[ids])
    assert torch.equal(y[:, :, :cu[0]], before[:, :, :cu[0]]) and torch.equal(y[:, :, cu[-1]:], before[:, :, cu[-1]:])
    for i in range(n):
        if cu[i] == cu[i + 1]:
            assert torch.equal(pool[ids[i]], start[ids[i]])
    rest = [i for i in range(n + 3) if i not in ids.tolist()]
    assert torch.equal(pool[rest], start[rest])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_not_a_number_stays_in_its_sequence(dtype):
    """A sequence of NaN and infinities beside others whose tiles reach into it."""
    H, T, d = 2, 500, 64
    cu = [0, 70, 200, 340, 500]
    q, k, v = (rand((1, H, T, d), dtype, i) for i in range(3))
    for t, x in zip((q, k, v), (float("nan"), float("inf"), float("-inf"))):
        t[:, :, 70:200] = x
    dy = rand((1, H, T, d), dtype, 8)
    y, g = torch.empty_like(q), gammas(H)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    lib.retention_forward(q, k, v, g, y, cu_seqlens=c)
    grads = [torch.empty_like(q) for _ in range(3)]
    lib.retention_backward(q, k, v, g, dy, *grads, cu_seqlens=c)
    clean = [t.clone() for t in (q, k, v)]
    for t in clean:
        t[:, :, 70:200] = 0
    y0, grads0 = torch.empty_like(q), [torch.empty_like(q) for _ in range(3)]
    lib.retention_forward(*clean, g, y0, cu_seqlens=c)
    lib.retention_backward(*clean, g, dy, *grads0, cu_seqlens=c)
    keep = torch.ones(T, dtype=torch.bool)
    keep[70:200] = False
    for a, b in zip([y] + grads, [y0] + grads0):
        assert torch.equal(a[:, :, keep], b[:, :, keep])
        assert torch.isfinite(a[:, :, keep].float()).all()


def test_slots_without_a_state():
    """Slots out of range and repeated ones: the sequence starts from zero and leaves the pool alone."""
    B, H, N, d = 5, 2, 140, 64
    q, k, v = (rand((B, H, N, d), BF, i) for i in range(3))
    pool, y = rand((4, H, d, d), F32, 3), torch.empty(B, H, N, d, dtype=BF, device="cuda")
    start = pool.clone()
    slots = torch.tensor([2, -1, 4, 2, 0], dtype=torch.int32, device="cuda")
    lib.retention_forward(q, k, v, gammas(H), y, states=pool, slots=slots, load_state=True)
    zero = torch.zeros_like(start[0])
    check_forward(q, k, v, gammas(H), y, 1.0, "identity", start=[start[2], zero, zero, zero, start[0]])
    assert torch.equal(pool[[1, 3]], start[[1, 3]])
    check_forward(q[:1], k[:1], v[:1], gammas(H), y[:1], 1.0, "identity", start=[start[2]], final=[pool[2]])


def check_backward(q, k, v, g, dy, grads, scale, feature, cu=None):
    dt = q.dtype
    for i, (b, lo, hi) in enumerate(ranges(cu, q.shape[0], q.shape[2])):
        if lo == hi:
            continue
        x = [to_f64(t[b, :, lo:hi]) for t in (q, k, v)]
        args = (to_f64(g), to_f64(dy[b, :, lo:hi]), scale, feature)
        ref, mag = ro.retention_backward(*x, *args), ro.retention_backward(*x, *args, magnitude=True)
        for name, got, r, m in zip(("dq", "dk", "dv"), grads, ref, mag):
            check(got[b, :, lo:hi], r, m, dt, hi - lo, rounded(dt, feature, 2), f"{name} of sequence {i}")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("N", [1, 64, 127, 129, 777])
def test_backward_lengths(N, d, dtype):
    B, H = 2, 5
    q, k, v, dy = (rand((B, H, N, d), dtype, 10 * N + i) for i in range(4))
    grads = [torch.full_like(q, 5.0) for _ in range(3)]
    lib.retention_backward(q, k, v, gammas(H), dy, *grads, scale=d ** -0.5)
    check_backward(q, k, v, gammas(H), dy, grads, d ** -0.5, "identity")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("feature", ["elu1", "relu", "exp"])
def test_backward_features(feature, d, dtype):
    q, k, v, dy = (0.5 * rand((1, 5, 260, d), dtype, i, "bnhd") for i in range(4))
    q[0, 0, 3, :5] = 0.0   # the corner: phi'(0) = 0 for ReLU, 1 for the others
    grads = [torch.empty_like(q) for _ in range(3)]
    lib.retention_backward(q, k, v, gammas(5), dy, *grads, scale=-0.25, feature=feature)
    check_backward(q, k, v, gammas(5), dy, grads, -0.25, feature)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("cu", PACKED + [[0, 5000, 5001, 9000]])
def test_backward_packed(cu, dtype):
    H, T, d = 3, max(720, cu[-1] + 7), 64
    q, k, v, dy = (rand((1, H, T, d), dtype, i, "slice") for i in range(4))
    fused = torch.full((1, T, 3, H, d), 2.0, dtype=dtype, device="cuda")  # the gradient of a fused projection
    grads = [fused[:, :, i].transpose(1, 2) for i in range(3)]
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    g = torch.tensor([1 - 2.0 ** -10, 0.97, 1.0], device="cuda")
    lib.retention_backward(q, k, v, g, dy, *grads, cu_seqlens=c, scale=0.2)
    check_backward(q, k, v, g, dy, grads, 0.2, "identity", cu)
    assert (fused[:, :cu[0]] == 2).all() and (fused[:, cu[-1]:] == 2).all()


def test_offsets_out_of_order_stay_in_bounds():
    """The host does not read cu_seqlens: whatever it holds, guards around the outputs and states are intact."""
    H, T, d = 2, 300, 64
    q, k, v, dy = (rand((1, H, T, d), BF, i) for i in range(4))
    for cu in ([0, 400, 100, 300], [-5, 20, 7, 1 << 30], [300, 0, 300, 0], [0, 300, 0, 300, 0, 300]):
        guard = torch.full((H * T * d * 3,), 9.0, dtype=BF, device="cuda")
        y = guard[H * T * d:2 * H * T * d].view(1, H, T, d)
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        lib.retention_forward(q, k, v, gammas(H), y, cu_seqlens=c)
        lib.retention_backward(q, k, v, gammas(H), dy, y, torch.empty_like(q), torch.empty_like(q), cu_seqlens=c)
        torch.cuda.synchronize()
        assert (guard[:H * T * d] == 9).all() and (guard[2 * H * T * d:] == 9).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (70, 4)])
def test_step(B, H, d, dtype):
    pool = rand((B + 3, H, d, d), F32, 1)
    start = pool.clone()
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(B))[:B].int().cuda()
    x = torch.randn(B, 3, H, d, generator=torch.Generator().manual_seed(d)).to(dtype).cuda()
    q, k, v = x.unbind(1)
    out, g = torch.empty(B, H, d, dtype=dtype, device="cuda"), gammas(H)
    lib.retention_step(q, k, v, g, pool, out, slots=slots, scale=0.2, feature="elu1")
    ids = slots.long()
    for b in range(B):
        args = [to_f64(t[b])[:, None] for t in (q, k, v)] + [to_f64(g), 0.2, "elu1", to_f64(start[ids[b]])]
        (ry, rs), (my, ms) = ro.retention(*args), ro.retention(*args, magnitude=True)
        check(out[b][:, None], ry, my, dtype, 1, 0.0, "out")   # no operand is rounded
        check(pool[ids[b]], rs, ms, F32, 1, 0.0, "state")
    rest = [i for i in range(B + 3) if i not in ids.tolist()]
    assert torch.equal(pool[rest], start[rest])


def test_step_leaves_rows_without_a_slot_alone():
    B, H, d = 6, 2, 64
    q, k, v = (rand((B, H, 1, d), BF, i)[:, :, 0] for i in range(3))
    pool, out = rand((4, H, d, d), F32, 3), torch.full((B, H, d), 7.0, dtype=BF, device="cuda")
    start = pool.clone()
    lib.retention_step(q, k, v, gammas(H), pool, out,
                       slots=torch.tensor([1, -1, 4, 1, 0, -2 ** 31], dtype=torch.int32, device="cuda"))
    assert (out[[1, 2, 3, 5]] == 7).all() and torch.equal(pool[[2, 3]], start[[2, 3]])
    ref, want = start.clone()[[1, 0]].contiguous(), torch.empty(2, H, d, dtype=BF, device="cuda")
    lib.retention_step(q[[0, 4]], k[[0, 4]], v[[0, 4]], gammas(H), ref, want)
    assert torch.equal(out[[0, 4]], want) and torch.equal(pool[[1, 0]], ref)


def test_step_without_slots_and_a_short_pool():
    """slots None: row b uses state b; rows behind the pool are left out."""
    B, H, d = 4, 3, 32
    q, k, v = (rand((B, H, 1, d), F32, i)[:, :, 0] for i in range(3))
    pool, out = rand((2, H, d, d), F32, 3), torch.full((B, H, d), 7.0, device="cuda")
    lib.retention_step(q, k, v, gammas(H), pool, out)
    assert (out[2:] == 7).all() and not (out[:2] == 7).any()


def copied(pool, src, dst):
    new = pool.clone()
    for s, t in zip(src, dst):
        if s < pool.shape[0] and 0 <= t < pool.shape[0]:
            new[t] = pool[s] if s >= 0 else 0
    return new


@pytest.mark.parametrize("H,d", [(1, 16), (3, 32), (5, 64), (2, 128)])
def test_copy_states(H, d):
    n = 11
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(d)).tolist()
    for src, dst in [
        ([4] * 6, [0, 1, 2, 3, 5, 4]),                      # fork, onto itself too
        (perm, list(range(n))),                             # a permutation: every slot source and target
        ([1, 0], [0, 1]),                                   # exchange
        ([9, 10, -1, -1], [0, 1, 9, 10]),                   # compact, then clear what was moved
        ([-1], [3]),
        ([2, 5, -7, 0, 11, 3], [6, 6, 8, 11, 2, -1]),       # one target twice, pairs out of range
        ([1, 2, 99], [4, 4, 4]),                            # the last valid one of three counts
    ]:
        pool = rand((n, H, d, d), F32, 1)
        want = copied(pool, src, dst)
        lib.retention_copy_states(pool, *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (src, dst)))
        assert torch.equal(pool, want), (src, dst)


@pytest.mark.parametrize("n", [255, 256, 257, 1024])
def test_copy_many_states(n):
    pool = torch.randn(1030, 1, 32, 32, generator=torch.Generator().manual_seed(n)).cuda()
    g = torch.Generator().manual_seed(n + 1)
    src, dst = torch.randint(-3, 1033, (n,), generator=g).int(), torch.randint(-3, 1033, (n,), generator=g).int()
    want = copied(pool, src.tolist(), dst.tolist())
    lib.retention_copy_states(pool, src.cuda(), dst.cuda())
    assert torch.equal(pool, want)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_request_from_prompt_to_parallel_samples(dtype):
    """As a server uses them: a prompt in two packed calls, its state forked to three samples, single
    tokens for all, then the finished slots compacted and one cleared: the outputs are those of the
    uninterrupted sequences."""
    H, d, P1, P2, T = 3, 64, 150, 77, 5
    g = gammas(H)
    tok = [rand((1, H, P1 + P2, d), dtype, i) for i in range(3)]
    new = [rand((3, H, T, d), dtype, 20 + i) for i in range(3)]
    pool = rand((6, H, d, d), F32, 7)
    y = torch.empty_like(tok[0])
    lib.retention_copy_states(pool, *(torch.tensor([x], dtype=torch.int32, device="cuda") for x in (-1, 4)))
    slot = torch.tensor([4], dtype=torch.int32, device="cuda")
    for lo, hi in ((0, P1), (P1, P1 + P2)):
        c = torch.tensor([lo, hi], dtype=torch.int32, device="cuda")
        lib.retention_forward(*tok, g, y, cu_seqlens=c, states=pool, slots=slot, load_state=True, scale=0.2)
    check_forward(*tok, g, y, 0.2, "identity", final=pool[4:5])
    lib.retention_copy_states(pool, torch.tensor([4, 4], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    slots = torch.tensor([2, 4, 0], dtype=torch.int32, device="cuda")
    out = torch.empty_like(new[0])
    for t in range(T):
        lib.retention_step(*(x[:, :, t] for x in new), g, pool, out[:, :, t], slots=slots, scale=0.2)
    whole = [torch.cat([a.expand(3, -1, -1, -1), b], 2) for a, b in zip(tok, new)]
    ref = [ro.retention(*(to_f64(x[b]) for x in whole), to_f64(g), 0.2) for b in range(3)]
    mag = [ro.retention(*(to_f64(x[b]) for x in whole), to_f64(g), 0.2, magnitude=True) for b in range(3)]
    sx = 2.0 ** -16 * 1.02 if dtype == BF else 0.0
    for b, s in enumerate([2, 4, 0]):
        check(out[b], ref[b][0][:, -T:], mag[b][0][:, -T:], dtype, 300, sx, "out")
        check(pool[s], ref[b][1], mag[b][1], F32, 300, sx, "state")
    kept = pool[[2, 0]].clone()
    lib.retention_copy_states(pool, torch.tensor([2, 0, -1], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool[:2], kept) and (pool[4] == 0).all()


@pytest.mark.parametrize("gamma", [1.0, 0.99])
def test_one_decay_equals_the_causal_forward_without_normaliser(gamma):
    """The library's scalar decay (fp32) is this operator with the same gamma in every head."""
    B, H, N, d = 2, 3, 384, 64
    q, k, v = (0.3 * rand((B, H, N, d), F32, i) for i in range(3))
    want, y = torch.empty_like(q), torch.empty_like(q)
    lib.mhla_forward_ex(q, k, v, None, want, 128, causal=1, normalise=False, gamma=gamma)
    lib.retention_forward(q, k, v, torch.full((H,), gamma, device="cuda"), y, feature="elu1")
    for b in range(B):
        mag = ro.retention(*(to_f64(x[b]) for x in (q, k, v)), [gamma] * H, 1.0, "elu1", magnitude=True)[0]
        assert (np.abs(to_f64(y[b]) - to_f64(want[b])) <= 2 * tol_sum(N) * mag).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_streams_workspaces_and_graphs(dtype):
    """A call on another stream; one workspace for calls of different sizes; captured calls replayed on new
    inputs, two graphs with a workspace each."""
    H, d = 4, 64
    g = gammas(H)
    need = max(lib.retention_workspace_bytes(1, H, 9000, d, backward=True), lib.retention_workspace_bytes(3, H, 600, d))
    ws = [lib.new_workspace(need, "cuda") for _ in range(2)]
    x = [rand((1, H, 9000, d), dtype, i) for i in range(4)]
    small = [t[:, :, :600].reshape(1, H, 3, 200, d)[0].transpose(0, 1).contiguous() for t in x]
    y, ys = torch.empty_like(x[0]), torch.empty_like(small[0])
    grads = [torch.empty_like(x[0]) for _ in range(3)]

    def calls(w):
        lib.retention_forward(*x[:3], g, y, workspace=w, scale=0.1)
        lib.retention_forward(*small[:3], g, ys, workspace=w, scale=0.1)
        lib.retention_backward(*x[:3], g, x[3], *grads, workspace=w, scale=0.1)

    calls(ws[0])
    want = [t.clone() for t in [y, ys] + grads]
    side = torch.cuda.Stream()
    for t in [y, ys] + grads:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(ws[0])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip([y, ys] + grads, want))
    graphs = []
    for w in ws:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            calls(w)
    for t in x:
        t.mul_(0.5)
    calls(ws[1])
    want = [t.clone() for t in [y, ys] + grads]
    for gr in graphs + graphs:
        for t in [y, ys] + grads:
            t.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([y, ys] + grads, want))
    assert all(binding.mhla_query_status(w) == 0 for w in ws)


def test_rows_past_32_bits():
    """Element offsets beyond 2^31: a batch stride that takes the second entry there."""
    H, N, d = 2, 130, 64
    far = (1 << 31) + 4096
    buf = torch.zeros(far + H * N * d, dtype=BF, device="cuda")
    base = rand((2, H, N, d), BF, 1)
    t = torch.as_strided(buf, (2, H, N, d), (far, N * d, d, 1))
    t.copy_(base)
    k, v, y = rand((2, H, N, d), BF, 2), rand((2, H, N, d), BF, 3), torch.empty(2, H, N, d, dtype=BF, device="cuda")
    lib.retention_forward(t, k, v, gammas(H), y)
    check_forward(base, k, v, gammas(H), y, 1.0, "identity")
    lib.retention_forward(k, k, v, gammas(H), t)                 # an output there
    check_forward(k, k, v, gammas(H), t, 1.0, "identity")


def test_tensors_on_a_device_that_is_not_current():
    """The call runs on its tensors' device (one GPU here: the binding makes it current itself)."""
    q, k, v = (rand((1, 2, 64, 64), BF, i) for i in range(3))
    y = torch.empty_like(q)
    with torch.cuda.device(q.device):
        lib.retention_forward(q, k, v, gammas(2), y)
    check_forward(q, k, v, gammas(2), y, 1.0, "identity")


def test_wait_limit_gives_up_then_the_next_call_is_right():
    """With every device-side wait at its shortest the tensor-core passes give up and the status says so;
    the same workspace serves the next call."""
    H, N, d = 3, 4000, 64
    q, k, v, dy = (rand((1, H, N, d), BF, i) for i in range(4))
    g, y = torch.full((H,), 0.98, device="cuda"), torch.zeros(1, H, N, d, dtype=BF, device="cuda")
    grads = [torch.zeros_like(q) for _ in range(3)]
    ws = lib.new_workspace(lib.retention_workspace_bytes(1, H, N, d, backward=True), "cuda")
    for call in (lambda: lib.retention_forward(q, k, v, g, y, workspace=ws),
                 lambda: lib.retention_backward(q, k, v, g, dy, *grads, workspace=ws)):
        binding.mhla_debug_set_wait_limit_ns(1)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            binding.mhla_debug_set_wait_limit_ns(0)
        assert binding.mhla_query_status(ws) == binding.MHLA_ERR_TIMEOUT
        assert binding.mhla_query_status(ws) == binding.MHLA_OK
        call()
        assert binding.mhla_query_status(ws) == binding.MHLA_OK
    check_forward(q, k, v, g, y, 1.0, "identity")
    check_backward(q, k, v, g, dy, grads, 1.0, "identity")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("feature", ["elu1", "exp"])
@pytest.mark.parametrize("d", [16, 32, 128])
def test_features_with_states_of_every_width(d, feature, dtype):
    """A feature map under a returned state, in every chunk and for every decay."""
    B, H, N = 2, 5, 430
    q, k, v = (0.5 * rand((B, H, N, d), dtype, i) for i in range(3))
    g, y, st = gammas(H), torch.empty(B, H, N, d, dtype=dtype, device="cuda"), rand((B, H, d, d), F32, 4)
    start = st.clone()
    lib.retention_forward(q, k, v, g, y, states=st, load_state=True, feature=feature, scale=0.5)
    check_forward(q, k, v, g, y, 0.5, feature, start=start, final=st)


def many(n, longest, seed):
    """Offsets of n sequences of 0 .. 40 tokens, one of them of `longest`."""
    lens = torch.randint(0, 41, (n,), generator=torch.Generator().manual_seed(seed))
    lens[n // 3] = longest
    return [3] + (3 + lens.cumsum(0)).tolist()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [64, 65, 700])
def test_many_packed_sequences(n, dtype):
    """More sequences than are put in order, and more than a block has threads; one is cut into segments."""
    H, d, cu = 2, 64, many(n, 9000, n)
    T = cu[-1] + 5
    q, k, v, dy, y = (rand((1, H, T, d), dtype, i, "bnhd") for i in range(5))
    before, c = y.clone(), torch.tensor(cu, dtype=torch.int32, device="cuda")
    g = torch.tensor([1.0, 0.75], device="cuda")
    pool = rand((n, H, d, d), F32, 6)
    start = pool.clone()
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(n)).int().cuda()
    lib.retention_forward(q, k, v, g, y, cu_seqlens=c, states=pool, slots=slots, load_state=True, scale=0.3)
    ids = slots.long()
    check_forward(q, k, v, g, y, 0.3, "identity", cu, start[ids], pool[ids])
    assert torch.equal(y[:, :, :3], before[:, :, :3]) and torch.equal(y[:, :, cu[-1]:], before[:, :, cu[-1]:])
    grads = [torch.empty_like(q) for _ in range(3)]
    lib.retention_backward(q, k, v, g, dy, *grads, cu_seqlens=c, scale=0.3)
    check_backward(q, k, v, g, dy, grads, 0.3, "identity", cu)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 128])
def test_packed_sequences_in_segments_with_states(d, dtype):
    """Split and whole sequences in one call, states taken and left in place, one slot out of range and one
    asked for twice; the same again bit for bit."""
    H, cu = 2, [0, 100, 7000, 7000, 12500, 12501, 17000]
    T, n = cu[-1], len(cu) - 1
    q, k, v = (rand((1, H, T, d), dtype, i) for i in range(3))
    g, y = torch.tensor([1 - 2.0 ** -10, 1.0], device="cuda"), torch.empty(1, H, T, d, dtype=dtype, device="cuda")
    pool = rand((8, H, d, d), F32, 6)
    start = pool.clone()
    slots = torch.tensor([5, 2, 0, 7, 8, 2], dtype=torch.int32, device="cuda")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    lib.retention_forward(q, k, v, g, y, cu_seqlens=c, states=pool, slots=slots, load_state=True, scale=0.2)
    zero = torch.zeros_like(start[0])
    check_forward(q, k, v, g, y, 0.2, "identity", cu, [start[5], start[2], start[0], start[7], zero, zero])
    check_forward(q[:, :, :12500], k[:, :, :12500], v[:, :, :12500], g, y, 0.2, "identity", cu[:5],
                  [start[i] for i in (5, 2, 0, 7)], [pool[i] for i in (5, 2, 0, 7)])
    assert torch.equal(pool[[0, 1, 3, 4, 6]], start[[0, 1, 3, 4, 6]])
    again, pool2 = torch.empty_like(y), start.clone()
    lib.retention_forward(q, k, v, g, again, cu_seqlens=c, states=pool2, slots=slots, load_state=True, scale=0.2)
    assert torch.equal(y, again) and torch.equal(pool, pool2)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [100, 6000])
def test_more_sequences_than_slots(N, dtype):
    """No slot numbers: sequences behind the pool start from zero and keep nothing."""
    B, H, d = 3, 1, 64
    q, k, v = (rand((B, H, N, d), dtype, i) for i in range(3))
    pool, y = rand((2, H, d, d), F32, 3), torch.empty(B, H, N, d, dtype=dtype, device="cuda")
    start, g = pool.clone(), torch.tensor([0.999], device="cuda")
    lib.retention_forward(q, k, v, g, y, states=pool, load_state=True)
    check_forward(q, k, v, g, y, 1.0, "identity", start=[start[0], start[1], torch.zeros_like(start[0])])
    check_forward(q[:2], k[:2], v[:2], g, y, 1.0, "identity", start=start, final=pool)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_captured_token_loop(dtype):
    """A copy, a prompt and tokens in one graph: slots and offsets are read when it is replayed."""
    H, d, T = 3, 64, 300
    g = gammas(H)
    x = [rand((1, H, T, d), dtype, i) for i in range(3)]
    t = [rand((2, H, 1, d), dtype, 10 + i)[:, :, 0] for i in range(3)]
    pool, y = torch.zeros(6, H, d, d, device="cuda"), torch.zeros(1, H, T, d, dtype=dtype, device="cuda")
    out = torch.zeros(2, H, d, dtype=dtype, device="cuda")
    ints = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 2, 2, 3)]
    src, dst, slots, cu = ints
    ws = lib.new_workspace(lib.retention_workspace_bytes(2, H, T, d), "cuda")

    def calls():
        lib.retention_copy_states(pool, src, dst)
        lib.retention_forward(*x, g, y, cu_seqlens=cu, states=pool, slots=slots, load_state=True, workspace=ws)
        lib.retention_step(*t, g, pool, out, slots=slots)

    calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for values in ([[3, -1], [0, 1], [0, 1], [0, 130, 300]], [[1, 1], [5, 2], [5, 2], [7, 7, 260]], [[9, 2], [4, 2], [-1, 2], [0, 300, 300]]):
        fill = rand((6, H, d, d), F32, 30)
        for a, b in zip(ints, values):
            a.copy_(torch.tensor(b, dtype=torch.int32))
        results = []
        for run in (calls, graph.replay):
            pool.copy_(fill)
            y.zero_()
            out.zero_()
            run()
            results.append([z.clone() for z in (pool, y, out)])
        assert all(torch.equal(a, b) for a, b in zip(*results))
        assert results[0][0].abs().sum() > 0 and results[0][2].abs().sum() > 0


@pytest.mark.parametrize("dtype", [F32, BF])
def test_two_streams_at_once(dtype):
    """Calls of every entry on two streams given by name, side by side, workspaces left to the calls."""
    H, d, N = 3, 64, 5000
    g = torch.tensor([0.9, 0.999, 1.0], device="cuda")
    x = [[rand((1, H, N, d), dtype, 10 * s + i) for i in range(4)] for s in range(2)]
    src, dst = (torch.tensor([i], dtype=torch.int32, device="cuda") for i in range(2))

    def buffers():
        return [torch.zeros_like(x[0][0]) for _ in range(4)] + [torch.zeros(2, H, d, d, device="cuda"),
                                                               torch.zeros(1, H, d, dtype=dtype, device="cuda")]

    def calls(s, o, stream):
        q, k, v, dy = x[s]
        lib.retention_forward(q, k, v, g, o[0], states=o[4], scale=0.1, stream=stream)
        lib.retention_backward(q, k, v, g, dy, *o[1:4], scale=0.1, stream=stream)
        lib.retention_copy_states(o[4], src, dst, stream=stream)
        lib.retention_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, o[4], o[5], scale=0.1, stream=stream)

    want, got = [buffers(), buffers()], [buffers(), buffers()]
    for s in range(2):
        calls(s, want[s], None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s in range(2):
            calls(s, got[s], streams[s])
        torch.full((1 << 20,), 0xff, dtype=torch.uint8, device="cuda")  # memory of this stream, not of those
    torch.cuda.synchronize()
    for a, b in zip(got[0] + got[1], want[0] + want[1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,H,N,d,feature", [(4, 3, 1832, 32, "identity"), (1, 6, 3769, 64, "identity"),
                                             (1, 4, 6000, 128, "elu1")])
def test_states_of_long_sequences_keep_fp32(B, H, N, d, feature):
    """Returned states of bf16 calls, over all decays: terms carry three bf16 parts, 2^-24, unless the decay
    leaves at most 2^-2.75 of them: then two, 2^-17 of a term, so 2^-19.75 of the state; sums in fp32 stay
    below 2^-20 of it (random signs): 2^-19 in all, relative to the states' norm."""
    g = 1 - 2.0 ** -torch.linspace(5, 9, H)
    q, k, v = (rand((B, H, N, d), BF, i) for i in range(3))
    y, st = torch.empty_like(q), torch.zeros(B, H, d, d, device="cuda")
    lib.retention_forward(q, k, v, g.cuda(), y, states=st, feature=feature, scale=0.2)
    got = to_f64(st)
    ref = np.stack([ro.retention(*(to_f64(t[b]) for t in (q, k, v)), to_f64(g), 0.2, feature)[1] for b in range(B)])
    assert np.linalg.norm(got - ref) <= 2.0 ** -19 * np.linalg.norm(ref)
