"""Linear cross attention on the GPU against the float64 oracle.

Tolerances, elementwise, relative to the oracle's ``magnitudes`` (the sums of the terms' absolute values), with half a
step of the output's type (bf16 2^-8, fp32 2^-24) of the value itself:
  * sums in 32 bits: n 2^-24 for n terms one after another, n <= tokens + d + 32, once for each sum that a result goes
    through (S or dS, the product with a row, the denominator): 4 of them at most;
  * the features' exponentials and the reciprocal of the denominator: at most 2^-20 together, three features a term;
  * bf16 calls may round operands of the tensor cores to bf16: phi(q) or phi(k) (2^-8) and S or dS (2^-8);
    the fp32 sums S and z of bf16 calls take phi(k) as three bf16 numbers (2^-24).
"""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import cross_oracle as co
from token_level_head_gb300.build import build_library

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
FORMS = [("elu1", True), ("relu", True), ("exp", True), ("identity", False), ("elu1", False)]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()


def rand(shape, dtype, seed, layout="bhnd", scale=1.0):
    """[B, H, N, d] of N(0, 1) in the layout's storage."""
    B, H, N, d = shape
    g = torch.Generator().manual_seed(seed)
    if layout == "bhnd":
        return (scale * torch.randn(B, H, N, d, generator=g)).to(dtype).cuda()
    if layout == "bnhd":
        return (scale * torch.randn(B, N, H, d, generator=g)).to(dtype).cuda().transpose(1, 2)
    return (scale * torch.randn(B, N, 3, H, d, generator=g)).to(dtype).cuda()[:, :, 1].transpose(1, 2)


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def check(got, ref, mag, dtype, n, rounded, what):
    """`rounded` operands rounded to bf16 where the call's type is bf16 (counted by the caller)."""
    got = to_f64(got)
    tol = half_step(dtype) * np.abs(ref) + (4 * (n + 160) * 2.0 ** -24 + 3 * 2.0 ** -20 + rounded * 2.0 ** -8) * 1.02 * mag + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / tol):.2f} x"


class Call:
    """One problem: inputs, their sequences, the calls and the comparison."""

    def __init__(self, B, H, Hk, nq, nk, d, dtype, feature="elu1", normalise=True, eps=1e-6, layout="bhnd", cu_q=None,
                 cu_k=None, lens=None, scale=1.0):
        self.B, self.H, self.Hk, self.d, self.dtype = B, H, Hk, d, dtype
        self.kw = dict(feature=feature, normalise=normalise)
        self.eps, self.cu_q, self.cu_k, self.lens = eps, cu_q, cu_k, lens
        bq, bk = 1 if cu_q else B, 1 if cu_k else B
        self.q, self.dy = rand((bq, H, nq, d), dtype, 1, layout, scale), rand((bq, H, nq, d), dtype, 2)
        self.k, self.v = rand((bk, Hk, nk, d), dtype, 3, layout, scale), rand((bk, Hk, nk, d), dtype, 4, layout)
        self.S = torch.full((B, Hk, d, d), 7.0, device="cuda")
        self.z = torch.full((B, Hk, d), 7.0, device="cuda")
        self.y, self.dq = (torch.full((bq, H, nq, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        self.dk, self.dv = (torch.full((bk, Hk, nk, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))

    def dev(self, x):
        return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")

    def run(self, backward=True, workspace=None):
        cq, ck, lens = self.dev(self.cu_q), self.dev(self.cu_k), self.dev(self.lens)
        lib.linattn_cross_states(self.k, self.v, self.S, self.z, cu_seqlens=ck, lens=lens, workspace=workspace, **self.kw)
        lib.linattn_cross_read(self.q, self.S, self.z, self.y, cu_seqlens=cq, eps=self.eps, workspace=workspace, **self.kw)
        if backward:
            lib.linattn_cross_backward(self.q, self.k, self.v, self.S, self.z, self.dy, self.dq, self.dk, self.dv,
                                       cu_seqlens_q=cq, cu_seqlens_k=ck, lens=lens, eps=self.eps, workspace=workspace, **self.kw)
        return self

    def rows(self, i):
        """(batch, rows) of sequence i's queries and keys."""
        rq = (0, slice(self.cu_q[i], self.cu_q[i + 1])) if self.cu_q else (i, slice(None))
        rk = (0, slice(self.cu_k[i], self.cu_k[i + 1])) if self.cu_k else (i, slice(0, None if self.lens is None else max(0, min(self.lens[i], self.k.shape[2]))))
        return rq, rk

    def check(self, backward=True, sequences=None):
        f, normalise = self.kw["feature"], self.kw["normalise"]
        bf = self.dtype == BF
        for i in range(self.B) if sequences is None else sequences:
            (bq, rq), (bk, rk) = self.rows(i)
            q, dy = to_f64(self.q[bq, :, rq]), to_f64(self.dy[bq, :, rq])
            k, v = to_f64(self.k[bk, :, rk]), to_f64(self.v[bk, :, rk])
            n = q.shape[1] + k.shape[1]
            S, z = co.states(k, v, f)
            args = (f, normalise, self.eps)
            mS, mz, my, mdq, mdk, mdv = co.magnitudes(q, k, v, dy, *args)
            check(self.S[i], S, mS, F32, k.shape[1], 0, f"S of {i}")
            check(self.z[i], z, mz, F32, k.shape[1], 0, f"z of {i}")
            check(self.y[bq, :, rq], co.read(q, S, z, *args), my, self.dtype, n, 2 * bf, f"y of {i}")
            if not backward:
                continue
            dq, dk, dv = co.backward(q, k, v, dy, *args)
            check(self.dq[bq, :, rq], dq, mdq, self.dtype, n, 2 * bf, f"dq of {i}")
            check(self.dk[bk, :, rk], dk, mdk, self.dtype, n, 2 * bf, f"dk of {i}")
            check(self.dv[bk, :, rk], dv, mdv, self.dtype, n, 2 * bf, f"dv of {i}")
        return self


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("nq,nk", [(1, 1), (2, 3), (63, 129), (64, 64), (65, 1), (127, 300), (128, 128), (129, 31), (400, 1000)])
def test_lengths(nq, nk, d, dtype):
    Call(2, 3, 3, nq, nk, d, dtype).run().check()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("feature,normalise", FORMS)
def test_features(feature, normalise, d, dtype):
    Call(1, 2, 2, 300, 260, d, dtype, feature, normalise, eps=1e-3 if feature == "relu" else 1e-6).run().check()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("H,Hk", [(4, 1), (6, 2), (8, 4)])
def test_shared_key_heads(H, Hk, d, dtype):
    Call(2, H, Hk, 200, 150, d, dtype).run().check()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cu_q,cu_k", [([0, 1], [0, 700]), ([0, 5, 5, 300, 301], [0, 130, 131, 131, 400]),
                                       ([3, 130, 260, 700], [2, 2, 1000, 1001]), ([0, 0], [0, 50]), ([0, 50], [0, 0])], ids=str)
def test_packed(cu_q, cu_k, d, dtype):
    """Both sides packed, empty sequences on either, rows of no sequence (not-a-number) on either."""
    c = Call(len(cu_q) - 1, 4, 2, cu_q[-1] + 9, cu_k[-1] + 9, d, dtype, cu_q=cu_q, cu_k=cu_k)
    for t, cu in ((c.q, cu_q), (c.dy, cu_q), (c.k, cu_k), (c.v, cu_k)):
        t[0, :, :cu[0]] = float("nan")
        t[0, :, cu[-1]:] = float("nan")
    c.run().check()
    for t, cu in ((c.y, cu_q), (c.dq, cu_q), (c.dk, cu_k), (c.dv, cu_k)):
        assert (t[0, :, :cu[0]] == 7).all() and (t[0, :, cu[-1]:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_padded(d, dtype):
    """Encoder rows of other lengths, none and more than there is among them; not-a-number and infinities behind them."""
    c = Call(6, 2, 2, 77, 300, d, dtype, lens=[300, 0, 1, 129, 5000, -3])
    for i, n in enumerate([300, 0, 1, 129, 300, 0]):
        c.k[i, :, n:], c.v[i, :, n:] = float("nan"), float("inf")
    c.run().check()
    for i, n in enumerate([300, 0, 1, 129, 300, 0]):
        assert not c.dk[i, :, n:].any() and not c.dv[i, :, n:].any()
        if n == 0:
            assert not c.S[i].any() and not c.z[i].any() and not c.y[i].any() and not c.dq[i].any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_packed_queries_on_a_padded_encoder_and_the_other_way_round(dtype):
    Call(3, 2, 2, 500, 200, 64, dtype, cu_q=[0, 100, 100, 500], lens=[200, 7, 0]).run().check()
    Call(3, 2, 2, 90, 500, 64, dtype, cu_k=[0, 100, 100, 500]).run().check()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_nothing_summed_without_eps(dtype):
    """den = 0: zeros, not not-a-number."""
    for d in (32, 64, 128):
        c = Call(2, 2, 2, 70, 90, d, dtype, eps=0.0, lens=[0, 90]).run().check()
        assert not c.y[0].any() and not c.dq[0].any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("layout", ["bnhd", "slice"])
def test_strides(layout, d, dtype):
    """Token-major tensors and slices of a fused projection; outputs beside one another in one tensor."""
    B, H, nq, nk = 2, 3, 140, 200
    c = Call(B, H, H, nq, nk, d, dtype, layout=layout)
    o = torch.full((B, nk, 3, H, d), 7.0, dtype=dtype, device="cuda")
    c.dk, c.dv = o[:, :, 0].transpose(1, 2), o[:, :, 2].transpose(1, 2)
    c.y, c.dq = (torch.full((B, nq, H, d), 7.0, dtype=dtype, device="cuda").transpose(1, 2) for _ in range(2))
    c.run().check()
    assert (o[:, :, 1] == 7).all()


def test_keys_shared_by_stride_zero():
    """One encoder for every sequence and head: expanded inputs, gradients of the full shape."""
    c = Call(3, 2, 2, 60, 150, 64, BF)
    c.k, c.v = c.k[:1, :1].expand(3, 2, 150, 64), c.v[:1, :1].expand(3, 2, 150, 64)
    c.run().check()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_slots(dtype):
    """States to slots of a larger pool; a slot twice, or out of range, is not kept; several rows may read one."""
    B, H, N, d = 5, 2, 300, 64
    c = Call(B, H, H, N, N, d, dtype)
    pool, zp = torch.full((6, H, d, d), 5.0, device="cuda"), torch.full((6, H, d), 5.0, device="cuda")
    slots = torch.tensor([3, -1, 3, 0, 6], dtype=torch.int32, device="cuda")
    lib.linattn_cross_states(c.k, c.v, pool, zp, slots=slots)
    c.run(backward=False)
    assert torch.equal(pool[3], c.S[0]) and torch.equal(pool[0], c.S[3])
    assert torch.equal(zp[3], c.z[0]) and torch.equal(zp[0], c.z[3])
    assert (pool[[1, 2, 4, 5]] == 5).all() and (zp[[1, 2, 4, 5]] == 5).all()
    read = torch.tensor([3, 3, -2, 0, 6], dtype=torch.int32, device="cuda")
    y = torch.full_like(c.y, 7.0)
    lib.linattn_cross_read(c.q, pool, zp, y, slots=read)
    c.check(backward=False)
    assert torch.equal(y[0], c.y[0]) and torch.equal(y[3], c.y[3]) and (y[[2, 4]] == 7).all()
    one = torch.full_like(c.y, 7.0)[:, :, :1]
    lib.linattn_cross_read(c.q[:, :, :1], pool, zp, one, slots=read)
    assert (one[[2, 4]] == 7).all() and (one[[0, 1, 3]] != 7).any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hk,feature", [(2, 2, "elu1"), (8, 2, "exp"), (3, 1, "identity"), (3, 3, "relu")])
def test_steps(H, Hk, feature, d, dtype):
    """Single queries, some rows on the same slot."""
    B, n = 7, 90
    normalise = feature != "identity"
    k, v = rand((3, Hk, n, d), dtype, 1), rand((3, Hk, n, d), dtype, 2)
    S, z = torch.empty(3, Hk, d, d, device="cuda"), torch.empty(3, Hk, d, device="cuda")
    lib.linattn_cross_states(k, v, S, z, feature=feature, normalise=normalise)
    slots = [2, 0, 1, 1, 2, 0, 0]
    q = rand((B, H, 1, d), dtype, 3, "bnhd")
    y = torch.full((B, H, 1, d), 7.0, dtype=dtype, device="cuda")
    lib.linattn_cross_read(q, S, z, y, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), feature=feature,
                           normalise=normalise, eps=1e-3)
    for b, s in enumerate(slots):
        args = (feature, normalise, 1e-3)
        ref = co.read(to_f64(q[b]), to_f64(S[s]), to_f64(z[s]), *args)
        mag = np.abs(to_f64(S[s]))
        num = co.read(to_f64(q[b]), mag, np.abs(to_f64(z[s])), *args) if feature != "identity" else co.read(np.abs(to_f64(q[b])), mag, None, *args)
        check(y[b], ref, np.abs(num), dtype, d, 0, f"row {b}")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_not_a_number_stays_in_its_sequence(dtype):
    for d in (32, 64, 128):
        c = Call(3, 2, 2, 200, 300, d, dtype).run()
        clean = [t.clone() for t in (c.S, c.z, c.y, c.dq, c.dk, c.dv)]
        c.k[1, 0, 17, 3], c.v[1, 1, 5, 2], c.q[2, 0, 100, 1] = float("nan"), float("inf"), float("nan")
        c.run()
        for t, r in zip((c.S, c.z, c.y, c.dq, c.dk, c.dv), clean):
            assert torch.equal(t[0], r[0])
        keep = torch.arange(200, device="cuda") != 100                  # a query's not-a-number stays in its row of y and dq
        assert torch.equal(c.y[2][:, keep], clean[2][2][:, keep]) and torch.equal(c.dq[2][:, keep], clean[3][2][:, keep])
        assert torch.isnan(c.y[2, 0, 100]).any() and torch.isnan(c.S[1, 0]).any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
def test_many_and_long_sequences(d, dtype):
    """Sequences cut into segments on both sides, few heads; and more heads than blocks run at once."""
    Call(1, 2, 1, 5000, 9000, d, dtype).run().check()
    Call(70, 8, 8, 130, 40, d, dtype).run().check(sequences=[0, 33, 69])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_equal_calls_give_equal_bits(dtype):
    outs = []
    for _ in range(3):
        c = Call(2, 4, 2, 700, 1500, 64, dtype).run()
        outs.append((c.S, c.z, c.y, c.dq, c.dk, c.dv))
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def test_offsets_that_break_their_contract():
    """Out of range and out of order: no row outside the tensors is touched."""
    T, d = 300, 64
    for dtype in (F32, BF):
        for cu in ([-5, 100, 900, 250, 10 ** 9], [200, 100, 50], [10 ** 9, 10 ** 9 + 5], [-(10 ** 9), -5, 5]):
            c = Call(len(cu) - 1, 2, 2, T, T, d, dtype)
            big = [torch.full((1, 2, T + 200, d), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
            c.q, c.dy, c.k, c.v = (rand((1, 2, T, d), dtype, i) for i in range(4))
            c.y, c.dq, c.dk, c.dv = (b[:, :, 100:100 + T] for b in big)
            c.cu_q = c.cu_k = cu
            c.run()
            for b in big:
                assert (b[:, :, :100] == 7).all() and (b[:, :, 100 + T:] == 7).all()


def test_captured_training_steps_on_one_workspace():
    """States, read and gradients captured on a side stream, replayed on new inputs, twice on one workspace."""
    c = Call(2, 4, 2, 600, 900, 64, BF)
    ws = lib.new_workspace(lib.linattn_cross_workspace_bytes(2, 4, 2, 1200, 1800, 64, backward=True), "cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.stream(side):
        c.run(workspace=ws)
        for g in graphs:
            with torch.cuda.graph(g, stream=side):
                c.run(workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (11, 12):
        c.q.copy_(rand(tuple(c.q.shape), BF, seed))
        c.k.copy_(rand(tuple(c.k.shape), BF, seed + 50))
        for g in graphs:
            for t in (c.S, c.z, c.y, c.dq, c.dk, c.dv):
                t.fill_(7.0)
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                g.replay()
            torch.cuda.synchronize()
            c.check()
    assert lib.mhla_query_status(ws) == 0


def test_a_decoder_layer_step_by_step():
    """The two mixers of a decoder together: a gated scan over its tokens, whose output queries an encoder's sums; prompt
    and then single tokens on the kept states, against the whole sequence in one call."""
    B, H, d, n, m, steps = 2, 4, 64, 50, 120, 5
    D = H * d
    x, g = rand((1, B, n + steps, D), F32, 1)[0], rand((1, B, n + steps, D), F32, 2)[0] + 2
    k, v = rand((B, H, m, d), F32, 3), rand((B, H, m, d), F32, 4)
    S, z = torch.empty(B, H, d, d, device="cuda"), torch.empty(B, H, d, device="cuda")
    lib.linattn_cross_states(k, v, S, z)
    whole, y = torch.empty_like(x), torch.empty_like(x)
    lib.gated_scan_forward(x, g, whole)
    heads = lambda t: t.view(B, -1, H, d).transpose(1, 2)  # noqa: E731
    lib.linattn_cross_read(heads(whole), S, z, heads(y))
    state, h, out = torch.empty(B, D, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    lib.gated_scan_forward(x[:, :n], g[:, :n], h[:, :n], states=state)
    lib.linattn_cross_read(h[:, :n].unflatten(2, (H, d)).transpose(1, 2), S, z, out[:, :n].unflatten(2, (H, d)).transpose(1, 2))
    for t in range(n, n + steps):
        lib.gated_scan_step(x[:, t], g[:, t], state, h[:, t])
        lib.linattn_cross_read(h[:, t:t + 1].unflatten(2, (H, d)).transpose(1, 2), S, z,
                               out[:, t:t + 1].unflatten(2, (H, d)).transpose(1, 2))
    # two orders of the same fp32 sums, of 170 terms at most; the outputs are means of |v| < 6
    assert (h - whole).abs().max() <= 2.0 ** -18 * whole.abs().max()
    assert (out - y).abs().max() <= 2.0 ** -14


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("feature", ["elu1", "exp"])
@pytest.mark.parametrize("nk,eps", [(1, 1e-6), (2, 1e-6), (1, 0.5), (2, 40.0)])
def test_gradients_where_a_sequence_s_values_are_equal(nk, eps, feature, d):
    """One value in all of a sequence's keys: without eps dq and dk vanish, as differences of equal terms, so the bf16 calls must
    not leave the roundings of S there.  dq, relative to its terms: S takes 3 nk products, each cut by at most 2^-23, and S - z m^T
    one more rounding; that comes in with u and with phi(q) . u, each at most its share of the terms: (3 nk + 2) 2^-22, and 16 more
    steps of 2^-24 for what eps leaves (sums of d values of m . dy, split in eight, and products).  dk: its sum over 2 d products of dS
    and the same of dS m, (2 d + 40) 2^-23, and the above.  Each with half a step of the value."""
    B, nq = 3, 200
    c = Call(B, 4, 2, nq, B * nk, d, BF, feature, eps=eps, cu_k=[i * nk for i in range(B + 1)])
    for i in range(B):
        c.v[0, :, i * nk:(i + 1) * nk] = c.v[0, :, i * nk:i * nk + 1]
    c.run()
    for i in range(B):
        (bq, rq), (bk, rk) = c.rows(i)
        q, dy, k, v = (to_f64(t) for t in (c.q[bq, :, rq], c.dy[bq, :, rq], c.k[bk, :, rk], c.v[bk, :, rk]))
        args = (feature, True, eps)
        _, _, _, mdq, mdk, _ = co.magnitudes(q, k, v, dy, *args)
        dq, dk, _ = co.backward(q, k, v, dy, *args)
        near = (3 * nk + 2) * 2.0 ** -22 + 16 * 2.0 ** -24
        # eps itself gives terms of the size of eps / den of the others; they are rounded as the rest of a bf16 call
        share = eps / (eps + co.states(k, v, feature)[1].min())
        for got, ref, mag, tol in ((c.dq[bq, :, rq], dq, mdq, near), (c.dk[bk, :, rk], dk, mdk, near + (2 * d + 40) * 2.0 ** -23)):
            bad = np.abs(to_f64(got) - ref) > 2.0 ** -8 * np.abs(ref) + (tol + 3 * 2.0 ** -8 * share) * mag + 1e-37
            assert not bad.any(), (i, bad.sum(), np.max(np.abs(to_f64(got) - ref) / mag) / tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("feature", ["elu1", "exp"])
def test_vanishing_gradients_are_as_small_as_in_32_bits(feature, d):
    """Sequences of one key, whose dq and dk are what eps leaves of differences of equal terms: a bf16 call's are off by no more,
    in the mean, than the formulas evaluated in 32 bits: twice that for dq; for dk, which sums 2 d products in the accumulators of
    the tensor cores (each step cut by 2^-23, not rounded by 2^-24) where the formula sums d, eight times."""
    B, nq = 8, 100
    c = Call(B, 4, 2, nq, 1, d, BF, feature).run()
    off = {"dq": 0.0, "dk": 0.0, "dq32": 0.0, "dk32": 0.0}
    phi = lambda x: np.exp(x) if feature == "exp" else np.where(x > 0, x + 1, np.exp(np.minimum(x, 0)))  # noqa: E731
    slope = lambda x: np.exp(x) if feature == "exp" else np.exp(np.minimum(x, 0))  # noqa: E731
    for i in range(B):
        q, dy, k, v = (to_f64(t[i]) for t in (c.q, c.dy, c.k, c.v))
        dq, dk, _ = co.backward(q, k, v, dy, feature, True, c.eps)
        q, dy, k, v = (t.astype(np.float32) for t in (q, dy, k, v))
        fq, fk = phi(q), np.repeat(phi(k), 2, 0)
        S, z = np.swapaxes(fk, 1, 2) @ np.repeat(v, 2, 0), fk.sum(1)[:, None]
        den = (fq * z).sum(-1, keepdims=True) + np.float32(c.eps)
        u = dy @ np.swapaxes(S, 1, 2)
        dden = -(fq * u).sum(-1, keepdims=True) / (den * den)
        dS, dz = np.swapaxes(fq / den, 1, 2) @ dy, (fq * dden).sum(1)
        dS, dz = (t.reshape(2, 2, *t.shape[1:]).sum(1) for t in (dS, dz))
        dq32, dk32 = slope(q) * (u / den + dden * z), slope(k) * (v @ np.swapaxes(dS, 1, 2) + dz[:, None])
        for name, got, ref in (("dq", to_f64(c.dq[i]), dq), ("dk", to_f64(c.dk[i]), dk), ("dq32", dq32, dq), ("dk32", dk32, dk)):
            off[name] += ((got - ref) ** 2).sum()
    assert off["dq"] <= 2 ** 2 * off["dq32"] and off["dk"] <= 8 ** 2 * off["dk32"], off


@pytest.mark.parametrize("feature,normalise", [("elu1", True), ("exp", True), ("identity", False)])
def test_gradients_are_the_differences(feature, normalise):
    """fp32 calls against central differences of the calls themselves: sum(dy y) for small moves of q, k and v."""
    c = Call(2, 4, 2, 40, 33, 16, F32, feature, normalise, cu_q=[0, 25, 40], scale=0.5).run()
    grads, x = [t.double() for t in (c.dq, c.dk, c.dv)], [c.q, c.k, c.v]

    def value(q, k, v):
        c.q, c.k, c.v = q, k, v
        c.run(backward=False)
        return (c.dy.double() * c.y.double()).sum(), (c.dy.double() * c.y.double()).abs().sum()

    for n in range(3):
        for seed in range(3):
            m = rand(x[n].shape, F32, 10 + seed)
            step = 2.0 ** -8
            lo, hi = list(x), list(x)
            lo[n], hi[n] = lo[n] - step * m, hi[n] + step * m
            (a, size), (b, _) = value(*hi), value(*lo)
            grad = (grads[n] * m.double()).sum()
            terms = (grads[n] * m.double()).abs().sum()
            # what a difference leaves out: step^2 / 6 of the third derivative, whose terms are the first's times at most
            # 8 |m|^2 (|m| < 5) through phi and the quotient; where ELU + 1 changes its form the second derivative jumps by
            # at most 1, for the 2 x 5 step of the values that a move takes there: step / 4 of the terms.  fp32 values of y:
            # 2^-18 of their sum over the 2 steps
            assert abs((a - b) / (2 * step) - grad) <= terms * (step ** 2 * 40 + step / 4 * (feature == "elu1")) + size * 2.0 ** -18 / step
