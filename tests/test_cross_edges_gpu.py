"""Linear cross attention on the GPU at its edges, against the float64 oracle; tolerances as in ``test_cross_gpu``."""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import cross_oracle as co
from test_cross_gpu import BF, F32, Call, check
from token_level_head_gb300.build import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()


@pytest.mark.parametrize("d,H,n", [(64, 24, 4800), (128, 8, 1500), (128, 8, 4096)])
def test_reads_of_many_tiles(d, H, n):
    """Segments of four tiles of 128 queries and more, neighbouring tiles with denominators of other sizes: a row divided by
    another tile's denominator is off by a multiple of itself.  Equal calls give equal bits."""
    c = Call(8, H, H, n, 90, d, BF)
    tile = torch.arange(n, device="cuda") // 128 % 5
    c.q += torch.tensor([0.0, 60.0, 4.0, 200.0, 15.0], device="cuda")[tile][:, None].to(BF)
    c.run(backward=False).check(backward=False, sequences=[0, 7])
    want = c.y.clone()
    for _ in range(10):
        c.y.fill_(7.0)
        c.run(backward=False)
        assert torch.equal(c.y, want)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_packed_sides_without_a_token(d, dtype):
    """Tensors of no rows at all: S and z become zeros (in their slots, others stay), dq is zero, dk and dv of no queries are."""
    B, H, Hk, n = 3, 4, 2, 150
    c = Call(B, H, Hk, n, 0, d, dtype, cu_q=[0, 100, 100, n], cu_k=[0, 0, 0, 0]).run()
    assert not c.S.any() and not c.z.any() and not c.y.any() and not c.dq.any()
    pool, zp = torch.full((5, Hk, d, d), 5.0, device="cuda"), torch.full((5, Hk, d), 5.0, device="cuda")
    slots = torch.tensor([4, -1, 1], dtype=torch.int32, device="cuda")
    lib.linattn_cross_states(c.k, c.v, pool, zp, cu_seqlens=c.dev(c.cu_k), slots=slots)
    assert not pool[[1, 4]].any() and not zp[[1, 4]].any() and (pool[[0, 2, 3]] == 5).all() and (zp[[0, 2, 3]] == 5).all()
    c = Call(B, H, Hk, 0, n, d, dtype, cu_q=[0, 0, 0, 0], cu_k=[0, 100, 100, n]).run()
    for i in range(B):
        k, v = (to_f64(t[0, :, c.cu_k[i]:c.cu_k[i + 1]]) for t in (c.k, c.v))
        (S, z), (mS, mz) = co.states(k, v), co.states(k, np.abs(v))
        check(c.S[i], S, mS, F32, n, 0, f"S of {i}")
        check(c.z[i], z, mz, F32, n, 0, f"z of {i}")
    assert not c.dk.any() and not c.dv.any()
    c = Call(B, H, Hk, 0, 0, d, dtype, cu_q=[0, 0, 0, 0], cu_k=[0, 0, 0, 0]).run()
    assert not c.S.any() and not c.z.any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_no_query_head(d, dtype):
    """No head of queries on two of keys: the gradients of keys and values are zeros."""
    for cu in (None, [0, 100, 150]):
        c = Call(2, 0, 2, 150, 150, d, dtype, cu_q=cu, cu_k=cu)
        c.run()
        assert not c.dk.any() and not c.dv.any() and c.S.any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_denominators_near_the_least_numbers(d, dtype):
    """An eps of 1e-40 beside nothing summed, and sums of d e^-91.5 (2.3e-38 for d = 128): a denominator below 2^-120 (7.5e-37)
    counts as 0; prompts, single queries and gradients have no infinity and no not-a-number."""
    c = Call(2, 2, 2, 70, 90, d, dtype, eps=1e-40, lens=[0, 90]).run().check()
    assert not c.y[0].any() and not c.dq[0].any() and not c.dk[0].any()
    one = torch.full_like(c.y[:, :, :1], 7.0)
    lib.linattn_cross_read(c.q[:, :, :1], c.S, c.z, one, eps=1e-40)
    assert not one[0].any() and torch.isfinite(one).all()
    c = Call(2, 2, 2, 70, 1, d, dtype, "exp", eps=0.0)
    c.q.fill_(-45.5)
    c.k.fill_(-46.0)
    c.run()
    lib.linattn_cross_read(c.q[:, :, :1], c.S, c.z, one, feature="exp", eps=0.0)
    for t in (c.y, one, c.dq, c.dk, c.dv):
        assert not t.any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_large_denominators(d, dtype):
    """exp features whose denominators are about 10^20, 10^33 and just below the largest number, 1 / den among the numbers below the
    normal ones: one key, so that y is its value (up to the rounding of phi(q) in numerator and denominator alike, and 2^-20
    for the steps of 1 / den, 2^-149 wide at 2^-127)."""
    for shift in (22.0, 37.0, 41.5 + 0.5 * (d == 64) + 0.75 * (d == 16)):
        c = Call(2, 2, 2, 150, 1, d, dtype, "exp")
        c.q.fill_(shift)
        c.k.fill_(41.5 if shift > 40 else shift)
        c.v.uniform_(-1.0, 1.0, generator=torch.Generator(device="cuda").manual_seed(5))
        c.run()
        want = c.v.float().expand_as(c.y)
        assert ((c.y.float() - want).abs() <= (2.0 ** -7 if dtype == BF else 2.0 ** -18) * want.abs()).all(), shift
    c = Call(1, 2, 2, 150, 200, d, dtype, "exp")
    c.q += 22
    c.k += 22
    c.run().check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("feature,normalise", [("elu1", True), ("exp", True), ("elu1", False)])
def test_dk_is_off_by_its_own_rounding(feature, normalise, d):
    """bf16 calls: dk = phi'(k) (dS v + dz) takes k and v as they are; dS, the w that it is summed from and S less z m^T, which dz
    goes through, are sums of two bf16 numbers, each off by 2^-17 of its terms.  Where those are some ten times dk, that adds
    (10 x 3 x 2^-17 / 2^-9)^2 < 1.5 % to the mean square of dk's own rounding; a phi' that is rounded itself would add half of it
    (ELU + 1, whose phi' is 1 for half of the keys: a fifth)."""
    c = Call(2, 4, 2, 700, 900, d, BF, feature, normalise).run()
    off = own = 0.0
    for i in range(2):
        q, dy, k, v = (to_f64(t[i]) for t in (c.q, c.dy, c.k, c.v))
        dk = co.backward(q, k, v, dy, feature, normalise, c.eps)[1]
        off += ((to_f64(c.dk[i]) - dk) ** 2).sum()
        own += ((to_f64(torch.from_numpy(dk).to(BF)) - dk) ** 2).sum()
    assert off <= 1.03 * own, off / own
