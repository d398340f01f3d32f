"""Sizes at the ends of the retention entries' range (CPU: every call is refused before the library touches CUDA)."""

import ctypes

import pytest
import torch

from token_level_head_gb300 import binding
from token_level_head_gb300.build import build_library

OK, INVALID, UNSUPPORTED = 0, 1, 2
BF16 = 1
P = 1 << 24  # fake, aligned "device" addresses; never dereferenced
MOST = (1 << 31) - 128  # tokens of a call


@pytest.fixture(scope="module")
def lib():
    build_library()
    return binding.load()


def forward(lib, B, H, N, d, cu=None, wsb=1 << 40):
    return lib.retention_forward(P, None, P, None, P, None, P, P, None, B, H, N, d, cu, None, None, 0, 0, BF16, None,
                                 P, wsb, None)


def backward(lib, B, H, N, d, cu=None, wsb=1 << 40):
    return lib.retention_backward(*[P, None] * 3, P, P, None, *[P, None] * 3, B, H, N, d, cu, BF16, None, P, wsb, None)


@pytest.mark.parametrize("back", [False, True])
def test_workspace_of_the_longest_calls(lib, back):
    """The states of a few hundred segments, as for shorter calls: the segment counts do not wrap."""
    w = binding.retention_workspace_bytes
    for d in (16, 128):
        half = w(1, 1, MOST // 2, d, backward=back)
        for tokens in (MOST - 100000, MOST - 1, MOST):
            for B in (1, 2, 1000):
                assert 0 < w(B, 1, tokens, d, backward=back) <= 8 * half, (B, tokens, d)


def test_more_tokens_than_a_call_takes(lib):
    for back in (False, True):
        assert binding.retention_workspace_bytes(1, 1, MOST + 1, 16, backward=back) == 0
    for call in (forward, backward):
        for cu in (None, 2 * P):
            assert call(lib, 1, 1, MOST + 1, 16, cu) == UNSUPPORTED
            assert call(lib, 1, 1, MOST, 16, cu, wsb=64) == INVALID  # (the workspace)
        assert call(lib, 2, 1, 1 << 30, 16) == UNSUPPORTED


def strides(*s):
    return ctypes.byref(binding._Strides(*s))


def test_sizes_that_no_memory_holds(lib):
    """Products of sizes and strides past 2^63, where a wrapped span would look apart from everything."""
    far = [0x10 * P, 0x20 * P, 0x30 * P, 0x40 * P, 0x50 * P]

    def fwd(B, H, N, d, s=None, ys=None, n_slots=0, states=None, dt=BF16):
        return lib.retention_forward(far[0], s, far[1], s, far[2], s, P, far[3], ys, B, H, N, d, None, states, None,
                                     n_slots, 0, dt, None, far[4], 1 << 62, None)

    wide = strides(1 << 36, 64, 64)                                        # (B - 1) x 2^36 = 2^64 and more
    assert fwd((1 << 28) + 1, 1, 1, 64, s=wide, ys=wide) == INVALID
    assert fwd(1, 1 << 29, (1 << 31) - 128, 128) in (INVALID, UNSUPPORTED)
    assert fwd(1, 8, 4, 128, states=2 * P, n_slots=(1 << 31) - 1) == INVALID
    s = strides(1 << 36, 64, 0)
    assert lib.retention_step(far[0], s, far[1], s, far[2], s, P, far[4], None, 4, far[3], s, (1 << 28) + 1, 1, 64,
                              BF16, None, None) == INVALID
    assert lib.retention_step(far[0], None, far[1], None, far[2], None, P, far[4], None, (1 << 31) - 1, far[3], None,
                              2, 4, 128, BF16, None, None) == INVALID
    assert lib.retention_copy_states(P, (1 << 31) - 1, 1 << 10, 128, far[3], far[4], 3, None) == INVALID


def test_no_workspace_size_for_calls_that_are_refused(lib):
    w = binding.retention_workspace_bytes
    for B, H, N in [((1 << 31) - 1, 1 << 20, 1000), (1 << 20, 1 << 20, 1 << 30), (1 << 30, 2, 1 << 30)]:
        assert w(B, H, N, 128) == 0 and w(B, H, N, 128, backward=True) == 0
        assert forward(lib, B, H, N, 128, cu=2 * P, wsb=1 << 62) == UNSUPPORTED


def test_sizes_past_an_int_are_not_cut():
    """The binding refuses what the C entries' ints do not hold (expanded CPU tensors: nothing is allocated)."""
    n = (1 << 32) + 8
    w = binding.retention_workspace_bytes
    assert w(1, 1, n, 16) == 0 and w(n, 1, 8, 16) == 0 and w(8, n, 8, 16, backward=True) == 0
    g = torch.zeros(1)
    x = torch.zeros(16).expand(1, 1, n, 16)
    for call in (lambda: binding.retention_forward(x, x, x, g, x), lambda: binding.retention_backward(x, x, x, g, x, x, x, x)):
        with pytest.raises(ValueError, match="N: 4294967304"):
            call()
    t = torch.zeros(16).expand(n, 1, 16)
    pool = torch.zeros(16, 16).expand(n, 1, 16, 16)
    with pytest.raises(ValueError, match="B: 4294967304"):
        binding.retention_step(t, t, t, g, pool, t)
    with pytest.raises(ValueError, match="slots: 4294967304"):
        binding.retention_step(t[:2], t[:2], t[:2], g, pool, t[:2])
    e = torch.as_strided(torch.zeros(1), (1, 1, 4, (1 << 32) + 64), (0, 0, 0, 0))
    with pytest.raises(ValueError, match="d: 4294967360"):
        binding.retention_forward(e, e, e, g, e)
    with pytest.raises(ValueError, match="d: 4294967360"):
        binding.retention_step(e[0], e[0], e[0], g, pool, e[0])
    y = torch.zeros(16).expand(2, 1, 4, 16)
    with pytest.raises(ValueError, match="slots: 4294967304"):
        binding.retention_forward(y, y, y, g, y, states=pool)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="slots: 4294967304"):
        binding.retention_copy_states(pool, i, i)
    with pytest.raises(ValueError, match="n: 4294967304"):
        binding.retention_copy_states(pool[:2], i.expand(n), i.expand(n))
    with pytest.raises(ValueError, match="B: 4294967303"):
        binding.retention_forward(x[:, :, :4], x[:, :, :4], x[:, :, :4], g, x[:, :, :4], cu_seqlens=i.expand(n))
