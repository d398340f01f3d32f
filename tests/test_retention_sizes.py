"""Sizes at the ends of the retention entries' range (CPU: every call is refused before the library touches CUDA)."""

import pytest

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
