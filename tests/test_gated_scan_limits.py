"""Sizes of the gated scan next to 2^31 (CPU: every call is refused before the library touches CUDA)."""

import pytest

from test_gated_scan_abi import BF16, F32, UNSUPPORTED, bwd, fwd, lib, step  # noqa: F401

FAR = 1 << 45  # addresses apart whatever the sizes


@pytest.mark.parametrize("D", [(1 << 31) - 8, (1 << 31) - 32, (1 << 31) - 1024 + 8])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_channels_whose_pieces_have_no_int(lib, D, dt):  # noqa: F811
    """More than 2^31 - 1024 channels: the last piece of a row would end behind 2^31."""
    assert fwd(lib, x=FAR, g=2 * FAR, y=3 * FAR, B=1, N=1, D=D, dt=dt, states=None, kept=None) == UNSUPPORTED
    assert bwd(lib, x=FAR, g=2 * FAR, dy=3 * FAR, kept=4 * FAR, dx=5 * FAR, dg=6 * FAR, B=1, N=1, D=D, dt=dt, h0=None, dl=None,
               dh0=None) == UNSUPPORTED
    assert step(lib, x=FAR, g=2 * FAR, states=3 * FAR, out=4 * FAR, n_slots=1, B=1, D=D, dt=dt) == UNSUPPORTED
