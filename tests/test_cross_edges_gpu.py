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
