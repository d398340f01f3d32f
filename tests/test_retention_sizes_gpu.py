"""The retention operators on the GPU at the largest sizes and with offsets that claim more than there is."""

import numpy as np
import pytest
import torch

import token_level_head_gb300 as lib
from gpu_util import to_f64
from oracle import retention_oracle as ro
from token_level_head_gb300.build import build_library

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_library()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("packed", [False, True])
def test_the_longest_sequence(packed):
    """2^31 - 128 tokens of one head: zeros but for the last 300, which are as if they stood alone.  q, k and v are
    one tensor.  Tolerance: scores and the state's copy in bf16, 2^-8 each of a term, and the result's rounding."""
    T, d, n = (1 << 31) - 128, 16, 300
    if torch.cuda.mem_get_info()[0] < 5 * T * d:
        pytest.skip("needs 160 GiB of free device memory")
    x, y = (torch.empty(1, 1, T, d, dtype=BF, device="cuda") for _ in range(2))
    x.zero_()
    y.fill_(7.0)
    tail = torch.randn(1, 1, n, d, generator=torch.Generator().manual_seed(1)).to(BF)
    x[:, :, T - n:] = tail.cuda()
    g = torch.tensor([0.9], device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if packed else None
    lib.retention_forward(x, x, x, g, y, cu_seqlens=cu)
    assert (y[:, :, :T - n:9973] == 0).all()
    assert (y[:, :, T - n - 200000:T - n] == 0).all()
    args = [to_f64(tail[0])] * 3 + [to_f64(g)]
    ref, mag = ro.retention(*args)[0], ro.retention(*args, magnitude=True)[0]
    assert (np.abs(to_f64(y[0, :, T - n:]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.05 * 2.0 ** -8 * mag).all()
