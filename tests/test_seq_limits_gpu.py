"""Sequence operators at the ends of their sizes, on the GPU."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cf():
    import implicit_gemm_convolution_conv2d_b200 as mod
    return mod


def test_more_sequences_than_half_of_31_bits(cf):
    """2^30 + 3 packed sequences, two of them not empty: the search for a row's sequence adds no two of their numbers."""
    n, rows, C = 2 ** 30 + 3, 100, 8
    torch.manual_seed(0)
    x, dy, w = torch.randn(rows, C, device="cuda"), torch.randn(rows, C, device="cuda"), torch.randn(C, 4, device="cuda")
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    few = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    for first in (0, n // 2 + 1, n - 2):  # the sequence of rows 0 .. 39; the last one's are 40 .. 99
        cu[: first + 1] = 0
        cu[first + 1 :] = 40
        cu[-1] = rows
        assert torch.equal(cf.conv_causal(x, w, cu_seqlens=cu), cf.conv_causal(x, w, cu_seqlens=few))
        for a, b in zip(cf.conv_causal_grad(x, w, dy, cu_seqlens=cu)[:2], cf.conv_causal_grad(x, w, dy, cu_seqlens=few)[:2]):
            assert torch.equal(a, b)
