"""Rows of x as a user cuts them out of other tensors."""
import numpy as np
import pytest
import torch

import w4_ref as ref
from gpu_util import dev
from test_w4 import _pack, _tokens


@pytest.mark.gpu
def test_the_stride_of_a_single_row_means_nothing(cuda_device):
    # one row of a tensor whose rows are an odd number of elements apart
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(4)
    N, K = 72, 96
    w = ref.random_weight(rng, N, K, 32, True)
    w4, x = _pack(w, 32), dev(_tokens(rng, 1, K))
    wide = torch.full((3, K + 3), float("nan"), dtype=torch.float16, device="cuda")
    wide[0, :K] = x[0]
    row = wide[:1, :K]
    new = lambda: torch.empty((1, N), dtype=torch.float16, device="cuda")
    want = sq.sq_w4a16_linear(x, w4, new())
    assert torch.equal(sq.sq_w4a16_linear(row, w4, new()), want) and torch.equal(sq.W4Linear(w4)(row), want)
    we = sq.W4Weight(w4.packed, N, K, 32, True, experts=1)
    off, order = dev(np.array([0, 1], np.int32)), dev(np.zeros(1, np.int32))
    assert torch.equal(sq.sq_w4a16_experts(row, we, off, order, new()), want)
