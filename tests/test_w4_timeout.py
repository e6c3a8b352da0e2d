"""Waits of the 4-bit products that run out: the status word says so, and nothing unfinished is stored."""
import glob
import os
import re

import numpy as np
import pytest
import torch

import w4_ref as ref
from gpu_util import dev
from test_w4 import _pack, _tokens

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_int8_linear_channel_b200", "csrc")


def test_no_wait_is_made_without_asking_how_it_ended():
    # mbar_wait_bounded records nothing, so a call that drops its answer hides a time-out
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            assert not re.search(r"^\s*mbar_wait_bounded\(", f.read(), re.M), path


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,f32", [(16, 4096, 8192, False), (60, 4090, 4096, True), (200, 4096, 4096, True),
                                       (384, 9000, 2048, False), (1930, 3904, 528, True), (1930, 3900, 528, False)])
def test_a_wait_that_runs_out_stores_nothing_unfinished(cuda_device, M, N, K, f32):
    """With the smallest wait budget and cold caches a call may give up.  Every element is then either
    what it was before the call or the right one, and with status 0 all are the right ones."""
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(M)
    w = ref.random_weight(rng, N, K, 128, False)
    x = dev(_tokens(rng, M, K))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    if f32:  # the experts' form: rows by cp.async, fp32 out
        w4 = _pack(tuple(None if t is None else t[None] for t in w), 128)
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        order = torch.arange(M, dtype=torch.int32, device="cuda")
        call = lambda y: sq.sq_w4a16_experts(x, w4, off, order, y)
    else:
        w4 = _pack(w, 128)
        call = lambda y: sq.sq_w4a16_linear(x, w4, y)
    new = lambda: torch.full((M, N), -777.0, dtype=torch.float32 if f32 else torch.float16, device="cuda")
    good = call(new())
    assert sq.sq_poll_status() == 0
    for _ in range(4):
        y = new()
        try:
            flush.zero_()
            sq.sq_set_wait_budget_ns(1000)
            call(y)
            status = sq.sq_poll_status()
        finally:
            sq.sq_set_wait_budget_ns(2_000_000_000)
        assert status in (0, 8)
        right = y == good
        assert bool((right | (y == -777.0)).all())
        assert status == 8 or bool(right.all())
    assert torch.equal(call(new()), good) and sq.sq_poll_status() == 0
