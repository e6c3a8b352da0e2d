"""Packed weights whose scales have all eleven bits of fp16, as another quantizer's have."""
import numpy as np
import pytest

import w4_ref as ref
from gpu_util import host
from test_w4 import _pack, _tokens
from test_w4_variants import FLAT, Product, _form_here, linear


def _weight(rng, N, K, group, zero, std=0.005):
    codes, _, zeros = ref.random_weight(rng, N, K, group, zero)
    scales = (rng.uniform(0.2, 1.0, (N, -(-K // group))) * std).astype(np.float16)
    return codes, scales, zeros


@pytest.mark.gpu
@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("form,M,N,K,s", FLAT)
def test_linear(cuda_device, form, M, N, K, s, group, zero):
    """Few tokens multiply by the scale in fp32, so the weight is (q - z) * s itself; many see it rounded to
    fp16 once, as sq_w4_dequantize shows it.  Within the same bounds as any weight either way: a product of an
    fp16 token and q - z has at most 15 bits and its group's sum is scaled in fp32."""
    assert _form_here(M, N, K) == form
    rng = np.random.default_rng(M + N + K + group)
    w = _weight(rng, N, K, group, zero)
    W = ref.values(*w, group)
    rounded = W.astype(np.float16).astype(np.float64)
    assert (W != rounded).any()
    x, w4 = _tokens(rng, M, K), _pack(w, group)
    p = Product(x, W if form == "stream" else rounded)
    p.check(linear(x, w4))


@pytest.mark.gpu
@pytest.mark.parametrize("zero", [False, True])
def test_values_past_the_range_of_fp16(cuda_device, zero):
    """(q - z) * s past 65504 is a number for few tokens and Inf for many, as sq_w4_dequantize shows it."""
    import torch
    import w8a8_int8_linear_channel_b200 as sq
    N, K, group = 9000, 2064, 128
    codes = np.full((N, K), 9, np.uint8)
    codes[5, 7] = 15
    scales = np.full((N, 17), 2.0**-4, np.float16)
    scales[5, 0] = 30000.0
    zeros = np.full((N, 17), 8, np.uint8) if zero else None
    w4 = _pack((codes, scales, zeros), group)
    out = host(sq.sq_w4_dequantize(w4, torch.empty((N, K), dtype=torch.float16, device="cuda")))
    assert np.isinf(out[5, 7]) and np.isfinite(out).sum() == out.size - 1
    for M in (1, 10, 80, 2500):
        assert (_form_here(M, N, K) == "stream") == (M == 1)
        x = np.zeros((M, K), np.float16)
        x[0, 7] = 2.0**-4
        x[M - 1, 200] = 1.0
        y = host(linear(x, w4))
        # 7 * 30000 / 16 in one, Inf / 16 in the other; and Inf * 0 in the other tokens' row
        want = np.float16(7 * 30000 / 16) if M == 1 else np.float16(np.inf)
        assert y[0, 5] == want
        if M > 1:
            assert np.isnan(y[1:, 5]).all()
        rest = np.delete(y, 5, 1)
        assert np.isfinite(rest).all() and (rest[M - 1] == np.float16(2.0**-4 + (2.0**-8 if M == 1 else 0))).all()
