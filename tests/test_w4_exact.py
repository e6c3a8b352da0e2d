"""4-bit products whose every fp32 sum is exact, compared for equality: a k that is lost, read twice or
meets the wrong scale shows at any K, in any kernel and slice.

Tokens are -2 .. 2, scales 1/8 .. 1 by powers of two, so every product is a multiple of 1/8 and no larger than 2 * 15:
in eighths a sum of K terms stays below 240 K, less than 2^24 up to K = 69905, whatever its order."""
import numpy as np
import pytest
import torch

import w4_ref as ref
from gpu_util import dev
from test_w4 import _pack
from test_w4_variants import FLAT, _ceil, _form_here, linear


def _weight(rng, N, K, group, zero, lead=()):
    G = _ceil(K, group)
    codes = rng.integers(0, 16, lead + (N, K)).astype(np.uint8)
    scales = np.exp2(rng.integers(-3, 1, lead + (N, G))).astype(np.float16)
    return codes, scales, rng.integers(0, 16, lead + (N, G)).astype(np.uint8) if zero else None


def _whole(rng, *shape):
    return rng.integers(-2, 3, shape).astype(np.float16)


LONG = [("stream", 1, 100, 49152, None), ("stream", 8, 64, 69888, None), ((64, 1), 16, 1000, 49152, None),
        ((64, 1), 64, 300, 49152, None), ((128, 1), 128, 256, 49152, None), ((128, 1), 96, 520, 69888, None)]


@pytest.mark.gpu
@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("form,M,N,K,s", FLAT + LONG)
def test_linear(cuda_device, form, M, N, K, s, group, zero):
    assert _form_here(M, N, K) == form
    rng = np.random.default_rng(M + N + K + group)
    w = _weight(rng, N, K, group, zero)
    x, w4 = _whole(rng, M, K), _pack(w, group)
    bias = (rng.integers(-80, 81, N) / 8).astype(np.float16)
    want = dev(x).double() @ dev(ref.values(*w, group)).T
    assert torch.equal(linear(x, w4), want.half())
    assert torch.equal(linear(x, w4, bias, True, True), (want + dev(bias).double()).clamp(min=0.0).half())


def experts_form(P, E, N, sms):
    tokens, nt = _ceil(P, E), _ceil(N, 128)
    if tokens <= 10:
        return "stream"
    if tokens <= 16:
        return 64, 1
    blocks = min(P, _ceil(P, 128) + E)
    return (128, 2) if blocks * _ceil(nt, 2) >= sms else (128, 1)


EXPERTS = [("stream", 7, 4, 16, 130, 12304), ("stream", 60, 4, 24, 1100, 528), ((64, 1), 40, 3, 9, 300, 8208),
           ((64, 1), 36, 4, 9, 2100, 592), ((128, 1), 60, 3, 4, 130, 12304), ((128, 1), 500, 2, 5, 700, 336),
           ((128, 2), 500, 2, 8, 4001, 336), ((128, 2), 1100, 3, 6, 3000, 272)]


@pytest.mark.parametrize("form,T,topk,E,N,K", EXPERTS)
def test_the_cases_reach_their_form(form, T, topk, E, N, K):
    assert experts_form(T * topk, E, N, 148) == form


@pytest.mark.gpu
@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("form,T,topk,E,N,K", EXPERTS)
def test_experts(cuda_device, form, T, topk, E, N, K, group, zero):
    import w8a8_int8_linear_channel_b200 as sq
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert experts_form(T * topk, E, N, sms) == form
    rng = np.random.default_rng(T + N + K + group)
    w = _weight(rng, N, K, group, zero, (E,))
    x, w4, W = _whole(rng, T, K), _pack(w, group), dev(ref.values(*w, group))
    bias = (rng.integers(-80, 81, (E, N)) / 8).astype(np.float16)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)]).astype(np.int32)
    ids[rng.random(ids.shape) < 0.1] = -1
    P = ids.size
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(P, dtype=torch.int32, device="cuda")
    sq.sq_moe_plan(dev(ids), off, order)
    xd, flat = dev(x).double(), ids.reshape(-1)
    want = torch.full((P, N), -777.0, dtype=torch.float64, device="cuda")  # rows that no expert takes stay
    for e in range(E):
        pairs = dev(np.nonzero(flat == e)[0])
        want[pairs] = (xd[pairs // topk] @ W[e].T + dev(bias[e]).double()).clamp(min=0.0)
    for dtype in (torch.float32, torch.float16):
        y = torch.full((P, N), -777.0, dtype=dtype, device="cuda")
        sq.sq_w4a16_experts(dev(x), w4, off, order, y, topk, bias=dev(bias), relu=True)
        assert sq.sq_poll_status() == 0
        assert torch.equal(y, want.to(dtype))
