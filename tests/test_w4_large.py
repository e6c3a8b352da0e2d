"""Tensors whose offsets pass 32 bits.  Sums are exact (as in test_w4_exact), so samples compare for equality."""
import numpy as np
import pytest
import torch

import w4_ref as ref
from gpu_util import host

pytestmark = pytest.mark.gpu


def _whole(gen, *shape):
    return torch.randint(-2, 3, shape, generator=gen, device="cuda").half()


def _packed(gen, N, K, group, experts=None):
    """A packed weight of random codes and scales 1/8 .. 1, and its values of chosen channels in 64 bits."""
    import w8a8_int8_linear_channel_b200 as sq
    lead = () if experts is None else (experts,)
    codes = torch.empty(lead + (N, K), dtype=torch.uint8, device="cuda").random_(0, 16, generator=gen)
    scales = torch.exp2(torch.randint(-3, 1, lead + (N, -(-K // group)), generator=gen, device="cuda").float()).half()
    w4 = sq.sq_w4_pack(codes, scales, sq.new_w4_weight(N, K, group, experts=experts))
    at = torch.arange(K, device="cuda") // group
    return w4, lambda *i: (codes[i].double() - 8.0) * scales[i].double()[..., at]


@pytest.fixture
def gen(cuda_device):
    yield torch.Generator(device="cuda").manual_seed(7)
    torch.cuda.empty_cache()


def test_output_of_more_than_2_31_elements(gen):
    import w8a8_int8_linear_channel_b200 as sq
    M, N, K, period = 70_001, 32_776, 32, 1000
    w4, values = _packed(gen, N, K, 32)
    x = _whole(gen, period, K)
    x = x.repeat(-(-M // period), 1)[:M].contiguous()
    y = sq.sq_w4a16_linear(x, w4, torch.empty((M, N), dtype=torch.float16, device="cuda"))
    want = (x[:period].double() @ values(slice(None)).T).half()
    assert y.numel() > 2**31
    for a in range(0, M, period):
        assert torch.equal(y[a:a + period], want[:M - a])


@pytest.mark.parametrize("M", [3, 20, 200])
def test_packed_weight_of_more_than_4_gigabytes(gen, M):
    import w8a8_int8_linear_channel_b200 as sq
    N, K = 8_388_480 - 5, 1040
    w4, values = _packed(gen, N, K, 128)
    assert w4.packed.numel() > 2**32
    x = _whole(gen, M, K)
    y = sq.sq_w4a16_linear(x, w4, torch.empty((M, N), dtype=torch.float16, device="cuda"))
    for a in [0, N - 3000] + [int(v) for v in np.random.default_rng(M).integers(0, N - 3000, 12)]:
        part = slice(a, a + 3000)
        assert torch.equal(y[:, part], (x.double() @ values(part).T).half())
    out = torch.empty((N, K), dtype=torch.float16, device="cuda")
    sq.sq_w4_dequantize(w4, out)
    for a in (0, N // 2, N - 3000):
        assert torch.equal(out[a:a + 3000].double(), values(slice(a, a + 3000)))


@pytest.mark.parametrize("M,N", [(5, 700), (12, 9000), (12, 200)])
def test_rows_of_x_far_apart(gen, M, N):
    import w8a8_int8_linear_channel_b200 as sq
    K, ld = 2064, 2**29 + 8
    w4, values = _packed(gen, N, K, 64)
    buf = torch.empty((M - 1) * ld + K, dtype=torch.float16, device="cuda")
    x = buf.as_strided((M, K), (ld, 1))
    assert (M - 1) * ld * 2 > 2**32
    x.copy_(_whole(gen, M, K))
    y = sq.sq_w4a16_linear(x, w4, torch.empty((M, N), dtype=torch.float16, device="cuda"))
    assert torch.equal(y, (x.double() @ values(slice(None)).T).half())


def test_expert_rows_of_more_than_2_31_elements(gen):
    import w8a8_int8_linear_channel_b200 as sq
    E, topk, T, N, K = 5, 4, 20_003, 28_672, 32
    P = T * topk
    assert P * N > 2**31
    w4, values = _packed(gen, N, K, 32, E)
    x = _whole(gen, T, K)
    ids = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :topk].int().contiguous()
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(P, dtype=torch.int32, device="cuda")
    sq.sq_moe_plan(ids, off, order)
    y = sq.sq_w4a16_experts(x, w4, off, order, torch.empty((P, N), dtype=torch.float32, device="cuda"), topk)
    W = values(slice(None))
    for p in [0, P - 1] + [int(v) for v in np.random.default_rng(0).integers(0, P, 200)]:
        assert torch.equal(y[p].double(), W[int(ids[p // topk, p % topk])] @ x[p // topk].double())
    w = torch.exp2(torch.randint(-2, 1, (T, topk), generator=gen, device="cuda").float())
    out = sq.sq_moe_combine(y, ids, w, E, torch.empty((T, N), dtype=torch.float16, device="cuda"))
    for t in [0, T - 1] + [int(v) for v in np.random.default_rng(1).integers(0, T, 50)]:
        assert torch.equal(out[t], (w[t].double() @ y[t * topk:(t + 1) * topk].double()).half())


def test_logits_of_more_than_2_31_elements(gen):
    import w8a8_int8_linear_channel_b200 as sq
    T, E, topk = 4_300_000, 512, 4
    l = torch.empty((T, E), dtype=torch.float16, device="cuda").normal_(generator=gen)
    ids = torch.empty((T, topk), dtype=torch.int32, device="cuda")
    w = torch.empty((T, topk), dtype=torch.float32, device="cuda")
    sq.sq_moe_route(l, ids, w)
    for a in (0, T // 2, T - 300):
        rid, rw = ref.route(host(l[a:a + 300]), topk)
        assert np.array_equal(host(ids[a:a + 300]), rid)
        assert (np.abs(host(w[a:a + 300]) - rw) <= (2.0**-24 + 2.0**-40) * rw).all()
