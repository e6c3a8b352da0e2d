"""Expert routing and the pair plan where a shortcut could differ from the definition."""
import numpy as np
import pytest
import torch

import w4_ref as ref
from gpu_util import dev, host

from test_moe import _check_route, _route


@pytest.mark.gpu
def test_route_group_scores_that_cancel(cuda_device):
    # 1000 + p and p - 1000: the scores 1.2822052 and 1.2821990 differ by less than the rounding of
    # their parts in 32 bits
    l = np.array([[-0.37785533, 1.9510481, 0.55182946, 0.60867757]], np.float32)
    bias = np.array([1000, -1000, 1000, -1000], np.float32)
    ids, _ = _route(l, 1, bias, score="sigmoid", n_group=2, topk_group=1, group_top=2)
    assert ids.tolist() == [[0]]


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,topk", [(4, 2, 1, 1), (8, 2, 1, 3), (32, 4, 2, 6), (256, 8, 4, 8)])
@pytest.mark.parametrize("size", [30.0, 1000.0, 1e5])
def test_route_groups_under_a_large_bias_of_either_sign(cuda_device, E, n_group, topk_group, topk, score, size):
    # the first of every group's experts far up, the others far down: a group's score is what is left
    rng = np.random.default_rng(int(E + size))
    l = (rng.standard_normal((3000, E)) * 1.5).astype(np.float32)
    bias = np.where(np.arange(E) % (E // n_group) == 0, size, -size).astype(np.float32)
    _check_route(l, topk, bias, score=score, n_group=n_group, topk_group=topk_group, group_top=2)


def test_plan_workspace_does_not_grow_with_the_pairs():
    # every CTA reads the whole workspace, so with a chunk per 2048 pairs the work grew with their square
    import w8a8_int8_linear_channel_b200 as sq
    assert sq.sq_moe_plan_workspace_bytes(2**31 - 1, 512) <= 512 * 512 * 4
    assert sq.sq_moe_plan_workspace_bytes(65536, 256) == 32 * 256 * 4


@pytest.mark.gpu
@pytest.mark.parametrize("pairs,E", [(2048 * 512, 64), (2048 * 512 + 1, 3), (2048 * 1024 + 1, 512), (5_000_001, 40),
                                     (8_388_611, 257)])
def test_plan_many_pairs(cuda_device, pairs, E):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(pairs)
    skewed = np.minimum(rng.geometric(0.3, pairs) - 1, E)  # some past the experts
    for ids in (rng.integers(-1, E, pairs), skewed, np.full(pairs, -1), np.full(pairs, E - 1)):
        ids = ids.astype(np.int32)
        off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
        order = torch.full((pairs,), -7, dtype=torch.int32, device="cuda")
        sq.sq_moe_plan(dev(ids), off, order)
        r_off, r_order = ref.plan(ids, E)
        assert np.array_equal(host(off), r_off) and np.array_equal(host(order), r_order)


def test_plan_refuses_a_workspace_whose_bytes_are_not_its_own():
    # an expanded tensor counts 4 MB and owns one byte
    import w8a8_int8_linear_channel_b200 as sq
    ids, off = torch.zeros(100000, dtype=torch.int32), torch.zeros(65, dtype=torch.int32)
    byte = torch.zeros(1, dtype=torch.uint8)
    for ws in (byte.expand(1 << 22), torch.zeros(1 << 23, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            sq.sq_moe_plan(ids, off, torch.empty_like(ids), workspace=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,E", [(np.float16, 60), (np.float16, 13), (np.float32, 6)])
def test_route_a_slice_of_rows(cuda_device, dtype, E):
    # rows of 120 bytes and the like: a slice of a batch starts off 16 bytes
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(E)
    T, topk = 9, 4
    l = rng.standard_normal((T, E)).astype(dtype)
    bias = dev((rng.standard_normal(E) * 0.1).astype(np.float32))
    full = dev(l)
    layer = sq.W4Experts.from_float(dev((rng.standard_normal((E, 64, 32)) * 0.1).astype(np.float16)),
                                    dev((rng.standard_normal((E, 32, 64)) * 0.1).astype(np.float16)), topk,
                                    group=32, router_bias=bias)
    x = dev(rng.standard_normal((T, 32)).astype(np.float16))
    side = torch.cuda.Stream()
    for a in range(1, 8):
        part = full[a:]
        assert part.data_ptr() % 16 or a % 2 == 0
        ids = torch.empty((T - a, topk), dtype=torch.int32, device="cuda")
        w = torch.empty((T - a, topk), dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        sq.sq_moe_route(part, ids, w, bias=bias, stream=side)
        torch.cuda.synchronize()
        rid, rw = ref.route(l[a:], topk, host(bias))
        assert np.array_equal(host(ids), rid)
        assert (np.abs(host(w) - rw) <= (2.0**-24 + 2.0**-40) * rw).all()
        assert torch.equal(layer(x[a:], part), layer(x[a:], part.clone()))


def test_route_refuses_host_logits_off_16_bytes():
    import w8a8_int8_linear_channel_b200 as sq
    l = torch.zeros(3 * 60 + 1, dtype=torch.float16)[1:].view(3, 60)
    ids, w = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    with pytest.raises(ValueError, match="CUDA tensors"):
        sq.sq_moe_route(l, ids, w)
