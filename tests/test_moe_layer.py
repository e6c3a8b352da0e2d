"""The expert layer is its documented calls, its hidden rows in fp16."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from test_w4 import _tokens


def _by_calls(sq, layer, x, logits):
    """The layer by the public calls; also its hidden rows."""
    T, K = x.shape
    E, F, topk = layer.up.experts, layer.up.N, layer.topk
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")
    ids, w = new(T, topk, dtype=torch.int32), new(T, topk)
    sq.sq_moe_route(logits, ids, w)
    off, order = new(E + 1, dtype=torch.int32), new(T * topk, dtype=torch.int32)
    sq.sq_moe_plan(ids, off, order)
    h = sq.sq_w4a16_experts(x, layer.up, off, order, new(T * topk, F, dtype=torch.float16), topk, relu=True)
    z = sq.sq_w4a16_experts(h, layer.down, off, order, new(T * topk, K))
    return sq.sq_moe_combine(z, ids, w, E, new(T, K, dtype=torch.float16)), h


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 90, 700])
def test_layer_is_its_calls(cuda_device, T):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(T)
    E, topk, K, F = 10, 3, 272, 336
    layer = sq.W4Experts.from_float(dev((rng.standard_normal((E, F, K)) * 0.05).astype(np.float16)),
                                    dev((rng.standard_normal((E, K, F)) * 0.05).astype(np.float16)), topk)
    x, logits = dev(_tokens(rng, T, K)), dev(rng.standard_normal((T, E)).astype(np.float32))
    y, _ = _by_calls(sq, layer, x, logits)
    assert torch.equal(layer(x, logits), y)


@pytest.mark.gpu
def test_a_hidden_value_past_fp16_is_inf_in_its_token_only(cuda_device):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(1)
    E, topk, K, F, T = 4, 2, 128, 64, 6
    layer = sq.W4Experts.from_float(dev(np.full((E, F, K), 0.5, np.float16)),
                                    dev((rng.standard_normal((E, K, F)) * 0.05).astype(np.float16)), topk)
    x = np.ones((T, K), np.float16)
    x[3] = 60000.0
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    y, h = _by_calls(sq, layer, dev(x), logits)
    assert bool(torch.isinf(h[3 * topk:4 * topk]).all())
    got = layer(dev(x), logits)
    assert not bool(torch.isfinite(got[3]).any())
    keep = [t for t in range(T) if t != 3]
    assert bool(torch.isfinite(got[keep]).all()) and torch.equal(got[keep], y[keep])
