"""Expert routing, the pair plan, the experts' products and the layer built from them."""
import ctypes

import numpy as np
import pytest
import torch

import w4_ref as ref
from gpu_util import dev, host
from test_w4 import _pack, _tokens

FAKE = ctypes.c_void_p(0x10000)
FAKE_ODD = ctypes.c_void_p(0x10004)


def _lib():
    import w8a8_int8_linear_channel_b200 as sq
    return sq._L


# ------------------------------------------------------------- refusals (CPU) ----
def test_route_refuses_on_the_host():
    f = _lib().sq_moe_route
    names = ["logits", "half", "T", "E", "ld", "bias", "sigmoid", "n_group", "topk_group", "group_top", "topk",
             "renorm", "scale", "ids", "weights", "stream"]
    good = dict(zip(names, [FAKE, 0, 4, 64, 64, None, 0, 1, 1, 1, 8, 1, 1.0, FAKE, FAKE, None]))
    call = lambda **kw: f(*[{**good, **kw}[n] for n in names])
    for kw in [dict(logits=None), dict(ids=None), dict(weights=None), dict(T=0), dict(E=0), dict(topk=0), dict(ld=63),
               dict(topk=33, E=32, ld=32), dict(n_group=3), dict(n_group=0), dict(n_group=8, topk_group=9),
               dict(n_group=8, topk_group=0), dict(group_top=3), dict(group_top=0), dict(scale=float("inf")),
               dict(n_group=8, topk_group=1, topk=9), dict(n_group=64, topk_group=8, group_top=2)]:
        assert call(**kw) == 1, kw
    for kw in [dict(E=513, ld=513), dict(topk=33), dict(T=1 << 30), dict(n_group=64, topk_group=8)]:
        assert call(**kw) == 3, kw
    for kw in [dict(logits=FAKE_ODD), dict(bias=FAKE_ODD), dict(ids=FAKE_ODD), dict(weights=FAKE_ODD)]:
        assert call(**kw) == 2, kw


def test_plan_experts_and_combine_refuse_on_the_host():
    L = _lib()
    f = L.sq_moe_plan
    assert f(None, 8, 4, FAKE, FAKE, None, 0, None) == 1
    assert f(FAKE, 0, 4, FAKE, FAKE, None, 0, None) == 1
    assert f(FAKE, 8, 0, FAKE, FAKE, None, 0, None) == 1
    assert f(FAKE, 8, 513, FAKE, FAKE, None, 0, None) == 3
    assert f(FAKE_ODD, 8, 4, FAKE, FAKE, None, 0, None) == 2
    need = L.sq_moe_plan_workspace_bytes(100000, 64)
    assert need > 0 and L.sq_moe_plan_workspace_bytes(64, 64) == 0 and L.sq_moe_plan_workspace_bytes(0, 64) == 0
    assert f(FAKE, 100000, 64, FAKE, FAKE, None, 0, None) == 5
    assert f(FAKE, 100000, 64, FAKE, FAKE, FAKE, need - 1, None) == 5
    f = L.sq_w4a16_experts
    good = [FAKE, 4, 64, FAKE, 8, 32, 64, 32, 0, None, 0, FAKE, FAKE, 8, 2, FAKE, 0, None]

    def with_(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    for i in (0, 3, 11, 12, 15):
        assert with_(**{f"_{i}": None}) == 1
    assert with_(_1=0) == 1 and with_(_4=0) == 1 and with_(_13=0) == 1 and with_(_14=0) == 1
    assert with_(_13=9) == 1                      # pair 8 would read row 4 of 4
    assert with_(_2=56) == 1 and with_(_2=68) == 2 and with_(_4=513) == 3 and with_(_7=31) == 3
    assert with_(_11=FAKE_ODD) == 2 and with_(_12=FAKE_ODD) == 2 and with_(_9=FAKE_ODD) == 2
    f = L.sq_moe_combine
    assert f(None, 0, FAKE, FAKE, 4, 2, 64, 8, FAKE, None) == 1
    assert f(FAKE, 0, FAKE, FAKE, 0, 2, 64, 8, FAKE, None) == 1
    assert f(FAKE, 0, FAKE, FAKE, 4, 33, 64, 8, FAKE, None) == 3
    assert f(FAKE_ODD, 0, FAKE, FAKE, 4, 2, 64, 8, FAKE, None) == 2


def test_binding_refuses():
    import w8a8_int8_linear_channel_b200 as sq
    l, ids, w = torch.zeros((3, 8)), torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    with pytest.raises(ValueError, match="CUDA tensors"):
        sq.sq_moe_route(l, ids, w)
    with pytest.raises(ValueError, match="score"):
        sq.sq_moe_route(l, ids, w, score="relu")
    with pytest.raises(ValueError):
        sq.sq_moe_route(l.double(), ids, w)
    with pytest.raises(ValueError, match="ids"):
        sq.sq_moe_route(l, ids[:2], w)
    up, down = (sq.new_w4_weight(n, k, 32, experts=4, device="cpu") for n, k in ((32, 64), (64, 48)))
    with pytest.raises(ValueError, match="up / down"):
        sq.W4Experts(up, down, 2)
    layer = sq.W4Experts(up, sq.new_w4_weight(64, 32, 32, experts=4, device="cpu"), 2)
    with pytest.raises(ValueError, match="x / logits"):
        layer(torch.zeros((3, 64), dtype=torch.float16), torch.zeros((2, 4)))
    with pytest.raises(ValueError, match="several experts"):
        sq.sq_w4a16_experts(torch.zeros((3, 64), dtype=torch.float16), up[0], ids, ids, w)


# ------------------------------------------------------------------- routing ----
def _route(logits, topk, bias=None, ld=None, **kw):
    import w8a8_int8_linear_channel_b200 as sq
    T, E = logits.shape
    l = dev(logits)
    if ld is not None:
        wide = torch.full((T, ld), float("inf"), dtype=l.dtype, device="cuda")
        wide[:, :E] = l
        l = wide[:, :E]
    ids = torch.full((T, topk), 77777, dtype=torch.int32, device="cuda")
    w = torch.full((T, topk), float("nan"), dtype=torch.float32, device="cuda")
    sq.sq_moe_route(l, ids, w, bias=dev(bias), **kw)
    return host(ids), host(w)


def _check_route(logits, topk, bias=None, ld=None, **kw):
    ids, w = _route(logits, topk, bias, ld, **kw)
    rid, rw = ref.route(logits, topk, bias, **kw)
    assert np.array_equal(ids, rid)
    # 64-bit scores, one rounding to fp32 (and 2^-40 for two 64-bit evaluations)
    assert (np.abs(w - rw) <= (2.0**-24 + 2.0**-40) * np.abs(rw) + 2.0**-150).all()


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (3, 7, 7), (5, 32, 4), (33, 33, 8), (16, 64, 6), (100, 160, 32),
                                      (257, 256, 8), (9, 512, 16)])
def test_route(cuda_device, T, E, topk, score):
    rng = np.random.default_rng(T * E)
    l = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    _check_route(l, topk, score=score)
    _check_route(l, topk, bias, score=score, renormalize=False, scale=2.5, ld=E + 5)
    _check_route(l.astype(np.float16), topk, bias, score=score, ld=E + 3)


@pytest.mark.gpu
@pytest.mark.parametrize("n_group,topk_group,group_top,E,topk", [(2, 1, 1, 8, 4), (8, 4, 2, 256, 8), (4, 4, 2, 64, 6),
                                                                (32, 3, 1, 32, 3), (32, 5, 2, 512, 16), (3, 2, 2, 51, 5)])
def test_route_groups(cuda_device, n_group, topk_group, group_top, E, topk):
    rng = np.random.default_rng(E + topk)
    l = (rng.standard_normal((65, E)) * 2).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        _check_route(l, topk, bias, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
        l2 = l.copy()
        l2[:, rng.integers(0, E, E // 2)] = -np.inf
        _check_route(l2, topk, None, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)


@pytest.mark.gpu
def test_route_ties_take_the_lowest_index(cuda_device):
    l = np.zeros((4, 70), np.float32)
    l[1, 69] = l[1, 3] = l[1, 40] = 1
    l[2] = np.repeat(np.arange(7), 10)
    l[3] = -5
    for score in ("softmax", "sigmoid"):
        ids, _ = _route(l, 8, score=score)
        assert ids[0].tolist() == list(range(8)) == ids[3].tolist()
        assert ids[1].tolist() == [3, 40, 69, 0, 1, 2, 4, 5] and ids[2].tolist() == list(range(60, 68))
        _check_route(l, 8, score=score, n_group=7, topk_group=3, group_top=2)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_different_logits_whose_64_bit_scores_tie(cuda_device, score):
    rng = np.random.default_rng(23)
    E, topk = 64, 6
    step = np.stack([rng.permutation(E) for _ in range(7)]).astype(np.float32)
    l = np.stack([step[0] * np.float32(1e-20),                  # next to 0: exp(l) == 1
                  -800 - step[1],                               # sigmoids and exponentials that are 0 ...
                  np.where(step[2] < 3, step[2], -800 - step[2]),  # ... for some of the chosen
                  50 + step[3],                                 # sigmoids that are 1
                  25 + step[4] * np.float32(2.0**-19),          # and some that 64 bits can hardly tell apart
                  np.where(step[5] < 60, -5 - step[5], step[5] * np.float32(1e-21)),
                  np.where(step[6] % 2 == 0, np.float32(0.0), np.float32(-0.0))]).astype(np.float32)
    _check_route(l, topk, score=score)
    _check_route(l, topk, score=score, renormalize=False)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_and_nonfinite(cuda_device, score):
    rng = np.random.default_rng(11)
    E, topk = 40, 4
    l = rng.standard_normal((8, E)).astype(np.float32)
    l[0] = -np.inf                       # nothing left
    l[1] = np.nan
    l[2, 2:] = -np.inf                   # fewer than topk left
    l[3, 7] = np.inf                     # certain
    l[4, [3, 9]] = np.inf
    l[5, ::2] = np.nan
    l[6] = np.finfo(np.float32).min      # the type's lowest value is a score like any other
    l[7, 5] = -np.finfo(np.float32).max
    _check_route(l, topk, score=score)
    _check_route(l, topk, score=score, renormalize=False)
    _check_route(l, topk, score=score, n_group=4, topk_group=2, group_top=2)
    bias = np.zeros(E, np.float32)
    bias[3], bias[9], bias[20] = -np.inf, np.nan, 5.0
    _check_route(l, topk, bias, score=score)
    ids, w = _route(l, topk, score=score)
    assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[2, 2:] == -1).all() and ids[3, 0] == 7
    assert np.isfinite(w).all()


# ------------------------------------------------------------- plan, combine ----
@pytest.mark.gpu
@pytest.mark.parametrize("pairs,E", [(1, 1), (8, 64), (31, 3), (2048, 512), (2049, 64), (5000, 7), (65536, 256),
                                     (70001, 512)])
def test_plan(cuda_device, pairs, E):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(pairs)
    for ids in (rng.integers(0, E, pairs), rng.integers(-2, E + 2, pairs), np.full(pairs, E - 1), np.full(pairs, -1)):
        ids = ids.astype(np.int32)
        off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
        order = torch.full((pairs,), -7, dtype=torch.int32, device="cuda")
        sq.sq_moe_plan(dev(ids), off, order)
        r_off, r_order = ref.plan(ids, E)
        assert np.array_equal(host(off), r_off) and np.array_equal(host(order), r_order)


@pytest.mark.gpu
@pytest.mark.parametrize("T,topk,N", [(1, 1, 1), (3, 8, 130), (17, 2, 4096), (5, 32, 33)])
@pytest.mark.parametrize("f32", [False, True])
def test_combine(cuda_device, T, topk, N, f32):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(T + N)
    E = 40
    rows = rng.standard_normal((T * topk, N)).astype(np.float32 if f32 else np.float16)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)]).astype(np.int32)
    ids[0, -1], ids[-1, 0] = -1, E
    skip = (ids < 0) | (ids >= E)
    rows.reshape(T, topk, N)[skip] = np.nan          # never written, so never read
    w = rng.uniform(0, 1, (T, topk)).astype(np.float32)
    y = torch.empty((T, N), dtype=torch.float16, device="cuda")
    got = host(sq.sq_moe_combine(dev(rows), dev(ids), dev(w), E, y)).astype(np.float64)
    terms = np.where(skip[..., None], 0.0, w[..., None].astype(np.float64) * np.nan_to_num(rows.astype(np.float64)).reshape(T, topk, N))
    want = terms.sum(1)
    bound = topk * 2.0**-24 * np.abs(terms).sum(1) * (1 + ref.F16_HALF) + ref.F16_HALF * np.abs(want) + ref.F16_TINY
    assert (np.abs(got - want) <= bound).all()


# -------------------------------------------------------- the experts' products ----
def _experts(x, w, group, ids, E, div, bias=None, relu=False, f32=False):
    import w8a8_int8_linear_channel_b200 as sq
    P, N = ids.size, w[0].shape[1]
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(P, dtype=torch.int32, device="cuda")
    sq.sq_moe_plan(dev(ids.astype(np.int32)), off, order)
    y = torch.full((P, N), 777.0, dtype=torch.float32 if f32 else torch.float16, device="cuda")
    sq.sq_w4a16_experts(dev(x), _pack(w, group), off, order, y, div, bias=dev(bias), relu=relu)
    assert sq.sq_poll_status() == 0
    got = host(y).astype(np.float64)
    W = ref.values(*w, group)
    flat = ids.reshape(-1)
    for e in range(-1, E):
        pairs = np.nonzero(flat == e)[0] if e >= 0 else np.nonzero((flat < 0) | (flat >= E))[0]
        if len(pairs) == 0:
            continue
        if e < 0:
            assert (got[pairs] == 777.0).all()   # left as they were
            continue
        want, bound = ref.linear(x[pairs // div], W[e], None if bias is None else bias[e], relu, f32)
        assert (np.abs(got[pairs] - want) <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,topk,E,N,K,group,zero", [(1, 1, 1, 40, 48, 32, False), (1, 4, 16, 130, 272, 64, True),
                                                     (7, 3, 5, 128, 512, 128, False), (40, 4, 6, 200, 144, 32, True),
                                                     (64, 2, 3, 260, 256, 128, True), (300, 4, 8, 96, 528, 64, False),
                                                     (700, 2, 2, 136, 128, 128, False), (20, 2, 2, 130, 4112, 32, True),
                                                     (512, 2, 4, 3400, 1040, 64, True),
                                                     (48, 2, 8, 300, 528, 32, True), (400, 8, 150, 140, 144, 64, False)])
def test_experts(cuda_device, T, topk, E, N, K, group, zero):
    rng = np.random.default_rng(T + N)
    w = ref.random_weight(rng, N, K, group, zero, lead=(E,))
    x = _tokens(rng, T, K)
    ids = np.stack([rng.permutation(max(E, topk))[:topk] for _ in range(T)])
    bias = rng.standard_normal((E, N)).astype(np.float16)
    _experts(x, w, group, ids, E, topk, bias, relu=True)
    ids[rng.random(ids.shape) < 0.2] = -1
    _experts(x, w, group, ids, E, topk, f32=True)
    _experts(_tokens(rng, T * topk, K), w, group, ids, E, 1)         # a product on an earlier product's rows
    _experts(x, w, group, np.full_like(ids, E - 1), E, topk)          # every pair on one expert
    _experts(x, w, group, np.full_like(ids, -1), E, topk)             # and on none


@pytest.mark.gpu
@pytest.mark.parametrize("T,topk,E,N,K", [(1024, 8, 64, 512, 2048), (24, 4, 64, 512, 4096), (200, 4, 32, 640, 2048)])
def test_experts_back_to_back(cuda_device, T, topk, E, N, K):
    """Many launches in a row, overlapping at their ends, over weights that do not stay in L2: the
    same bits as from single launches."""
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(T)
    P = T * topk
    w4 = [_pack(ref.random_weight(np.random.default_rng(i), N, K, 128, False, lead=(1,)), 128) for i in range(2)]
    ws = []
    for i in range(4):  # four packed weights of E experts each, made of two experts' bytes in turn
        w = sq.new_w4_weight(N, K, 128, experts=E)
        n = w.packed.numel() // E
        for e in range(E):
            w.packed[e * n:(e + 1) * n] = w4[(e + i) & 1].packed
        ws.append(w)
    x = dev(_tokens(rng, T, K))
    ids = dev(np.stack([rng.permutation(E)[:topk] for _ in range(T)]).astype(np.int32))
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(P, dtype=torch.int32, device="cuda")
    sq.sq_moe_plan(ids, off, order)
    want = []
    for w in ws:
        want.append(sq.sq_w4a16_experts(x, w, off, order, torch.empty((P, N), dtype=torch.float16, device="cuda"), topk))
        torch.cuda.synchronize()
    junk = torch.empty(200 << 20, dtype=torch.uint8, device="cuda")
    outs = [torch.empty((P, N), dtype=torch.float16, device="cuda") for _ in range(40)]
    junk.fill_(1)
    for i, y in enumerate(outs):
        sq.sq_w4a16_experts(x, ws[i % 4], off, order, y, topk)
    assert sq.sq_poll_status() == 0
    for i, y in enumerate(outs):
        assert torch.equal(y, want[i % 4])
    W = ref.values(*ref.random_weight(np.random.default_rng(0), N, K, 128, False, lead=(1,)), 128)[0]
    pairs = np.nonzero(host(ids).reshape(-1) == 0)[0][:8]
    y0, bound = ref.linear(host(x)[pairs // topk], W)
    assert (np.abs(host(want[0])[pairs].astype(np.float64) - y0) <= bound).all()


@pytest.mark.gpu
def test_experts_skip_entries_no_plan_wrote(cuda_device):
    """Offsets and orders outside the pairs lead nowhere: nothing is read or written for them."""
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(2)
    w4 = _pack(ref.random_weight(rng, 64, 64, 32, False, lead=(3,)), 32)
    x = dev(_tokens(rng, 4, 64))
    order = torch.tensor([5, -3, 900, 1 << 30, 2, -(1 << 31), 0, 7], dtype=torch.int32, device="cuda")
    for off in ([0, 8, 8, 8], [-9, 4, 1 << 30, 3], [8, 0, 0, 0], [1 << 30, -(1 << 30), 5, 6]):
        y = torch.full((8, 64), 777.0, dtype=torch.float16, device="cuda")
        sq.sq_w4a16_experts(x, w4, torch.tensor(off, dtype=torch.int32, device="cuda"), order, y, 2)
        assert sq.sq_poll_status() == 0
        got = host(y)
        assert (got[[1, 3, 4, 6]] == 777.0).all()
    y = torch.full((8, 64), 777.0, dtype=torch.float16, device="cuda")
    sq.sq_w4a16_experts(x, w4, torch.tensor([0, 8, 8, 8], dtype=torch.int32, device="cuda"), order, y, 2)
    assert (host(y)[[0, 2, 5, 7]] != 777.0).any(axis=1).all()


# ------------------------------------------------------------------- the layer ----
def _layer_ref(layer_args, x, logits, up, down, group, topk, up_bias, down_bias):
    """The layer in 64 bits and its bound: the hidden rows are rounded to fp16 (the tensor core's
    input), which the down product carries on as |W| times that error; then the fp32 rows' own bound,
    the weighted sum and the output's rounding."""
    ids, wt = ref.route(logits, topk, **layer_args)
    Wu, Wd = ref.values(*up, group), ref.values(*down, group)
    y, tol = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(x.shape[0]):
        for j in range(topk):
            e = ids[t, j]
            if e < 0:
                continue
            h, hb = ref.linear(x[t:t + 1], Wu[e], None if up_bias is None else up_bias[e], True)
            z, zb = ref.linear(h, Wd[e], None if down_bias is None else down_bias[e], False, True)
            zb = zb * (1 + ref.F16_HALF) + hb @ np.abs(Wd[e]).T
            y[t] += wt[t, j] * z[0]
            tol[t] += wt[t, j] * (zb[0] + (topk + 2) * 2.0**-24 * np.abs(z[0]))
    return y, tol * (1 + ref.F16_HALF) + ref.F16_HALF * np.abs(y) + ref.F16_TINY


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 33, 150])
def test_layer(cuda_device, T):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(T)
    E, topk, K, F, group = 12, 3, 144, 208, 64
    w_up = (rng.standard_normal((E, F, K)) * 0.05).astype(np.float16)
    w_down = (rng.standard_normal((E, K, F)) * 0.05).astype(np.float16)
    ub = (rng.standard_normal((E, F)) * 0.1).astype(np.float16)
    db = (rng.standard_normal((E, K)) * 0.1).astype(np.float16)
    rb = (rng.standard_normal(E) * 0.1).astype(np.float32)
    args = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=1.5)
    layer = sq.W4Experts.from_float(dev(w_up), dev(w_down), topk, group=group, zero_point=True, router_bias=dev(rb),
                                    up_bias=dev(ub), down_bias=dev(db), **args)
    up = tuple(np.stack(p) for p in zip(*[ref.quantize(w, group, True) for w in w_up]))
    down = tuple(np.stack(p) for p in zip(*[ref.quantize(w, group, True) for w in w_down]))
    x = _tokens(rng, T, K)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[0] = -np.inf                                 # a token that no expert takes: its output is zero
    y = layer(dev(x)[None], dev(l)[None])
    assert tuple(y.shape) == (1, T, K)
    want, bound = _layer_ref(dict(args, bias=rb), x, l, up, down, group, topk, ub, db)
    got = host(y)[0].astype(np.float64)
    assert (np.abs(got - want) <= bound).all()
    assert (got[0] == 0).all()
    assert layer(dev(x)[:0], dev(l)[:0]).shape == (0, K)


@pytest.mark.gpu
def test_layer_captured_and_on_two_streams(cuda_device):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(9)
    E, topk, K, F = 16, 4, 256, 512
    layer = sq.W4Experts.from_float(dev((rng.standard_normal((E, F, K)) * 0.05).astype(np.float16)),
                                    dev((rng.standard_normal((E, K, F)) * 0.05).astype(np.float16)), topk)
    for T in (2, 700):                             # 2800 pairs: the plan takes its workspace
        xs = [dev(_tokens(rng, T, K)) for _ in range(2)]
        ls = [dev(rng.standard_normal((T, E)).astype(np.float32)) for _ in range(2)]
        want = [layer(x, l) for x, l in zip(xs, ls)]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        outs = []
        for _ in range(5):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    outs.append((i, layer(xs[i], ls[i])))
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i]) for i, y in outs)
        graphs = []
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                y = layer(xs[i], ls[i])
            graphs.append((g, y))
        torch.cuda.synchronize()
        for _ in range(3):
            for (g, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for (_, y), w in zip(graphs, want))


# ----------------------------------------------------------------- guard bands ----
class _Guard:
    """Tensors between margins of a byte pattern that every call has to leave alone."""
    MARGIN = 4096

    def __init__(self):
        self.buffers = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 2 * self.MARGIN,), 0x5A, dtype=torch.uint8, device="cuda")
        self.buffers.append((buf, n))
        return buf[self.MARGIN:self.MARGIN + n].view(dtype).view(shape)

    def check(self):
        for buf, n in self.buffers:
            assert bool((buf[:self.MARGIN] == 0x5A).all()) and bool((buf[self.MARGIN + n:] == 0x5A).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,topk,K,F,group", [(1, 5, 2, 48, 72, 32), (37, 6, 3, 272, 136, 64), (300, 4, 2, 144, 400, 128),
                                                (700, 3, 2, 1040, 4000, 128)])
def test_outputs_inside_guard_bands(cuda_device, T, E, topk, K, F, group):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(T)
    g, P = _Guard(), T * topk
    w = dev((rng.standard_normal((E, F, K)) * 0.05).astype(np.float16))
    w4 = sq.W4Weight(g((sq.sq_w4_packed_bytes(F, K, group, True) * E,), torch.uint8), F, K, group, True, E)
    sq.sq_quantize_weight_w4(w, w4)
    back = g((F, K), torch.float16)
    sq.sq_w4_dequantize(w4[E - 1], back)
    step = float(w.float().abs().max()) / 15 * 2
    assert float((back.float() - w[E - 1].float()).abs().max()) <= step
    x = dev(_tokens(rng, T, K))
    ids, wt = g((T, topk), torch.int32), g((T, topk), torch.float32)
    sq.sq_moe_route(dev(rng.standard_normal((T, E)).astype(np.float32)), ids, wt)
    off, order = g((E + 1,), torch.int32), g((P,), torch.int32)
    need = sq.sq_moe_plan_workspace_bytes(P, E)
    sq.sq_moe_plan(ids, off, order, workspace=g((need,), torch.uint8) if need else None)
    for dtype in (torch.float16, torch.float32):
        y = g((P, F), dtype)
        sq.sq_w4a16_experts(x, w4, off, order, y, topk)
        out = g((T, F), torch.float16)
        sq.sq_moe_combine(y, ids, wt, E, out)
        assert bool(torch.isfinite(out).all())
    torch.cuda.synchronize()
    assert sq.sq_poll_status() == 0
    g.check()
