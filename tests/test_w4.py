"""4-bit weights with group scales: the quantizer, the packed form and the linear."""
import ctypes

import numpy as np
import pytest
import torch

import w4_ref as ref
from gpu_util import dev, host

FAKE = ctypes.c_void_p(0x10000)
FAKE_ODD = ctypes.c_void_p(0x10004)


def _lib():
    import w8a8_int8_linear_channel_b200 as sq
    return sq._L


# ------------------------------------------------------------- refusals (CPU) ----
def test_packed_bytes():
    f = _lib().sq_w4_packed_bytes
    assert f(128, 128, 128, 0) == 8192 + 256
    assert f(129, 144, 32, 1) == 4 * (8192 + 1024 + 512)
    for bad in [(0, 128, 128, 0), (128, 120, 128, 0), (128, 0, 64, 0), (128, 128, 48, 0), (128, 133152, 32, 0), (8388481, 16, 32, 0)]:
        assert f(*bad) == 0


def test_weight_entry_points_refuse_on_the_host():
    L = _lib()
    q = L.sq_quantize_weight_w4
    assert q(None, 8, 64, None, 32, 0, FAKE, None) == 1
    assert q(FAKE, 8, 64, None, 32, 0, None, None) == 1
    assert q(FAKE, 0, 64, None, 32, 0, FAKE, None) == 1
    assert q(FAKE, 8, 72, None, 32, 0, FAKE, None) == 3
    assert q(FAKE, 8, 64, None, 16, 0, FAKE, None) == 3
    assert q(FAKE, 8, 133152, None, 32, 0, FAKE, None) == 4
    assert q(FAKE, 8, 64, FAKE_ODD, 32, 0, FAKE, None) == 2
    assert q(FAKE_ODD, 8, 64, None, 32, 0, FAKE, None) == 2
    p = L.sq_w4_pack
    assert p(None, FAKE, None, 8, 64, 32, FAKE, None) == 1
    assert p(FAKE, None, None, 8, 64, 32, FAKE, None) == 1
    assert p(FAKE, FAKE, FAKE_ODD, 8, 64, 32, FAKE, None) == 2
    assert p(FAKE, FAKE, None, 8, 64, 256, FAKE, None) == 3
    d = L.sq_w4_dequantize
    assert d(FAKE, 8, 64, 32, 0, None, None) == 1
    assert d(FAKE, 8, 64, 32, 0, FAKE_ODD, None) == 2
    assert d(FAKE_ODD, 8, 64, 32, 0, FAKE, None) == 2


def test_linear_refuses_on_the_host():
    f = _lib().sq_w4a16_linear
    good = [FAKE, 4, 64, FAKE, 8, 64, 32, 0, None, 0, FAKE, None]

    def with_(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert with_(_0=None) == 1 and with_(_3=None) == 1 and with_(_10=None) == 1
    assert with_(_1=0) == 1 and with_(_4=0) == 1 and with_(_2=56) == 1     # M, N, ldx < K
    assert with_(_2=68) == 2 and with_(_0=FAKE_ODD) == 2 and with_(_8=FAKE_ODD) == 2 and with_(_10=FAKE_ODD) == 2
    assert with_(_5=40) == 3 and with_(_6=100) == 3 and with_(_1=1 << 31) == 3 and with_(_4=8388481) == 3
    assert with_(_5=133152, _2=133152) == 4


def test_binding_refuses():
    import w8a8_int8_linear_channel_b200 as sq
    with pytest.raises(ValueError, match="4-bit form"):
        sq.new_w4_weight(8, 40, 32, device="cpu")
    with pytest.raises(ValueError, match="4-bit form"):
        sq.new_w4_weight(8, 64, 48, device="cpu")
    with pytest.raises(ValueError, match="experts"):
        sq.new_w4_weight(8, 64, 32, experts=513, device="cpu")
    w = sq.new_w4_weight(8, 64, 32, device="cpu")
    e = sq.new_w4_weight(8, 64, 32, experts=3, device="cpu")
    x, y = torch.zeros((2, 64), dtype=torch.float16), torch.zeros((2, 8), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensors"):
        sq.sq_w4a16_linear(x, w, y)
    with pytest.raises(ValueError, match="single weight"):
        sq.sq_w4a16_linear(x, e, y)
    with pytest.raises(ValueError, match="need"):
        sq.sq_w4a16_linear(x[:, :48], w, y)
    with pytest.raises(ValueError):
        sq.sq_w4a16_linear(x.float(), w, y)
    with pytest.raises(ValueError, match="zeros"):
        sq.sq_w4_pack(torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((8, 2), dtype=torch.float16), w,
                      zeros=torch.zeros((8, 2), dtype=torch.uint8))
    with pytest.raises(IndexError):
        e[3]
    with pytest.raises(ValueError, match="packed"):
        sq.W4Weight(torch.zeros(7, dtype=torch.uint8), 8, 64, 32, False)
    with pytest.raises(ValueError, match="x: need"):
        sq.W4Linear(w)(torch.zeros((2, 48), dtype=torch.float16))


def test_scaled_codes_are_fp16_numbers():
    # the reason for 8 (7) significant bits in the quantizer's scales: every value of a weight it
    # makes is exactly an fp16 number
    rng = np.random.default_rng(3)
    for zero in (False, True):
        w = (rng.standard_normal((64, 256)) * 0.02).astype(np.float16)
        c, s, z = ref.quantize(w, 32, zero)
        v = ref.values(c, s, z, 32)
        assert np.array_equal(v, v.astype(np.float16).astype(np.float64))


# ------------------------------------------------------------------------ GPU ----
def _pack(w, group):
    import w8a8_int8_linear_channel_b200 as sq
    codes, scales, zeros = w
    lead = codes.shape[0] if codes.ndim == 3 else None
    w4 = sq.new_w4_weight(codes.shape[-2], codes.shape[-1], group, zeros is not None, experts=lead)
    w4.packed.fill_(0xA5)
    return sq.sq_w4_pack(dev(codes), dev(scales), w4, zeros=dev(zeros))


def _tokens(rng, M, K):
    x = rng.standard_normal((M, K))
    x[:, rng.integers(0, K, 2)] *= 30
    return x.astype(np.float16)


SHAPES = [(1, 16), (3, 32), (16, 48), (100, 112), (128, 128), (129, 144), (300, 1040), (257, 4112)]


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K", SHAPES)
def test_pack_and_dequantize(cuda_device, N, K, group, zero):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(N * K + group)
    w = ref.random_weight(rng, N, K, group, zero)
    out = torch.full((N, K), float("nan"), dtype=torch.float16, device="cuda")
    sq.sq_w4_dequantize(_pack(w, group), out)
    assert np.array_equal(host(out).astype(np.float64), ref.values(*w, group))


@pytest.mark.gpu
def test_pack_experts_on_another_stream(cuda_device):
    # experts whose scales start off 16 bytes, filled in on the call's stream only after a while
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(3)
    E, N, K, group = 3, 5, 48, 32
    c, s, z = (dev(a) for a in ref.random_weight(rng, N, K, group, True, lead=(E,)))
    want = sq.sq_w4_pack(c, s, sq.new_w4_weight(N, K, group, True, experts=E), z).packed
    c2, s2, z2 = (torch.zeros_like(t) for t in (c, s, z))
    w4 = sq.new_w4_weight(N, K, group, True, experts=E)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        c2.copy_(c), s2.copy_(s), z2.copy_(z)
    sq.sq_w4_pack(c2, s2, w4, z2, stream=side)
    side.synchronize()
    assert torch.equal(w4.packed, want)


@pytest.mark.gpu
def test_more_blocks_than_a_grid_holds_is_refused(cuda_device):
    # refused before any launch, and no error stays behind for the next call
    x = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    a = x.data_ptr()
    assert _lib().sq_w4a16_linear(a, 0x7fffffff, 64, a, 8388480, 64, 32, 0, None, 0, a, None) == 3
    torch.cuda.synchronize()
    assert float(x.sum()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("fold", [False, True])
@pytest.mark.parametrize("N,K", SHAPES)
def test_quantize(cuda_device, N, K, group, zero, fold):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(N + K + group)
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float16)
    w[0, : K // 2] = 0                                      # a group of zeros
    w[-1, 1::2] = np.abs(w[-1, 1::2])                       # and one-sided ranges
    w[N // 2] = rng.integers(-15, 16, K) * np.float16(2.0**-7)  # many ties
    s = rng.uniform(0.5, 4.0, K).astype(np.float32) if fold else None
    w4 = sq.new_w4_weight(N, K, group, zero)
    w4.packed.fill_(0xA5)
    sq.sq_quantize_weight_w4(dev(w), w4, s=dev(s))
    c, sc, z = ref.quantize(w, group, zero, s)
    # the packed bytes themselves: scales, zero points, padding and all
    assert torch.equal(w4.packed, _pack((c, sc, z), group).packed)
    out = torch.empty((N, K), dtype=torch.float16, device="cuda")
    sq.sq_w4_dequantize(w4, out)
    assert np.array_equal(host(out).astype(np.float64), ref.values(c, sc, z, group))


@pytest.mark.gpu
@pytest.mark.parametrize("zero", [False, True])
def test_quantize_nonfinite_and_extreme(cuda_device, zero):
    import w8a8_int8_linear_channel_b200 as sq
    K, group = 128, 32
    w = np.zeros((8, K), np.float16)
    w[:] = np.linspace(-1, 1, K).astype(np.float16)
    w[0, 5] = np.nan
    w[1, 40] = np.inf
    w[2, 40] = -np.inf
    w[3] = 65504.0
    w[4] = np.float16(2.0**-24)                  # smallest subnormal: the scale rounds to 0 or one step
    w[5, 64:96] = np.nan
    w[6] = np.arange(K) % 23 * 2.0**-24 - 11 * 2.0**-24      # subnormal scales: -8 has to be clamped to -7
    w[7] = (np.arange(K) % 31 - 10) * 2.0**-23
    w4 = sq.new_w4_weight(8, K, group, zero)
    sq.sq_quantize_weight_w4(dev(w), w4)
    out = torch.empty((8, K), dtype=torch.float16, device="cuda")
    with np.errstate(invalid="ignore"):
        want = ref.values(*ref.quantize(w, group, zero), group)
    got = host(sq.sq_w4_dequantize(w4, out)).astype(np.float64)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isnan(got[1, 32:64]).all() and not np.isnan(got[0]).any() and (got[5, 64:96] == 0).all()


def _check_linear(x, w, group, bias=None, relu=False, w4=None, ldx=None):
    import w8a8_int8_linear_channel_b200 as sq
    M, K = x.shape
    N = w[0].shape[0]
    w4 = _pack(w, group) if w4 is None else w4
    xd = dev(x)
    if ldx is not None:  # rows inside a wider tensor whose other columns are NaN
        wide = torch.full((M, ldx), float("nan"), dtype=torch.float16, device="cuda")
        wide[:, :K] = xd
        xd = wide[:, :K]
    y = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    sq.sq_w4a16_linear(xd, w4, y, bias=dev(bias), relu=relu)
    want, bound = ref.linear(x, ref.values(*w, group), bias, relu)
    err = np.abs(host(y).astype(np.float64) - want)
    assert (err <= bound).all(), f"worst {np.nanmax(err / bound)} of the bound"
    assert sq.sq_poll_status() == 0
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 100, 129, 257, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (100, 112), (129, 144), (300, 1040)])
def test_linear(cuda_device, M, N, K, group, zero):
    rng = np.random.default_rng(M * 1000 + N + K)
    w = ref.random_weight(rng, N, K, group, zero)
    bias = rng.standard_normal(N).astype(np.float16) if M % 2 else None
    _check_linear(_tokens(rng, M, K), w, group, bias, relu=M % 3 == 0, ldx=K + 24 if M % 4 else None)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("M,N,K", [(10, 5000, 2064), (33, 2100, 2320), (64, 1000, 5008), (65, 1100, 2192),
                                   (130, 777, 2320), (500, 900, 592), (1000, 3000, 272)])
def test_linear_many_tokens(cuda_device, M, N, K, group, zero):
    # enough work for the kernel of many tokens whatever their number: odd sizes, one and two weight tiles
    rng = np.random.default_rng(M * 1000 + N + K)
    w = ref.random_weight(rng, N, K, group, zero)
    bias = rng.standard_normal(N).astype(np.float16) if M % 2 else None
    _check_linear(_tokens(rng, M, K), w, group, bias, relu=M % 3 == 0, ldx=K + 24 if M % 4 else None)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (4, 64, 49152), (16, 1000, 12288), (32, 49152, 256),
                                   (128, 512, 4096), (1000, 777, 4112), (2048, 256, 512), (640, 7700, 144),
                                   (1280, 4000, 1040), (40, 130, 8208)])
def test_linear_larger(cuda_device, M, N, K):
    rng = np.random.default_rng(M + N + K)
    _check_linear(_tokens(rng, M, K), ref.random_weight(rng, N, K, 128, M % 3 == 1), 128)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3, 140, 272), (16, 140, 272), (40, 140, 272), (200, 140, 272),
                                   (40, 2100, 2320), (200, 2100, 528), (1500, 2100, 272)])
def test_linear_nonfinite_tokens_stay_in_their_row(cuda_device, M, N, K):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(M)
    group = 64
    w = ref.random_weight(rng, N, K, group, True)
    x = _tokens(rng, M, K)
    y0 = host(_check_linear(x, w, group))
    x[1, K - 2], x[2, 0] = np.nan, np.inf
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    sq.sq_w4a16_linear(dev(x), _pack(w, group), y)
    got = host(y)
    assert np.isnan(got[1]).all() and not np.isfinite(got[2]).any()
    keep = [m for m in range(M) if m not in (1, 2)]
    assert np.array_equal(got[keep].view(np.uint16), y0[keep].view(np.uint16))
    sq.sq_w4a16_linear(dev(x), _pack(w, group), y, relu=True)
    assert (host(y)[1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 130), (24, 130), (150, 130), (24, 25000), (150, 8000), (500, 8000)])
def test_linear_overflow_and_zero_scales(cuda_device, M, N):
    # sums past 65504 become Inf; groups of scale 0 contribute nothing
    import w8a8_int8_linear_channel_b200 as sq
    K, group = 160, 32
    codes = np.full((N, K), 15, np.uint8)
    scales = np.full((N, 5), 64.0, np.float16)
    scales[1] = 0
    x = np.full((M, K), 100.0, np.float16)
    x[0] = 0
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    got = host(sq.sq_w4a16_linear(dev(x), _pack((codes, scales, None), group), y))
    assert (got[:, 1] == 0).all() and (got[0] == 0).all()
    assert np.isinf(got[1:, [0, 2, 129]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 520), (13, 520), (30, 520), (90, 520), (300, 520), (20, 8001), (128, 8008)])
def test_linear_streams_graphs_and_repeats(cuda_device, M, N):
    """The same bits from: a repeated call, another stream, two streams at once, a captured and
    replayed call whose input changed, and an output inside guard bands."""
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(M)
    K, group = 2064, 128
    w4 = _pack(ref.random_weight(rng, N, K, group, True), group)
    xa, xb = dev(_tokens(rng, M, K)), dev(_tokens(rng, M, K))
    new = lambda: torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    ya, yb = sq.sq_w4a16_linear(xa, w4, new()), sq.sq_w4a16_linear(xb, w4, new())
    assert torch.equal(sq.sq_w4a16_linear(xa, w4, new()), ya)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(new(), new()) for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in outs:
        sq.sq_w4a16_linear(xa, w4, a, stream=s1)
        sq.sq_w4a16_linear(xb, w4, b, stream=s2)
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, ya) and torch.equal(b, yb)
    x, y = xa.clone(), new()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sq.sq_w4a16_linear(x, w4, y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ya)
    x.copy_(xb)
    y.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, yb)
    band = torch.full((M * N + 4096,), 0x5A5A, dtype=torch.int16, device="cuda")
    inner = band[2048:2048 + M * N].view(torch.float16).view(M, N)
    sq.sq_w4a16_linear(xa, w4, inner)
    assert torch.equal(inner, ya)
    assert bool((band[:2048] == 0x5A5A).all()) and bool((band[2048 + M * N:] == 0x5A5A).all())


@pytest.mark.gpu
def test_w4_linear_layer(cuda_device):
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(5)
    N, K = 200, 320
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float16)
    s = rng.uniform(0.5, 2.0, K).astype(np.float32)
    bias = rng.standard_normal(N).astype(np.float16)
    layer = sq.W4Linear.from_float(dev(w), group=64, zero_point=True, s=dev(s), bias=dev(bias), relu=True)
    x = _tokens(rng, 6, K)
    y = layer(dev(x).view(2, 3, K))
    assert tuple(y.shape) == (2, 3, N)
    want, bound = ref.linear(x, ref.values(*ref.quantize(w, 64, True, s), 64), bias, True)
    assert (np.abs(host(y).reshape(6, N).astype(np.float64) - want) <= bound).all()
    assert layer(dev(x)[:0]).shape == (0, N)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 40, 300])
def test_wait_that_runs_out_is_reported(cuda_device, M):
    """With the smallest wait budget a call may give up; it must say so or be right."""
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(8)
    w = ref.random_weight(rng, 2048, 4096, 128, False)
    w4, x = _pack(w, 128), dev(_tokens(rng, M, 4096))
    good = sq.sq_w4a16_linear(x, w4, torch.empty((M, 2048), dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()
    try:
        sq.sq_set_wait_budget_ns(1000)
        y = sq.sq_w4a16_linear(x, w4, torch.empty_like(good))
        assert sq.sq_poll_status() in (0, 8)
    finally:
        sq.sq_set_wait_budget_ns(2_000_000_000)
    y = sq.sq_w4a16_linear(x, w4, torch.empty_like(good))
    assert sq.sq_poll_status() == 0 and torch.equal(y, good)


@pytest.mark.gpu
def test_products_beside_the_int8_linear(cuda_device):
    """4-bit and INT8 linears on two streams at once, whose CTAs share SMs and tensor memory: the bits
    of each running alone."""
    import w8a8_int8_linear_channel_b200 as sq
    rng = np.random.default_rng(12)
    N, K = 2048, 2064
    w = dev((rng.standard_normal((N, K)) * 0.05).astype(np.float16))
    calib = dev(_tokens(rng, 64, K))
    int8, w4 = sq.SmoothQuantLinear.from_float(w, calib), sq.W4Linear.from_float(w)
    xs = [dev(_tokens(rng, M, K)) for M in (1, 40, 100, 500, 1200)]
    alone = [(int8(x).clone(), w4(x).clone()) for x in xs]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a, b = [], []
        for x in xs:
            with torch.cuda.stream(s1):
                a.append(w4(x))
            with torch.cuda.stream(s2):
                b.append(int8(x).clone())
        torch.cuda.synchronize()
        assert sq.sq_poll_status() == 0
        for (y8, y4), p, q in zip(alone, a, b):
            assert torch.equal(y4, p) and torch.equal(y8, q)
