"""Every form of the 4-bit products against the definition.  Which form a call takes follows from its
sizes and the number of SMs; the rule is restated here, so that a test knows what it reached."""
import numpy as np
import pytest
import torch

import w4_ref as ref
from gpu_util import dev
from test_w4 import _pack, _tokens


def _ceil(a, b):
    return -(-a // b)


def dense_form(M, N, K, sms):
    """"stream" or (tokens per block, weight tiles per CTA) of sq_w4a16_linear."""
    nt, kt = _ceil(N, 128), _ceil(K, 128)
    if M <= 8 or _ceil(M, 8) * 2 * nt * kt <= 32 * sms:
        return "stream"
    if M <= 64:
        return 64, 1
    blocks = _ceil(M, 128)
    pairs = blocks * _ceil(nt, 2)
    small, large = _ceil(blocks * nt, sms), _ceil(pairs, sms)
    return (128, 2) if pairs >= sms and large * 100 <= small * 53 else (128, 1)


def slices(M, N, K, sms):
    """CTAs along K of the tcgen05 form of sq_w4a16_linear."""
    bt, rt = dense_form(M, N, K, sms)
    if rt == 2:
        return 1
    units, kt, best, out = _ceil(N, 128) * _ceil(M, bt), _ceil(K, 128), None, 1
    for s in range(1, 9):
        if s > 1 and kt // s < 4:
            break
        per_sm = _ceil(units * s, sms if s <= 2 else sms - sms // 8)
        cost = (per_sm + 1) // 2 * _ceil(kt, s) * (39 if bt == 64 else 59) + per_sm * (450 if s == 1 else 850)
        if best is None or cost < best:
            best, out = cost, s
    return out


# (M, N, K, slices or None), by form; odd channels, an odd number of weight tiles, ragged last blocks, a last K tile
# of 16, 64 or 80 k, rows of 16 bytes and not (the two ways an output is stored), one slice and several
CASES = {
    (64, 1): [(10, 9000, 2064, 1), (33, 3200, 2320, None), (17, 25001, 592, 1), (16, 1000, 32784, None),
              (64, 1000, 5008, None), (49, 20008, 272, 1), (32, 777, 12368, None)],
    (128, 1): [(65, 2100, 4176, None), (100, 3200, 2128, None), (130, 1501, 4112, None), (500, 1600, 1104, 1),
               (257, 6000, 592, 1), (193, 12345, 272, 1), (72, 130, 33008, None)],
    (128, 2): [(1930, 3904, 272, 1), (1930, 3900, 272, 1), (1930, 3901, 80, 1), (1664, 4737, 144, 1),
               (3841, 2000, 144, 1)],
    "stream": [(1, 4096, 4096, None), (3, 777, 12368, None), (8, 12345, 592, None), (24, 520, 2064, None),
               (300, 130, 272, None)],
}
FLAT = [(form, *c) for form, cs in CASES.items() for c in cs]


@pytest.mark.parametrize("form,M,N,K,s", FLAT)
def test_the_cases_reach_their_form(form, M, N, K, s):
    assert dense_form(M, N, K, 148) == form
    if form != "stream":
        n = slices(M, N, K, 148)
        assert n > 1 if s is None else n == s


class Product:
    """x W^T in 64 bits, on the GPU, with what the bounds need."""

    def __init__(self, x, W):
        self.x, self.W = dev(x).double(), dev(W)
        self.y = self.x @ self.W.T
        self.S = self.x.abs() @ self.W.abs().T
        self.K = x.shape[1]
        self.squares = float((self.x.square() @ self.W.square().T).sum())

    def expect(self, bias=None, relu=False, f32=False):
        """(y, a bound for every element, a bound for the root of the squared errors' sum).

        Elements: as in w4_ref.linear.  That bound grows with K and would hide a lost K tile among
        many; the norm's does not: every one of K additions is off by at most one fp32 step, 2^-23,
        of a partial sum.  For weights of random sign a partial sum's mean square is that of its
        terms, so over all outputs the errors' norm is at most K 2^-23 times the norm of the terms
        (the triangle inequality: no luck assumed among the errors), and half a step of the output.
        One K tile lost of 384 changes 1 / sqrt(384) = 5% of the norm; with K = 49152 the bound is 0.6%."""
        y, S, squares = self.y, self.S, self.squares
        if bias is not None:
            b = dev(bias).double()
            y, S, squares = y + b, S + b.abs(), squares + float(b.square().sum()) * y.shape[0]
        if relu:
            y = y.clamp(min=0.0)
        last = 2.0**-24 * y.abs() if f32 else ref.F16_HALF * y.abs() + ref.F16_TINY
        bound = (self.K + 2 * (self.K // 32 + 1) + 16) * 2.0**-23 * S * (1 + ref.F16_HALF) + last
        return y, bound, (self.K + 16) * 2.0**-23 * squares**0.5 + float(last.norm())

    def check(self, got, *args, **kw):
        y, bound, norm = self.expect(*args, **kw)
        err = (got.double() - y).abs()
        assert bool((err <= bound).all()), f"worst {float((err / bound).nan_to_num(9e9).max())} of the bound"
        assert float(err.norm()) <= norm, f"{float(err.norm()) / norm} of the norm's bound"


def linear(x, w4, bias=None, relu=False, wide=False):
    import w8a8_int8_linear_channel_b200 as sq
    M, K = x.shape
    xd = dev(x)
    if wide:  # rows inside a wider tensor whose other columns are NaN
        t = torch.full((M, K + 24), float("nan"), dtype=torch.float16, device="cuda")
        t[:, :K] = xd
        xd = t[:, :K]
    y = torch.full((M, w4.N), float("nan"), dtype=torch.float16, device="cuda")
    sq.sq_w4a16_linear(xd, w4, y, bias=dev(bias), relu=relu)
    assert sq.sq_poll_status() == 0
    return y


def _form_here(M, N, K):
    return dense_form(M, N, K, torch.cuda.get_device_properties(0).multi_processor_count)


@pytest.mark.gpu
@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (64, True), (128, False), (128, True), (32, False)])
@pytest.mark.parametrize("form,M,N,K,s", FLAT)
def test_random_weights(cuda_device, form, M, N, K, s, group, zero):
    assert _form_here(M, N, K) == form
    rng = np.random.default_rng(M + N + K + group)
    w = ref.random_weight(rng, N, K, group, zero)
    x, w4 = _tokens(rng, M, K), _pack(w, group)
    bias = rng.standard_normal(N).astype(np.float16)
    p = Product(x, ref.values(*w, group))
    p.check(linear(x, w4))
    p.check(linear(x, w4, bias, True, True), bias, True)
