"""4-bit weights with group scales, and mixture-of-experts layers on them.

The ctypes binding of the ``sq_w4*`` and ``sq_moe_*`` entry points of
``include/sq.h`` (argument marshalling only, like the rest of the package) and
the two layers built from them: ``W4Linear`` beside ``SmoothQuantLinear`` for
layers whose time is the weight's bytes, and ``W4Experts``, a routed
feed-forward layer (up, ReLU, down) over 4-bit experts.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _L, _check, _p, _rows, _vec

MOE_MAX_EXPERTS = 512
MOE_MAX_TOPK = 32
GROUPS = (32, 64, 128)


# These calls take a few microseconds on the GPU, so their host side counts: one
# look at the current device per call, plain integers as pointers, and the
# current stream's handle without a Stream object where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_F16, _F32, _I32 = torch.float16, torch.float32, torch.int32


def _ptrs(*tensors):
    """Device addresses (None stays None); a host tensor or one on another GPU is refused as by _p."""
    dev = -2
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if dev == -2 and t.is_cuda:
            dev = _current_device()
        out.append(t.data_ptr() if t.get_device() == dev else _p(t))
    return out


def _stream(stream) -> int:
    return _raw_stream(_current_device()) if stream is None else stream.cuda_stream


def _realigned(logits: torch.Tensor, stream=None) -> torch.Tensor:
    """Rows that start off 16 bytes (a slice of a batch may) copied, contiguous, in the stream's order."""
    with torch.cuda.stream(stream):
        return logits.clone(memory_format=torch.contiguous_format)


class W4Weight:
    """A packed 4-bit weight [N, K] (or one per expert): the library's buffer and its shape."""

    def __init__(self, packed: torch.Tensor, N: int, K: int, group: int, zero_point: bool,
                 experts: Optional[int] = None):
        need = sq_w4_packed_bytes(N, K, group, zero_point) * (1 if experts is None else experts)
        if packed.dtype != torch.uint8 or not packed.is_contiguous() or packed.numel() != need or need == 0:
            raise ValueError(f"packed: need a contiguous uint8 tensor of {need} bytes")
        self.packed, self.N, self.K = packed, N, K
        self.group, self.zero_point, self.experts = group, bool(zero_point), experts

    def __getitem__(self, e: int) -> "W4Weight":
        """Expert e's weight (a view)."""
        if self.experts is None or not 0 <= e < self.experts:
            raise IndexError(f"expert {e} of {self.experts}")
        n = self.packed.numel() // self.experts
        return W4Weight(self.packed[e * n:(e + 1) * n], self.N, self.K, self.group, self.zero_point)


def sq_w4_packed_bytes(N: int, K: int, group: int, zero_point: bool) -> int:
    return int(_L.sq_w4_packed_bytes(N, K, group, int(bool(zero_point))))


def new_w4_weight(N: int, K: int, group: int = 128, zero_point: bool = False, experts: Optional[int] = None,
                  device=None) -> W4Weight:
    """An empty packed weight, to be filled by sq_quantize_weight_w4 or sq_w4_pack."""
    n = sq_w4_packed_bytes(N, K, group, zero_point)
    if n == 0 or (experts is not None and not 1 <= experts <= MOE_MAX_EXPERTS):
        raise ValueError(f"no packed 4-bit form of N={N}, K={K}, group={group}, experts={experts} "
                         f"(K % 16 == 0, group one of {GROUPS}, at most {MOE_MAX_EXPERTS} experts)")
    packed = torch.empty(n * (experts or 1), dtype=torch.uint8, device=device or "cuda")
    return W4Weight(packed, N, K, group, zero_point, experts)


def _dense(w4: W4Weight, what: str) -> None:
    if w4.experts is not None:
        raise ValueError(f"{what}: a single weight is needed, this one holds {w4.experts} experts")


def _tensor(t: torch.Tensor, dtype, shape: tuple, name: str) -> None:
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous {dtype} {tuple(shape)} tensor")


def sq_quantize_weight_w4(w: torch.Tensor, w4: W4Weight, s=None, stream=None) -> W4Weight:
    """Quantize fp16 w [N, K] ([E, N, K] for experts), folded by s [K] when given, into w4."""
    lead = () if w4.experts is None else (w4.experts,)
    _tensor(w, torch.float16, lead + (w4.N, w4.K), "w")
    _vec(s, w4.K, torch.float32, "s")
    for src, dst in ((w, w4),) if w4.experts is None else ((w[e], w4[e]) for e in range(w4.experts)):
        a, b, c = _ptrs(src, s, dst.packed)
        _check(_L.sq_quantize_weight_w4(a, w4.N, w4.K, b, w4.group, w4.zero_point, c, _stream(stream)),
               "sq_quantize_weight_w4")
    return w4


def sq_w4_pack(codes: torch.Tensor, scales: torch.Tensor, w4: W4Weight, zeros=None, stream=None) -> W4Weight:
    """Pack uint8 codes [N, K], fp16 scales and uint8 zeros [N, ceil(K / group)] (each with a leading
    [E] for experts) into w4; zeros exactly when w4 has zero points."""
    lead = () if w4.experts is None else (w4.experts,)
    G = -(-w4.K // w4.group)
    _tensor(codes, torch.uint8, lead + (w4.N, w4.K), "codes")
    _tensor(scales, torch.float16, lead + (w4.N, G), "scales")
    if (zeros is not None) != w4.zero_point:
        raise ValueError("zeros: given exactly when the weight has zero points")
    if zeros is not None:
        _tensor(zeros, torch.uint8, lead + (w4.N, G), "zeros")
    if w4.experts is None:
        parts = [(codes, scales, zeros, w4)]
    else:
        parts = [(codes[e], scales[e], None if zeros is None else zeros[e], w4[e]) for e in range(w4.experts)]
    for c, s, z, dst in parts:
        if s.data_ptr() % 16 or (z is not None and z.data_ptr() % 16):  # an expert's slice may start off 16 bytes
            with torch.cuda.stream(stream):  # copied, and the copy's memory reused, in this stream's order
                s, z = s.clone(), None if z is None else z.clone()
        pc, ps, pz, pw = _ptrs(c, s, z, dst.packed)
        _check(_L.sq_w4_pack(pc, ps, pz, w4.N, w4.K, w4.group, pw, _stream(stream)), "sq_w4_pack")
    return w4


def sq_w4_dequantize(w4: W4Weight, out: torch.Tensor, stream=None) -> torch.Tensor:
    """out fp16 [N, K] = the values of a packed weight."""
    _dense(w4, "sq_w4_dequantize")
    _tensor(out, torch.float16, (w4.N, w4.K), "out")
    pw, po = _ptrs(w4.packed, out)
    _check(_L.sq_w4_dequantize(pw, w4.N, w4.K, w4.group, w4.zero_point, po, _stream(stream)), "sq_w4_dequantize")
    return out


def sq_w4a16_linear(x: torch.Tensor, w4: W4Weight, y: torch.Tensor, bias=None, relu: bool = False,
                    stream=None) -> torch.Tensor:
    """y fp16 [M, N] = fp16(x @ W^T + bias) with a packed 4-bit W; ReLU optional."""
    if w4.experts is not None:
        _dense(w4, "sq_w4a16_linear")
    shape = x.shape
    if x.dtype != _F16 or len(shape) != 2:
        _rows(x, _F16, "x")
    M, K = shape
    ld, inner = x.stride()
    N = w4.N
    if K != w4.K or inner != 1:
        raise ValueError(f"x: need [M, {w4.K}] with a unit inner stride, got {tuple(shape)}")
    if M == 1:
        ld = K  # the stride of a single row means nothing
    if y.dtype != _F16 or y.shape != (M, N) or not y.is_contiguous():
        _tensor(y, _F16, (M, N), "y")
    if bias is not None:
        _vec(bias, N, _F16, "bias")
    packed = w4.packed
    dev = x.get_device()
    if dev < 0 or dev != packed.get_device() or dev != y.get_device() or (
            bias is not None and dev != bias.get_device()) or dev != _current_device():
        _ptrs(x, packed, y, bias)  # says what is wrong
    status = _L.sq_w4a16_linear(x.data_ptr(), M, ld, packed.data_ptr(), N, K, w4.group, w4.zero_point,
                                None if bias is None else bias.data_ptr(), bool(relu), y.data_ptr(),
                                _raw_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status, "sq_w4a16_linear")
    return y


_SCORES = {"softmax": 0, "sigmoid": 1}


def sq_moe_route(logits: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, bias=None, score: str = "softmax",
                 n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                 scale: float = 1.0, stream=None):
    """The topk experts of every token (ids int32 [T, topk], largest choice first) and their weights
    (fp32 [T, topk]) from router logits, fp32 or fp16 [T, E] (copied first when they start off 16 bytes)."""
    half = logits.dtype == _F16
    if not half and logits.dtype != _F32:
        raise ValueError("logits: fp32 or fp16")
    if score not in _SCORES:
        raise ValueError(f"score: one of {sorted(_SCORES)}")
    if logits.dim() != 2:
        _rows(logits, logits.dtype, "logits")
    T, E = logits.shape
    ld, inner = logits.stride()
    if inner != 1:
        _rows(logits, logits.dtype, "logits")
    shape = ids.shape
    if len(shape) != 2 or shape[0] != T:
        raise ValueError(f"ids: need [{T}, topk]")
    if ids.dtype != _I32 or not ids.is_contiguous():
        _tensor(ids, _I32, shape, "ids")
    if weights.dtype != _F32 or weights.shape != shape or not weights.is_contiguous():
        _tensor(weights, _F32, shape, "weights")
    if bias is not None:
        _vec(bias, E, _F32, "bias")
    if logits.data_ptr() % 16:
        logits, ld = _realigned(logits, stream), E
    dev = logits.get_device()
    if dev < 0 or dev != ids.get_device() or dev != weights.get_device() or (
            bias is not None and dev != bias.get_device()) or dev != _current_device():
        _ptrs(logits, ids, weights, bias)  # says what is wrong
    status = _L.sq_moe_route(logits.data_ptr(), half, T, E, E if T == 1 else ld,
                             None if bias is None else bias.data_ptr(), _SCORES[score], n_group, topk_group,
                             group_top, shape[1], bool(renormalize), scale, ids.data_ptr(), weights.data_ptr(),
                             _raw_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status, "sq_moe_route")
    return ids, weights


def sq_moe_plan_workspace_bytes(pairs: int, experts: int) -> int:
    return int(_L.sq_moe_plan_workspace_bytes(pairs, experts))


def sq_moe_plan(ids: torch.Tensor, offsets: torch.Tensor, order: torch.Tensor, workspace=None, stream=None):
    """The (token, slot) pairs of ids (int32, any shape) stably sorted by expert: offsets int32
    [E + 1], order int32 [ids.numel()].  Without a workspace one is allocated for the call."""
    pairs, E = ids.numel(), offsets.numel() - 1
    if ids.dtype != _I32 or not ids.is_contiguous():
        raise ValueError("ids: need a contiguous int32 tensor")
    if offsets.dtype != _I32 or not offsets.is_contiguous():
        _vec(offsets, E + 1, _I32, "offsets")
    if order.dtype != _I32 or order.numel() != pairs or not order.is_contiguous():
        _vec(order, pairs, _I32, "order")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: need a contiguous tensor")
    if workspace is None:
        need = int(_L.sq_moe_plan_workspace_bytes(pairs, E))
        if need:
            with torch.cuda.stream(stream):  # freed memory is reused in this stream's order
                workspace = torch.empty(need, dtype=torch.uint8, device=ids.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    dev = ids.get_device()
    if dev < 0 or dev != offsets.get_device() or dev != order.get_device() or (
            workspace is not None and dev != workspace.get_device()) or dev != _current_device():
        _ptrs(ids, offsets, order, workspace)  # says what is wrong
    status = _L.sq_moe_plan(ids.data_ptr(), pairs, E, offsets.data_ptr(), order.data_ptr(),
                            None if workspace is None else workspace.data_ptr(), ws_bytes,
                            _raw_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status, "sq_moe_plan")
    return offsets, order


def sq_w4a16_experts(x: torch.Tensor, w4: W4Weight, offsets: torch.Tensor, order: torch.Tensor, y: torch.Tensor,
                     pairs_per_row: int = 1, bias=None, relu: bool = False, stream=None) -> torch.Tensor:
    """y [pairs, N] (fp16 or fp32): pair p, which the plan lists under expert e, gets
    x[p // pairs_per_row] @ W_e^T + bias[e]; rows the plan leaves out keep their contents."""
    if w4.experts is None:
        raise ValueError("w4: need a weight of several experts")
    rows, K, ld = _rows(x, torch.float16, "x")
    if K != w4.K:
        raise ValueError(f"x: need [rows, {w4.K}], got {tuple(x.shape)}")
    if rows == 1:
        ld = K
    pairs = order.numel()
    _vec(offsets, w4.experts + 1, torch.int32, "offsets")
    _vec(order, pairs, torch.int32, "order")
    if bias is not None:
        _tensor(bias, torch.float16, (w4.experts, w4.N), "bias")
    if y.dtype not in (torch.float16, torch.float32):
        raise ValueError("y: fp16 or fp32")
    _tensor(y, y.dtype, (pairs, w4.N), "y")
    px, pw, pb, pf, po, py = _ptrs(x, w4.packed, bias, offsets, order, y)
    _check(_L.sq_w4a16_experts(px, rows, ld, pw, w4.experts, w4.N, K, w4.group, w4.zero_point, pb, bool(relu), pf, po,
                               pairs, pairs_per_row, py, y.dtype == torch.float32, _stream(stream)),
           "sq_w4a16_experts")
    return y


def sq_moe_combine(y_pairs: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, experts: int, y: torch.Tensor,
                   stream=None) -> torch.Tensor:
    """y fp16 [T, N] = the weighted sum of every token's rows of y_pairs [T * topk, N] (fp16 or fp32)."""
    if y_pairs.dtype not in (torch.float16, torch.float32):
        raise ValueError("y_pairs: fp16 or fp32")
    if ids.dim() != 2:
        raise ValueError("ids: need [T, topk]")
    T, topk = ids.shape
    N = y_pairs.shape[-1]
    _tensor(ids, torch.int32, (T, topk), "ids")
    _tensor(weights, torch.float32, (T, topk), "weights")
    _tensor(y_pairs, y_pairs.dtype, (T * topk, N), "y_pairs")
    _tensor(y, torch.float16, (T, N), "y")
    pz, pi, pw, py = _ptrs(y_pairs, ids, weights, y)
    _check(_L.sq_moe_combine(pz, y_pairs.dtype == torch.float32, pi, pw, T, topk, N, experts, py, _stream(stream)),
           "sq_moe_combine")
    return y


# ------------------------------------------------------------- layer API ----
class W4Linear:
    """A linear layer with a packed 4-bit weight: fp16 [..., K] -> fp16 [..., N]."""

    def __init__(self, w4: W4Weight, bias: Optional[torch.Tensor] = None, relu: bool = False):
        _dense(w4, "W4Linear")
        self.w4, self.bias, self.relu = w4, bias, relu

    @classmethod
    def from_float(cls, w: torch.Tensor, group: int = 128, zero_point: bool = False, s=None, bias=None,
                   relu: bool = False) -> "W4Linear":
        """Quantize an fp16 weight [N, K].  With s (fp32 [K], e.g. from sq_smooth_fold) the weight is
        folded by it first; the layer's input is then the smoothed one, x / s."""
        w4 = new_w4_weight(w.shape[0], w.shape[1], group, zero_point, device=w.device)
        return cls(sq_quantize_weight_w4(w, w4, s=s), bias, relu)

    def forward(self, x: torch.Tensor, y: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Leading dimensions are flattened into tokens; an empty batch launches nothing."""
        N, K = self.w4.N, self.w4.K
        if x.dim() < 1 or x.shape[-1] != K:
            raise ValueError(f"x: need [..., {K}], got {tuple(x.shape)}")
        lead = tuple(x.shape[:-1])
        x2 = x if x.dim() == 2 else x.reshape(-1, K)
        if y is None:
            y = x.new_empty(lead + (N,), dtype=_F16)
        elif tuple(y.shape) not in (lead + (N,), (x2.shape[0], N)) or not y.is_contiguous():
            raise ValueError(f"y: need a contiguous fp16 {lead + (N,)} tensor")
        if x2.shape[0]:
            sq_w4a16_linear(x2, self.w4, y.view(-1, N), self.bias, self.relu)
        return y

    __call__ = forward


class W4Experts:
    """A mixture-of-experts feed-forward layer on packed 4-bit weights.

    up [E, F, K] and down [E, K, F]: y[t] = sum_j weight[t, j] * down_e(relu(up_e(x[t]))) over the
    topk experts e that sq_moe_route picks for token t from its router logits.

    The hidden rows relu(up_e(x)) are fp16, like every activation of the library, since the down
    product takes fp16 tokens: one rounding of 2^-11 at most, and Inf past 65504.  (fp32 ones would have to
    be split in two for the tensor cores, twice the down product's MMAs.)  The down product's rows are fp32, so the
    output is rounded once.  With outputs of random weights the layer is within 2.9e-4 of a 64-bit one, relative over
    the whole output; exact hidden rows would leave 2.1e-4, the output's own rounding."""

    def __init__(self, up: W4Weight, down: W4Weight, topk: int, score: str = "softmax", router_bias=None,
                 n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                 scale: float = 1.0, up_bias=None, down_bias=None):
        if up.experts is None or up.experts != down.experts or (up.N, up.K) != (down.K, down.N):
            raise ValueError("up / down: need [E, F, K] and [E, K, F] of the same experts")
        if score not in _SCORES:
            raise ValueError(f"score: one of {sorted(_SCORES)}")
        _vec(router_bias, up.experts, torch.float32, "router_bias")
        for t, w, name in ((up_bias, up, "up_bias"), (down_bias, down, "down_bias")):
            if t is not None:
                _tensor(t, torch.float16, (w.experts, w.N), name)
        self.up, self.down, self.topk = up, down, topk
        self.score, self.router_bias = score, router_bias
        self.n_group, self.topk_group, self.group_top = n_group, topk_group, group_top
        self.renormalize, self.scale = bool(renormalize), scale
        self.up_bias, self.down_bias = up_bias, down_bias

    @classmethod
    def from_float(cls, w_up: torch.Tensor, w_down: torch.Tensor, topk: int, group: int = 128,
                   zero_point: bool = False, **kw) -> "W4Experts":
        """Quantize fp16 expert weights [E, F, K] and [E, K, F]; other arguments as in the constructor."""
        packed = []
        for w in (w_up, w_down):
            w4 = new_w4_weight(w.shape[1], w.shape[2], group, zero_point, experts=w.shape[0], device=w.device)
            packed.append(sq_quantize_weight_w4(w, w4))
        return cls(packed[0], packed[1], topk, **kw)

    def forward(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """x fp16 [..., K] and router logits [..., E] (fp32 or fp16) -> y fp16 [..., K]."""
        up, down, topk = self.up, self.down, self.topk
        E, F, K = up.experts, up.N, up.K
        shape, lshape = x.shape, logits.shape
        if not shape or shape[-1] != K or lshape[-1:] != (E,) or lshape[:-1] != shape[:-1]:
            raise ValueError(f"x / logits: need [..., {K}] and [..., {E}], got {tuple(shape)}, {tuple(lshape)}")
        half = logits.dtype == _F16
        if x.dtype != _F16 or not (half or logits.dtype == _F32):
            raise ValueError("x: fp16; logits: fp32 or fp16")
        x2, l2 = (x, logits) if len(shape) == 2 else (x.reshape(-1, K), logits.reshape(-1, E))
        (T, _), (ldx, inner), (ldl, linner) = x2.shape, x2.stride(), l2.stride()
        if inner != 1 or linner != 1:
            raise ValueError("x / logits: need a unit inner stride")
        if l2.data_ptr() % 16:
            l2, ldl = _realigned(l2), E
        y = x.new_empty(shape)
        if T == 0:
            return y
        if T == 1:
            ldx, ldl = K, E  # the stride of a single row means nothing
        P = T * topk
        # The whole layer is a few tens of microseconds for a few tokens, so the calls below pass
        # addresses inside one allocation instead of tensors cut from it.
        plan_ws = _L.sq_moe_plan_workspace_bytes(P, E)
        at, end = [], 0
        for n in (4 * P, 4 * P, 4 * (E + 1), 4 * P, plan_ws, 2 * P * F, 4 * P * K):
            at.append(end)
            end += -(-n // 256) * 256
        buf = x.new_empty(end // 2)
        px, pl, prb, pu, pub, pd, pdb, pbuf, py = _ptrs(x2, l2, self.router_bias, up.packed, self.up_bias, down.packed,
                                                        self.down_bias, buf, y)
        ids, weights, offsets, order, ws, h, z = [pbuf + a for a in at]
        st = _raw_stream(x2.get_device())
        status = _L.sq_moe_route(pl, half, T, E, ldl, prb, _SCORES[self.score], self.n_group, self.topk_group,
                                 self.group_top, topk, self.renormalize, self.scale, ids, weights, st)
        if status:
            _check(status, "sq_moe_route")
        status = _L.sq_moe_plan(ids, P, E, offsets, order, ws, plan_ws, st)
        if status:
            _check(status, "sq_moe_plan")
        status = _L.sq_w4a16_experts(px, T, ldx, pu, E, F, K, up.group, up.zero_point, pub, True, offsets, order, P,
                                     topk, h, False, st)
        if status:
            _check(status, "sq_w4a16_experts")
        # fp32 rows, so that the layer's output is rounded once
        status = _L.sq_w4a16_experts(h, P, F, pd, E, K, F, down.group, down.zero_point, pdb, False, offsets, order, P,
                                     1, z, True, st)
        if status:
            _check(status, "sq_w4a16_experts")
        status = _L.sq_moe_combine(z, True, ids, weights, T, topk, K, E, py, st)
        if status:
            _check(status, "sq_moe_combine")
        return y

    __call__ = forward
