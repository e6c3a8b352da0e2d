"""Plain 64-bit forms of the 4-bit weight and expert-routing operators (numpy, from the formulas in
include/sq.h), and their error bounds."""
import numpy as np

F16_HALF = 2.0**-11   # half a step of fp16, relative
F16_TINY = 2.0**-25   # half a step of its subnormals


def round_bits(v, n):
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 2.0**n), e - n)


def groups_of(K, group):
    return [(k, min(K, k + group)) for k in range(0, K, group)]


def quantize(w, group, zero, s=None):
    """codes uint8 [N, K], scales fp16 [N, G], zeros uint8 [N, G] or None of an fp16 weight."""
    if s is not None:
        w = (w.astype(np.float32) * s.astype(np.float32)).astype(np.float16)
    w = w.astype(np.float64)
    N, K = w.shape
    parts = groups_of(K, group)
    codes = np.empty((N, K), np.uint8)
    scales = np.empty((N, len(parts)), np.float16)
    zeros = np.empty((N, len(parts)), np.uint8)
    for g, (a, b) in enumerate(parts):
        v = w[:, a:b]
        finite = np.where(np.isnan(v), 0.0, v)
        if zero:
            lo, hi = np.minimum(finite.min(1), 0.0), np.maximum(finite.max(1), 0.0)
            sc = round_bits((hi - lo) / 15.0, 7).astype(np.float16)
        else:
            sc = round_bits(np.abs(finite).max(1) / 7.0, 8).astype(np.float16)
        d = np.where((sc == 0) | np.isinf(sc), 1.0, sc.astype(np.float64))
        ok = ((sc > 0) & np.isfinite(sc))[:, None] & ~np.isnan(v)
        fv = np.where(ok, v, 0.0)
        if zero:
            z = np.where(ok.any(1), np.minimum(np.rint(-np.where(np.isfinite(lo), lo, 0.0) / d), 15), 0)
            q = np.where(ok, np.clip(np.rint(fv / d[:, None]) + z[:, None], 0, 15), z[:, None])
        else:
            z = np.full(N, 8)
            q = np.where(ok, np.clip(np.rint(fv / d[:, None]), -7, 7) + 8, 8)
        codes[:, a:b], scales[:, g], zeros[:, g] = q, sc, z
    return codes, scales, zeros if zero else None


def values(codes, scales, zeros, group):
    """fp64 [..., N, K]."""
    K = codes.shape[-1]
    idx = np.arange(K) // group
    z = 8.0 if zeros is None else zeros.astype(np.float64)[..., idx]
    return (codes.astype(np.float64) - z) * scales.astype(np.float64)[..., idx]


def random_weight(rng, N, K, group, zero, lead=(), std=0.02):
    G = -(-K // group)
    codes = rng.integers(0, 16, lead + (N, K)).astype(np.uint8)
    scales = round_bits(rng.uniform(0.2, 1.0, lead + (N, G)) * std / 4, 7).astype(np.float16)
    zeros = rng.integers(0, 16, lead + (N, G)).astype(np.uint8) if zero else None
    return codes, scales, zeros


def linear(x, W, bias=None, relu=False, out_f32=False):
    """(y, bound): the product in 64 bits and how far a kernel with fp32 sums may be from it.

    Every product of an fp16 x and an fp16-exact weight is exact in fp32 (at most 22 bits).  A sum of
    K terms takes at most K additions, each off by at most one fp32 step, 2^-23 (the tensor core
    truncates), of a partial sum no larger than S = sum |x||W| + |bias|; scaling a group's sum and
    adding it are two more.  The last rounding is half a step of the output's type."""
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        y = x @ W.T
        S = np.abs(x) @ np.abs(W).T
    if bias is not None:
        y = y + bias.astype(np.float64)
        S = S + np.abs(bias.astype(np.float64))
    if relu:
        y = np.where(y > 0, y, 0.0)
    sums = (x.shape[1] + 2 * (x.shape[1] // 32 + 1) + 16) * 2.0**-23 * S
    last = 2.0**-24 * np.abs(y) if out_f32 else F16_HALF * np.abs(y) + F16_TINY
    return y, sums * (1 + F16_HALF) + last


def route(logits, topk, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    l = logits.astype(np.float64)
    T, E = l.shape
    ids = np.full((T, topk), -1, np.int64)
    weights = np.zeros((T, topk))
    for t in range(T):
        masked = np.isnan(l[t]) | (l[t] == -np.inf)
        p = np.zeros(E)
        if not masked.all():
            if score == "softmax":
                top = l[t][~masked].max()
                with np.errstate(invalid="ignore"):
                    e = np.where(masked, 0.0, np.where(l[t] == top, 1.0, np.exp(np.where(masked, -1e300, l[t]) - top)))
                p = e / e.sum()
            else:
                with np.errstate(over="ignore"):
                    p = np.where(masked, 0.0, 1.0 / (1.0 + np.exp(-np.where(masked, 0.0, l[t]))))
        c = p + (0.0 if bias is None else bias.astype(np.float64))
        c = np.where(masked | np.isnan(c), -np.inf, c)
        if topk_group < n_group:
            per = E // n_group
            gs = np.full(n_group, -np.inf)
            for g in range(n_group):
                best = np.sort(c[g * per:(g + 1) * per])[::-1]
                gs[g] = best[0]
                if group_top == 2 and best[1] > -np.inf:
                    gs[g] = best[0] + best[1]
            keep = [g for g in np.argsort(-gs, kind="stable")[:topk_group] if gs[g] > -np.inf]
            c = np.where(np.isin(np.arange(E) // per, keep), c, -np.inf)
        order = [e for e in np.argsort(-c, kind="stable")[:topk] if c[e] > -np.inf]
        w = p[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        ids[t, :len(order)] = order
        weights[t, :len(order)] = w * scale
    return ids, weights


def plan(ids, E):
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")
    counts = np.bincount(flat[ok], minlength=E)
    order = np.where(np.arange(len(flat)) < counts.sum(), order, -1)
    return np.concatenate([[0], np.cumsum(counts)]), order
