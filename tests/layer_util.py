"""Plain 64-bit forms of block_norm, lora_linear and moe_route on host arrays,
with bounds on what fp32 arithmetic may leave between them and the kernels."""
import numpy as np
import torch

from tests.kv_util import bf16_values

U32 = 2.0 ** -24                 # half a step of fp32, relative
U16 = 2.0 ** -8                  # half a step of bf16, relative
TINY16 = 2.0 ** -133             # a step of bf16's subnormal numbers


def host(t):
    """A tensor's values, or None."""
    return None if t is None else t.detach().double().cpu().numpy()


def _normed(v, ev, weight, bias, layer, eps):
    """norm(v) * weight + bias along the rows, and its bound given v's `ev`: a
    changed mean and root mean square to first order (times 1.01 for the rest),
    and four fp32 roundings of the product, one of the sum."""
    with np.errstate(all="ignore"):
        c, ec = v, ev
        if layer:
            c = v - v.mean(axis=1, keepdims=True)
            ec = ev + ev.mean(axis=1, keepdims=True)
        q = (c * c).mean(axis=1, keepdims=True) + eps
        r = 1.0 / np.sqrt(q)
        er = r * (2 * np.abs(c) * ec + ec * ec).mean(axis=1, keepdims=True) / (2 * q) * 1.01
        y = c * r * weight
        e = np.abs(weight) * (ec * r + np.abs(c) * er) + 4 * U32 * np.abs(y)
        if bias is not None:
            y = y + bias
            e = e + U32 * (np.abs(y) + np.abs(bias)) + U32 * np.abs(y)
    return y, e


def block_norm(block, residual, weight, bias=None, post_weight=None, post_bias=None, gate=None,
               route_weights=None, routes=1, layer=False, eps=1e-6, residual_scale=1.0,
               block_scale=1.0, weight_offset=0.0):
    """(h, bound of h before its rounding, out, bound of out before its rounding)."""
    eps, rs, bs, off = (float(np.float32(x)) for x in (eps, residual_scale, block_scale, weight_offset))
    some = residual if residual is not None else block
    width = some.shape[1]
    h, eh = np.zeros((1, 1)), np.zeros((1, 1))
    with np.errstate(all="ignore"):
        if block is not None:
            rows = block.shape[0] // routes
            parts = block.reshape(rows, routes, width)
            w = np.ones((rows, routes)) if route_weights is None else route_weights
            b = (parts * w[:, :, None]).sum(axis=1)
            eb = np.zeros_like(b)
            if routes > 1 or route_weights is not None:
                eb = routes * U32 * (np.abs(parts) * np.abs(w[:, :, None])).sum(axis=1)
            if post_weight is not None:
                b, eb = _normed(b, eb, off + post_weight, post_bias, layer, eps)
            if gate is not None:
                b, eb = b * gate, eb * np.abs(gate) + U32 * np.abs(b * gate)
            h = bs * b
            eh = np.abs(bs) * eb + 2 * U32 * np.abs(h)
        if residual is not None:
            eh = eh + 2 * U32 * (np.abs(rs * residual) + np.abs(h))
            h = h + rs * residual
        out, eo = _normed(h, eh, np.ones(width) if weight is None else off + weight, bias, layer, eps)
    return h, eh, out, eo


def near(got, want, bound, half=U16, tiny=TINY16):
    """Whether got is want after `bound` and one rounding; infinities and NaN alike."""
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape
    fine = np.isfinite(want)
    # A row with an infinity has no bound (inf - inf): its finite values are exact zeros.
    bound = np.where(np.isnan(bound), 0.0, bound) + np.zeros_like(want)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    bad = ~fine & ~np.isnan(want)
    np.testing.assert_array_equal(got[bad], want[bad])
    off = np.abs(got - want)[fine]
    limit = (bound + half * (np.abs(want) + bound) + tiny)[fine]
    worst = float((off / limit).max()) if off.size else 0.0
    assert worst <= 1.0, f"worst error {worst:.3g} of the bound"
    return worst


def lora(x, ids, base, a, b, ranks, scale):
    """(y, its bound before rounding) for host arrays; a and b lists of slices
    (None without adapters, b then the width).  A x: K products and their sums in
    any order (2^-23 each: matrix units need not round to nearest); its split into
    two bf16 numbers 2^-16; the products with B likewise; one fp32 sum."""
    y, e, at = base.copy(), np.zeros_like(base), 0
    U = 2 * U32
    for p, q in zip(a, b):
        n = q if p is None else q.shape[1]
        for t, i in enumerate(ids):
            if p is None or not 0 <= i < p.shape[0]:
                continue
            r = p.shape[1] if ranks is None else min(max(int(ranks[i]), 0), p.shape[1])
            s = 1.0 if scale is None else scale[i]
            A, B = p[i, :r], q[i, :, :r]
            v = A @ x[t]
            ev = (x.shape[1] + 8) * U * (np.abs(A) @ np.abs(x[t]))
            v, ev = v * s, ev * abs(s) + U * np.abs(v * s)
            size = np.abs(B) @ np.abs(v)
            y[t, at:at + n] += B @ v
            e[t, at:at + n] = np.abs(B) @ ev + (2.0 ** -16 + 2 * (r + 1) * U) * size + \
                U * (np.abs(base[t, at:at + n]) + size)
        at += n
    return y, e


def route(logits, topk, sigmoid, bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """(ids, weights), row by row and choice by choice."""
    T, E = logits.shape
    ids, weights = np.zeros((T, topk), np.int64), np.zeros((T, topk))
    each = E // groups
    for t in range(T):
        l = np.where(np.isnan(logits[t]), -np.inf, logits[t])
        l = np.minimum(l, float(np.finfo(np.float32).max))
        with np.errstate(all="ignore"):
            if sigmoid:
                s = np.where(l >= 0, 1 / (1 + np.exp(-l)), np.exp(l) / (1 + np.exp(l)))
                s = np.where(l == -np.inf, 0.0, s)
            elif np.all(l == -np.inf):
                s = np.zeros(E)
            else:
                s = np.exp(l - l.max())
                s = s / s.sum()
            c = l if bias is None else s + bias
        c = np.where(np.isnan(c), -np.inf, c)
        open_to = list(range(E))
        if groups > 1:
            worth = []
            for g in range(groups):
                top = sorted(c[g * each:(g + 1) * each], reverse=True)
                with np.errstate(all="ignore"):
                    w = top[0] + top[1] if bias is not None and each > 1 else top[0]
                worth.append(-np.inf if np.isnan(w) else w)
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            open_to = [e for e in open_to if e // each in kept]
        chosen = sorted(open_to, key=lambda e: (-c[e], e))[:topk]
        w = s[chosen]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(topk)
        ids[t], weights[t] = chosen, w * float(np.float32(scale))
    return ids, weights


def values(t):
    """bf16 or fp32 device tensor -> fp64 host values."""
    if t.dtype is torch.bfloat16:
        return bf16_values(t.cpu().view(torch.int16).numpy().view(np.uint16))
    return t.double().cpu().numpy()
