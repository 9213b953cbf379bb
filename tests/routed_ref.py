"""Plain 64-bit forms of the routed-expert operators (torch, CPU), for the tests."""
import math

import torch

BLOCK = 128
FLOOR = 2.0 ** -100
CLOSED_FROM = -3.3895313892515355e38


def blocks(n):
    return -(-n // BLOCK)


def e4m3(v):
    """Nearest e4m3 value of v (float64), ties to even."""
    exponent = (torch.frexp(v).exponent - 1).clamp_min(-6)
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.round(v / step) * step


def rounded(x):
    """(q, scale) of x [.., K] float64 in blocks of 1 x 128 along K."""
    q = torch.empty_like(x)
    s = torch.empty(*x.shape[:-1], blocks(x.shape[-1]), dtype=torch.float64)
    for b in range(s.shape[-1]):
        v = x[..., b * BLOCK:(b + 1) * BLOCK]
        a = v.abs().amax(-1, keepdim=True).clamp_min(FLOOR)
        q[..., b * BLOCK:(b + 1) * BLOCK] = e4m3(448.0 * v / a)
        s[..., b:b + 1] = a / 448.0
    return q, s


def spread_rows(q, s):
    """q [.., K] times its scales [.., K / 128]."""
    return q * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def weight(q, s):
    """The matrix [N, K] that e4m3 values q and block scales s stand for."""
    N, K = q.shape
    return q.double() * s.double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def route(logits, top_k, scoring, bias=None, n_group=1, topk_group=1, group_top=2, renormalise=True, scale=1.0):
    """(ids, weights, gap): gap[t] is the smallest distance between choices that decide row t."""
    l = logits.double()
    T, E = l.shape
    ids = torch.full((T, top_k), -1, dtype=torch.int32)
    w = torch.zeros(T, top_k, dtype=torch.float64)
    gap = torch.full((T,), math.inf)
    for t in range(T):
        open_ = [e for e in range(E) if l[t, e] > CLOSED_FROM]
        if not open_:
            continue
        if scoring == "sigmoid":
            score = {e: 1.0 / (1.0 + math.exp(-l[t, e])) for e in open_}
        else:
            top = max(float(l[t, e]) for e in open_)
            ex = {e: math.exp(float(l[t, e]) - top) for e in open_}
            score = {e: v / sum(ex.values()) for e, v in ex.items()}
        choice = {e: score[e] + (float(bias[e]) if bias is not None else 0.0) for e in open_}
        kept = open_
        if n_group > 1:
            size = E // n_group
            value = []
            for g in range(n_group):
                best = sorted((choice[e] for e in open_ if e // size == g), reverse=True)[:group_top]
                value.append((sum(best) if best else -math.inf, -g))
            order = sorted(value, reverse=True)
            if topk_group < n_group and math.isfinite(order[topk_group][0]):
                gap[t] = min(gap[t], order[topk_group - 1][0] - order[topk_group][0])
            groups = {-g for _, g in order[:topk_group]}
            kept = [e for e in open_ if e // size in groups]
        order = sorted(((choice[e], -e) for e in kept), reverse=True)
        for a, b in zip(order[:top_k], order[1:top_k + 1]):
            gap[t] = min(gap[t], a[0] - b[0])
        for j, (_, e) in enumerate(order[:top_k]):
            ids[t, j] = -e
            w[t, j] = score[-e]
        if renormalise and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale, gap


def experts(x, ids, weights, wgu, sgu, wd, sd, first=0, shared=None):
    """y [T, H] float64; wgu [E, 2I, H] and wd [E, H, I] e4m3 values, sgu and sd their scales."""
    I = wd.shape[2]
    nb = blocks(I)
    xr = spread_rows(*rounded(x.double()))
    gate = [weight(wgu[e, :I], sgu[e, :nb]) for e in range(wd.shape[0])]
    up = [weight(wgu[e, I:], sgu[e, nb:]) for e in range(wd.shape[0])]
    down = [weight(wd[e], sd[e]) for e in range(wd.shape[0])]
    y = torch.zeros_like(xr) if shared is None else shared.double().clone()
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j]) - first
            if not 0 <= e < wd.shape[0]:
                continue
            g = gate[e] @ xr[t]
            u = up[e] @ xr[t]
            h = spread_rows(*rounded(g / (1 + torch.exp(-g)) * u))
            y[t] += weights[t, j].double() * (down[e] @ h)
    return y
