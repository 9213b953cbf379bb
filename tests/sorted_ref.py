"""Plain 64-bit forms of the sorted rows and of the products in 8-bit integers (torch, CPU), for the tests."""
import torch

FLOOR = 2.0 ** -100


def sort(ids, E, first=0):
    """(place [T, k], pairs in sorted order, offsets) of a rank's pairs, one after another."""
    T, k = ids.shape
    place = torch.full((T, k), -1, dtype=torch.int32)
    order, offsets = [], [0]
    for e in range(E):
        for i in torch.nonzero(ids.flatten().long() - first == e).flatten().tolist():
            place[i // k, i % k] = len(order)
            order.append(i)
        offsets.append(len(order))
    return place, order, torch.tensor(offsets, dtype=torch.int32)


def unsort(rows, place, weights=None, base=None):
    """(y, sum of the terms' magnitudes): float64."""
    T, k = place.shape
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64) if base is None else base.double().clone()
    size = y.abs()
    for j in range(k):
        for t in range(T):
            at = int(place[t, j])
            if 0 <= at < rows.shape[0]:
                term = rows[at].double() * (1.0 if weights is None else weights[t, j].double())
                y[t] += term
                size[t] += term.abs()
    return y, size


def unsort_backward(dy, place, rows=None, weights=None, n=None):
    """(drows, dweights, sum of the products' magnitudes)."""
    T, k = place.shape
    n = rows.shape[0] if rows is not None else n
    drows = torch.zeros(n, dy.shape[1], dtype=torch.float64)
    dw, size = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            at = int(place[t, j])
            if 0 <= at < n:
                drows[at] = dy[t].double() * (1.0 if weights is None else weights[t, j].double())
                if rows is not None:
                    p = rows[at].double() * dy[t].double()
                    dw[t, j], size[t, j] = p.sum(), p.abs().sum()
    return drows, dw, size


def quantised(x):
    """(q, scale in 32 bits) of rows x, float64 values; NaN and infinities: q 0, scale NaN."""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True).clamp_min(FLOOR)
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    q = torch.where(bad, 0.0, torch.round(127.0 * x / a))
    scale = torch.where(bad[..., 0], torch.nan, (a[..., 0].float() / torch.tensor(127.0)).double())
    return q, scale.float()


def swiglu(x):
    g, u = x.double().chunk(2, -1)
    return g / (1.0 + torch.exp(-g)) * u


def product(xq, xs, wq, ws):
    """The integer sum, rounded to fp32, times xs, times ws, each product rounded: fp32 [T, N].  (Sums below 2^53 are exact here.)"""
    acc = (xq.double() @ wq.double().transpose(-1, -2)).float()
    return acc * xs[:, None] * ws
