"""Plain 64-bit forms of the training operators and bounds on what their documented arithmetic may leave of them.

half(t), SUM and close are dense_ref's: a rounding to t is off by at most half(t) of the value, a fp32 sum of n
terms in any order by at most n 2^-23 of the sum of their magnitudes.
"""
import torch

from tests.dense_ref import SUM, close, half, rnd  # noqa: F401

U = 2.0 ** -24  # one fp32 rounding


def chain(d):
    """Longest chain of additions in a row's sum: 512 threads at least from 8192 values on, else 16 values a lane and
    more threads, then the lanes' and the warps' tree."""
    return d / 512 + 40


def norm_forward(x, w, b, eps, ty):
    """{name: (value, bound)} of y (rounded to ty), mean and rstd."""
    x = x.double()
    w = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = c.square().mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    k = 2 * U * chain(x.shape[1])
    e_mean = k * x.abs().mean(1, keepdim=True) + U * mean.abs()
    # (x - mean)^2 with mean off by e: its mean is off by e^2 at most (the linear part adds up to nothing), and each
    # difference by U of itself
    e_var = e_mean.square() + 2 * U * c.abs().mean(1, keepdim=True) * e_mean + (k + 4 * U) * var
    e_rstd = rstd * (0.5 * e_var / (var + eps) * 1.01 + 6 * U)
    xh = c * rstd
    y = xh * w + b
    e = w.abs() * (rstd * (e_mean + U * (c.abs() + e_mean)) + (c.abs() + e_mean) * e_rstd + 3 * U * xh.abs()) + 3 * U * (xh * w).abs() + 2 * U * y.abs()
    return {"y": (y, e + rnd(y.abs() + e, ty)), "mean": (mean[:, 0], e_mean[:, 0] + U * mean.abs()[:, 0]),
            "rstd": (rstd[:, 0], e_rstd[:, 0])}


def norm_backward(dy, x, mean, rstd, w):
    """{name: (value, bound before the last rounding)} of dx, dw and db."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if w is None else w.double()
    xh = (x - mean) * rstd
    e_xh = 3 * U * xh.abs()
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    k = 2 * U * chain(x.shape[1]) + 6 * U
    e1, e2 = k * g.abs().mean(1, keepdim=True), k * (g * xh).abs().mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    e_dx = rstd * (8 * U * (g.abs() + m1.abs() + (xh * m2).abs()) + e1 + xh.abs() * e2 + e_xh * m2.abs())
    n = x.shape[0] + 8
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return {"dx": (dx, e_dx), "dw": (dw, (n * SUM) * (dy * xh).abs().sum(0) + (dy.abs() * e_xh).sum(0)),
            "db": (db, (n * SUM) * dy.abs().sum(0))}


def grouped(x, offsets, w):
    """(y [rows, n], bound before the last rounding), zeros for rows of no expert."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    e = torch.zeros_like(y)
    at = offsets.tolist()
    for m, i, j in zip(w, at[:-1], at[1:]):
        y[i:j] = x[i:j].double() @ m.double().T
        e[i:j] = (x[i:j].double().abs() @ m.double().abs().T) * (x.shape[1] * SUM)
    return y, e


def grouped_weights(dy, x, offsets):
    """(dW [E, n, k], bound before the last rounding)."""
    at = offsets.tolist()
    v, e = [], []
    for i, j in zip(at[:-1], at[1:]):
        p, q = dy[i:j].double(), x[i:j].double()
        v.append(p.T @ q)
        e.append((p.abs().T @ q.abs()) * ((j - i) * SUM))
    return torch.stack(v), torch.stack(e)


MUON = (3.4445, -4.7750, 2.0315)


def orthogonal(g, steps=5, coefficients=MUON):
    """The definition in 64 bits, one matrix."""
    a, b, c = coefficients
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    n = x.norm()
    x = x / n if n > 0 else x
    for _ in range(steps):
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.T if tall else x


def orthogonal_rounded(g, steps=5, coefficients=MUON):
    """The same with the roundings that the operator documents, its sums exact: what it may be off by is taken from
    here (one and a half times this form's distance, for the fp32 sums and other orders)."""
    a, b, c = coefficients

    def r(v):
        return (v * 1024).to(torch.float16).double() / 1024

    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    n = x.norm()
    x = x / n if n > 0 else x
    for i in range(steps):
        h = r(x)
        x = h + r(x - h) if i + 1 < steps else h
        p = r(h @ h.T)
        q = b * p + c * (p @ p)
        d = torch.diagonal(q).clone()
        x = a * x + d[:, None] * (x if i + 2 >= steps else h) + r(q - torch.diag(d)) @ h
    return x.T if tall else x


def dense_distance(a, b):
    """Norm of the difference over the norm of b (of a where b is zero)."""
    n = b.norm()
    return float((a.double() - b).norm() / n) if n > 0 else float(a.double().norm())


# Stacks (count, rows, cols) past the small kernel, and the way that A is made on: tiles of side x side, and shares of the long
# side whose sums are added up by a launch of their own (0: all tiles at once).  test_train_abi holds this against the
# library's workspaces, so that a change of the rule cannot take a way's cases away unseen.
ORTHO_WAYS = {(1, 301, 2007): (256, 8), (1, 2007, 301): (256, 8), (2, 301, 2007): (256, 4), (2, 2007, 301): (256, 4),
              (3, 301, 3007): (256, 4), (3, 3001, 304): (256, 4), (1, 520, 5000): (256, 8), (1, 5003, 520): (256, 8),
              (1, 16, 7168): (128, 16), (1, 7168, 16): (128, 16), (1, 4000, 100): (128, 16), (3, 100, 4001): (128, 16),
              (4, 4000, 100): (128, 16), (2, 64, 1500): (128, 12), (2, 1500, 65): (128, 12), (2, 520, 136): (256, 0),
              (2, 200, 520): (256, 0), (2, 330, 131): (256, 0), (1, 513, 129): (256, 0), (4, 2007, 301): (256, 0)}


def ortho_workspace(count, rows, cols, side, slices):
    """Bytes of a call's workspace, made that way: X in three parts, A and B, B's diagonal, sums of squares, A's partial
    sums."""
    def take(n):
        return (n + 255) // 256 * 256

    m = min(rows, cols)
    ldx, ldm, across = (cols + 7) // 8 * 8, (m + 7) // 8 * 8, (m + side - 1) // side
    return (3 * take(count * rows * ldx * 2) + 2 * take(count * m * ldm * 2) + take(count * ldm * 4) + take(count * 512 * 3 * 4)
            + take(count * (across * (across + 1) // 2) * slices * side * side * 4))
