"""Plain 64-bit forms of the dense operators and bounds on what 16-bit and fp32 arithmetic may
leave of them, for the tests.

A rounding to type t is off by at most half(t) of the value (half a step), or by half the smallest
subnormal.  A fp32 sum of n products, in any order, is off by at most n 2^-23 of the sum of
their magnitudes (2^-24 a rounding; twice that for a unit that cuts instead of rounding).
"""
import torch

SUM = 2.0 ** -23
FUN = 2.0 ** -20  # relative error allowed to sigmoid, products and sums of one element in fp32


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


SPLIT = 32  # calls of at most so many tokens keep intermediate values in two parts of type t


def kept(v, e, t, tokens):
    """Bound on a value of magnitude v, off by e, on its way into the next product: rounded to t, or
    to t and the rest to t again."""
    return e + (rnd(v + e, t) if tokens > SPLIT else 2 * half(t) ** 2 * (v + e) + tiny(t))


def rnd(v, t):
    """Bound on rounding values of magnitude at most v to type t."""
    return half(t) * v + tiny(t)


def close(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs().max()), float(tol.max()),
                           float(((got - ref).abs() / tol.clamp(min=1e-300)).max()))


def forward(x, wg, wu, wd, t):
    """{name: (value, bound)} for y before its own rounding, g and u before theirs, in fp64."""
    x, wg, wu, wd = (v.double() for v in (x, wg, wu, wd))
    g, u = x @ wg.T, x @ wu.T
    eg, eu = ((x.abs() @ w.abs().T) * (x.shape[1] * SUM) for w in (wg, wu))
    s = torch.sigmoid(g)
    a = g * s * u
    # |silu'| <= 1.1
    ea = 1.1 * eg * (u.abs() + eu) + (g * s).abs() * eu + FUN * a.abs()
    ea = kept(a.abs(), ea, t, x.shape[0])
    y = a @ wd.T
    ey = ea @ wd.abs().T + ((a.abs() + ea) @ wd.abs().T) * (wd.shape[1] * SUM)
    return {"g": (g, eg), "u": (u, eu), "a": (a, ea), "y": (y, ey)}


def backward(dy, x, g, u, wg, wu, wd, t):
    dy, x, g, u, wg, wu, wd = (v.double() for v in (dy, x, g, u, wg, wu, wd))
    s = torch.sigmoid(g)
    slope = s * (1 + g * (1 - s))
    da = dy @ wd
    eda = (dy.abs() @ wd.abs()) * (dy.shape[1] * SUM)
    a, du, dg = g * s * u, da * g * s, da * u * slope

    def into(v, e):
        return kept(v.abs(), e + FUN * v.abs(), t, x.shape[0])

    # the slope is a sum with cancellation: its own error is up to FUN of its terms
    ea, edu = into(a, torch.zeros_like(a)), into(du, eda * (g * s).abs())
    edg = into(dg, eda * (u * slope).abs() + FUN * (da * u).abs() * s * (1 + g.abs() * (1 - s)))

    def prod(p, ep, q, n):  # p^T q with p off by ep
        v = p.T @ q
        return v, ep.T @ q.abs() + ((p.abs() + ep).T @ q.abs()) * (n * SUM)

    T, f = x.shape[0], g.shape[1]
    dwg, dwu = prod(dg, edg, x, T), prod(du, edu, x, T)
    v, e = prod(a, ea, dy, T)
    dwd = v.T, e.T
    dx = dg @ wg + du @ wu
    edx = edg @ wg.abs() + edu @ wu.abs()
    edx = edx + ((dg.abs() + edg) @ wg.abs() + (du.abs() + edu) @ wu.abs()) * (2 * f * SUM)
    return {"dx": (dx, edx), "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}


# ---------------------------------------------------------------- microscaled 4-bit matrices

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def mx_exponent(big):
    """Shared exponent of blocks with the largest magnitudes big (fp64)."""
    _, ex = torch.frexp(big)  # big = m 2^ex, m in [0.5, 1)
    e = (ex - 1 - 2).clamp(min=-127)
    return torch.where(big == 0, torch.full_like(e, -127), e).double()


def mx_codes(v, e=None):
    """(codes 0..15 [rows, cols], scale bytes [rows, blocks]) of v by comparing each value with
    every E2M1 value; e: the blocks' exponents, if not taken from v."""
    rows, cols = v.shape
    b = v.double().reshape(rows, cols // 32, 32)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    if e is None:
        e = mx_exponent(b.abs().amax(-1))
    m = b.abs() * torch.exp2(-e)[..., None]
    grid = GRID.to(v.device)
    n = torch.zeros(m.shape, dtype=torch.int64, device=v.device)
    for i in range(1, 8):
        mid = (grid[i] + grid[i - 1]) / 2
        n = torch.where((m > mid) | ((m == mid) & (i % 2 == 0)), i, n)
    code = n + 8 * torch.signbit(b).long()
    code = torch.where(bad[..., None], torch.zeros_like(code), code)
    scale = torch.where(bad, torch.full_like(e, 255), e + 127).long()
    return code.reshape(rows, cols), scale


def mx_pack(code, scale):
    """Codes and scale bytes in the library's layout (loops over tiles)."""
    rows, cols = code.shape
    codes = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    kb, rt = -(-cols // 128), -(-rows // 128)
    full = torch.zeros(rt * 128, kb * 4, dtype=torch.uint8, device=code.device)
    full[:rows, :cols // 32] = scale.to(torch.uint8)
    out = torch.empty(rt, kb, 32, 4, 4, dtype=torch.uint8, device=code.device)
    for q in range(4):
        for k in range(4):
            out[:, :, :, q, k] = full.view(rt, 4, 32, kb, 4)[:, q, :, :, k].permute(0, 2, 1)
    return codes.contiguous(), out.reshape(-1)


def mx_values(code, scale):
    """fp64 values of codes and scale bytes."""
    v = GRID.to(code.device)[code % 8] * torch.where(code >= 8, -1.0, 1.0)
    p = torch.exp2(scale.double() - 127)
    p = torch.where(scale == 255, torch.full_like(p, float("nan")), p)
    return (v.reshape(code.shape[0], -1, 32) * p[..., None]).reshape(code.shape)


def mx_round(v):
    return mx_values(*mx_codes(v))


def mx_spread(a, ea):
    """What quantising a' may differ from quantising a, for any a' within ea of a."""
    rows, cols = a.shape
    base = mx_round(a)
    b, eb = a.reshape(rows, -1, 32).abs(), ea.reshape(rows, -1, 32)
    lo, hi = mx_exponent((b - eb).clamp(min=0).amax(-1)), mx_exponent((b + eb).amax(-1))
    worst = torch.zeros_like(a)
    for e in (lo, hi):
        for v in (a - ea, a + ea):
            c, s = mx_codes(v, e)
            worst = torch.maximum(worst, (mx_values(c, s) - base).abs())
    return worst
