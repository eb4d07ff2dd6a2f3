"""The operators that train the layer around the compressed experts, as they are measured.

  norm_forward      layer norm: y = (x - mean) rstd w + b over each row, mean and rstd kept if asked for
  norm_backward     its gradients: dx, and dw and db summed over the rows
  grouped_forward   products grouped by expert: y_r = x_r W_e^T for the rows r of each expert e
  grouped_backward  their gradients: dx_r = dy_r W_e, dW_e = sum over e's rows of dy_r^T x_r
  orthogonalize     a gradient made orthogonal by Newton-Schulz products: X = G / |G|, then `steps` times
                    X <- a X + (b A + c A^2) X with A = X X^T (X^T X on the other side where G is tall);
                    out = scale X, or added to the weights

Sizes are those of the package's workloads (hidden size 7168, expert width 1536, 384 or 64 experts, 16
experts a token, and the small 256 x 128 layer of 8), one token to a long batch.  Rows arrive sorted by
expert: the rows of expert e are offsets[e] .. offsets[e + 1] - 1.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_COEFFICIENTS = (3.4445, -4.7750, 2.0315)
_EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the hidden state of one decoded token, before the router and the experts
        {"name": "norm token", "op": "norm_forward", "T": 1, "d": 7168, "type": "fp32", "out": "fp32", "save": False},
        # a training batch's forward
        {"name": "norm train forward", "op": "norm_forward", "T": 16384, "d": 7168, "type": "bf16", "out": "bf16", "save": True},
        # the same batch's gradients
        {"name": "norm train backward", "op": "norm_backward", "T": 16384, "d": 7168, "type": "bf16"},
        # fine-tuning a small layer on a ragged batch, rows of an odd length
        {"name": "norm odd backward", "op": "norm_backward", "T": 333, "d": 1001, "type": "fp16"},
        # one decoded token's 16 rows, each of another expert of 64: the weights' way from memory
        {"name": "grouped token", "op": "grouped_forward", "T": 1, "top": 16, "E": 64, "k": 7168, "n": 1536, "type": "bf16"},
        # 128 decoding sequences over 384 experts of uneven popularity: most get a few rows, some none
        {"name": "grouped batch", "op": "grouped_forward", "T": 128, "top": 16, "E": 384, "k": 7168, "n": 1536, "type": "bf16"},
        # a training batch through the down projection
        {"name": "grouped train forward", "op": "grouped_forward", "T": 2048, "top": 16, "E": 64, "k": 1536, "n": 7168, "type": "bf16"},
        # a training batch's gradients of the gate or up projection
        {"name": "grouped train backward", "op": "grouped_backward", "T": 2048, "top": 16, "E": 64, "k": 7168, "n": 1536, "type": "bf16"},
        # the small layer, a few tokens: latency
        {"name": "grouped small backward", "op": "grouped_backward", "T": 77, "top": 2, "E": 8, "k": 256, "n": 128, "type": "fp16"},
        # every gate matrix of the small layer at once
        {"name": "orthogonalize small", "op": "orthogonalize", "count": 8, "rows": 128, "cols": 256, "type": "fp32", "weights": ""},
        # the gradient of one expert's gate matrix
        {"name": "orthogonalize wide", "op": "orthogonalize", "count": 1, "rows": 1536, "cols": 7168, "type": "bf16", "weights": ""},
        # the down matrices of four experts, the update added to their weights
        {"name": "orthogonalize tall", "op": "orthogonalize", "count": 4, "rows": 7168, "cols": 1536, "type": "fp32", "weights": "bf16"},
    ]


def _spread(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "grouped_forward", "grouped_backward", "orthogonalize"])
    half = rng.choice(["bf16", "fp16"])
    if op == "norm_forward":
        return {"op": op, "T": _spread(rng, 1, 16384), "d": _spread(rng, 32, 7168), "type": rng.choice(["bf16", "fp16", "fp32"]),
                "out": half, "save": rng.random() < 0.5}
    if op == "norm_backward":
        return {"op": op, "T": _spread(rng, 1, 16384), "d": _spread(rng, 32, 7168), "type": rng.choice(["bf16", "fp16", "fp32"])}
    if op != "orthogonalize":
        E = _spread(rng, 1, 64)
        top = min(E, rng.choice([1, 2, 4, 8, 16]))
        return {"op": op, "T": _spread(rng, 1, 8192 // top), "top": top, "E": E, "k": _spread(rng, 64, 7168, 8),
                "n": _spread(rng, 64, 1536, 8), "type": half}
    rows, cols = _spread(rng, 16, 1536), _spread(rng, 16, 7168)
    if rng.random() < 0.5:
        rows, cols = cols, rows
    return {"op": op, "count": rng.choice([1, 1, 2, 4]), "rows": rows, "cols": cols, "type": rng.choice(["bf16", "fp32"]),
            "weights": rng.choice(["", "bf16"])}


def _sizes(T, top, E):
    """Rows of the experts in order of popularity (which falls as 1 / rank^1.1): T * top in all, none over T."""
    share = [(r + 1) ** -1.1 for r in range(E)]
    rows, low, high = T * top, 0.0, float(T) / share[-1]
    for _ in range(60):
        mid = (low + high) / 2
        low, high = (mid, high) if sum(min(T, int(mid * v)) for v in share) <= rows else (low, mid)
    n = [min(T, int(low * v)) for v in share]
    left = rows - sum(n)
    for r in range(E):  # what rounding down left over
        more = min(T - n[r], left, 1)
        n[r] += more
        left -= more
    for r in range(E):
        more = min(T - n[r], left)
        n[r] += more
        left -= more
    return n


def work(case):
    op, s = case["op"], _SIZE[case["type"]]
    if op == "norm_forward":
        T, d = case["T"], case["d"]
        return {"bytes": (s + _SIZE[case["out"]]) * T * d + 2 * s * d + (8 * T if case["save"] else 0), "flops": 8 * T * d}
    if op == "norm_backward":
        T, d = case["T"], case["d"]
        return {"bytes": 3 * s * T * d + s * d + 8 * d + 8 * T, "flops": 16 * T * d}
    if op == "orthogonalize":
        c, m, n = case["count"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        out = 2 * _SIZE[case["weights"]] if case["weights"] else 2
        # A and A^2 are symmetric: half of each
        return {"bytes": c * m * n * (s + out), "flops": c * 5 * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)}
    n = _sizes(case["T"], case["top"], case["E"])
    rows, used, w = sum(n), sum(1 for v in n if v), case["k"] * case["n"]
    if op == "grouped_forward":
        return {"bytes": s * (rows * (case["k"] + case["n"]) + used * w), "flops": 2 * rows * w}
    return {"bytes": s * (rows * (2 * case["k"] + case["n"]) + (used + case["E"]) * w), "flops": 4 * rows * w}


# ---------------------------------------------------------------- inputs

def _randn(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 29)
    op, t = case["op"], _TYPES[case["type"]]
    s = dict(case)
    if op in ("norm_forward", "norm_backward"):
        T, d = case["T"], case["d"]
        # hidden states: some columns much larger than the rest, rows of a mean other than zero
        x = _randn(gen, T, d) * torch.exp(_randn(gen, 1, d)) + _randn(gen, T, 1, scale=0.5)
        s["x"] = x.to(t)
        s["w"], s["b"] = (1 + _randn(gen, d, scale=0.1)).to(t), _randn(gen, d, scale=0.1).to(t)
        if op == "norm_forward":
            s["y"] = torch.empty(T, d, dtype=_TYPES[case["out"]], device="cuda")
            s["mean"], s["rstd"] = (torch.empty(T, device="cuda") if case["save"] else None for _ in range(2))
        else:
            v = s["x"].float()  # what the forward of this step kept
            s["mean"] = v.mean(1)
            s["rstd"] = torch.rsqrt((v - s["mean"][:, None]).square().mean(1) + _EPS)
            s["dy"] = _randn(gen, T, d).to(t)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"], s["db"] = (torch.empty(d, device="cuda") for _ in range(2))
    elif op == "orthogonalize":
        c, m, n = case["count"], case["rows"], case["cols"]
        # a gradient of some hundred tokens, of falling weight, and the noise of the rest
        r = min(m, n, 256)
        fall = torch.exp(-3 * torch.arange(r, device="cuda") / r)
        g = (_randn(gen, c, m, r) * fall) @ _randn(gen, c, r, n) + _randn(gen, c, m, n, scale=0.5)
        s["g"] = (g * 1e-3).to(t)
        if case["weights"]:
            s["out"] = _randn(gen, c, m, n, scale=max(m, n) ** -0.5).to(_TYPES[case["weights"]])
        else:
            s["out"] = torch.empty(c, m, n, dtype=torch.bfloat16, device="cuda")
    else:
        E, k, n = case["E"], case["k"], case["n"]
        sizes = torch.tensor(_sizes(case["T"], case["top"], E))
        host = torch.Generator()
        host.manual_seed(int(seed) * 7919 + 3)
        sizes = sizes[torch.randperm(E, generator=host)]
        ends = sizes.cumsum(0)
        rows = int(ends[-1])
        s["most"] = int(sizes.max())
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).cuda()
        s["w"] = torch.empty(E, n, k, dtype=t, device="cuda")
        for e in range(E):
            s["w"][e] = _randn(gen, n, k, scale=k ** -0.5).to(t)
        s["x"] = _randn(gen, rows, k).to(t)
        if op == "grouped_forward":
            s["y"] = torch.empty(rows, n, dtype=t, device="cuda")
        else:
            s["dy"] = _randn(gen, rows, n).to(t)
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    return s


# ---------------------------------------------------------------- plain forms

def _padded(v, offsets, most):
    """fp32 rows [rows, c] sorted by expert -> [E, most, c], zeros behind each expert's last, and their places."""
    first, end = offsets[:-1].long(), offsets[1:].long()
    at = first[:, None] + torch.arange(most, device=v.device)
    there = at < end[:, None]
    out = v[torch.where(there, at, 0)].float()
    return torch.where(there[..., None], out, 0.0), there


def _plain(s):
    op, t = s["op"], _TYPES[s["type"]]
    if op == "norm_forward":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        x = x - mean
        rstd = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + _EPS)
        y = (x * rstd * s["w"].float() + s["b"].float()).to(_TYPES[s["out"]])
        return [y, mean[:, 0], rstd[:, 0]] if s["save"] else [y]
    if op == "norm_backward":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["w"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        return [dx.to(t), (dy * xhat).sum(0), dy.sum(0)]
    if op == "grouped_forward":
        x, there = _padded(s["x"], s["offsets"], s["most"])
        return [(x @ s["w"].float().transpose(1, 2))[there].to(t)]
    if op == "grouped_backward":
        dy, there = _padded(s["dy"], s["offsets"], s["most"])
        dx = (dy @ s["w"].float())[there].to(t)
        x, _ = _padded(s["x"], s["offsets"], s["most"])
        return [dx, (dy.transpose(1, 2) @ x).to(t)]
    g = s["g"].float()
    tall = g.shape[1] > g.shape[2]
    x = g / torch.linalg.vector_norm(g, dim=(1, 2), keepdim=True)
    x = x.transpose(1, 2) if tall else x
    a, b, c = _COEFFICIENTS
    for _ in range(5):
        p = x @ x.transpose(1, 2)
        x = a * x + (b * p + c * (p @ p)) @ x
    x = x.transpose(1, 2) if tall else x
    if s["weights"]:
        return [s["out"].copy_(s["out"].float() - 0.02 * x)]
    return [x.to(torch.bfloat16)]


# ---------------------------------------------------------------- the framework's calls

def _kept(s):
    """What the program makes once and keeps: the layer's norm, its experts' matrices, the update's workspace."""
    if "kept" not in s:
        from rvq_compressed_expert_gb300 import grouped, norm, ortho

        op = s["op"]
        if op in ("norm_forward", "norm_backward"):
            s["kept"] = norm.LayerNorm(s["w"], s["b"], eps=_EPS)
        elif op in ("grouped_forward", "grouped_backward"):
            s["kept"] = grouped.GroupedLinear(s["w"])
        else:
            s["kept"] = ortho.NewtonSchulz(s["count"], s["rows"], s["cols"], steps=5, coefficients=_COEFFICIENTS)
    return s["kept"]


def _own(s):
    op, k = s["op"], _kept(s)
    if op == "norm_forward":
        k.forward(s["x"], s["y"], s["mean"], s["rstd"])
        return [s["y"], s["mean"], s["rstd"]] if s["save"] else [s["y"]]
    if op == "norm_backward":
        k.backward(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"])
        return [s["dx"], s["dw"], s["db"]]
    if op == "grouped_forward":
        k.forward(s["x"], s["offsets"], s["y"])
        return [s["y"]]
    if op == "grouped_backward":
        k.backward(s["dy"], s["x"], s["offsets"], s["dx"], s["dw"])
        return [s["dx"], s["dw"]]
    if s["weights"]:
        k.orthogonalize(s["g"], s["out"], scale=-0.02, mode=1)
    else:
        k.orthogonalize(s["g"], s["out"])
    return [s["out"]]


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_forward":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + _EPS) ** -0.5
        y = torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double())
        return [y, mean, rstd] if case["save"] else [y]
    if op == "norm_backward":
        x, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        mean, rstd, d = s["mean"].double(), s["rstd"].double(), case["d"]
        h = torch.einsum("td,t->td", x - mean[:, None], rstd)
        one, two = torch.einsum("td,d->t", dy, w) / d, torch.einsum("td,d,td->t", dy, w, h) / d
        dx = torch.einsum("td,t->td", dy * w - one[:, None] - h * two[:, None], rstd)
        return [dx, torch.einsum("td,td->d", dy, h), torch.einsum("td->d", dy)]
    if op == "orthogonalize":
        a, b, c = _COEFFICIENTS
        out = []
        for g in s["g"]:
            x = g.double() if g.shape[0] <= g.shape[1] else g.double().t()
            x = x / x.square().sum().sqrt()
            for _ in range(5):
                p = torch.einsum("ik,jk->ij", x, x)
                px = torch.einsum("ij,jk->ik", p, x)
                x = a * x + b * px + c * torch.einsum("ij,jk->ik", p, px)
            out.append(x if g.shape[0] <= g.shape[1] else x.t())
        x = torch.stack(out)
        return [s["out"].double() - 0.02 * x if case["weights"] else x]
    at = s["offsets"].tolist()
    spans = list(zip(at[:-1], at[1:]))
    if op == "grouped_forward":
        return [torch.cat([torch.einsum("rk,nk->rn", s["x"][i:j].double(), w.double()) for w, (i, j) in zip(s["w"], spans)])]
    dx = torch.cat([torch.einsum("rn,nk->rk", s["dy"][i:j].double(), w.double()) for w, (i, j) in zip(s["w"], spans)])
    dw = torch.empty(s["w"].shape, dtype=torch.float64, device="cuda")
    for e, (i, j) in enumerate(spans):
        dw[e] = torch.einsum("rn,rk->nk", s["dy"][i:j].double(), s["x"][i:j].double())
    return [dx, dw]
