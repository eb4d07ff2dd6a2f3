"""The dense operators beside the routed experts, as they are measured.

  ffn_forward    gated feed-forward block: y = (silu(x Wg^T) * (x Wu^T)) Wd^T
  ffn_backward   its gradients: dx, dWg, dWu, dWd from dy and the saved g, u
  mx4_roundtrip  a matrix quantised to microscaled 4-bit floats and read back
  mx4_matmul     the product A B^T of two microscaled 4-bit matrices
  mx4_ffn        the gated block with its weights in microscaled 4-bit floats

Sizes are those of the package's workloads (hidden size 7168, expert width 1536, and the small
256 x 128 layer), one token to a long prompt.

Microscaled 4-bit floats: blocks of 32 values along a row share a power of two (E8M0, one byte),
each value is an E2M1 code (two codes a byte, the lower column in the low half).  The scale
bytes stand in tiles of 128 rows x 4 blocks: the byte of row r, block k is at
((r // 128) * ceil(K / 128) + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through a dense expert beside the routed ones
        {"name": "ffn token", "op": "ffn_forward", "T": 1, "d": 7168, "f": 1536, "type": "bf16", "save": False},
        # a batch of decoding sequences, of no round number
        {"name": "ffn batch", "op": "ffn_forward", "T": 131, "d": 7168, "f": 1536, "type": "fp16", "save": False},
        # a training step's forward, g and u kept for the backward
        {"name": "ffn train forward", "op": "ffn_forward", "T": 4096, "d": 7168, "f": 1536, "type": "bf16", "save": True},
        # the same step's gradients
        {"name": "ffn train backward", "op": "ffn_backward", "T": 4096, "d": 7168, "f": 1536, "type": "bf16"},
        # fine-tuning a small expert on a ragged batch
        {"name": "ffn small backward", "op": "ffn_backward", "T": 333, "d": 1032, "f": 264, "type": "fp16"},
        # the hidden state of one token made 4-bit
        {"name": "mx4 token roundtrip", "op": "mx4_roundtrip", "rows": 1, "cols": 7168, "type": "fp32"},
        # a long prompt's hidden states, or a large weight, with an odd number of rows
        {"name": "mx4 large roundtrip", "op": "mx4_roundtrip", "rows": 16383, "cols": 7168, "type": "bf16"},
        # one token against one projection
        {"name": "mx4 token matmul", "op": "mx4_matmul", "M": 1, "N": 1536, "K": 7168, "type": "fp32"},
        # a prompt chunk against one projection
        {"name": "mx4 chunk matmul", "op": "mx4_matmul", "M": 509, "N": 7168, "K": 1536, "type": "bf16"},
        # a long prompt against a square projection of the hidden size
        {"name": "mx4 large matmul", "op": "mx4_matmul", "M": 4096, "N": 7168, "K": 7168, "type": "bf16"},
        # one decoded token through a 4-bit expert
        {"name": "mx4 ffn token", "op": "mx4_ffn", "T": 1, "d": 7168, "f": 1536, "type": "bf16"},
        # a prompt through a 4-bit expert
        {"name": "mx4 ffn prompt", "op": "mx4_ffn", "T": 2048, "d": 7168, "f": 1536, "type": "bf16"},
    ]


def _spread(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["ffn_forward", "ffn_backward", "mx4_roundtrip", "mx4_matmul", "mx4_ffn"])
    half = rng.choice(["bf16", "fp16"])
    if op == "ffn_forward":
        return {"op": op, "T": _spread(rng, 1, 4096), "d": _spread(rng, 256, 7168, 8), "f": _spread(rng, 128, 1536, 8),
                "type": half, "save": rng.random() < 0.5}
    if op == "ffn_backward":
        return {"op": op, "T": _spread(rng, 1, 4096), "d": _spread(rng, 256, 7168, 8), "f": _spread(rng, 128, 1536, 8),
                "type": half}
    if op == "mx4_roundtrip":
        return {"op": op, "rows": _spread(rng, 1, 16383), "cols": _spread(rng, 32, 7168, 32),
                "type": rng.choice(["bf16", "fp16"])}
    if op == "mx4_matmul":
        return {"op": op, "M": _spread(rng, 1, 4096), "N": _spread(rng, 64, 7168), "K": _spread(rng, 128, 7168, 32),
                "type": rng.choice(["bf16", "fp32"])}
    return {"op": op, "T": _spread(rng, 1, 2048), "d": _spread(rng, 256, 7168, 32), "f": _spread(rng, 128, 1536, 32),
            "type": "bf16"}


def work(case):
    op, s = case["op"], _SIZE[case["type"]]
    if op in ("ffn_forward", "ffn_backward", "mx4_ffn"):
        T, d, f = case["T"], case["d"], case["f"]
        if op == "ffn_forward":
            return {"bytes": s * (2 * T * d + 3 * f * d + (2 * T * f if case["save"] else 0)), "flops": 6 * T * f * d}
        if op == "ffn_backward":
            return {"bytes": s * (3 * T * d + 2 * T * f + 6 * f * d), "flops": 12 * T * f * d}
        return {"bytes": 2 * s * T * d + 3 * f * d * 17 / 32, "flops": 6 * T * f * d}
    if op == "mx4_roundtrip":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * s * n + 2 * n * 17 / 32, "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": (M + N) * K * 17 / 32 + s * M * N, "flops": 2 * M * N * K}


# ---------------------------------------------------------------- inputs

def _randn(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * scale


def _code_table():
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    return torch.cat([half, -half])


def _scale_places(rows, blocks):
    """Where the scale byte of (row, block) stands."""
    r = torch.arange(rows, device="cuda")[:, None]
    k = torch.arange(blocks, device="cuda")[None, :]
    return ((r // 128) * -(-blocks // 4) + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4


def _mx4_parts(v):
    """fp32 [rows, cols] -> (code numbers [rows, cols], power of two's exponent + 127 [rows, blocks])."""
    b = v.reshape(v.shape[0], -1, 32)
    big = b.abs().amax(-1)
    e = (torch.frexp(big).exponent - 3).clamp(-127, 127)
    e = torch.where(big == 0, torch.full_like(e, -127), e)
    x = torch.ldexp(b.abs(), -e[..., None])
    step = torch.where(x < 2, 0.5, torch.where(x < 4, 1.0, 2.0))
    q = (torch.round(x / step) * step).clamp(max=6.0)
    table = _code_table()[:8]
    code = torch.searchsorted(table, q) + 8 * torch.signbit(b)
    return code.reshape(v.shape).to(torch.uint8), (e + 127).to(torch.uint8)


def _mx4_pack(v):
    """What a program keeps of a 4-bit matrix: its packed codes and its scale tiles."""
    rows, cols = v.shape
    code, e = _mx4_parts(v)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = torch.zeros(-(-rows // 128) * -(-cols // 128) * 512, dtype=torch.uint8, device="cuda")
    scales[_scale_places(rows, cols // 32)] = e
    return codes.contiguous(), scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    op, t = case["op"], _TYPES[case["type"]]
    s = dict(case)
    if op == "ffn_forward" or op == "ffn_backward":
        T, d, f = case["T"], case["d"], case["f"]
        s["x"] = _randn(gen, T, d).to(t)
        s["w_gate"], s["w_up"] = (_randn(gen, f, d, scale=d ** -0.5).to(t) for _ in range(2))
        s["w_down"] = _randn(gen, d, f, scale=f ** -0.5).to(t)
        if op == "ffn_forward":
            s["out"] = torch.empty(T, d, dtype=t, device="cuda")
            s["g"], s["u"] = (torch.empty(T, f, dtype=t, device="cuda") if case["save"] else None for _ in range(2))
        else:
            # what the forward of this step kept: the projections, of unit size here
            s["g"], s["u"] = (_randn(gen, T, f).to(t) for _ in range(2))
            s["dy"] = _randn(gen, T, d).to(t)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = [torch.empty_like(s[n]) for n in ("w_gate", "w_up", "w_down")]
    elif op == "mx4_roundtrip":
        # values over several binades, as hidden states have: a few columns much larger than the rest
        v = _randn(gen, case["rows"], case["cols"])
        v *= torch.exp(_randn(gen, 1, case["cols"], scale=1.5))
        s["x"] = v.to(t)
        s["out"] = torch.empty_like(s["x"])
    elif op == "mx4_matmul":
        s["a"] = _mx4_pack(_randn(gen, case["M"], case["K"]))
        s["b"] = _mx4_pack(_randn(gen, case["N"], case["K"], scale=case["K"] ** -0.5))
        s["out"] = torch.empty(case["M"], case["N"], dtype=t, device="cuda")
    else:
        T, d, f = case["T"], case["d"], case["f"]
        s["x"] = _randn(gen, T, d).to(t)
        s["w_gate"], s["w_up"] = (_mx4_pack(_randn(gen, f, d, scale=d ** -0.5)) for _ in range(2))
        s["w_down"] = _mx4_pack(_randn(gen, d, f, scale=f ** -0.5))
        s["out"] = torch.empty(T, d, dtype=t, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _values(m, cols):
    """fp32 values of a packed 4-bit matrix."""
    codes, scales = m
    rows = codes.shape[0]
    table = _code_table()
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).reshape(rows, cols // 32, 32)
    e = scales[_scale_places(rows, cols // 32)].int() - 127
    return torch.ldexp(v, e[..., None]).reshape(rows, cols)


def _requantised(v):
    """The values that v's 4-bit form stands for, in fp32."""
    code, e = _mx4_parts(v)
    b = _code_table()[code.int()].reshape(v.shape[0], -1, 32)
    return torch.ldexp(b, e.int()[..., None] - 127).reshape(v.shape)


def _plain(s):
    op, t = s["op"], _TYPES[s["type"]]
    if op == "ffn_forward":
        x, wg, wu, wd = (s[n].float() for n in ("x", "w_gate", "w_up", "w_down"))
        g, u = x @ wg.t(), x @ wu.t()
        y = (g * torch.sigmoid(g) * u) @ wd.t()
        return [y.to(t), g.to(t), u.to(t)] if s["save"] else [y.to(t)]
    if op == "ffn_backward":
        x, wg, wu, wd, g, u, dy = (s[n].float() for n in ("x", "w_gate", "w_up", "w_down", "g", "u", "dy"))
        sg = torch.sigmoid(g)
        da = dy @ wd
        du = da * g * sg
        dg = da * u * sg * (1 + g * (1 - sg))
        out = [dg @ wg + du @ wu, dg.t() @ x, du.t() @ x, dy.t() @ (g * sg * u)]
        return [o.to(t) for o in out]
    if op == "mx4_roundtrip":
        return [_requantised(s["x"].float()).to(t)]
    if op == "mx4_matmul":
        return [(_values(s["a"], s["K"]) @ _values(s["b"], s["K"]).t()).to(t)]
    x = _requantised(s["x"].float())
    g, u = x @ _values(s["w_gate"], s["d"]).t(), x @ _values(s["w_up"], s["d"]).t()
    a = _requantised(g * torch.sigmoid(g) * u)
    return [(a @ _values(s["w_down"], s["f"]).t()).to(t)]


# ---------------------------------------------------------------- the framework's calls

def _kept(s):
    """What the program makes once from its weights and keeps: the expert, the 4-bit matrices."""
    if "kept" not in s:
        from rvq_compressed_expert_gb300 import dense, mx4

        op = s["op"]
        if op in ("ffn_forward", "ffn_backward"):
            s["kept"] = dense.DenseExpert(s["w_gate"], s["w_up"], s["w_down"], max_tokens=s["T"])
        elif op == "mx4_roundtrip":
            s["kept"] = mx4.Mx4Matrix.empty(s["rows"], s["cols"])
        elif op == "mx4_matmul":
            s["kept"] = [mx4.Mx4Matrix(s["M"], s["K"], *s["a"]), mx4.Mx4Matrix(s["N"], s["K"], *s["b"])]
        else:
            d, f = s["d"], s["f"]
            s["kept"] = mx4.Mx4Expert(mx4.Mx4Matrix(f, d, *s["w_gate"]), mx4.Mx4Matrix(f, d, *s["w_up"]),
                                      mx4.Mx4Matrix(d, f, *s["w_down"]), max_tokens=s["T"])
    return s["kept"]


def _own(s):
    op, k = s["op"], _kept(s)
    if op == "ffn_forward":
        k.forward(s["x"], s["out"], save_g=s["g"], save_u=s["u"])
        return [s["out"], s["g"], s["u"]] if s["save"] else [s["out"]]
    if op == "ffn_backward":
        k.backward(s["dy"], s["x"], s["g"], s["u"], s["dx"], *s["dw"])
        return [s["dx"], *s["dw"]]
    if op == "mx4_roundtrip":
        k.quantize(s["x"])
        k.dequantize(s["out"])
    elif op == "mx4_matmul":
        from rvq_compressed_expert_gb300 import mx4

        mx4.matmul(k[0], k[1], s["out"])
    else:
        k.forward(s["x"], s["out"])
    return [s["out"]]


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------- 64 bits, from the definitions

def _grid64(v):
    """The nearest microscaled 4-bit value of each entry of v [rows, cols], in 64 bits."""
    b = v.double().reshape(-1, 32)
    big = b.abs().amax(1, keepdim=True)
    e = torch.floor(torch.log2(big.clamp(min=2.0 ** -300)))
    e = e + (torch.exp2(e + 1) <= big).double() - (torch.exp2(e) > big).double()
    p = torch.exp2((e - 2).clamp(-127, 127))
    x = b.abs() / p
    # borders between neighbouring values; a value on a border goes to the even code
    q = torch.zeros_like(x)
    for border, up, even in ((0.25, 0.5, False), (0.75, 1.0, True), (1.25, 1.5, False), (1.75, 2.0, True),
                             (2.5, 3.0, False), (3.5, 4.0, True), (5.0, 6.0, False)):
        q = torch.where((x >= border) if even else (x > border), torch.full_like(q, up), q)
    return (torch.sign(b) * q * p).reshape(v.shape)


def _unpacked64(m, rows, cols):
    codes, scales = m
    n = torch.empty(rows, cols, dtype=torch.int64, device="cuda")
    n[:, 0::2], n[:, 1::2] = (codes % 16).long(), (codes // 16).long()
    exponent, mantissa = (n % 8) // 2, (n % 2).double()
    size = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.exp2(exponent.double() - 1))
    # tiles of [row tile][block tile][row % 32][row // 32 % 4][block % 4], read back in row order
    t = scales.reshape(-(-rows // 128), -(-cols // 128), 32, 4, 4).permute(0, 3, 2, 1, 4)
    t = t.reshape(-(-rows // 128) * 128, -1)[:rows, : cols // 32].double()
    return (torch.where(n >= 8, -size, size).reshape(rows, -1, 32) * torch.exp2(t - 127)[..., None]).reshape(rows, cols)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ffn_forward":
        x = s["x"].double()
        g, u = torch.einsum("td,fd->tf", x, s["w_gate"].double()), torch.einsum("td,fd->tf", x, s["w_up"].double())
        y = torch.einsum("tf,df->td", g / (1 + torch.exp(-g)) * u, s["w_down"].double())
        return [y, g, u] if case["save"] else [y]
    if op == "ffn_backward":
        x, g, u, dy = (s[n].double() for n in ("x", "g", "u", "dy"))
        e = torch.exp(-g)
        silu, slope = g / (1 + e), (1 + e + g * e) / (1 + e) ** 2
        da = torch.einsum("td,df->tf", dy, s["w_down"].double())
        dg, du = da * u * slope, da * silu
        dx = torch.einsum("tf,fd->td", dg, s["w_gate"].double()) + torch.einsum("tf,fd->td", du, s["w_up"].double())
        return [dx, torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x),
                torch.einsum("td,tf->df", dy, silu * u)]
    if op == "mx4_roundtrip":
        return [_grid64(s["x"])]
    if op == "mx4_matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return [torch.einsum("mk,nk->mn", _unpacked64(s["a"], M, K), _unpacked64(s["b"], N, K))]
    T, d, f = case["T"], case["d"], case["f"]
    x = _grid64(s["x"])
    g = torch.einsum("td,fd->tf", x, _unpacked64(s["w_gate"], f, d))
    u = torch.einsum("td,fd->tf", x, _unpacked64(s["w_up"], f, d))
    a = _grid64(g / (1 + torch.exp(-g)) * u)
    return [torch.einsum("tf,df->td", a, _unpacked64(s["w_down"], d, f))]
