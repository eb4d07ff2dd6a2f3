"""The dense operators' C ABI without a GPU: declared, exported, bound, and bad arguments refused on
the host before anything is launched."""
import os
import re

import pytest
import torch

from rvq_compressed_expert_gb300 import _build
from rvq_compressed_expert_gb300 import binding as B
from tests import dense_ref as R

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "waste_dense.h")
P = 4096  # an aligned address that a refused call never reads


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return B.load()


class Bytes:
    """Stands in for a workspace tensor."""

    def __init__(self, n, at=P):
        self.n, self.at = n, at

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n


def test_header_matches_binding_and_library(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(waste_(?:dense|ffn|mx4)_\w+)\s*\(", text)))
    assert names == sorted(B.EXPORTED_DENSE)
    out = os.popen(f"nm -D --defined-only {B.LIB_PATH}").read()
    for n in names:
        assert re.search(rf"\bT {n}$", out, re.M), n


def refused(f, *a, **k):
    with pytest.raises(B.WasteError) as ei:
        f(*a, **k)
    assert ei.value.status == -1 and ei.value.message


def cfg(d=64, f=32, dtype=B.ACT_BF16, abi=B.ABI_VERSION):
    return B.waste_ffn_config(abi, d, f, dtype)


def test_workspace_sizes():
    assert B.waste_ffn_workspace(cfg(64, 32), 0) == 0
    assert B.waste_ffn_workspace(cfg(64, 32), 1) == 256
    # a call of T tokens may be followed by one of fewer in the same workspace
    for f in (8, 32, 1536):
        for back in (0, 1):
            n = [B.waste_ffn_workspace(cfg(64, f), T, back) for T in range(1, 40)]
            assert n == sorted(n) and all(v >= T * f * 2 * (3 if back else 1) and v % 256 == 0 for T, v in enumerate(n, 1))
    # past 32 bits
    assert B.waste_ffn_workspace(cfg(8, 1 << 20), 1 << 16) == 1 << 37
    assert B.waste_mx4_layout(0, 32) == (0, 0)
    assert B.waste_mx4_layout(1, 32) == (16, 512)
    assert B.waste_mx4_layout(129, 160) == (129 * 80, 2 * 2 * 512)
    assert B.waste_mx4_layout(1 << 20, 1 << 16) == (1 << 35, 1 << 31)


@pytest.mark.parametrize("c", [cfg(d=0), cfg(d=12), cfg(f=-8), cfg(f=20), cfg(dtype=B.ACT_F32), cfg(dtype=7),
                               cfg(abi=99)])
def test_ffn_bad_config(c):
    refused(B.waste_ffn_workspace, c, 1)
    refused(B.waste_ffn_forward, c, P, 1, P, P, P, P, B.ACT_BF16, 0, None, None, Bytes(1 << 20), stream=0)
    refused(B.waste_ffn_backward, c, P, 1, P, P, P, P, P, P, P, P, P, P, B.ACT_BF16, 0, Bytes(1 << 20), stream=0)


@pytest.mark.parametrize("change", [dict(x=None), dict(x=P + 8), dict(wg=None), dict(wu=P + 2), dict(wd=None),
                                    dict(out=None), dict(T=-1), dict(out_dtype=B.ACT_F16), dict(out_dtype=9),
                                    dict(mode=2), dict(mode=-1), dict(g=P), dict(u=P), dict(g=P, u=P + 4),
                                    dict(ws=Bytes(255)), dict(ws=Bytes(1 << 20, P + 128)),
                                    dict(ws=Bytes(1 << 20, None))])
def test_ffn_forward_refusals(change):
    a = dict(x=P, T=1, wg=P, wu=P, wd=P, out=P, out_dtype=B.ACT_BF16, mode=0, g=None, u=None, ws=Bytes(1 << 20))
    a.update(change)
    refused(B.waste_ffn_forward, cfg(), a["x"], a["T"], a["wg"], a["wu"], a["wd"], a["out"], a["out_dtype"],
            a["mode"], a["g"], a["u"], a["ws"], stream=0)


@pytest.mark.parametrize("change", [dict(dy=None), dict(x=P + 8), dict(g=None), dict(u=None), dict(wg=None),
                                    dict(wu=None), dict(wd=P + 1), dict(dx=P + 2), dict(dwg=None), dict(dwu=None),
                                    dict(dwd=None), dict(dwd=P + 8), dict(T=-1), dict(gt=B.ACT_F16), dict(acc=2),
                                    dict(ws=Bytes(3 * 256 - 1)), dict(ws=Bytes(1 << 20, P + 16))])
def test_ffn_backward_refusals(change):
    a = dict(dy=P, T=1, x=P, g=P, u=P, wg=P, wu=P, wd=P, dx=P, dwg=P, dwu=P, dwd=P, gt=B.ACT_BF16, acc=0,
             ws=Bytes(1 << 20))
    a.update(change)
    refused(B.waste_ffn_backward, cfg(), *(a[k] for k in ("dy", "T", "x", "g", "u", "wg", "wu", "wd", "dx", "dwg",
                                                          "dwu", "dwd", "gt", "acc", "ws")), stream=0)


def test_nothing_to_do_is_ok():
    """No tokens, or no output wanted: success without a launch."""
    w = Bytes(0, None)
    B.waste_ffn_forward(cfg(), None, 0, None, None, None, None, B.ACT_F32, 0, None, None, w, stream=0)
    B.waste_ffn_backward(cfg(), None, 0, None, None, None, None, None, None, None, None, None, None, B.ACT_F32, 0, w,
                         stream=0)
    B.waste_ffn_backward(cfg(), P, 3, P, P, P, P, P, P, None, None, None, None, B.ACT_F32, 0, w, stream=0)
    B.waste_mx4_quantize(None, B.ACT_F32, 0, 32, 32, None, None, stream=0)
    B.waste_mx4_dequantize(None, None, 0, 32, None, B.ACT_F32, 32, stream=0)
    B.waste_mx4_matmul(0, 1, 32, None, None, None, None, None, B.ACT_F32, stream=0)


@pytest.mark.parametrize("shape", [(-1, 32), (1, 0), (1, 16), (1, 48), (4, -32)])
def test_mx4_bad_shapes(shape):
    refused(B.waste_mx4_layout, *shape)
    refused(B.waste_mx4_quantize, P, B.ACT_F32, *shape, 64, P, P, stream=0)
    refused(B.waste_mx4_dequantize, P, P, *shape, P, B.ACT_F32, 64, stream=0)
    refused(B.waste_mx4_matmul, shape[0], 1, shape[1], P, P, P, P, P, B.ACT_F32, stream=0)


def test_sizes_past_the_limit():
    """Sizes past 2^30 are refused before any arithmetic on them."""
    big = (1 << 30) + 32
    refused(B.waste_ffn_workspace, cfg(), big)
    refused(B.waste_ffn_workspace, cfg(d=big), 1)
    refused(B.waste_mx4_layout, big, 32)
    refused(B.waste_mx4_layout, 1, big)
    refused(B.waste_mx4_matmul, 1, big, 32, P, P, P, P, P, B.ACT_F32, 0, stream=0)
    refused(B.waste_mx4_ffn_workspace, B.waste_mx4_ffn_config(B.ABI_VERSION, 32, big, P, P, P, P, P, P), 1)


def test_mx4_refusals():
    for a in ((None, B.ACT_F32, 1, 32, 32, P, P), (P + 4, B.ACT_F32, 1, 32, 32, P, P), (P, 3, 1, 32, 32, P, P),
              (P, B.ACT_F32, 1, 64, 32, P, P), (P, B.ACT_BF16, 2, 32, 36, P, P), (P, B.ACT_F32, 1, 32, 32, None, P),
              (P, B.ACT_F32, 1, 32, 32, P, None), (P, B.ACT_F32, 1, 32, 32, P + 8, P)):
        refused(B.waste_mx4_quantize, *a, stream=0)
    for a in ((None, P, 1, 32, P, B.ACT_F32, 32), (P, P, 1, 32, None, B.ACT_F32, 32), (P, P, 1, 32, P, -1, 32),
              (P, P, 1, 32, P, B.ACT_F16, 33), (P, P + 1, 1, 32, P, B.ACT_F16, 32)):
        refused(B.waste_mx4_dequantize, *a, stream=0)
    for a in ((1, 0, 32, P, P, P, P, P, B.ACT_F32, 0), (1, 1, 32, None, P, P, P, P, B.ACT_F32, 0),
              (1, 1, 32, P, P, P, P, None, B.ACT_F32, 0), (1, 1, 32, P, P, P, P, P, 5, 0),
              (1, 1, 32, P, P, P, P, P, B.ACT_F32, 2), (1, 1, 32, P, P + 4, P, P, P, B.ACT_F32, 0)):
        refused(B.waste_mx4_matmul, *a, stream=0)


def test_mx4_ffn_refusals():
    def c(d=64, f=32, abi=B.ABI_VERSION, **k):
        m = B.waste_mx4_ffn_config(abi, d, f, P, P, P, P, P, P)
        for n, v in k.items():
            setattr(m, n, v)
        return m

    for bad in (c(d=16), c(f=48), c(d=0), c(abi=0)):
        refused(B.waste_mx4_ffn_workspace, bad, 1)
        refused(B.waste_mx4_ffn_forward, bad, P, B.ACT_F32, 1, P, B.ACT_F32, 0, Bytes(1 << 20), stream=0)
    need = B.waste_mx4_ffn_workspace(c(), 1)
    for a in ((c(d_up_codes=None), P, 0, 1, P, 0, 0, Bytes(need)), (c(d_down_scales=P + 8), P, 0, 1, P, 0, 0, Bytes(need)),
              (c(), None, 0, 1, P, 0, 0, Bytes(need)), (c(), P, 4, 1, P, 0, 0, Bytes(need)),
              (c(), P, 0, 1, P, 4, 0, Bytes(need)), (c(), P, 0, 1, P, 0, 3, Bytes(need)),
              (c(), P, 0, -1, P, 0, 0, Bytes(need)), (c(), P, 0, 1, P, 0, 0, Bytes(need - 1)),
              (c(), P, 0, 1, P, 0, 0, Bytes(need, P + 16))):
        refused(B.waste_mx4_ffn_forward, *a, stream=0)
    B.waste_mx4_ffn_forward(c(), None, 0, 0, None, 0, 0, Bytes(0, None), stream=0)


def test_reference_codes_by_hand():
    """The 64-bit reference against values worked by hand: a block whose largest value is 7 has
    exponent 0; 7 saturates to 6, borders go to the even code, a small block to its own power."""
    v = torch.zeros(1, 32)
    v[0, :12] = torch.tensor([7.0, -0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, -0.0, -6.9])
    code, scale = R.mx_codes(v)
    assert scale.tolist() == [[127]]
    assert code[0, :12].tolist() == [7, 8, 1, 2, 2, 4, 4, 6, 6, 7, 8, 15]
    assert (R.mx_values(code, scale)[0, :4] == torch.tensor([6.0, 0.0, 0.5, 1.0])).all()
    code, scale = R.mx_codes(torch.full((1, 32), 3.0 * 2.0 ** -130, dtype=torch.float64))
    assert scale.tolist() == [[0]] and code.unique().tolist() == [1]  # 0.375 of 2^-127 goes to 0.5
    assert R.mx_codes(torch.full((1, 32), float("inf")))[1].tolist() == [[255]]
    codes, scales = R.mx_pack(*R.mx_codes(torch.eye(130, 160)))
    assert codes.shape == (130, 80) and scales.numel() == 2 * 2 * 512
    # row 129, block 4 (its one at column 129): second row tile, second tile of blocks; 1 = 4 x 2^-2
    assert scales[3 * 512 + 1 * 16 + 0 * 4 + 0] == 125 and codes[129, 64] == 6 << 4


def test_debug_wait_refusals():
    for a in ((-1, 0), ((1 << 18) + 1, 0), (1, 2), (1, -1)):
        refused(B.waste_dense_debug_wait, *a, stream=0)


# ---------------------------------------------------------------- memory that a call writes and something else of it

A = 1 << 40  # far from anything; never read


def overlap(f, *a):
    with pytest.raises(B.WasteError) as ei:
        f(*a, stream=0)
    assert ei.value.status == -1 and "overlaps" in ei.value.message, ei.value.message


def test_backward_overlaps():
    """dx over dy, over x, a gradient over its weight or another gradient, by their first and last 16 bytes."""
    T, d, f = 6, 64, 32
    size = dict(dy=T * d * 2, x=T * d * 2, g=T * f * 2, u=T * f * 2, wg=d * f * 2, wu=d * f * 2, wd=d * f * 2, dx=T * d * 2,
                dwg=d * f * 4, dwu=d * f * 4, dwd=d * f * 4)
    need = B.waste_ffn_workspace(cfg(d, f), T, 1)
    names = list(size)
    place = {n: A + (i << 20) for i, n in enumerate(names)}

    def call(p, ws):
        B.waste_ffn_backward(cfg(d, f), p["dy"], T, *(p[k] for k in names[1:]), B.ACT_F32, 0, Bytes(need, ws), stream=0)

    for out in ("dx", "dwg", "dwu", "dwd"):
        for other in names:
            if other == out:
                continue
            for at in (place[other], place[other] + size[other] - 16, place[other] - size[out] + 16):
                with pytest.raises(B.WasteError) as ei:
                    call({**place, out: at}, A - (1 << 30))
                assert ei.value.status == -1 and "overlaps" in ei.value.message
    for other in names:
        with pytest.raises(B.WasteError) as ei:
            call(place, (place[other] + size[other] - 1) // 256 * 256)
        assert "workspace overlaps" in ei.value.message


def test_forward_overlaps():
    T, d, f = 5, 64, 32
    c, need = cfg(d, f), B.waste_ffn_workspace(cfg(d, f), 5)
    w = [A + (i << 20) for i in range(8)]  # x wg wu wd out g u ws

    def call(**k):
        x, wg, wu, wd, out, g, u, ws = (k.get(n, v) for n, v in zip(("x", "wg", "wu", "wd", "out", "g", "u", "ws"), w))
        overlap(B.waste_ffn_forward, c, x, T, wg, wu, wd, out, B.ACT_F32, 0, g, u, Bytes(need, ws))

    for n in range(1, 4):
        call(out=w[n] + d * f * 2 - 16)
        call(g=w[n])
        call(ws=w[n])
    call(g=w[0])
    call(u=w[0] + 16)
    call(g=w[4] + T * d * 4 - 16)
    call(u=w[5] + 16)
    call(ws=w[0])
    call(ws=w[4])


def test_mx4_overlaps():
    M, N, K = 3, 5, 64
    ns = 512
    p = [A + (i << 20) for i in range(5)]
    for i, n in ((0, M * K // 2), (1, ns), (2, N * K // 2), (3, ns)):
        for at in (p[i], p[i] + (n - 1) // 16 * 16, p[i] - M * N * 4 // 16 * 16):
            overlap(B.waste_mx4_matmul, M, N, K, *p[:4], at, B.ACT_F32, 0)
    # strided rows: the gaps between them are the caller's
    rows, cols, ld = 4, 32, 96
    for at in (p[0], p[0] + 16, p[0] + 3 * ld * 4, p[0] + 3 * ld * 4 + 112):
        overlap(B.waste_mx4_quantize, p[0], B.ACT_F32, rows, cols, ld, at, p[1])
        overlap(B.waste_mx4_dequantize, at, p[1], rows, cols, p[0], B.ACT_F32, ld)
    overlap(B.waste_mx4_quantize, p[0], B.ACT_F32, rows, cols, ld, p[1], p[1] + 16)
    overlap(B.waste_mx4_dequantize, p[2], p[0] + 2 * ld * 4, rows, cols, p[0], B.ACT_F32, ld)
    m = B.waste_mx4_ffn_config(B.ABI_VERSION, 64, 32, *(A + (i << 20) for i in range(6)))
    need = B.waste_mx4_ffn_workspace(m, 2)
    for i in range(6):
        overlap(B.waste_mx4_ffn_forward, m, A - (1 << 20), 0, 2, A + (i << 20), 0, 0, Bytes(need, A - (1 << 24)))
        overlap(B.waste_mx4_ffn_forward, m, A - (1 << 20), 0, 2, A - (2 << 20), 0, 0, Bytes(need, A + (i << 20)))
    overlap(B.waste_mx4_ffn_forward, m, A - (1 << 20), 0, 2, A - (2 << 20), 0, 0, Bytes(need, A - (1 << 20)))
    overlap(B.waste_mx4_ffn_forward, m, A - (1 << 20), 0, 2, A - (2 << 20), 0, 0, Bytes(need, A - (2 << 20)))


@pytest.mark.parametrize("far", [(1 << 32) + 32, 1 << 31, (1 << 40) + 64, -(1 << 32) + 32])
def test_sizes_past_32_bits(far):
    """Sizes that would be other, valid ones once cut to 32 bits."""
    refused(B.waste_ffn_config, B.ABI_VERSION, far, 32, B.ACT_BF16)
    refused(B.waste_ffn_config, B.ABI_VERSION, 64, far, B.ACT_BF16)
    refused(B.waste_mx4_ffn_config, B.ABI_VERSION, far, 32, P, P, P, P, P, P)
    refused(B.waste_mx4_ffn_config, B.ABI_VERSION, 32, far, P, P, P, P, P, P)
    m, w = B.waste_mx4_ffn_config(B.ABI_VERSION, 64, 32, P, P, P, P, P, P), Bytes(1 << 40)
    refused(B.waste_ffn_workspace, cfg(), far)
    refused(B.waste_ffn_forward, cfg(), P, far, P, P, P, P, B.ACT_F32, 0, None, None, w, stream=0)
    refused(B.waste_ffn_backward, cfg(), P, far, P, P, P, P, P, P, P, P, P, P, B.ACT_F32, 0, w, stream=0)
    refused(B.waste_mx4_ffn_workspace, m, far)
    refused(B.waste_mx4_ffn_forward, m, P, 0, far, P, 0, 0, w, stream=0)
    for r, c in ((far, 32), (32, far)):
        refused(B.waste_mx4_layout, r, c)
        refused(B.waste_mx4_quantize, P, 0, r, c, max(far, 32), P, P, stream=0)
        refused(B.waste_mx4_dequantize, P, P, r, c, P, 0, max(far, 32), stream=0)
    for s in ((far, 32, 32), (32, far, 32), (32, 32, far)):
        refused(B.waste_mx4_matmul, *s, P, P, P, P, P, 0, stream=0)


def test_configs_take_fields_by_name():
    c = B.waste_ffn_config(abi_version=B.ABI_VERSION, d=64, f=32, dtype=B.ACT_F16)
    assert (c.d, c.f, c.dtype) == (64, 32, B.ACT_F16) and B.waste_ffn_config().d == 0
    m = B.waste_mx4_ffn_config(B.ABI_VERSION, 64, d_up_codes=P, f=32)
    assert (m.d, m.f, m.d_up_codes, m.d_gate_codes) == (64, 32, P, None)
    refused(lambda: B.waste_ffn_config(d=1 << 32))
    refused(lambda: B.waste_mx4_ffn_config(B.ABI_VERSION, 64, f=1 << 33))
