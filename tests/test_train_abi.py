"""The training operators' C ABI without a GPU: declared, exported, bound, and bad arguments refused on the host before
anything is launched."""
import os
import re

import pytest

from rvq_compressed_expert_gb300 import _build
from rvq_compressed_expert_gb300 import binding as B
from tests import train_ref as R

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "waste_train.h")
A = 1 << 40  # an address that a refused call never reads
F, H, BF = B.ACT_F32, B.ACT_F16, B.ACT_BF16


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return B.load()


class Bytes:
    """Stands in for a workspace tensor."""

    def __init__(self, n, at=A):
        self.n, self.at = n, at

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n


def refused(f, *a, word="", **k):
    with pytest.raises(B.WasteError) as ei:
        f(*a, **k)
    assert ei.value.status == -1 and ei.value.message and word in ei.value.message, ei.value.message


def test_header_matches_binding_and_library():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(waste_\w+)\s*\(", text)))
    assert names == sorted(B.EXPORTED_TRAIN)
    out = os.popen(f"nm -D --defined-only {B.LIB_PATH}").read()
    for n in names:
        assert re.search(rf"\bT {n}$", out, re.M), n


# ---------------------------------------------------------------- layer norm

def norm(d=64, x=F, y=F, w=F, eps=1e-5, abi=B.ABI_VERSION):
    return B.waste_norm_config(abi, d, x, y, w, eps)


def forward(c=None, **k):
    a = dict(x=A, ldx=64, T=3, w=A + (1 << 20), b=A + (2 << 20), y=A + (3 << 20), ldy=64, mean=None, rstd=None)
    a.update(k)
    B.waste_norm_forward(c or norm(), *a.values(), stream=0)


def backward(c=None, ws=Bytes(1 << 20, A + (9 << 20)), **k):
    a = dict(dy=A, lddy=64, x=A + (1 << 20), ldx=64, T=3, mean=A + (2 << 20), rstd=A + (3 << 20), w=A + (4 << 20),
             dx=A + (5 << 20), lddx=64, dw=A + (6 << 20), db=A + (7 << 20), gt=F, acc=0)
    a.update(k)
    B.waste_norm_backward(c or norm(), *a.values(), ws, stream=0)


@pytest.mark.parametrize("c", [norm(d=0), norm(d=-8), norm(x=3), norm(y=-1), norm(w=7), norm(eps=-1e-9), norm(eps=float("nan")),
                               norm(eps=float("inf")), norm(abi=2), norm(d=(1 << 30) + 1)])
def test_norm_bad_config(c):
    refused(forward, c)
    refused(backward, c)
    refused(B.waste_norm_workspace, c, 1)


def test_norm_refusals():
    for k in (dict(x=None), dict(y=None), dict(x=A + 2), dict(y=A + 1), dict(w=A + 2), dict(b=A + 3), dict(ldx=63), dict(ldy=0),
              dict(ldx=(1 << 40) + 1), dict(T=-1), dict(mean=A + (4 << 20)), dict(rstd=A + (4 << 20)),
              dict(mean=A + (4 << 20) + 2, rstd=A + (5 << 20))):
        refused(forward, **k)
    for k in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(rstd=A + 2), dict(w=A + 1), dict(dx=A + (5 << 20) + 2),
              dict(lddx=60), dict(lddy=1), dict(T=-2), dict(dw=A + (6 << 20) + 2), dict(gt=BF), dict(gt=9), dict(acc=2),
              dict(ws=Bytes(0)), dict(ws=Bytes(1 << 20, A + 128)), dict(ws=Bytes(1 << 20, None)), dict(ws=None)):
        refused(backward, **k)
    refused(backward, norm(w=BF), gt=H)


def test_norm_overlaps():
    n = 3 * 64 * 4
    for at in (A + 16, A - 16, A + n - 4):
        refused(forward, y=at, word="overlaps")
    refused(forward, norm(y=BF), y=A, word="overlaps")  # in place only where the types agree
    refused(forward, y=A, ldy=65, ldx=64, word="overlaps")
    refused(forward, mean=A + 64, rstd=A + (5 << 20), word="overlaps")
    refused(forward, mean=A + (5 << 20), rstd=A + (5 << 20) + 8, word="overlaps")
    refused(forward, y=A + (1 << 20) - n + 4, word="overlaps")  # over w
    for out in ("dx", "dw", "db"):
        for at in (A + (1 << 20), A + (2 << 20), A + (3 << 20) + 8, A + (4 << 20) + 252):
            refused(backward, **{out: at}, word="overlaps")
    for out in ("dw", "db"):
        refused(backward, **{out: A + n - 4}, word="overlaps")
    refused(backward, dx=A + 4, word="overlaps")
    refused(backward, norm(y=H, w=F), dx=A, word="overlaps")
    refused(backward, ws=Bytes(1 << 20, A + (1 << 20)), word="overlaps")
    refused(backward, db=A + (6 << 20) + 252, word="overlaps")
    # rows of one stride between each other's are apart, by one value less they are not
    refused(forward, ldx=128, ldy=128, y=A + 252, word="overlaps")
    refused(forward, ldx=128, ldy=128, y=A - 3 * 512 + 260, word="overlaps")


def test_norm_nothing_to_do():
    forward(T=0, x=None, y=None, w=None, b=None)
    backward(T=0, dw=None, db=None, dx=None, ws=None)
    backward(T=0, dw=None, db=None, x=None, dy=None, mean=None, rstd=None, ws=None)
    backward(dx=None, dw=None, db=None, ws=None)
    assert B.waste_norm_workspace(norm(), 0) == 0
    sizes = [B.waste_norm_workspace(norm(), T) for T in (1, 2, 16, 100, 1 << 30)]
    assert sizes == sorted(sizes) and sizes[0] >= 512


# ---------------------------------------------------------------- products grouped by expert

def group(E=4, k=64, n=32, t=BF, abi=B.ABI_VERSION):
    return B.waste_group_config(abi, E, k, n, t)


def gforward(c=None, **k):
    a = dict(x=A, rows=5, off=A + (1 << 20), w=A + (2 << 20), out=A + (3 << 20), t=BF, mode=0)
    a.update(k)
    B.waste_group_forward(c or group(), *a.values(), stream=0)


def gbackward(c=None, **k):
    a = dict(dy=A, x=A + (1 << 20), rows=5, off=A + (2 << 20), w=A + (3 << 20), dx=A + (4 << 20), dw=A + (5 << 20), t=BF, acc=0)
    a.update(k)
    B.waste_group_backward(c or group(), *a.values(), stream=0)


@pytest.mark.parametrize("c", [group(E=0), group(E=4097), group(k=0), group(k=12), group(n=-8), group(n=20), group(t=F), group(t=5),
                               group(abi=0), group(E=4096, k=1 << 19), group(E=4096, n=1 << 19)])
def test_group_bad_config(c):
    refused(gforward, c)
    refused(gbackward, c)


def test_group_refusals():
    for k in (dict(x=None), dict(x=A + 8), dict(off=None), dict(off=A + 2), dict(w=None), dict(w=A + 2), dict(out=None), dict(out=A + 4),
              dict(rows=-1), dict(rows=(1 << 30) + 1), dict(t=H), dict(t=4), dict(mode=2), dict(mode=-1)):
        refused(gforward, **k)
    for k in (dict(dy=None), dict(dy=A + 8), dict(x=None), dict(off=None), dict(w=None), dict(dx=A + (4 << 20) + 8),
              dict(dw=A + (5 << 20) + 2), dict(rows=-1), dict(t=H), dict(acc=2), dict(rows=0, dw=A + 1)):
        refused(gbackward, **k)
    for at in (A, A + 5 * 64 * 2 - 16, A + (1 << 20) + 16, A + (2 << 20) + 4 * 64 * 32 * 2 - 16):
        refused(gforward, out=at, word="overlaps")
    for out in ("dx", "dw"):
        for at in (A, A + (2 << 20), A + (3 << 20) + 16):
            refused(gbackward, **{out: at}, word="overlaps")
    refused(gbackward, dw=A + (1 << 20), word="overlaps")
    refused(gbackward, dw=A + (4 << 20) + 16, word="overlaps")


def test_group_nothing_to_do():
    gforward(rows=0, x=None, w=None, out=None)
    gbackward(dx=None, dw=None, x=None, w=None)
    gbackward(rows=0, dy=None, x=None, w=None, dw=None)
    gbackward(rows=0, dy=None, x=None, w=None, acc=1)


# ---------------------------------------------------------------- orthogonalised updates

MUON = (3.4445, -4.7750, 2.0315)


def ortho(count=2, rows=32, cols=48, steps=5, abc=MUON, abi=B.ABI_VERSION):
    return B.waste_ortho_config(abi, count, rows, cols, steps, *abc)


def update(c=None, ws=Bytes(1 << 30, A + (1 << 32)), **k):
    a = dict(g=A, gt=F, out=A + (1 << 20), ot=BF, scale=1.0, mode=0)
    a.update(k)
    B.waste_ortho_update(c or ortho(), *a.values(), ws, stream=0)


@pytest.mark.parametrize("c", [ortho(count=-1), ortho(count=65536), ortho(rows=0), ortho(cols=-3), ortho(rows=40000, cols=40000),
                               ortho(count=60000, rows=30000, cols=2), ortho(steps=0), ortho(steps=33), ortho(abi=3),
                               ortho(abc=(9.0, 0.0, 0.0)), ortho(abc=(3.4445, 4.775, 2.0315)), ortho(abc=(float("nan"), 0.0, 0.0)),
                               ortho(abc=(2.0, 0.0, 0.0)), ortho(abc=(1.0, float("inf"), 1.0)), ortho(abc=(7.9, 0.0, 0.0), steps=2),
                               ortho(abc=(1.0, -9.0, 50.0))])
def test_ortho_bad_config(c):
    refused(B.waste_ortho_workspace, c)
    refused(update, c)


def test_ortho_refusals():
    for k in (dict(g=None), dict(g=A + 8), dict(out=None), dict(out=A + (1 << 20) + 4), dict(gt=3), dict(ot=F), dict(ot=H), dict(ot=9, mode=1),
              dict(mode=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=Bytes(1 << 10, A + (1 << 32))),
              dict(ws=Bytes(1 << 30, A + (1 << 32) + 16)), dict(ws=Bytes(1 << 30, None))):
        refused(update, **k)
    need = B.waste_ortho_workspace(ortho())
    for at in (A, A + 16, A - 16, A + 2 * 32 * 48 * 4 - 16):
        refused(update, out=at, word="overlaps")
    refused(update, ws=Bytes(need, A), word="overlaps")
    refused(update, ws=Bytes(need, A + (1 << 20) - need // 256 * 256 + 256), word="overlaps")
    update(ortho(count=0), g=None, out=None, ws=Bytes(0, None))


def test_ortho_accepts():
    """Coefficients in use: the quintic of the default, the cubic and the quintic that converge, one step, a row, a column."""
    for abc in (MUON, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5)):
        assert B.waste_ortho_workspace(ortho(abc=abc)) > 0
    for r, c in ((1, 1), (1, 9), (9, 1), (32768, 40000), (5, 1 << 29)):
        assert B.waste_ortho_workspace(ortho(count=1, rows=r, cols=c, steps=1)) >= 6 * r * c


@pytest.mark.parametrize("far", [(1 << 32) + 32, 1 << 31, -(1 << 32) + 32])
def test_sizes_past_32_bits(far):
    """Sizes that would be other, valid ones once cut to 32 bits."""
    refused(B.waste_norm_config, B.ABI_VERSION, far, F, F, F, 1e-5)
    refused(B.waste_group_config, B.ABI_VERSION, 4, far, 32, BF)
    refused(B.waste_ortho_config, B.ABI_VERSION, 1, far, 32, 5, *MUON)
    refused(lambda: B.waste_ortho_config(abi_version=B.ABI_VERSION, cols=far))
    refused(forward, T=far)
    refused(backward, T=far)
    refused(B.waste_norm_workspace, norm(), far)
    refused(gforward, rows=far)
    refused(gbackward, rows=far)


def test_ortho_ways():
    """Which way each of the GPU tests' stacks takes: its workspace's size tells.  Wide and tall, one matrix and several,
    both sizes of tiles, shares and all at once are among them."""
    for (count, rows, cols), (side, slices) in R.ORTHO_WAYS.items():
        assert B.waste_ortho_workspace(ortho(count, rows, cols)) == R.ortho_workspace(count, rows, cols, side, slices), (count, rows, cols)
    ways = {(rows > cols, count > 1, side, slices > 0) for (count, rows, cols), (side, slices) in R.ORTHO_WAYS.items()}
    assert {(tall, many, side, True) for tall in (False, True) for many in (False, True) for side in (128, 256)} <= ways
    assert {(tall, True, 256, False) for tall in (False, True)} <= ways


def test_debug_wait_refusals():
    for a in ((-1, 64, 0), (3, 64, 0), (0, -1, 0), (1, (1 << 18) + 1, 0), (2, 64, 2), (2, 64, -1)):
        refused(B.waste_train_debug_wait, *a, stream=0)
