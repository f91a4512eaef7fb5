"""The feed-forward block's bf16 kernels where their loops go on: blocks that
take a second and third tile, with K longer than the ring of stages, and the
few-rows kernel with its second row tile, its matrix form and several column
tiles a block.  Sizes are large enough that the 64-bit definition is computed
on the device.

Tolerances are those of test_gpu_expert_ffn.py: K steps of 2^-24 of the
terms' magnitudes for a product of K terms, 2^-8 for each value rounded to
bf16 before the next product, 64 fp32 roundings for the activation, and half
a step of the output."""

import math

import pytest
import torch

from co_activation_amd import ops
from gpu_util import say
from layer_ref import HALF_STEP, U32

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8
CUS = 256


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib):
    assert torch.cuda.is_available()
    return built_lib


def _up(a, b):
    return -(-a // b)


def _row_tiles(counts, R, cols):
    """The tile that a product over the rows takes (its rule restated), and
    how many of them there are."""
    E = len(counts)
    most = lambda bm: R // bm + min(R, E)  # noqa: E731
    if R >= 512 * E and R // 256 * _up(cols, 256) >= CUS // 2:
        bm, bn = 256, 256
    elif most(128) * _up(cols, 256) >= CUS // 2:
        bm, bn = 128, 256
    else:
        bm, bn = 128, 64
    return (bm, bn), sum(_up(c, bm) for c in counts) * _up(cols, bn)


def _inputs(counts, H, F, seed, gap=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, R = len(counts), sum(counts) + gap
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    first = (count.cumsum(0) - count).int()
    s = {"x": rnd(R, H).bfloat16(), "dy": rnd(R, H).bfloat16(),
         "w_in": (rnd(E, 2 * F, H) / math.sqrt(H)).bfloat16(),
         "w_down": (rnd(E, H, F) / math.sqrt(F)).bfloat16(), "first": first, "count": count}
    s["x"][R - gap:], s["dy"][R - gap:] = float("nan"), float("nan")  # rows of no expert
    return s


def _bound(got, want, tol, name):
    off = (got.double() - want).abs()
    bad = ~(off <= HALF_STEP[got.dtype] * want.abs() * (1 + BF16) + tol + 1e-37)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()} out of tolerance, worst off by "
                                 f"{float(off.nan_to_num(1e9).max()):.3g}")


def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    p = 0.5 * torch.special.erfc(-g / math.sqrt(2))
    return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def _check(s, counts, act, f, b=None):
    H, F = s["x"].shape[1], s["w_down"].shape[2]
    lo = 0
    for e, c in enumerate(counts):
        rows, lo = slice(lo, lo + c), lo + c
        if c == 0:
            if b is not None:
                assert not bool(b["dw_in"][e].any()) and not bool(b["dw_down"][e].any()), e
            continue
        x, wi, wd = s["x"][rows].double(), s["w_in"][e].double(), s["w_down"][e].double()
        p, err = x @ wi.t(), H * U32 * (x.abs() @ wi.abs().t())
        g, u = p[:, :F], p[:, F:]
        if f["gu"] is not None:
            _bound(f["gu"][rows], p, err, f"gu of {e}")
        a = _act(act, g)[0] * u
        a_err = 1.13 * u.abs() * err[:, :F] + g.abs() * err[:, F:] + 64 * U32 * (g.abs() + 0.2) * u.abs()
        _bound(f["a"][rows], a, a_err, f"a of {e}")
        y_err = (a_err + BF16 * a.abs()) @ wd.abs().t() + F * U32 * (a.abs() @ wd.abs().t())
        _bound(f["y"][rows], a @ wd.t(), y_err, f"y of {e}")
        if b is None:
            continue
        dy, p, a = s["dy"][rows].double(), f["gu"][rows].double(), f["a"][rows].double()
        g, u = p[:, :F], p[:, F:]
        value, slope = _act(act, g)
        da, da_err = dy @ wd, H * U32 * (dy.abs() @ wd.abs())
        dgu = torch.cat((da * u * slope, da * value), 1)
        few = torch.cat((64 * U32 * da.abs() * u.abs() * (1 + g.abs()),
                         64 * U32 * da.abs() * (g.abs() + 0.2)), 1)
        dgu_err = torch.cat((da_err * (u * slope).abs(), da_err * value.abs()), 1) + few + BF16 * dgu.abs()
        _bound(b["dx"][rows], dgu @ wi, dgu_err @ wi.abs() + 2 * F * U32 * (dgu.abs() @ wi.abs()), f"dx of {e}")
        _bound(b["dw_in"][e], dgu.t() @ x, dgu_err.t() @ x.abs() + c * U32 * (dgu.abs().t() @ x.abs()),
               f"dw_in of {e}")
        _bound(b["dw_down"][e], dy.t() @ a, c * U32 * (dy.abs().t() @ a.abs()), f"dw_down of {e}")


def _forward(s, act, save=True):
    R, H, F = s["x"].shape[0], s["x"].shape[1], s["w_down"].shape[2]
    out = {"y": (R, H), "a": (R, F), "gu": (R, 2 * F)}
    out = {k: torch.full(v, 7.0, dtype=torch.bfloat16, device="cuda") for k, v in out.items()}
    err = ops.new_error_word()
    f = ops.expert_ffn(s["x"], s["w_in"], s["w_down"], s["first"], s["count"], act=act, save=save, out=out,
                       d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return f


def _backward(s, act, f):
    out = {"dw_in": torch.full_like(s["w_in"], float("nan")),
           "dw_down": torch.full_like(s["w_down"], float("nan")), "dx": torch.full_like(s["x"], 7.0)}
    b = ops.expert_ffn_backward(s["dy"], s["x"], s["w_in"], s["w_down"], f["gu"], f["a"], s["first"],
                                s["count"], act=act, out=out)
    torch.cuda.synchronize()
    return b


@pytest.mark.parametrize("counts,H,F,act,tile,most", [
    # 256 x 256: up and its gradient take two and three tiles a block
    ([4000, 3200, 0, 3700], 328, 1928, "silu", (256, 256), {"up": 2, "act": 1}),
    # 256 x 256: down and dx
    ([4000, 0, 3200, 3700], 4104, 200, "gelu", (256, 256), {"down": 2, "dx": 2}),
    # 128 x 256: up and its gradient; a short second tile in most experts
    ([200 + 13 * (e % 9) - 160 * (e % 5 == 0) for e in range(32)], 520, 1032, "silu", (128, 256),
     {"up": 2, "act": 1}),
    # 128 x 256: down and dx
    ([200 + 13 * (e % 9) - 160 * (e % 5 == 0) for e in range(32)], 2056, 392, "gelu", (128, 256),
     {"down": 2, "dx": 2}),
])
def test_blocks_take_several_row_tiles(counts, H, F, act, tile, most):
    say("expert_ffn row tiles", counts[:4], H, F, act)
    cols = {"up": 2 * F, "down": H, "act": F, "dx": H}
    for product, turns in most.items():  # every block has that many tiles, some have one more
        chosen, n = _row_tiles(counts, sum(counts), cols[product])
        assert chosen == tile and n > turns * CUS, (product, chosen, n)
    s = _inputs(counts, H, F, seed=H + F)
    f = _forward(s, act)
    _check(s, counts, act, f, _backward(s, act, f))


def test_blocks_take_several_weight_tiles_in_ranges():
    """Too few panels to be dealt out: an XCD has a range of tiles, and its
    blocks a second one, with and without rows."""
    counts = [0 if e % 4 == 1 else 150 + 7 * e for e in range(40)]
    H, F = 520, 264
    say("expert_ffn weight tiles", len(counts), H, F)
    tiles = len(counts) * _up(2 * F, 256) * _up(H, 256)
    assert CUS < tiles and _up(len(counts) * _up(2 * F, 256), 4) < 64
    s = _inputs(counts, H, F, seed=1)
    f = _forward(s, "silu")
    _check(s, counts, "silu", f, _backward(s, "silu", f))


def test_blocks_take_several_weight_tiles_dealt_out():
    """Four and five tiles a block, of 0 to 19 steps, in any order."""
    g = torch.Generator().manual_seed(3)
    counts = [(c > 180) * (c - 50) for c in torch.randint(0, 640, (128,), generator=g).tolist()]
    H, F = 520, 264
    say("expert_ffn weight tiles dealt", len(counts), H, F)
    assert 20 < sum(c == 0 for c in counts) < 60
    tiles = len(counts) * _up(2 * F, 256) * _up(H, 256)
    assert 4 * CUS < tiles and _up(len(counts) * _up(2 * F, 256), 4) >= 64
    s = _inputs(counts, H, F, seed=2)
    f = _forward(s, "gelu")
    _check(s, counts, "gelu", f, _backward(s, "gelu", f))


def _few(E, at):
    counts = [0] * E
    for e, c in at.items():
        counts[e] = c
    return counts


FEW = [
    _few(1, {0: 1}),
    _few(64, {3: 33, 10: 17, 20: 1, 63: 5}),       # up to three row tiles of an expert
    _few(64, {0: 4, 5: 5, 7: 16, 9: 2, 40: 31}),
    _few(256, {0: 33, 1: 17, 2: 16, 50: 5, 51: 4, 130: 1, 200: 48, 255: 20}),
]


@pytest.mark.parametrize("H,F", [(1032, 520), (264, 1032), (520, 136), (72, 24)])
@pytest.mark.parametrize("counts", FEW, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("act,save", [("silu", True), ("gelu", False)])
def test_few_rows(counts, H, F, act, save):
    """No more rows than experts: dot products up to four rows, the matrix
    form above; with 256 experts a block has several column tiles."""
    say("expert_ffn few rows", len(counts), sum(counts), H, F, act, save)
    gap = len(counts) - sum(counts)
    assert gap >= 0
    s = _inputs(counts, H, F, seed=H, gap=gap)
    f = _forward(s, act, save)
    assert (f["gu"] is not None) == save
    _check(s, counts, act, f)
    n = sum(counts)
    for k, v in f.items():
        assert v is None or bool((v[n:] == 7.0).all()), f"{k}: rows of no expert were written"


def test_few_rows_of_a_wide_layer():
    """Column tiles of many K batches, and a last batch that ends inside."""
    counts = _few(64, {1: 3, 8: 12, 30: 20, 31: 1, 60: 4})
    say("expert_ffn few rows wide")
    s = _inputs(counts, 4104, 2008, seed=9, gap=24)
    _check(s, counts, "silu", _forward(s, "silu"))
