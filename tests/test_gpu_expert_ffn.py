"""The experts' feed-forward block and its backward pass against the
definitions in 64 bits.

Tolerances.  A product of K terms summed in fp32 is off by at most K steps of
2^-24 of the sum of the terms' magnitudes (any order).  bf16 rows: a, dg and
du are rounded to bf16 (half a step, 2^-8 each) before the next product, so
that product is off by 2^-8 of its terms' magnitudes as well; the
activation adds a few fp32 roundings (64 counted, of act(g) u's terms).
Every output adds its own half step."""

import math

import pytest
import torch

from co_activation_amd import ops
from gpu_util import say
from layer_ref import HALF_STEP, U32, d

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib):
    assert torch.cuda.is_available()
    return built_lib


def _inputs(counts, H, F, dtype, seed=0, gap=3, order=None, wide=1.0):
    """Rows of len(counts) experts, `gap` rows of no expert between the
    blocks, which lie in the given order."""
    g = torch.Generator().manual_seed(seed)
    dt, E = DT[dtype], len(counts)
    first = [0] * E
    at = gap
    for e in order if order is not None else range(E):
        first[e] = at
        at += counts[e] + gap
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = {"x": (wide * rnd(at, H)).to(dt), "w_in": (rnd(E, 2 * F, H) / math.sqrt(H)).to(dt),
         "w_down": (rnd(E, H, F) / math.sqrt(F)).to(dt), "dy": rnd(at, H).to(dt),
         "first": torch.tensor(first, dtype=torch.int32),
         "count": torch.tensor(counts, dtype=torch.int32)}
    owned = torch.zeros(at, dtype=torch.bool)
    for f, c in zip(first, counts):
        owned[f:f + c] = True
    s["x"][~owned] = float("nan")   # rows of no expert are not read
    s["dy"][~owned] = float("nan")
    return s, owned


def _act(name, g):
    return g * torch.sigmoid(g) if name == "silu" else g * 0.5 * (1 + torch.erf(g / math.sqrt(2)))


def _slope(name, g):
    if name == "silu":
        p = torch.sigmoid(g)
        return p + g * p * (1 - p)
    return 0.5 * (1 + torch.erf(g / math.sqrt(2))) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def _bound(got, want, tol, name):
    bad = ~((d(got) - want).abs() <= HALF_STEP[got.dtype] * want.abs() * (1 + 2.0 ** -8) + tol + 1e-37)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()} out of tolerance, worst off by "
                                 f"{float((d(got) - want).abs().nan_to_num(1e9).max()):.3g}")


def _check_forward(s, got, act, save):
    step = HALF_STEP[s["x"].dtype]
    mid = step if s["x"].dtype == torch.bfloat16 else 0.0
    H, F = s["x"].shape[1], s["w_down"].shape[2]
    for e, (f, c) in enumerate(zip(s["first"].tolist(), s["count"].tolist())):
        if c == 0:
            continue
        x, wi, wd = d(s["x"][f:f + c]), d(s["w_in"][e]), d(s["w_down"][e])
        p, pa = x @ wi.t(), x.abs() @ wi.abs().t()
        g, u = p[:, :F], p[:, F:]
        err = H * U32 * pa  # of g and u
        a = _act(act, g) * u
        # |act'| <= 1.13 and |act(g)| <= |g|
        a_err = 1.13 * u.abs() * err[:, :F] + g.abs() * err[:, F:] + 64 * U32 * (g.abs() + 0.2) * u.abs()
        if save:
            _bound(got["gu"][f:f + c], p, err, "gu")
        _bound(got["a"][f:f + c], a, a_err, "a")
        y = a @ wd.t()
        y_err = (a_err + mid * a.abs()) @ wd.abs().t() + F * U32 * (a.abs() @ wd.abs().t())
        _bound(got["y"][f:f + c], y, y_err, "y")


def _check_backward(s, gu, a_saved, got, act):
    mid = 2.0 ** -8 if s["x"].dtype == torch.bfloat16 else 0.0
    H, F = s["x"].shape[1], s["w_down"].shape[2]
    for e, (f, c) in enumerate(zip(s["first"].tolist(), s["count"].tolist())):
        if c == 0:
            assert not bool(got["dw_in"][e].any()) and not bool(got["dw_down"][e].any())
            continue
        x, wi, wd = d(s["x"][f:f + c]), d(s["w_in"][e]), d(s["w_down"][e])
        dy, p, a = d(s["dy"][f:f + c]), d(gu[f:f + c]), d(a_saved[f:f + c])
        g, u = p[:, :F], p[:, F:]
        da, da_err = dy @ wd, H * U32 * (dy.abs() @ wd.abs())
        value, slope = _act(act, g), _slope(act, g)
        dgu = torch.cat((da * u * slope, da * value), 1)
        # fp32 roundings of the slope and value, whose terms are at most
        # 1 + |g| and |g|
        few = torch.cat((64 * U32 * da.abs() * u.abs() * (1 + g.abs()),
                         64 * U32 * da.abs() * (g.abs() + 0.2)), 1)
        dgu_err = torch.cat((da_err * (u * slope).abs(), da_err * value.abs()), 1) + few + mid * dgu.abs()
        _bound(got["dx"][f:f + c], dgu @ wi,
               dgu_err @ wi.abs() + 2 * F * U32 * (dgu.abs() @ wi.abs()), "dx")
        _bound(got["dw_in"][e], dgu.t() @ x,
               dgu_err.t() @ x.abs() + c * U32 * (dgu.abs().t() @ x.abs()), "dw_in")
        _bound(got["dw_down"][e], dy.t() @ a, c * U32 * (dy.abs().t() @ a.abs()), "dw_down")


def _run(s, owned, act, save=True, backward=True):
    c = {k: v.cuda() for k, v in s.items()}
    R, H, F = c["x"].shape[0], c["x"].shape[1], c["w_down"].shape[2]
    err = ops.new_error_word()
    out = {"y": (R, H), "a": (R, F), "gu": (R, 2 * F), "dx": (R, H)}
    out = {k: torch.full(v, 7.0, dtype=c["x"].dtype, device="cuda") for k, v in out.items()}
    got = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"], act=act, save=save,
                         out=out, d_err=err)
    _check_forward(s, got, act, save)
    names = ["y", "a"] + (["gu"] if save else [])
    if backward:
        grad = ops.expert_ffn_backward(c["dy"], c["x"], c["w_in"], c["w_down"], got["gu"], got["a"],
                                       c["first"], c["count"], act=act, out=out, d_err=err)
        _check_backward(s, got["gu"], got["a"], grad, act)
        names.append("dx")
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for k in names:
        assert bool((out[k].cpu()[~owned] == 7.0).all()), f"{k}: rows of no expert were written"
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,H,F,act", [
    ([1], 8, 8, "silu"),                        # the smallest call
    ([0, 3, 0, 17, 1], 72, 40, "gelu"),         # odd widths, empty experts, two tiles
    ([5, 0, 16, 15, 2, 1, 33, 0], 264, 136, "silu"),
    ([70, 1, 64, 129], 200, 328, "gelu"),       # K and N tails of every tile
    ([100, 300, 0, 150], 520, 264, "silu"),
    # (as few tiles as here are 128 x 64; test_gpu_expert_tiles.py has the wide ones)
    ([700, 513], 136, 392, "silu"),             # the widest row tiles
    ([257], 1024, 512, "gelu"),
    ([3100], 40, 24, "silu"),                   # the rows of a weight gradient in ranges
    ([2500, 0, 900], 96, 136, "gelu"),
])
def test_forward_and_backward(dtype, counts, H, F, act):
    say("expert_ffn", dtype, counts, H, F, act)
    s, owned = _inputs(counts, H, F, dtype, seed=sum(counts))
    _run(s, owned, act)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_experts_in_another_order(dtype):
    """256 experts, blocks in a shuffled order, from none to a few rows."""
    g = torch.Generator().manual_seed(2)
    counts = torch.randint(0, 6, (256,), generator=g).tolist()
    order = torch.randperm(256, generator=g).tolist()
    say("expert_ffn 256 experts", dtype)
    s, owned = _inputs(counts, 64, 32, dtype, seed=5, gap=0, order=order)
    _run(s, owned, "silu")


@pytest.mark.parametrize("counts", [[40, 200, 90], [130, 20, 400, 7]])
def test_every_row_tile(counts):
    """The tile a launch takes goes by the rows an expert has on average:
    uneven experts fill it badly and stay right."""
    # (all of these are few enough to be 128 x 64; test_gpu_expert_tiles.py has the others)
    for pad in (0, 1500):  # more rows of no expert: another tile
        s, owned = _inputs(counts, 96, 160, "bf16", seed=pad, gap=pad // len(counts))
        say("expert_ffn tiles", counts, pad)
        _run(s, owned, "silu")


def test_inference_writes_no_gu():
    s, owned = _inputs([9, 30], 128, 64, "bf16", seed=4)
    got = _run(s, owned, "silu", save=False, backward=False)
    assert got["gu"] is None


def test_large_gates_saturate():
    """Gates of several hundred: act is g or 0, and no exponential overflow
    reaches the result."""
    s, owned = _inputs([20, 40], 64, 64, "bf16", seed=6, wide=200.0)
    for act in ("silu", "gelu"):
        _run(s, owned, act)


def test_a_value_that_is_not_finite_stays_in_its_row():
    s, owned = _inputs([20, 40], 64, 64, "bf16", seed=7)
    c = {k: v.cuda() for k, v in s.items()}
    clean = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"])["y"]
    row = int(s["first"][1]) + 5
    c["x"][row, 3] = float("inf")
    got = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"])["y"]
    keep = owned.clone()
    keep[row] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
    assert bool(got[row].isnan().any())


def test_an_expert_whose_weights_are_nan_stays_alone():
    """Column tiles and k tails end inside an expert's weights: the next
    expert's are not touched."""
    s, owned = _inputs([20, 40, 9], 72, 40, "bf16", seed=8)
    c = {k: v.cuda() for k, v in s.items()}
    args = (c["x"], c["w_in"], c["w_down"], c["first"], c["count"])
    clean = ops.expert_ffn(*args)["y"].clone()
    c["w_in"][1], c["w_down"][1] = float("nan"), float("nan")
    got = ops.expert_ffn(*args)["y"].cpu()
    for e in (0, 2):
        f, n = int(s["first"][e]), int(s["count"][e])
        assert torch.equal(got[f:f + n], clean.cpu()[f:f + n])


@pytest.mark.parametrize("first,count", [([0, -1], [4, 4]), ([0, 30], [4, 4]), ([0, 4], [4, -2]),
                                         ([0, 4], [4, 1000]), ([0, 2 ** 31 - 1], [4, 2 ** 31 - 1])])
def test_rows_outside_the_buffer_are_reported(first, count):
    """Such an expert counts as without rows; the other one is computed."""
    s, _ = _inputs([4, 4], 64, 32, "bf16", seed=9, gap=0)
    s = {k: v.cuda() for k, v in s.items()}
    want = ops.expert_ffn(s["x"], s["w_in"], s["w_down"], s["first"], s["count"], save=True)
    grad = ops.expert_ffn_backward(s["dy"], s["x"], s["w_in"], s["w_down"], want["gu"], want["a"],
                                   s["first"], s["count"])
    bad = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (first, count)]
    err = ops.new_error_word()
    got = ops.expert_ffn(s["x"], s["w_in"], s["w_down"], *bad, d_err=err)
    assert ops.decode_errors(int(err.item())) == ["EXPERT_ROWS"]
    assert torch.equal(got["y"][:4], want["y"][:4])
    err.zero_()
    back = ops.expert_ffn_backward(s["dy"], s["x"], s["w_in"], s["w_down"], want["gu"], want["a"],
                                   *bad, d_err=err)
    assert ops.decode_errors(int(err.item())) == ["EXPERT_ROWS"]
    assert torch.equal(back["dx"][:4], grad["dx"][:4])
    assert torch.equal(back["dw_in"][0], grad["dw_in"][0]) and not bool(back["dw_in"][1].any())


def test_no_rows():
    s, _ = _inputs([0, 0], 64, 32, "bf16", gap=0)
    s = {k: v.cuda() for k, v in s.items()}
    got = ops.expert_ffn(s["x"], s["w_in"], s["w_down"], s["first"], s["count"], save=True)
    assert got["y"].shape == (0, 64)
    grad = ops.expert_ffn_backward(s["dy"], s["x"], s["w_in"], s["w_down"], got["gu"], got["a"],
                                   s["first"], s["count"])
    assert not bool(grad["dw_in"].any()) and not bool(grad["dw_down"].any())


def test_gradients_against_differences():
    """<y, dy> along random directions: central differences of the 64-bit
    definition against the engine's fp32 gradients."""
    s, _ = _inputs([6, 0, 11], 24, 20, "f32", seed=10, gap=0)
    c = {k: v.cuda() for k, v in s.items()}
    f = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"], act="gelu", save=True)
    grad = ops.expert_ffn_backward(c["dy"], c["x"], c["w_in"], c["w_down"], f["gu"], f["a"],
                                   c["first"], c["count"], act="gelu")
    base = {"x": d(s["x"]), "w_in": d(s["w_in"]), "w_down": d(s["w_down"])}

    def value(p):
        total = 0.0
        for e, (r, n) in enumerate(zip(s["first"].tolist(), s["count"].tolist())):
            z = p["x"][r:r + n] @ p["w_in"][e].t()
            y = (_act("gelu", z[:, :20]) * z[:, 20:]) @ p["w_down"][e].t()
            total += float((y * d(s["dy"][r:r + n])).sum())
        return total

    g = torch.Generator().manual_seed(3)
    for n, key in (("x", "dx"), ("w_in", "dw_in"), ("w_down", "dw_down")):
        step = torch.randn(base[n].shape, generator=g).double()
        e = 1e-5
        want = (value(dict(base, **{n: base[n] + e * step})) - value(dict(base, **{n: base[n] - e * step}))) / (2 * e)
        terms = d(grad[key]) * step
        # e^2 truncation, 2^-53 over e, and fp32 gradients
        assert abs(float(terms.sum()) - want) <= 1e-5 * float(terms.abs().sum() + 1), n


def test_runs_are_the_same_and_graphs_replay():
    """Bit-identical from run to run, and a captured forward and backward
    that follows its inputs, with eager work between the replays."""
    s, _ = _inputs([300, 20, 150], 256, 192, "bf16", seed=11, gap=0)
    c = {k: v.cuda() for k, v in s.items()}
    R = c["x"].shape[0]
    ws = torch.empty(ops.expert_ffn_workspace_bytes(R, 256, 192, 3, torch.bfloat16), dtype=torch.uint8, device="cuda")

    def both(out, w):
        f = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"], save=True, out=out)
        b = ops.expert_ffn_backward(c["dy"], c["x"], c["w_in"], c["w_down"], f["gu"], f["a"],
                                    c["first"], c["count"], out=out, ws=w)
        return {**f, **b}

    out = both(None, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(out, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(out, ws)
    for i in range(4):
        c["x"].copy_(torch.randn(c["x"].shape, generator=torch.Generator().manual_seed(i)))
        cut = [100 * i, 470 - 100 * i, 0]
        c["count"].copy_(torch.tensor(cut))
        c["first"].copy_(torch.tensor([0, cut[0], 470]))
        graph.replay()
        torch.cuda.synchronize()
        fresh = both(None, None)
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], fresh[k]), (i, k)


def test_bound_calls_and_another_stream():
    s, _ = _inputs([30, 20], 128, 64, "bf16", seed=12, gap=0)
    c = {k: v.cuda() for k, v in s.items()}
    args = (c["x"], c["w_in"], c["w_down"], c["first"], c["count"])
    r, fwd = ops.expert_ffn(*args, save=True, bind=True)
    ws = torch.empty(ops.expert_ffn_workspace_bytes(50, 128, 64, 2, torch.bfloat16), dtype=torch.uint8, device="cuda")
    q, bwd = ops.expert_ffn_backward(c["dy"], *args[:3], r["gu"], r["a"], *args[3:], ws=ws, bind=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    fwd(st.cuda_stream)
    bwd(st.cuda_stream)
    st.synchronize()
    want = ops.expert_ffn(*args, save=True)
    grad = ops.expert_ffn_backward(c["dy"], *args[:3], want["gu"], want["a"], *args[3:])
    for k in r:
        assert torch.equal(r[k], want[k]), k
    for k in q:
        assert torch.equal(q[k], grad[k]), k


def test_binding_refuses():
    s, _ = _inputs([4, 4], 64, 32, "bf16", gap=0)
    c = {k: v.cuda() for k, v in s.items()}
    f = lambda **kw: ops.expert_ffn(  # noqa: E731
        *[kw.pop(n, c[n]) for n in ("x", "w_in", "w_down", "first", "count")], **kw)
    with pytest.raises(TypeError):
        f(x=c["x"].half())
    with pytest.raises(TypeError):
        f(w_in=c["w_in"].float())
    with pytest.raises(TypeError):
        f(count=c["count"].long())
    with pytest.raises(ValueError, match="shape"):
        f(w_in=c["w_in"][:, :32].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        f(w_down=c["w_down"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="act"):
        f(act="relu")
    with pytest.raises(ops._lib.MoeError):
        f(out={"y": c["x"]})
    with pytest.raises(ValueError):
        ops.expert_ffn_backward(c["dy"], c["x"], c["w_in"], c["w_down"], c["x"], c["x"], c["first"],
                                c["count"])
    odd = torch.zeros(8, 60, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ops._lib.MoeError):
        ops.expert_ffn(odd, torch.zeros(2, 64, 60, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(2, 60, 32, dtype=torch.bfloat16, device="cuda"), c["first"], c["count"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_expert_has_rows(dtype):
    """A buffer with room for rows and none in it: nothing is read, the
    weight gradients are zero, the rows' outputs stay."""
    say("expert_ffn all empty", dtype)
    s, owned = _inputs([0, 0, 0], 64, 48, dtype, gap=40)
    assert not bool(owned.any())
    c = {k: v.cuda() for k, v in s.items()}
    R = c["x"].shape[0]
    keep = {"y": torch.full((R, 64), 5.0, dtype=DT[dtype], device="cuda")}
    got = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"], save=True, out=keep)
    dx = torch.full_like(keep["y"], 6.0)
    grad = ops.expert_ffn_backward(c["dy"], c["x"], c["w_in"], c["w_down"], got["gu"], got["a"],
                                   c["first"], c["count"], out={"dx": dx})
    torch.cuda.synchronize()
    assert bool((keep["y"] == 5.0).all()) and bool((dx == 6.0).all())
    assert not bool(grad["dw_in"].any()) and not bool(grad["dw_down"].any())


@pytest.mark.parametrize("E", [1, 2])
def test_rows_past_32_bit_offsets(E):
    """The rows of the last expert lie more than 4 GiB into the buffers."""
    R, H, F, n = 600_000, 4096, 64, 300
    say("expert_ffn far rows", E)
    s, _ = _inputs([n], H, F, "bf16", gap=0)
    first = torch.tensor([0] * (E - 1) + [R - n], dtype=torch.int32, device="cuda")
    count = torch.tensor([0] * (E - 1) + [n], dtype=torch.int32, device="cuda")
    big = {k: torch.empty(R, H, dtype=torch.bfloat16, device="cuda") for k in ("x", "dy", "y", "dx")}
    big["x"][R - n:] = s["x"].cuda()
    big["dy"][R - n:] = s["dy"].cuda()
    w_in = s["w_in"].cuda().repeat(E, 1, 1)
    w_down = s["w_down"].cuda().repeat(E, 1, 1)
    got = ops.expert_ffn(big["x"], w_in, w_down, first, count, save=True, out={"y": big["y"]})
    grad = ops.expert_ffn_backward(big["dy"], big["x"], w_in, w_down, got["gu"], got["a"], first, count,
                                   out={"dx": big["dx"]})
    torch.cuda.synchronize()
    _check_forward(s, {k: got[k][R - n:].cpu() for k in ("gu", "a", "y")}, "silu", True)
    _check_backward(s, got["gu"][R - n:].cpu(), got["a"][R - n:].cpu(),
                    {"dx": grad["dx"][R - n:].cpu(), "dw_in": grad["dw_in"][E - 1:].cpu(),
                     "dw_down": grad["dw_down"][E - 1:].cpu()}, "silu")


@pytest.mark.parametrize("counts,H,F", [([700, 30, 0, 900], 64, 40), ([3000], 136, 72),
                                        ([520, 0, 511, 1], 512, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_in_ranges_and_products_in_one_launch(counts, H, F, dtype):
    """Few tiles: each expert's rows in several ranges, both weight gradients
    (fp32: dx too) in one launch; what lies behind the workspace stays."""
    say("expert_ffn ranges", counts, H, F, dtype)
    s, owned = _inputs(counts, H, F, dtype, seed=H)
    c = {k: v.cuda() for k, v in s.items()}
    R, E = c["x"].shape[0], len(counts)
    need = ops.expert_ffn_workspace_bytes(R, H, F, E, DT[dtype])
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    f = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"], save=True)
    grad = ops.expert_ffn_backward(c["dy"], c["x"], c["w_in"], c["w_down"], f["gu"], f["a"], c["first"],
                                   c["count"], ws=ws)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xA5).all())
    gu, a = f["gu"].cpu(), f["a"].cpu()
    _check_backward(s, gu, a, {k: v.cpu() for k, v in grad.items()}, "silu")


def test_a_bound_backward_needs_its_workspace():
    s, _ = _inputs([5], 64, 48, "bf16")
    c = {k: v.cuda() for k, v in s.items()}
    f = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"], save=True)
    with pytest.raises(ValueError, match="workspace"):
        ops.expert_ffn_backward(c["dy"], c["x"], c["w_in"], c["w_down"], f["gu"], f["a"], c["first"],
                                c["count"], bind=True)


@pytest.mark.parametrize("E,H,F", [(254, 64, 40), (256, 272, 24), (33, 264, 1032)])
def test_weight_tiles_dealt_out(E, H, F):
    """Enough tiles that panels of them are dealt out one by one, the last
    panel short; every tile is written."""
    say("expert_ffn dealt", E, H, F)
    counts = [(7 * e) % 23 for e in range(E)]
    s, owned = _inputs(counts, H, F, "bf16", seed=E)
    c = {k: v.cuda() for k, v in s.items()}
    f = ops.expert_ffn(c["x"], c["w_in"], c["w_down"], c["first"], c["count"], save=True)
    out = {"dw_in": torch.full_like(c["w_in"], float("nan")),
           "dw_down": torch.full_like(c["w_down"], float("nan"))}
    grad = ops.expert_ffn_backward(c["dy"], c["x"], c["w_in"], c["w_down"], f["gu"], f["a"], c["first"],
                                   c["count"], out=out)
    torch.cuda.synchronize()
    _check_backward(s, f["gu"].cpu(), f["a"].cpu(), {k: v.cpu() for k, v in grad.items()}, "silu")


@pytest.mark.parametrize("rows", [1, 9, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gelu_keeps_its_digits_in_the_tail(dtype, rows):
    """The gates themselves as weights and a row of 1, 0, 0, ...: a is act(g)
    and the first column of dw_in act'(g), each within a relative tolerance.
    The exponential of -g^2 / 2 is off by the rounding of its argument, of the
    argument in base 2 and of that base's constant, g^2 / 2 half steps each, and
    its own; with the rest of the formula's roundings (64 counted) that is (2
    g^2 + 64) half steps of Phi(g) and of |g| times the density."""
    say("expert_ffn gelu tail", dtype, rows)
    H, F = 8, 256
    g = torch.cat((torch.linspace(-12, 4, F - 6), torch.tensor([0.0, -0.0, -1e-6, 1e-6, 40.0, 300.0])))
    g = g.to(DT[dtype])
    w_in = torch.zeros(1, 2 * F, H, dtype=DT[dtype])
    w_in[0, :F, 0], w_in[0, F:, 0] = g, 1.0
    w_down = torch.zeros(1, H, F, dtype=DT[dtype])
    w_down[0, 0] = 1.0
    x, dy = (torch.zeros(rows, H, dtype=DT[dtype]) for _ in range(2))
    x[:, 0], dy[0, 0] = 1.0, 1.0
    x, dy, w_in, w_down = (t.cuda() for t in (x, dy, w_in, w_down))
    first, count = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, rows))
    f = ops.expert_ffn(x, w_in, w_down, first, count, act="gelu", save=True)
    b = ops.expert_ffn_backward(dy, x, w_in, w_down, f["gu"], f["a"], first, count, act="gelu")
    torch.cuda.synchronize()
    gd = g.double()
    phi = 0.5 * torch.special.erfc(-gd / math.sqrt(2))
    dens = torch.exp(-gd * gd / 2) / math.sqrt(2 * math.pi)
    few = (2 * gd * gd + 64) * U32
    for r in (0, rows - 1):
        _bound(f["a"][r], gd * phi, few * gd.abs() * phi, "a")
    value, slope = b["dw_in"][0, F:, 0], b["dw_in"][0, :F, 0]
    again = HALF_STEP[DT[dtype]]  # [dg | du] lies in the workspace in the rows' type
    _bound(value, gd * phi, (few + again) * gd.abs() * phi, "act")
    _bound(slope, phi + gd * dens, few * (phi + gd.abs() * dens) + again * (phi + gd * dens).abs(), "slope")
