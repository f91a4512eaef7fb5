"""The closing combine and its backward pass against the definitions in 64
bits, at the sizes, masks and options where they can go wrong.

Tolerances: half a step of the output's type, plus fp32 roundings counted
against the size of the terms a result is summed from.  Forward: k products
of b, at most 32 sequential and 6 + 8 tree additions for a mean, its square
root (2) and the final products (4): below 64.  Backward: the same for the
second norm's statistic, then for D, b, the two sums and the products that
follow, each at most 64: 256; a weight gradient adds at most T tokens in
sequence per block and 16 + blocks / 16 partial sums."""

import math
from fractions import Fraction

import pytest
import torch

from co_activation_amd import ops
from gpu_util import say
from layer_ref import close_grad_ref, close_ref, close_to, d

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib):
    assert torch.cuda.is_available()
    return built_lib


def _inputs(T, H, k, dtype, seed=0, weighted=True, gated=True, drop=0.3, spare=3):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = {"x": rnd(T, H).to(dt), "w_post": 1 + 0.2 * rnd(H), "w_next": 1 + 0.2 * rnd(H),
         "dy": rnd(T, H).to(dt), "dh": rnd(T, H).to(dt)}
    s["gate"] = torch.rand(T, generator=g) if gated else None
    n = T * k + spare
    s["z"] = rnd(n, H).to(dt)
    rows = torch.randperm(n, generator=g)[:T * k].reshape(T, k).to(torch.int32)
    rows[torch.rand(T, k, generator=g) < drop] = -1
    if T > 2:
        rows[T // 2] = -1          # a token without rows
        rows[T // 3, 1:] = -1      # a token with at most one
    s["rows"] = rows
    s["row_weight"] = torch.rand(n, generator=g) + 0.1 if weighted else None
    return s


def _gpu(s):
    return {k: None if v is None else v.cuda() for k, v in s.items()}


def _check_forward(s, got, scale, eps, opens=True):
    ref = close_ref(d(s["z"]), s["rows"], d(s["row_weight"]), d(s["x"]), d(s["w_post"]),
                    d(s["w_next"]) if opens else None, d(s["gate"]), scale, eps)
    close_to(got["y"], ref["y"], ref["y_size"], 64, "y")
    if opens:
        close_to(got["h"], ref["h"], ref["h_size"], 128, "h")
    return ref


def _check_backward(s, y, got, scale, eps, with_dy=True, with_dh=True):
    ref = close_grad_ref(d(s["dy"]) if with_dy else None, d(s["dh"]) if with_dh else None,
                         d(s["z"]), s["rows"], d(s["row_weight"]), d(y), d(s["w_post"]),
                         d(s["w_next"]), d(s["gate"]), scale, eps)
    T = s["x"].shape[0]
    close_to(got["dx"], ref["dx"], ref["dx_size"], 128, "dx")
    if with_dh:
        close_to(got["dw_next"], ref["dw_next"], ref["dw_next_size"], 256 + T, "dw_next")
    if s["rows"] is None:
        return
    listed = torch.zeros(s["z"].shape[0], dtype=torch.bool)
    listed[s["rows"][s["rows"] >= 0].long()] = True
    close_to(got["dz"].cpu()[listed], ref["dz"][listed], ref["dz_size"][listed], 256, "dz")
    close_to(got["dw_post"], ref["dw_post"], ref["dw_post_size"], 256 + T, "dw_post")
    if s["gate"] is not None:
        close_to(got["d_gate"], ref["d_gate"], ref["d_gate_size"], 256, "d_gate")
    if s["row_weight"] is not None:
        close_to(got["d_row_weight"].cpu()[listed], ref["d_row_weight"][listed],
                 ref["d_row_weight_size"][listed], 256, "d_row_weight")


def _run(s, scale=0.75, eps=1e-6, with_dy=True, with_dh=True):
    c = _gpu(s)
    err = ops.new_error_word()
    got = ops.combine_norm(c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"], c["w_next"],
                           gate=c["gate"], residual_scale=scale, eps=eps, d_err=err)
    grad = ops.combine_norm_backward(
        c["dy"] if with_dy else None, c["dh"] if with_dh else None, c["z"], c["rows"],
        c["row_weight"], got["y"], c["w_post"], c["w_next"], gate=c["gate"], residual_scale=scale,
        eps=eps, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return got, grad


@pytest.mark.parametrize("T,H,k,dtype", [
    (1, 8, 1, "bf16"), (1, 4, 1, "f32"), (5, 136, 3, "bf16"), (7, 132, 8, "f32"),
    (130, 512, 2, "bf16"), (33, 1024, 6, "bf16"), (33, 1032, 6, "bf16"), (9, 512, 4, "f32"),
    (9, 516, 5, "f32"), (40, 2048, 2, "bf16"), (6, 4096, 8, "bf16"), (5, 7168, 8, "bf16"),
    (3, 8192, 3, "bf16"), (3, 8200, 8, "bf16"), (2, 16384, 8, "bf16"), (3, 4100, 7, "f32"),
    (2, 8192, 2, "f32"), (800, 5120, 5, "bf16"),
])
def test_forward_and_backward(T, H, k, dtype):
    say("combine_norm", T, H, k, dtype)
    s = _inputs(T, H, k, dtype, seed=T + H)
    got, grad = _run(s)
    _check_forward(s, got, 0.75, 1e-6)
    _check_backward(s, got["y"], grad, 0.75, 1e-6)


@pytest.mark.parametrize("weighted,gated", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("H", [256, 4096])
def test_options(weighted, gated, H):
    s = _inputs(21, H, 4, "bf16", seed=3, weighted=weighted, gated=gated)
    say("combine_norm options", weighted, gated, H)
    got, grad = _run(s, scale=1.0)
    assert (grad["d_gate"] is None) == (not gated)
    assert (grad["d_row_weight"] is None) == (not weighted)
    _check_forward(s, got, 1.0, 1e-6)
    _check_backward(s, got["y"], grad, 1.0, 1e-6)


@pytest.mark.parametrize("with_dy,with_dh", [(True, False), (False, True)])
@pytest.mark.parametrize("H", [256, 4096])
def test_one_gradient_only(with_dy, with_dh, H):
    s = _inputs(2100, H, 2, "bf16", seed=4) if H == 256 else _inputs(40, H, 2, "bf16", seed=4)
    say("combine_norm one gradient", with_dy, with_dh, H)
    got, grad = _run(s, with_dy=with_dy, with_dh=with_dh)
    _check_backward(s, got["y"], grad, 0.75, 1e-6, with_dy, with_dh)


@pytest.mark.parametrize("T,H,dtype", [(1, 128, "f32"), (700, 256, "bf16"), (9000, 4096, "bf16"),
                                       (5, 7168, "bf16")])
def test_no_block(T, H, dtype):
    """rows = None: the norm that opens a layer, and a scaled residual."""
    s = _inputs(T, H, 1, dtype, seed=9, weighted=False, gated=False, spare=0)
    s["z"] = s["rows"] = s["w_post"] = None
    say("combine_norm without a block", T, H, dtype)
    got, grad = _run(s)
    x = d(s["x"])
    y = 0.75 * x
    close_to(got["y"], y, y.abs(), 4, "y")
    sigma = 1.0 / (y.pow(2).mean(1, keepdim=True) + 1e-6).sqrt()
    h = y * sigma * d(s["w_next"])
    close_to(got["h"], h, h.abs(), 128, "h")
    assert grad["dz"] is None and grad["dw_post"] is None
    _check_backward(s, got["y"], grad, 0.75, 1e-6)


@pytest.mark.parametrize("H", [64, 2048])
def test_many_tokens_a_block(H):
    """More tokens than the launch has blocks: each block walks several."""
    s = _inputs(4500, H, 2, "f32", seed=11)
    say("combine_norm many tokens", H)
    got, grad = _run(s)
    _check_forward(s, got, 0.75, 1e-6)
    _check_backward(s, got["y"], grad, 0.75, 1e-6)


def test_only_one_output():
    s = _gpu(_inputs(50, 512, 3, "bf16", seed=1))
    both = ops.combine_norm(s["z"], s["rows"], s["row_weight"], s["x"], s["w_post"], s["w_next"])
    y = ops.combine_norm(s["z"], s["rows"], s["row_weight"], s["x"], s["w_post"])
    h = ops.combine_norm(s["z"], s["rows"], s["row_weight"], s["x"], s["w_post"], s["w_next"],
                         with_y=False)
    assert y["h"] is None and h["y"] is None
    assert torch.equal(y["y"], both["y"]) and torch.equal(h["h"], both["h"])


@pytest.mark.parametrize("H", [256, 4096])
def test_n_valid_leaves_the_rest(H):
    """Tokens from n_valid on: not read, not written, nothing added."""
    s = _inputs(24, H, 2, "bf16", seed=6)
    c = _gpu(s)
    n = torch.tensor([17], dtype=torch.int32, device="cuda")
    c["x"][17:], c["dy"][17:], c["dh"][17:] = float("nan"), float("nan"), float("nan")
    out = {k: torch.full((24, H), 7.0, dtype=torch.bfloat16, device="cuda") for k in ("y", "h", "dx")}
    out["dz"] = torch.full_like(c["z"], 7.0)
    out["d_gate"] = torch.full((24,), 7.0, device="cuda")
    out["d_row_weight"] = torch.full((c["z"].shape[0],), 7.0, device="cuda")
    got = ops.combine_norm(c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"], c["w_next"],
                           gate=c["gate"], out=out, n_valid=n)
    grad = ops.combine_norm_backward(c["dy"], c["dh"], c["z"], c["rows"], c["row_weight"], got["y"],
                                     c["w_post"], c["w_next"], gate=c["gate"], out=out, n_valid=n)
    torch.cuda.synchronize()
    cut = {k: v if v is None or k in ("w_post", "w_next", "z", "row_weight") else v[:17]
           for k, v in s.items()}
    _check_forward(cut, {"y": got["y"][:17], "h": got["h"][:17]}, 1.0, 1e-6)
    part = dict(grad, dx=grad["dx"][:17], d_gate=grad["d_gate"][:17])
    _check_backward(cut, got["y"][:17], part, 1.0, 1e-6)
    for k in ("y", "h", "dx", "d_gate"):
        assert bool((out[k][17:] == 7.0).all()), k
    untouched = torch.ones(c["z"].shape[0], dtype=torch.bool)
    untouched[cut["rows"][cut["rows"] >= 0].long()] = False
    assert bool((out["dz"].cpu()[untouched] == 7.0).all())
    assert bool((out["d_row_weight"].cpu()[untouched] == 7.0).all())


def test_a_row_listed_twice_by_its_token():
    s = _inputs(6, 640, 3, "f32", seed=8, drop=0.0)
    s["rows"][0, 1] = s["rows"][0, 0]
    s["rows"][4, 2] = s["rows"][4, 0]
    got, grad = _run(s)
    _check_forward(s, got, 0.75, 1e-6)
    _check_backward(s, got["y"], grad, 0.75, 1e-6)


def test_a_bad_row_is_skipped_and_reported():
    s = _inputs(6, 256, 2, "bf16", seed=8, drop=0.0)
    want = dict(s, rows=s["rows"].clone())
    want["rows"][1, 0] = -1
    s["rows"][1, 0] = s["z"].shape[0] + 5
    c = _gpu(s)
    err = ops.new_error_word()
    got = ops.combine_norm(c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"], c["w_next"],
                           gate=c["gate"], d_err=err)
    assert ops.decode_errors(int(err.item())) == ["ROW_RANGE"]
    _check_forward(want, got, 1.0, 1e-6)
    err.zero_()
    grad = ops.combine_norm_backward(c["dy"], c["dh"], c["z"], c["rows"], c["row_weight"], got["y"],
                                     c["w_post"], c["w_next"], gate=c["gate"], d_err=err)
    assert ops.decode_errors(int(err.item())) == ["ROW_RANGE"]
    _check_backward(want, got["y"], grad, 1.0, 1e-6)


def test_values_that_are_not_finite_stay_in_their_token():
    """A NaN or an infinity in an unlisted row is never read; in a listed
    row it reaches its own token only."""
    s = _inputs(9, 512, 2, "bf16", seed=12, drop=0.0)
    used = set(s["rows"].flatten().tolist())
    free = [r for r in range(s["z"].shape[0]) if r not in used]
    s["z"][free] = float("nan")
    clean, _ = _run(s)
    _check_forward(s, clean, 0.75, 1e-6)
    s["z"][int(s["rows"][7, 0])] = float("inf")
    got, grad = _run(s)
    keep = [t for t in range(9) if t != 7]
    assert torch.equal(got["y"][keep], clean["y"][keep])
    assert bool(got["y"][7].isnan().any())
    assert bool(grad["dx"][keep].isfinite().all())


def test_runs_are_the_same_bit_for_bit():
    s = _inputs(3000, 1024, 3, "bf16", seed=13)
    _, a = _run(s)
    _, b = _run(s)
    listed = torch.zeros(s["z"].shape[0], dtype=torch.bool)
    listed[s["rows"][s["rows"] >= 0].long()] = True
    for k in a:
        x, y = (a[k].cpu()[listed], b[k].cpu()[listed]) if k in ("dz", "d_row_weight") else (a[k], b[k])
        assert torch.equal(x, y), k


def test_no_tokens():
    s = _gpu(_inputs(0, 256, 2, "bf16", seed=1, spare=4))
    got = ops.combine_norm(s["z"], s["rows"], s["row_weight"], s["x"], s["w_post"], s["w_next"])
    assert got["y"].shape == (0, 256)
    grad = ops.combine_norm_backward(s["dy"], s["dh"], s["z"], s["rows"], s["row_weight"], got["y"],
                                     s["w_post"], s["w_next"])
    assert bool((grad["dw_post"] == 0).all()) and bool((grad["dw_next"] == 0).all())


def test_gradients_against_differences():
    """A directional derivative of <y, dy> + <h, dh> by central differences
    of the 64-bit definition, against the engine's fp32 gradients."""
    T, H, k, scale, eps = 5, 64, 3, 0.5, 1e-3
    s = _inputs(T, H, k, "f32", seed=20, drop=0.0)
    got, grad = _run(s, scale=scale, eps=eps)
    names = {"z": "dz", "row_weight": "d_row_weight", "x": "dx", "w_post": "dw_post",
             "w_next": "dw_next", "gate": "d_gate"}
    base = {n: d(s[n]) for n in names}

    def value(p):
        r = close_ref(p["z"], s["rows"], p["row_weight"], p["x"], p["w_post"], p["w_next"],
                      p["gate"], scale, eps)
        return float((r["y"] * d(s["dy"])).sum() + (r["h"] * d(s["dh"])).sum())

    g = torch.Generator().manual_seed(1)
    for n, key in names.items():
        listed = torch.ones(base[n].shape[0], dtype=torch.bool)
        if n in ("z", "row_weight"):
            listed[:] = False
            listed[s["rows"][s["rows"] >= 0].long()] = True
        step = torch.randn(base[n].shape, generator=g).double()
        step[~listed] = 0
        e = 1e-5
        up = value(dict(base, **{n: base[n] + e * step}))
        down = value(dict(base, **{n: base[n] - e * step}))
        want = (up - down) / (2 * e)
        gv = d(grad[key])
        gv[~listed] = 0
        have = float((gv * step).sum())
        # e^2 truncation, 2^-53 cancellation over e, and fp32 gradients
        assert abs(have - want) <= 1e-5 * float((gv * step).abs().sum() + 1), (n, have, want)


def test_captured_and_replayed():
    """One graph with both directions; every replay against the eager run on
    the inputs of the moment, with eager work between."""
    c = _gpu(_inputs(300, 1024, 2, "bf16", seed=15))
    ws = torch.empty(ops.combine_norm_workspace_bytes(300, 1024, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    out = {k: torch.zeros(300, 1024, dtype=torch.bfloat16, device="cuda") for k in ("y", "h", "dx")}
    out.update(dz=torch.zeros_like(c["z"]), d_gate=torch.zeros(300, device="cuda"),
               d_row_weight=torch.zeros(c["z"].shape[0], device="cuda"),
               dw_post=torch.zeros(1024, device="cuda"), dw_next=torch.zeros(1024, device="cuda"))

    def both(o, w):
        f = ops.combine_norm(c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"], c["w_next"],
                             gate=c["gate"], out=o)
        b = ops.combine_norm_backward(c["dy"], c["dh"], c["z"], c["rows"], c["row_weight"], f["y"],
                                      c["w_post"], c["w_next"], gate=c["gate"], out=o, ws=w)
        return {**f, **b}

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
        for n in ("x", "z", "dy", "dh"):
            c[n].copy_(torch.randn(c[n].shape, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        fresh = {k: torch.zeros_like(v) for k, v in out.items()}
        both(fresh, None)
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], fresh[k]), (i, k)


def test_bound_calls():
    c = _gpu(_inputs(64, 512, 2, "bf16", seed=16))
    r, fwd = ops.combine_norm(c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"], c["w_next"],
                              gate=c["gate"], bind=True)
    dz, dw = torch.zeros_like(c["z"]), torch.zeros(c["z"].shape[0], device="cuda")
    ws = torch.empty(ops.combine_norm_workspace_bytes(64, 512, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    args = (c["dy"], c["dh"], c["z"], c["rows"], c["row_weight"], r["y"], c["w_post"], c["w_next"])
    q, bwd = ops.combine_norm_backward(*args, gate=c["gate"], ws=ws,
                                       out={"dz": dz, "d_row_weight": dw}, bind=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fwd(s.cuda_stream)
    bwd(s.cuda_stream)
    s.synchronize()
    want = ops.combine_norm(c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"], c["w_next"],
                            gate=c["gate"])
    grad = ops.combine_norm_backward(*args, gate=c["gate"],
                                     out={"dz": torch.zeros_like(dz), "d_row_weight": torch.zeros_like(dw)})
    for k in r:
        assert torch.equal(r[k], want[k]), k
    for k in q:
        assert torch.equal(q[k], grad[k]), k


def test_binding_refuses():
    c = _gpu(_inputs(8, 256, 2, "bf16", seed=17))
    f = lambda **kw: ops.combine_norm(  # noqa: E731
        *(kw.get(n, c[n]) for n in ("z", "rows", "row_weight", "x", "w_post", "w_next")),
        **{k: v for k, v in kw.items() if k not in ("z", "rows", "row_weight", "x", "w_post", "w_next")})
    with pytest.raises(TypeError):
        f(x=c["x"].half())
    with pytest.raises(TypeError):
        f(z=c["z"].float())
    with pytest.raises(TypeError):
        f(w_post=c["w_post"].bfloat16())
    with pytest.raises(ValueError, match="row_weight"):
        f(row_weight=c["row_weight"][:3].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        f(x=c["x"].t().contiguous().t())
    with pytest.raises(ValueError, match="block"):
        f(rows=None)
    with pytest.raises(ValueError):
        f(gate=torch.ones(9, device="cuda"))
    with pytest.raises(ValueError, match="nothing"):
        f(w_next=None, with_y=False)
    with pytest.raises(ops._lib.MoeError):
        f(eps=0.0)
    with pytest.raises(ops._lib.MoeError):
        f(out={"y": c["x"]})  # y over x: other blocks would read what is overwritten
    with pytest.raises(ValueError):
        ops.combine_norm_backward(None, None, c["z"], c["rows"], None, c["x"], c["w_post"])
    with pytest.raises(ValueError, match="w_next"):
        ops.combine_norm_backward(None, c["dh"], c["z"], c["rows"], None, c["x"], c["w_post"])
    with pytest.raises(ops._lib.MoeError):
        ops.combine_norm_backward(c["dy"], None, c["z"], c["rows"], None, None, c["w_post"],
                                  ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("H,k", [(64, 2), (1024, 8), (1032, 2), (2048, 8), (4104, 5), (5120, 8),
                                 (8192, 2), (10240, 8), (16384, 5)])
def test_backward_keeps_to_its_workspace(H, k):
    """Enough tokens for the most blocks; what lies behind the workspace's
    size, and rows that no token lists, stay."""
    T = 2100
    say("combine_norm workspace", H, k)
    need = ops.combine_norm_workspace_bytes(T, H, torch.bfloat16)
    ws = torch.full((need + 64 * 1024 * 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, device="cuda")
    z = torch.ones(T * k + 1, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    dz = torch.full_like(z, 7.0)
    y = ops.combine_norm(z, rows, None, x, w, w)["y"]
    ops.combine_norm_backward(x, x, z, rows, None, y, w, w, ws=ws, out={"dz": dz})
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xA5).all()) and bool((dz[-1] == 7.0).all())


def test_rows_past_32_bit_offsets():
    """Rows of z, and of the gradient, more than 4 GiB into their buffers."""
    T, H, k, z_rows = 40, 4096, 2, 600_000
    say("combine_norm far rows")
    s = _inputs(T, H, k, "bf16", seed=2)
    n = s["z"].shape[0]
    c = _gpu(s)
    z = torch.empty(z_rows, H, dtype=torch.bfloat16, device="cuda")
    z[z_rows - n:] = c["z"]
    w = torch.zeros(z_rows, device="cuda")
    w[z_rows - n:] = c["row_weight"][:n]
    rows = torch.where(c["rows"] >= 0, c["rows"] + (z_rows - n), c["rows"]).contiguous()
    dz = torch.empty_like(z)
    got = ops.combine_norm(z, rows, w, c["x"], c["w_post"], c["w_next"], gate=c["gate"], residual_scale=0.75)
    grad = ops.combine_norm_backward(c["dy"], c["dh"], z, rows, w, got["y"], c["w_post"], c["w_next"],
                                     gate=c["gate"], residual_scale=0.75, out={"dz": dz})
    near = ops.combine_norm(c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"], c["w_next"],
                            gate=c["gate"], residual_scale=0.75)
    near_grad = ops.combine_norm_backward(c["dy"], c["dh"], c["z"], c["rows"], c["row_weight"], near["y"],
                                          c["w_post"], c["w_next"], gate=c["gate"], residual_scale=0.75)
    torch.cuda.synchronize()
    listed = torch.unique(c["rows"][c["rows"] >= 0]).long()
    assert torch.equal(got["y"], near["y"]) and torch.equal(got["h"], near["h"])
    for name in ("dx", "d_gate", "dw_post", "dw_next"):
        assert torch.equal(grad[name], near_grad[name]), name
    assert torch.equal(dz[listed + (z_rows - n)], near_grad["dz"][listed])
    assert torch.equal(grad["d_row_weight"][listed + (z_rows - n)], near_grad["d_row_weight"][listed])


def test_a_bound_backward_needs_its_workspace():
    c = _gpu(_inputs(4, 64, 2, "f32"))
    with pytest.raises(ValueError, match="workspace"):
        ops.combine_norm_backward(c["dy"], c["dh"], c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"],
                                  c["w_next"], gate=c["gate"], bind=True)


def _exact_row_gradients(s, eps):
    """d_row_weight from dy in rational numbers, only the reciprocal norm's
    root rounded: a token's only row has 1 / (1 + mean(b^2) / eps) of its
    terms left, which 64-bit sums lose."""
    num = lambda v: [Fraction(float(x)) for x in v]  # noqa: E731
    dot = lambda a, b: sum(x * y for x, y in zip(a, b))  # noqa: E731
    H = s["x"].shape[1]
    out = torch.zeros(s["z"].shape[0], dtype=torch.float64)
    for t in range(s["rows"].shape[0]):
        ids = [r for r in s["rows"][t].tolist() if r >= 0]
        if not ids:
            continue
        z = {r: num(s["z"][r]) for r in ids}
        a = {r: Fraction(float(s["row_weight"][r])) for r in ids}
        b = [sum(a[r] * z[r][i] for r in ids) for i in range(H)]
        v = [x * y for x, y in zip(num(s["dy"][t]), num(s["w_post"]))]
        rho2 = 1 / (dot(b, b) / H + Fraction(eps))
        gate_rho = float(s["gate"][t]) * math.sqrt(rho2)
        for r in ids:
            out[r] = gate_rho * float(dot(v, z[r]) - dot(b, z[r]) * dot(v, b) * rho2 / H)
    return out


@pytest.mark.parametrize("size,eps", [(1e13, 1e-6), (1e16, 1e-6), (1e-15, 1e-30), (0.0, 1e-30)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_of_large_and_small_rows(size, eps, dtype):
    """Rows whose products with each other leave the range of fp32 when
    multiplied once more, and a reciprocal norm whose cube does."""
    say("combine_norm magnitudes", size, eps, dtype)
    s = _inputs(24, 136, 3, dtype, seed=31)
    s["z"] = (size * s["z"].double()).to(DT[dtype])
    _, grad = _run(s, eps=eps, with_dh=False)
    ref = close_grad_ref(d(s["dy"]), None, d(s["z"]), s["rows"], d(s["row_weight"]), None,
                         d(s["w_post"]), None, d(s["gate"]), 0.75, eps)
    listed = s["rows"][s["rows"] >= 0].long()
    close_to(grad["d_row_weight"].cpu()[listed], _exact_row_gradients(s, eps)[listed],
             ref["d_row_weight_size"][listed], 256, "d_row_weight")
    for n in ("dx", "dz", "dw_post", "d_gate"):
        at = listed if n == "dz" else slice(None)
        close_to(grad[n].cpu()[at], ref[n][at], ref[n + "_size"][at], 256 + 24, n)


@pytest.mark.parametrize("H", [256, 4096])
def test_the_next_norm_without_its_gradient(H):
    """h was formed but nothing uses it: its weight's gradient is zero, and
    what an earlier call left in the output is gone."""
    c = _gpu(_inputs(40, H, 2, "bf16", seed=41))
    y = ops.combine_norm(c["z"], c["rows"], c["row_weight"], c["x"], c["w_post"], c["w_next"])["y"]
    out = {"dw_next": torch.full((H,), 7.0, device="cuda")}
    args = (c["z"], c["rows"], c["row_weight"], y, c["w_post"], c["w_next"])
    got = ops.combine_norm_backward(c["dy"], None, *args, out=out)
    assert got["dw_next"] is out["dw_next"] and not bool(out["dw_next"].any())
    out["dw_next"].fill_(7.0)
    got = ops.combine_norm_backward(c["dy"], None, None, None, None, y, None, c["w_next"], out=out)
    assert not bool(out["dw_next"].any()) and got["dw_post"] is None
    plain = ops.combine_norm_backward(c["dy"], None, *args[:5])
    assert plain["dw_next"] is None


@pytest.mark.parametrize("H", [256, 4096])
def test_without_a_block_its_arguments_are_not_read(H):
    """k = 0: a gate shorter than the tokens and full of NaN, as the C
    interface may be given it, plays no part."""
    say("combine_norm k = 0", H)
    c = _gpu(_inputs(700, H, 1, "bf16", seed=43))
    want = ops.combine_norm(None, None, None, c["x"], None, c["w_next"], residual_scale=0.75)
    got = {n: torch.empty_like(c["x"]) for n in ("y", "h")}
    gate = torch.full((1,), float("nan"), device="cuda")
    st = ops._lib.lib().moe_combine_norm(
        None, 0, None, 0, None, c["x"].data_ptr(), gate.data_ptr(), None, c["w_next"].data_ptr(), 0.75,
        1e-6, 700, H, 1, got["y"].data_ptr(), got["h"].data_ptr(), None, None,
        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for n in got:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("H", [256, 4096])
@pytest.mark.parametrize("with_dh", [True, False])
def test_the_gate_gradient_without_a_block_is_zero(H, with_dh):
    """The C interface may ask for it: every token's is written, those from
    n_valid on stay."""
    say("combine_norm k = 0 d_gate", H, with_dh)
    T, n = 2500, 2311
    c = _gpu(_inputs(T, H, 1, "bf16", seed=44))
    d_gate = torch.full((T,), 7.0, device="cuda")
    n_valid = torch.tensor([n], dtype=torch.int32, device="cuda")
    dx, dw = torch.empty_like(c["x"]), torch.empty(H, device="cuda")
    ws = torch.empty(ops.combine_norm_workspace_bytes(T, H, torch.bfloat16), dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    st = ops._lib.lib().moe_combine_norm_backward(
        p(c["dy"]), p(c["dh"]) if with_dh else None, None, 0, None, 0, None, p(c["x"]), None, None,
        p(c["w_next"]), 0.75, 1e-6, T, H, 1, p(dx), None, None, p(d_gate), None, p(dw), p(n_valid),
        None, p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    assert not bool(d_gate[:n].any()) and bool((d_gate[n:] == 7.0).all())
