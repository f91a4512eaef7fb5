"""A whole layer, as it is used: dispatch plan, rows to the experts, the
experts' feed-forward block, replies, the closing combine, and all gradients.

Tolerances.  Stage by stage (bf16 and fp32): those of each operator, from
the stage's own device inputs.  End to end (fp32 only): a product over K
terms is off by at most K steps of 2^-24 of |A| |B|, which for factors with
independent signs is up to sqrt(K) |A B|; so the longest chain's sum of
K^1.5 times 2^-24 bounds the error, relative in the norm of each tensor."""

import math

import pytest
import torch

from co_activation_amd.pipeline import (ExpertLayerBackward, ExpertLayerStep, GraphStep, LayerStep,
                                        Pipeline, TwoLayerStep)
from gpu_util import dev, i32, say, x_tensor
from layer_ref import U32, close_grad_ref, close_ref, close_to, d
from test_gpu_expert_ffn import _act, _check_backward, _check_forward
from workloads import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib):
    assert torch.cuda.is_available()
    return built_lib


def _layer(w):
    z = torch.zeros(1, w.H, dtype=x_tensor(w).dtype, device="cuda")  # not read by these steps
    if w.topk2 is not None:
        return TwoLayerStep(i32(w.topk), i32(w.topk2), dev(w.gates2), i32(w.expert_rank2),
                            x_tensor(w), z, w.G, w.ranks_per_node, E1=w.E)
    # tokens that do not split evenly all come from the first source rank
    src = i32([0] + [w.T] * w.G) if w.T % w.G else None
    return LayerStep(i32(w.topk), dev(w.gates), i32(w.expert_rank), x_tensor(w), z, w.G,
                     w.ranks_per_node, src_offsets=src)


def _step(w, F, seed=0, act="silu", train=True, next_norm=True, weights=None):
    g = torch.Generator().manual_seed(seed)
    layer = _layer(w)
    dt, E, H, T = layer.x.dtype, w.E, w.H, w.T
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if weights is None:
        weights = [(rnd(E, 2 * F, H) / math.sqrt(H)).to(dt).cuda(),
                   (rnd(E, H, F) / math.sqrt(F)).to(dt).cuda(),
                   (1 + 0.1 * rnd(H)).cuda(), (1 + 0.1 * rnd(H)).cuda(), torch.rand(T, generator=g).cuda()]
    w_in, w_down, w_post, w_next, gate = weights
    res = None if w.topk2 is not None else rnd(T, H).to(dt).cuda()
    step = ExpertLayerStep(layer, w_in, w_down, w_post, w_next if next_norm else None, residual=res,
                           gate=gate, residual_scale=0.75, eps=1e-6, act=act, train=train)
    return step, weights


def _grads(step, seed):
    g = torch.Generator().manual_seed(seed)
    shape, dt = step.y.shape, step.y.dtype
    return [torch.randn(*shape, generator=g).to(dt).cuda() for _ in range(2)]


@pytest.mark.parametrize("cfg,T,H,F,act", [(1, 300, 64, 48, "silu"), (2, 200, 128, 96, "gelu"),
                                           (5, 260, 256, 128, "silu"), (4, 24, 128, 64, "silu")])
def test_stages(cfg, T, H, F, act):
    w = make(cfg, T=T, H=H)
    say("expert layer stages", cfg, T, H, F, act)
    step, _ = _step(w, F, seed=cfg, act=act)
    side, lp = step.side, step.layer.plan
    back = ExpertLayerBackward(step)
    dy, dh = _grads(step, 7)
    step.run()
    back.run(dy, dh)
    torch.cuda.synchronize()
    assert int(step.d_err.item()) == 0
    # the rows at their experts are the tokens' rows, bit for bit
    x = step.layer.x_s if w.topk2 is not None else step.layer.x
    erow = side.plan["erow"].cpu().long()
    rows = side.expert_in.cpu()
    assert (torch.sort(erow.flatten()).values == torch.arange(erow.numel())).all()
    for j in range(erow.shape[1]):
        assert torch.equal(rows[erow[:, j]], x.cpu())
    # the experts, forward and backward
    s = {"x": side.expert_in.cpu(), "w_in": step.w_in.cpu(), "w_down": step.w_down.cpu(),
         "dy": back.d_expert_out.cpu(), "first": side.out["expert_first"].cpu(),
         "count": side.out["expert_count"].cpu()}
    assert int(s["count"].sum()) == erow.numel()
    _check_forward(s, {"gu": step.gu, "a": step.a, "y": step.expert_out}, act, True)
    _check_backward(s, step.gu, step.a, {"dx": back.d_expert_in, "dw_in": back.dw_in,
                                         "dw_down": back.dw_down}, act)
    # the closing combine, forward and backward
    n = int(side.n_rows().item())
    tr = lp.token_rows.cpu()
    reply = d(side.reply)
    reply[n:] = 0
    ref = close_ref(reply, tr, None, d(step.residual), d(step.w_post), d(step.w_next), d(step.gate),
                    0.75, 1e-6)
    k, Hh = tr.shape[1], w.H
    close_to(step.y, ref["y"], ref["y_size"], k + Hh + 8, "y")
    ref = close_grad_ref(d(dy), d(dh), reply, tr, None, d(step.y), d(step.w_post), d(step.w_next),
                         d(step.gate), 0.75, 1e-6)
    R = 2 * (k + Hh) + 16
    close_to(back.d_residual, ref["dx"], ref["dx_size"], R, "d_residual")
    close_to(back.d_reply[:n], ref["dz"][:n], ref["dz_size"][:n], R, "d_reply")
    close_to(back.d_gate, ref["d_gate"], ref["d_gate_size"], R, "d_gate")
    close_to(back.dw_post, ref["dw_post"], ref["dw_post_size"], R + w.T, "dw_post")
    close_to(back.dw_next, ref["dw_next"], ref["dw_next_size"], R + w.T, "dw_next")
    # the gates' gradients: each slot's own dot
    out, dr = d(step.expert_out), d(back.d_reply)
    slot = lp.slot_row.cpu().long()
    want = (out[erow] * dr[slot]).sum(-1)
    size = (out[erow] * dr[slot]).abs().sum(-1)
    close_to(back.dw, want, size, Hh, "dw")


def _whole(w, step, dy, dh, topk, gates, x):
    """The layer in 64 bits from its definition, and autograd's gradients."""
    leaves = {k: d(v).requires_grad_() for k, v in
              dict(x=x, res=step.residual, gates=gates, w_in=step.w_in, w_down=step.w_down,
                   w_post=step.w_post, w_next=step.w_next, gate=step.gate).items()}
    F = step.w_down.shape[2]
    b = torch.zeros_like(leaves["x"])
    for e in range(step.w_down.shape[0]):
        t, j = torch.nonzero(topk == e, as_tuple=True)
        p = leaves["x"][t] @ leaves["w_in"][e].t()
        o = (_act(step.act, p[:, :F]) * p[:, F:]) @ leaves["w_down"][e].t()
        b = b.index_add(0, t, leaves["gates"][t, j][:, None] * o)
    norm = lambda v: v / (v.pow(2).mean(1, keepdim=True) + step.eps).sqrt()  # noqa: E731
    y = step.residual_scale * leaves["res"] + leaves["gate"][:, None] * norm(b) * leaves["w_post"]
    h = norm(y) * leaves["w_next"]
    ((y * d(dy)).sum() + (h * d(dh)).sum()).backward()
    return y.detach(), h.detach(), {k: v.grad for k, v in leaves.items()}


@pytest.mark.parametrize("T,H,F", [(96, 64, 48), (1, 32, 16), (700, 64, 80)])
def test_end_to_end(T, H, F):
    w = make(1, T=T, H=H)
    say("expert layer end to end", T, H, F)
    step, _ = _step(w, F, seed=T)
    back = ExpertLayerBackward(step)
    dy, dh = _grads(step, T + 1)
    step.run()
    back.run(dy, dh)
    torch.cuda.synchronize()
    assert int(step.d_err.item()) == 0
    y, h, want = _whole(w, step, dy, dh, torch.from_numpy(w.topk).long(), torch.from_numpy(w.gates),
                        step.layer.x)
    got = {"x": back.dx, "res": back.d_residual, "gates": back.dw, "w_in": back.dw_in,
           "w_down": back.dw_down, "w_post": back.dw_post, "w_next": back.dw_next,
           "gate": back.d_gate}
    terms = [H, F, w.k, H, H]                       # forward: up, down, replies, two norms
    tol_y = U32 * (sum(K ** 1.5 for K in terms) + 64)
    terms += [H, H, w.k, H, 2 * F, T]               # backward: two norms, gates, down, up, weights
    tol = U32 * (sum(K ** 1.5 for K in terms) + 192)
    for name, a, b, t in [("y", step.y, y, tol_y), ("h", step.h, h, tol_y)] + \
            [("d_" + n, got[n], want[n], tol) for n in got]:
        off = float((d(a) - b).norm() / b.norm())
        assert off <= t, f"{name}: off by {off:.3g} of its norm, allowed {t:.3g}"


def _outputs(step, back):
    return [t.clone() for t in (step.y, step.h, back.dx, back.d_residual, back.dw, back.dw_in,
                                back.dw_down, back.dw_post, back.dw_next, back.d_gate)]


class _Both:
    """Forward and backward as one step, for a graph."""

    def __init__(self, step, back, dy, dh):
        self.step, self.back, self.dy, self.dh = step, back, dy, dh

    def run(self):
        self.step.run()
        self.back.run(self.dy, self.dh)
        return self


def test_captured_and_replayed():
    w = make(2, T=256, H=128)
    say("expert layer graph")
    step, _ = _step(w, 64)
    back = ExpertLayerBackward(step)
    dy, dh = _grads(step, 3)
    both = _Both(step, back, dy, dh)
    graph = GraphStep(both)
    for seed in range(3):
        w2 = make(2, T=256, H=128, seed=seed + 5)   # another routing, rows and gates
        step.layer.topk.copy_(i32(w2.topk))
        step.layer.gates.copy_(dev(w2.gates))
        step.layer.x.copy_(x_tensor(w2))
        both.run()
        want = _outputs(step, back)
        for t in (step.y, step.h, back.dx, back.dw, back.dw_in, back.dw_down):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert int(step.d_err.item()) == 0
        for a, b in zip(_outputs(step, back), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("beside", ["combine", "move"])
def test_batches_through_a_pipeline(beside):
    ws = [make(5, T=192, H=128, seed=s) for s in (1, 2)]
    say("expert layer pipeline", beside)
    first, weights = _step(ws[0], 64, train=False)
    steps = [first, _step(ws[1], 64, train=False, weights=weights)[0]]
    want = []
    for st in steps:
        st.run()
        want.append((st.y.clone(), st.h.clone()))
    torch.cuda.synchronize()
    seen = []
    pipe = Pipeline(steps, beside)
    pipe.run(6, collect=lambda st, i: seen.append((i, st.y.clone(), st.h.clone())))
    torch.cuda.synchronize()
    assert all(int(st.d_err.item()) == 0 for st in steps)
    for i, y, h in seen:
        assert torch.equal(y, want[i % 2][0]) and torch.equal(h, want[i % 2][1])


def test_without_training_or_next_norm():
    w = make(1, T=130, H=64)
    say("expert layer inference")
    full, weights = _step(w, 48)
    step, _ = _step(w, 48, train=False, next_norm=False, weights=weights)
    step.residual.copy_(full.residual)
    full.run()
    step.run()
    torch.cuda.synchronize()
    assert step.h is None and step.gu is None and torch.equal(step.y, full.y)
    with pytest.raises(ValueError, match="train"):
        ExpertLayerBackward(step)
    with pytest.raises(ValueError):
        ExpertLayerStep(step.layer, step.w_in[:, :-1].contiguous(), step.w_down, step.w_post)
    with pytest.raises(TypeError):
        ExpertLayerStep(step.layer, step.w_in.double(), step.w_down, step.w_post)
    # the gradient of y alone, without the next layer's norm
    plain, _ = _step(w, 48, next_norm=False, weights=weights)
    plain.residual.copy_(full.residual)
    plain.run()
    full.run()
    dy, _ = _grads(plain, 2)
    a, b = ExpertLayerBackward(plain).run(dy), ExpertLayerBackward(full).run(dy)
    torch.cuda.synchronize()
    assert a.dw_next is None
    for n in ("dx", "d_residual", "dw", "dw_in", "dw_down", "dw_post", "d_gate"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_two_graphs_share_a_workspace_and_two_streams_do_not():
    """Backward calls captured into two graphs over one workspace, replayed in
    turn; then both at once on two streams with a workspace each."""
    from co_activation_amd import ops
    say("expert_ffn_backward graphs and streams")
    g = torch.Generator().manual_seed(1)
    H, F, E = 128, 96, 3
    w_in = (torch.randn(E, 2 * F, H, generator=g) / 11).bfloat16().cuda()
    w_down = (torch.randn(E, H, F, generator=g) / 10).bfloat16().cuda()
    cases = []
    for counts in ([300, 0, 900], [5, 700, 64]):
        R = sum(counts)
        x, dy = (torch.randn(R, H, generator=g).bfloat16().cuda() for _ in range(2))
        count = torch.tensor(counts, dtype=torch.int32, device="cuda")
        first = (count.cumsum(0) - count).int()
        f = ops.expert_ffn(x, w_in, w_down, first, count, save=True)
        args = (dy, x, w_in, w_down, f["gu"], f["a"], first, count)
        want = {k: v.clone() for k, v in ops.expert_ffn_backward(*args).items()}
        cases.append((args, want, {k: torch.empty_like(v) for k, v in want.items()},
                      ops.expert_ffn_workspace_bytes(R, H, F, E, torch.bfloat16)))
    ws = torch.empty(max(c[3] for c in cases), dtype=torch.uint8, device="cuda")
    graphs = []
    for args, _, out, _ in cases:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            ops.expert_ffn_backward(*args, out=out, ws=ws)
        graphs.append(graph)
    for _ in range(3):
        for graph, (_, want, out, _) in zip(graphs, cases):
            for t in out.values():
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for k in want:
                assert torch.equal(out[k], want[k]), k
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [torch.empty(c[3], dtype=torch.uint8, device="cuda") for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for stream, space, (args, _, out, _) in zip(streams, spaces, cases):
            with torch.cuda.stream(stream):
                ops.expert_ffn_backward(*args, out=out, ws=space)
    torch.cuda.synchronize()
    for _, want, out, _ in cases:
        for k in want:
            assert torch.equal(out[k], want[k]), k


def test_the_next_norm_gradient_of_an_earlier_run_does_not_stay():
    w = make(1, T=130, H=64)
    say("expert layer dw_next")
    step, _ = _step(w, 48)
    step.run()
    dy, dh = _grads(step, 2)
    back = ExpertLayerBackward(step)
    back.run(dy, dh)
    torch.cuda.synchronize()
    assert bool(back.dw_next.any())
    back.run(dy)
    torch.cuda.synchronize()
    assert not bool(back.dw_next.any())


def _balanced(w, seed, weights, fused):
    """cfg 5's routing with fp32 rows through a balanced two-layer step."""
    g = torch.Generator().manual_seed(seed)
    T, H, F, E = w.T, w.H, 48, w.E
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    layer = TwoLayerStep(i32(w.topk), i32(w.topk2), dev(w.gates2), i32(w.expert_rank2), rnd(T, H),
                         torch.zeros(1, H, device="cuda"), w.G, w.ranks_per_node, E1=w.E,
                         balanced=True, fused=fused)
    if weights is None:
        weights = [rnd(E, 2 * F, H) / math.sqrt(H), rnd(E, H, F) / math.sqrt(F), 1 + 0.1 * rnd(H),
                   1 + 0.1 * rnd(H), torch.rand(T, generator=g).cuda()]
    w_in, w_down, w_post, w_next, gate = weights
    return ExpertLayerStep(layer, w_in, w_down, w_post, w_next, gate=gate, residual_scale=0.75), weights


@pytest.mark.parametrize("beside", ["combine", "move"])
@pytest.mark.parametrize("fused", [True, False])
def test_balanced_two_layer_batches_through_a_pipeline(beside, fused):
    """Each batch against the layer in 64 bits over its own shuffled rows,
    forward and backward, then the same batches through a pipeline."""
    ws = [make(5, T=192, H=64, seed=s) for s in (3, 4)]
    say("expert layer balanced pipeline", beside, fused)
    first, weights = _balanced(ws[0], 1, None, fused)
    steps = [first, _balanced(ws[1], 2, weights, fused)[0]]
    H, F, T, k = 64, 48, 192, ws[0].k
    terms = [H, F, k, H, H]
    tol_y = U32 * (sum(K ** 1.5 for K in terms) + 64)
    terms += [H, H, k, H, 2 * F, T]
    tol = U32 * (sum(K ** 1.5 for K in terms) + 192)
    want = []
    for st in steps:
        st.run()
        back = ExpertLayerBackward(st)
        dy, dh = _grads(st, 5)
        back.run(dy, dh)
        torch.cuda.synchronize()
        assert int(st.d_err.item()) == 0
        layer = st.layer
        assert torch.equal(torch.sort(layer.shuffle["perm"]).values, torch.arange(T, device="cuda").int())
        assert torch.equal(layer.x_s, layer.x[layer.shuffle["perm"].long()])
        y, h, grads = _whole(None, st, dy, dh, layer.topk2_s.cpu().long(), layer.gates2_s, layer.x_s)
        got = {"x": back.dx, "res": back.d_residual, "gates": back.dw, "w_in": back.dw_in,
               "w_down": back.dw_down, "w_post": back.dw_post, "w_next": back.dw_next, "gate": back.d_gate}
        for name, a, b, t in [("y", st.y, y, tol_y), ("h", st.h, h, tol_y)] + \
                [("d_" + n, got[n], grads[n], tol) for n in got]:
            off = float((d(a) - b).norm() / b.norm())
            assert off <= t, f"{name}: off by {off:.3g} of its norm, allowed {t:.3g}"
        want.append((st.y.clone(), st.h.clone()))
    seen = []
    Pipeline(steps, beside).run(6, collect=lambda st, i: seen.append((i, st.y.clone(), st.h.clone())))
    torch.cuda.synchronize()
    assert all(int(st.d_err.item()) == 0 for st in steps) and len(seen) == 6
    for i, y, h in seen:
        assert torch.equal(y, want[i % 2][0]) and torch.equal(h, want[i % 2][1])


def test_a_captured_pipeline_follows_its_inputs():
    from co_activation_amd.pipeline import GraphPipeline
    say("expert layer graph pipeline")
    ws = [make(5, T=192, H=128, seed=s) for s in (6, 7)]
    first, weights = _step(ws[0], 64, train=False)
    steps = [first, _step(ws[1], 64, train=False, weights=weights)[0]]
    graph = GraphPipeline(Pipeline(steps), 4)
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        for st in steps:
            st.layer.x.copy_(torch.randn(st.layer.x.shape, generator=g))
        want = []
        for st in steps:
            st.run()
            want.append((st.y.clone(), st.h.clone()))
            st.y.zero_()
            st.h.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for st, (y, h) in zip(steps, want):
            assert int(st.d_err.item()) == 0
            assert torch.equal(st.y, y) and torch.equal(st.h, h)


@pytest.mark.parametrize("cfg", [1, 5])
def test_stage_timers_cover_every_stage(cfg):
    """The names that STAGES lists are those that a run records, each once,
    alone and in a pipeline."""
    from co_activation_amd.pipeline import StageTimers
    say("expert layer timers", cfg)
    first, weights = _step(make(cfg, T=192, H=64, seed=1), 48)
    timers = StageTimers(first.STAGES, 1)
    first.run(timers)
    back = ExpertLayerBackward(first)
    back_timers = StageTimers(back.STAGES, 1)
    back.run(*_grads(first, 1), timers=back_timers)
    torch.cuda.synchronize()
    assert timers.used == {n: 1 for n in first.STAGES} and len(timers.mean_ms()) == len(first.STAGES)
    assert back_timers.used == {n: 1 for n in back.STAGES}
    second, _ = _step(make(cfg, T=192, H=64, seed=2), 48, weights=weights)
    timers = StageTimers(first.STAGES, 6)
    Pipeline([first, second], "combine").run(6, timers)
    torch.cuda.synchronize()
    assert timers.used == {n: 6 for n in first.STAGES}
