"""A layer's forward and backward run from the grouped products and the rows' way, captured in a graph and replayed: every step of
the replay against the formula of that step on what it was given, in 64 bits, and the outputs and all gradients against the
layer's formula from the inputs.

Bounds.  A sum of n fp32 terms is off by at most n 2^-23 S, S the sum of the terms' magnitudes; storing it in bf16 adds 2^-8 of it.
A step given values that are off by at most E (elementwise) adds what the same step makes of E and the magnitudes of the
other side.
"""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import bf16, check, gen

pytestmark = pytest.mark.gpu

DEV = "cuda"
T, k, E, H, I = 96, 4, 16, 256, 128


def rounded(ref, S, terms, given=0.0, eps=2.0 ** -8):
    """The most that a stored sum is off: n 2^-23 of the magnitudes, what it was given, and its own rounding."""
    off = terms * 2.0 ** -23 * (S + given) + given
    return off + eps * (ref.abs() + off)


def within(name, got, ref, bound, most):
    """The largest error is in the bound, and the bound is a small part of the largest value, so that it says something."""
    worst, share = float(((got.double() - ref).abs() / bound).max()), float(bound.max() / ref.abs().max())
    print(f"[run] {name}: worst {worst:.3f} of the bound, which is {share:.4f} of the largest value", flush=True)
    assert worst <= 1 and share < most, name


@pytest.fixture(scope="module")
def run():
    """What the last of three replays gave, with its inputs."""
    g = gen(21)
    w1, w2 = bf16(g, E, I, H, scale=0.05), bf16(g, E, H, I, scale=0.05)
    router = bf16(g, E, H, scale=0.1)
    x, dout = torch.empty(T, H, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, device=DEV)
    M = qm.moe_align_capacity(T, k, E, 16)
    outs = {}

    def step():
        o = {}
        _, o["ids"], o["wts"] = qm.moe_route(x, router, None, k)
        al = qm.moe_align(o["ids"], E, 16)
        ranges = (al.offsets, al.counts, T * k)
        o["slots"] = qm.moe_pair_slots(o["ids"], al.sorted_ids, al.offsets, al.counts)
        o["rows"] = qm.moe_gather_rows(x, o["slots"], rows=M)
        o["a"] = qm.moe_grouped_mm(o["rows"], w1, *ranges)
        o["y"] = qm.moe_grouped_mm(o["a"], w2, *ranges)
        o["out"] = qm.moe_combine_rows(o["y"], o["slots"], o["wts"], out_dtype=torch.float32)
        o["dy"], o["dwts"] = qm.moe_combine_rows_grad(dout, o["y"], o["slots"], o["wts"])
        o["da"] = qm.moe_grouped_mm_dgrad(o["dy"], w2, *ranges)
        o["drows"] = qm.moe_grouped_mm_dgrad(o["da"], w1, *ranges)
        o["dx"] = qm.moe_combine_rows(o["drows"], o["slots"], out_dtype=torch.float32)
        o["dw1"] = qm.moe_grouped_mm_wgrad(o["da"], o["rows"], *ranges, out_dtype=torch.float32)
        o["dw2"] = qm.moe_grouped_mm_wgrad(o["dy"], o["a"], *ranges, out_dtype=torch.float32)
        return o

    def fill(seed):
        x.copy_(torch.randn(T, H, device=DEV, generator=gen(seed)))
        dout.copy_(torch.randn(T, H, device=DEV, generator=gen(seed + 100)))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2, 3):
        fill(seed)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("ids", "wts", "slots", "out", "dwts", "dx", "dw1", "dw2"):  # (the others have rows of nobody)
            assert torch.equal(outs[n], want[n]), (seed, n)
    ids = outs["ids"].cpu()
    pairs = [tuple(v.to(DEV) for v in torch.nonzero(ids == e, as_tuple=True)) for e in range(E)]
    assert sum(len(t) for t, _ in pairs) == T * k
    return dict(outs, graph=graph, x=x, dout=dout, w1=w1, w2=w2, pairs=[(e, t, j) for e, (t, j) in enumerate(pairs) if len(t)])


def test_every_step(run):
    """Each step on what the step before it gave."""
    r = run
    d = {n: r[n].double() for n in ("x", "dout", "w1", "w2", "rows", "a", "y", "wts", "dy", "da", "drows")}
    out, mag = torch.zeros(2, T, H, dtype=torch.float64, device=DEV)
    dx, dmag = torch.zeros(2, T, H, dtype=torch.float64, device=DEV)
    for e, t, j in r["pairs"]:
        s = r["slots"][t, j].long()
        assert torch.equal(r["rows"][s], r["x"][t])
        w1, w2, w = d["w1"][e], d["w2"][e], d["wts"][t, j][:, None]
        check("a", r["a"][s], d["rows"][s] @ w1.t(), d["rows"][s].abs() @ w1.abs().t(), H)
        check("y", r["y"][s], d["a"][s] @ w2.t(), d["a"][s].abs() @ w2.abs().t(), I)
        check("dy", r["dy"][s], w * d["dout"][t], (w * d["dout"][t]).abs(), 1)
        terms = d["y"][s] * d["dout"][t]
        check("dwts", r["dwts"][t, j], terms.sum(1), terms.abs().sum(1), H)
        check("da", r["da"][s], d["dy"][s] @ w2, d["dy"][s].abs() @ w2.abs(), H)
        check("drows", r["drows"][s], d["da"][s] @ w1, d["da"][s].abs() @ w1.abs(), I)
        check("dw1", r["dw1"][e], d["da"][s].t() @ d["rows"][s], d["da"][s].abs().t() @ d["rows"][s].abs(), len(t))
        check("dw2", r["dw2"][e], d["dy"][s].t() @ d["a"][s], d["dy"][s].abs().t() @ d["a"][s].abs(), len(t))
        for ref, m, v in ((out, mag, d["y"][s] * w), (dx, dmag, d["drows"][s])):
            ref.index_add_(0, t, v)
            m.index_add_(0, t, v.abs())
    check("out", r["out"], out, mag, k)
    check("dx", r["dx"], dx, dmag, k)


def test_outputs_and_gradients_from_the_inputs(run):
    """out = sum_j w_j W2 W1 x, and the gradients of sum(out * dout) for x, the weights and both matrices, by autograd in 64
    bits, with the roundings to bf16 on the way carried through."""
    r = run
    leaf = {n: r[n].double().requires_grad_() for n in ("x", "wts", "w1", "w2")}
    dout = r["dout"].double()
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e, t, j in r["pairs"]:
        y = leaf["x"][t] @ leaf["w1"][e].t() @ leaf["w2"][e].t()
        out = out.index_add(0, t, leaf["wts"][t, j][:, None] * y)
    (out * dout).sum().backward()
    out_off, dx_off, dw_off = [torch.zeros(n, dtype=torch.float64, device=DEV) for n in ((T, H), (T, H), (T, k))]
    for e, t, j in r["pairs"]:
        x, w1, w2, w = r["x"][t].double(), r["w1"][e].double(), r["w2"][e].double(), r["wts"][t, j].double()[:, None]
        d = dout[t]
        a = x @ w1.t()
        a_off = rounded(a, x.abs() @ w1.abs().t(), H)
        y = a @ w2.t()
        y_off = rounded(y, a.abs() @ w2.abs().t(), I, a_off @ w2.abs().t())
        out_off.index_add_(0, t, w * y_off + k * 2.0 ** -23 * w * (y.abs() + y_off))
        dw_off[t, j] = rounded((y * d).sum(1), (y * d).abs().sum(1), H, (y_off * d.abs()).sum(1), 2.0 ** -24)
        dy = w * d
        dy_off = rounded(dy, dy.abs(), 1)
        da = dy @ w2
        da_off = rounded(da, dy.abs() @ w2.abs(), H, dy_off @ w2.abs())
        dr = da @ w1
        dr_off = rounded(dr, da.abs() @ w1.abs(), I, da_off @ w1.abs())
        dx_off.index_add_(0, t, dr_off + k * 2.0 ** -23 * (dr.abs() + dr_off))
        n, g1, g2 = len(t), leaf["w1"].grad[e], leaf["w2"].grad[e]
        off = rounded(g1, da.abs().t() @ x.abs(), n, da_off.t() @ x.abs(), 2.0 ** -24)
        within(f"dw1 of {e}", r["dw1"][e], g1, off, 0.5)
        given = dy_off.t() @ (a.abs() + a_off) + dy.abs().t() @ a_off
        within(f"dw2 of {e}", r["dw2"][e], g2, rounded(g2, dy.abs().t() @ a.abs(), n, given, 2.0 ** -24), 0.5)
    within("out", r["out"], out.detach(), out_off, 0.5)
    within("dx", r["dx"], leaf["x"].grad, dx_off, 0.5)
    within("dwts", r["dwts"], leaf["wts"].grad, dw_off, 0.5)
