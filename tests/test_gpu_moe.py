"""A whole MoE layer step (-m gpu): router, route, dispatch, experts, combine, and
back, with the replicas' gradients reduced and an optimizer step, through EpLayer
and through autograd; against the same layer in fp64 from the same bf16 weights.

Between the stages rows are bf16, so against fp64 a result carries a few roundings
of 2^-9 of its terms' sizes: the comparison is by norm, and each stage by itself is
compared element by element in the stages' own tests."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


class Model:
    """Reference in fp64 with autograd; the routing (which experts) is given."""

    def __init__(self, x, logits, w13, w2, ids, score, scale):
        import torch
        leaf = lambda t: t.double().clone().requires_grad_(True)  # noqa: E731
        self.x, self.logits, self.w13, self.w2 = leaf(x), leaf(logits), leaf(w13), leaf(w2)
        T, K = ids.shape
        I = w2.shape[2]
        s = torch.sigmoid(self.logits) if score == "sigmoid" else torch.softmax(self.logits, 1)
        c = s.gather(1, ids.long())
        self.w = scale * c / c.sum(1, keepdim=True)
        out = torch.zeros_like(self.x)
        for e in range(w13.shape[0]):
            t, k = torch.nonzero(ids == e, as_tuple=True)
            if len(t) == 0:
                continue
            gu = self.x[t] @ self.w13[e].T
            h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
            out = out.index_add(0, t, self.w[t, k][:, None] * (h @ self.w2[e].T))
        self.out = out


def close(got, want, tol, what):
    """Distance by norm; tol in units of 2^-8."""
    d = float((got.double() - want).norm() / want.norm())
    assert d <= tol * 2.0 ** -8, f"{what}: {d:.3g}"


def make(R, S, K, E, H, I, seed=0, skew=1.5):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = r(R * S, H).to(torch.bfloat16)
    logits = r(R * S, E) + skew * r(E)
    w13 = (r(E, 2 * I, H) * H ** -0.5).to(torch.bfloat16)
    w2 = (r(E, H, I) * I ** -0.5).to(torch.bfloat16)
    dout = r(R * S, H).to(torch.bfloat16)
    return x, logits, w13, w2, dout


CASES = [(4, 64, 2, 16, 128, 72), (8, 128, 6, 64, 256, 128), (1, 40, 4, 8, 64, 64), (2, 1, 1, 2, 64, 8)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "R{}_S{}_K{}_E{}_H{}_I{}".format(*c))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_training_step_of_a_layer(case, score):
    import torch
    import token_dispatch_histogram_b200 as tdh
    from token_dispatch_histogram_b200.optim import EpAdamW
    R, S, K, E, H, I = case
    x, logits, w13, w2, dout = make(*case)
    layer = tdh.EpLayer(R, S, K, E, H, 4, grad_n=3 * H * I)
    P = layer.P
    kw = dict(score=score, renorm=True, scale=1.5)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, gu, y = torch.empty((P, I), **bf), torch.empty((P, 2 * I), **bf), torch.empty((P, H), **bf)
    dy, dgu, dx = torch.empty((P, H), **bf), torch.empty((P, 2 * I), **bf), torch.empty((R * S, H), **bf)
    dw, dlogits = torch.empty((R * S, K), device="cuda"), torch.empty_like(logits)
    layer.x.copy_(x)
    layer.router(logits, **kw)
    layer.route()
    layer.dispatch()
    layer.experts(w13, w2, h, gu, y)
    layer.combine(y=y)
    tdh.ep_combine_backward(dout, layer.w, y, layer.pos, dy, dw, layer.dev_status)
    tdh.ep_router_backward(dw, logits, layer.topk_ids, dlogits, dev_status=layer.dev_status, **kw)
    layer.experts_backward(dy, layer.buf, w13, w2, gu, dgu, h, dy)
    tdh.ep_dispatch_backward(dy, layer.pos, R * S, K, dx, layer.dev_status)
    layer.grad_reduce()
    assert layer.status() == 0
    ref = Model(x, logits, w13, w2, layer.topk_ids, score, 1.5)
    close(layer.out, ref.out, 2, "out")
    ref.out.backward(dout.double())
    close(layer.w, ref.w, 1e-3, "w")
    close(dx, ref.x.grad, 3, "dx")
    if K > 1:
        close(dlogits, ref.logits.grad, 4, "dlogits")
    (g13, g2), _ = layer.weight_grads(I)
    close(g2, ref.w2.grad, 3, "dw2")
    close(g13, ref.w13.grad, 3, "dw13")
    # the optimizer takes the reduced gradients where they are, and leaves the products' weights
    p13, p2 = w13.float(), w2.float()
    opt = EpAdamW([p13[e] for e in range(E)] + [p2[e] for e in range(E)],
                  [g13[e] for e in range(E)] + [g2[e] for e in range(E)], lr=1e-2, betas=(0.9, 0.95), eps=1e-8,
                  weight_decay=0.0, state_bits=8,
                  copies=[w13[e] for e in range(E)] + [w2[e] for e in range(E)])
    before = w2.float()
    opt.step()
    assert torch.equal(w13, p13.to(torch.bfloat16)) and torch.equal(w2, p2.to(torch.bfloat16))
    # a first step of AdamW is lr in the direction of the gradient
    moved = (p2 - before)[g2.abs() > 1e-6]
    assert torch.allclose(moved, -1e-2 * torch.sign(g2[g2.abs() > 1e-6]), rtol=0, atol=2e-4)


def test_the_buffer_of_a_layer_serves_in_place():
    """Serving: the experts write over the dispatched rows, and combine reads them there."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    R, S, K, E, H, I = 4, 32, 4, 16, 128, 64
    x, logits, w13, w2, _ = make(R, S, K, E, H, I, seed=3)
    layer = tdh.EpLayer(R, S, K, E, H, 4)
    h = torch.empty((layer.P, I), dtype=torch.bfloat16, device="cuda")
    layer.x.copy_(x)
    layer.router(logits, score="softmax")
    layer.route_dispatch()
    layer.experts(w13, w2, h)
    layer.combine()
    assert layer.status() == 0
    close(layer.out, Model(x, logits, w13, w2, layer.topk_ids, "softmax", 1.0).out, 2, "out")


def test_a_captured_layer_follows_its_inputs():
    import torch
    import token_dispatch_histogram_b200 as tdh
    R, S, K, E, H, I = 4, 64, 2, 16, 128, 72
    layer = tdh.EpLayer(R, S, K, E, H, 4)
    h = torch.empty((layer.P, I), dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros((R * S, E), device="cuda")
    x, first, w13, w2, _ = make(R, S, K, E, H, I, seed=1)
    layer.x.copy_(x)
    logits.copy_(first)

    def step():
        layer.router(logits, score="sigmoid")
        layer.route()
        layer.dispatch()
        layer.experts(w13, w2, h)
        layer.combine()

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 5):
        x, other, _, _, _ = make(R, S, K, E, H, I, seed=seed, skew=2.0)
        layer.x.copy_(x)
        logits.copy_(other)
        graph.replay()
        assert layer.status() == 0
        close(layer.out, Model(x, logits, w13, w2, layer.topk_ids, "sigmoid", 1.0).out, 2, "out")


@pytest.mark.parametrize("case", CASES[:2], ids=str)
def test_autograd_through_the_whole_layer(case):
    import torch
    import token_dispatch_histogram_b200 as tdh
    from token_dispatch_histogram_b200.autograd import ep_combine_fn, ep_dispatch_fn, ep_experts_fn, ep_router_fn
    R, S, K, E, H, I = case
    x, logits, w13, w2, dout = make(*case, seed=7)
    layer = tdh.EpLayer(R, S, K, E, H, 4, grad_n=3 * H * I)
    xt, lt = x.clone().requires_grad_(True), logits.clone().requires_grad_(True)
    w, ids = ep_router_fn(lt, K, score="sigmoid", scale=2.0, dev_status=layer.dev_status)
    layer.topk_ids.copy_(ids)
    layer.route()
    rows = ep_dispatch_fn(xt, layer.pos, K, torch.empty((layer.P, H), dtype=torch.bfloat16, device="cuda"))
    out = ep_combine_fn(ep_experts_fn(rows, w13, w2, layer), w, layer.pos)
    out.backward(dout)
    layer.grad_reduce()
    assert layer.status() == 0 and not ids.requires_grad
    ref = Model(x, logits, w13, w2, ids, "sigmoid", 2.0)
    close(out.detach(), ref.out, 2, "out")
    ref.out.backward(dout.double())
    close(xt.grad, ref.x.grad, 3, "dx")
    close(lt.grad, ref.logits.grad, 4, "dlogits")
    (g13, g2), _ = layer.weight_grads(I)
    close(g2, ref.w2.grad, 3, "dw2")
    close(g13, ref.w13.grad, 3, "dw13")
    # a second pass adds to what is there
    once = g13.clone(), g2.clone()
    w, ids = ep_router_fn(lt, K, score="sigmoid", scale=2.0)
    layer.g_rep.zero_()
    rows = ep_dispatch_fn(xt, layer.pos, K, torch.empty((layer.P, H), dtype=torch.bfloat16, device="cuda"))
    ep_combine_fn(ep_experts_fn(rows, w13, w2, layer, accumulate=True), w, layer.pos).backward(dout)
    layer.grad_reduce()
    for got, was in zip((g13, g2), once):
        assert torch.allclose(got, 2 * was, rtol=1e-5, atol=1e-5 * float(was.abs().max()))


def test_a_frozen_trunk_under_trained_experts():
    import torch
    import token_dispatch_histogram_b200 as tdh
    from token_dispatch_histogram_b200.autograd import ep_combine_fn, ep_dispatch_fn, ep_experts_fn, ep_router_fn
    R, S, K, E, H, I = case = 4, 64, 2, 16, 128, 72
    x, logits, w13, w2, dout = make(*case, seed=7)
    layer = tdh.EpLayer(R, S, K, E, H, 4, grad_n=3 * H * I)
    lt = logits.clone().requires_grad_(True)
    w, ids = ep_router_fn(lt, K, dev_status=layer.dev_status)
    layer.topk_ids.copy_(ids)
    layer.route()
    rows = ep_dispatch_fn(x, layer.pos, K, torch.empty((layer.P, H), dtype=torch.bfloat16, device="cuda"))
    ep_combine_fn(ep_experts_fn(rows, w13, w2, layer), w, layer.pos).backward(dout)
    layer.grad_reduce()
    ref = Model(x, logits, w13, w2, ids, "softmax", 1.0)
    ref.out.backward(dout.double())
    (g13, g2), _ = layer.weight_grads(I)
    close(lt.grad, ref.logits.grad, 4, "dlogits")
    close(g2, ref.w2.grad, 3, "dw2")
    close(g13, ref.w13.grad, 3, "dw13")
    # without gradient rows, and without grad mode, nothing is kept for a backward
    plain = tdh.EpLayer(R, S, K, E, H, 4)
    plain.topk_ids.copy_(ids)
    plain.route()
    assert not ep_experts_fn(rows, w13, w2, plain).requires_grad
    with torch.no_grad():
        assert not ep_experts_fn(rows, w13, w2, layer).requires_grad


def test_micro_batches_that_are_each_reduced():
    """Three micro-batches of their own routing: the sum of three separate gradients, replicas counted once each."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    R, S, K, E, H, I = case = 4, 64, 2, 16, 128, 72
    bf = dict(dtype=torch.bfloat16, device="cuda")
    layer = tdh.EpLayer(R, S, K, E, H, 4, grad_n=3 * H * I)
    P = layer.P
    h, gu, y = torch.empty((P, I), **bf), torch.empty((P, 2 * I), **bf), torch.empty((P, H), **bf)
    dy, dgu, dx, dw = (torch.empty((P, H), **bf), torch.empty((P, 2 * I), **bf), torch.empty((P, H), **bf),
                       torch.empty((R * S, K), device="cuda"))
    _, _, w13, w2, _ = make(*case)

    def backward(seed, accumulate):
        x, logits, _, _, dout = make(*case, seed=seed)
        layer.x.copy_(x)
        layer.router(logits)
        layer.route()
        assert layer.plan_view("n_rep", 1).item() > 0
        layer.dispatch()
        layer.experts(w13, w2, h, gu, y)
        tdh.ep_combine_backward(dout, layer.w, y, layer.pos, dy, dw, layer.dev_status)
        layer.experts_backward(dy, layer.buf, w13, w2, gu, dgu, h, dx, accumulate=accumulate)
        layer.grad_reduce()
        assert layer.status() == 0
        return layer.g_home.clone()

    want = sum(backward(seed, False).double() for seed in (1, 2, 3))
    backward(1, False)
    backward(2, True)
    got = backward(3, True)
    assert float((got.double() - want).norm() / want.norm()) <= 1e-6


def test_second_derivatives_are_refused():
    """Rather than left out of a sum that has other parts."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    from token_dispatch_histogram_b200.autograd import ep_experts_fn, ep_router_fn
    x = torch.randn(8, 16, device="cuda", requires_grad=True)
    w, _ = ep_router_fn(x, 2)
    (dx,) = torch.autograd.grad((w * w).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (dx.square().sum() + w.sum()).backward()
    R, S, K, E, H, I = case = 2, 16, 2, 4, 64, 8
    rows, logits, w13, w2, _ = make(*case)
    layer = tdh.EpLayer(R, S, K, E, H, 4, grad_n=3 * H * I)
    layer.router(logits)
    layer.route()
    rows = rows.repeat(2, 1).requires_grad_(True)
    y = ep_experts_fn(rows, w13, w2, layer).float()
    (dx,) = torch.autograd.grad(y.square().sum(), rows, create_graph=True)
    with pytest.raises(RuntimeError):
        (dx.float().square().sum() + y.sum()).backward()


@pytest.mark.parametrize("planner", ["exact", "quota"])
def test_a_ranks_slots_cover_its_rows(planner):
    """Each rank's products over its own buffer, with home weights and prefetched replicas' weights, equal the rows of
    the same products over the whole buffer; and its weight gradients the whole's home and replica rows."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    from token_dispatch_histogram_b200.ranks import EpRank
    R, S, K, E, H, I = 4, 64, 2, 16, 64, 40
    x, logits, w13, _, _ = make(R, S, K, E, H, I, seed=4)
    ids = torch.empty((R * S, K), dtype=torch.int32, device="cuda")
    w = torch.empty((R * S, K), device="cuda")
    tdh.ep_router(logits, ids, w)
    ranks = [EpRank(r, R, S, K, E, H, planner=planner, B=2, buf_rows=R * S * K if planner == "quota" else None,
                    grad_n=2 * I * H) for r in range(R)]
    for r, rk in enumerate(ranks):
        rk.topk_local.copy_(ids[r * S:(r + 1) * S])
        rk.x_local.copy_(x[r * S:(r + 1) * S])
        rk.count()
    counts = torch.stack([rk.counts_row for rk in ranks])
    peers = tdh.peer_table([rk.buf for rk in ranks])
    for rk in ranks:
        rk.counts.copy_(counts)
        rk.set_peers(peers)
        rk.plan_and_layout()
        rk.dispatch()
    torch.cuda.synchronize()
    ER, lay = E // R, ranks[0].plan_layout
    plan = ranks[0].plan
    view = lambda name, n: plan[lay[name]:lay[name] + n].tolist()  # noqa: E731
    n_rep = view("n_rep", 1)[0]
    assert n_rep > 0
    rep_e, rep_r = view("rep_expert", n_rep), view("rep_rank", n_rep)
    for r, rk in enumerate(ranks):
        mine = [m for m in range(n_rep) if rep_r[m] == r]
        table = torch.cat([w13[r * ER:(r + 1) * ER], w13[[rep_e[m] for m in mine]]])
        s = rk.slots()
        n_rows = int(s["cu_seqlens"].max())
        gu = torch.full((rk.buf.shape[0], 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
        tdh.ep_expert_gemm(rk.buf, table, y=gu, dev_status=rk.dev_status, **s)
        tdh.ep_expert_wgrad(gu, rk.buf, g_home=rk.g_home.unflatten(1, (2 * I, H)),
                            g_rep=rk.g_rep.unflatten(1, (2 * I, H)), dev_status=rk.dev_status, **s)
        assert rk.status() == 0
        # the expert of each of this rank's rows, from the pairs that were sent there
        seen = 0
        for e, rows in slots_of(s, table.shape[0]):
            want = rk.buf[rows].double() @ table[e].double().T
            assert torch.allclose(gu[rows].double(), want, rtol=2.0 ** -7, atol=1e-3)
            g = rk.g_home[e] if e < ER else rk.g_rep[e - ER]
            gw = gu[rows].double().T @ rk.buf[rows].double()
            assert torch.allclose(g.view(2 * I, H).double(), gw, rtol=1e-4, atol=1e-3)
            seen += len(range(*rows.indices(rk.buf.shape[0])))
        assert seen == n_rows and torch.all(gu[n_rows:] == 7.0)


def slots_of(s, n):
    cu, order = s["cu_seqlens"].tolist(), s["slot_order"].tolist()
    for i, e in enumerate(order):
        if e >= 0:
            assert e < n
            yield e, slice(cu[i], cu[i + 1])
