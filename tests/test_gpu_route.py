"""moe_route and moe_route_backward against the 64-bit definition: choices
exactly (ties, near ties, saturated scores, experts out of service), weights and
gradients within fp32 rounding bounds, and routed layers against their parts."""
import math

import pytest
import torch

import block_ref as R
import moe_inputs as mi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    from _lib import build_and_import
    return build_and_import()


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def run(M, logits, bias, K, **kw):
    T, E = logits.shape
    d = M.make_route(T, E, K, **kw)
    idx = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), float("nan"), device="cuda")
    M.moe_route(d, logits.cuda(), bias.cuda() if bias is not None else None, idx, w)
    return d, idx, w


def weight_tol(logits, idx, ref, scale, K):
    """s: expf (2 ulp = 4u), the rounding of l - max (|l - max| u), an add and a division;
    the sums of K or E scores add their depth; numerator and denominator both err."""
    l = logits.double()
    chosen = l.gather(1, idx)
    finite = torch.where(chosen > -math.inf, chosen, l.amax(dim=1, keepdim=True))
    span = (l.amax(dim=1, keepdim=True) - finite).abs().amax().item()
    span = span if math.isfinite(span) else 0.0
    return R.U32 * (2 * (8 + span) + K + 24) * ref.abs() + 1e-37 * abs(scale)


def check(M, logits, bias, K, score, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_top=group_top,
              renorm=renorm, scale=scale)
    _, idx, w = run(M, logits, bias, K, **kw)
    ref_idx, ref_w = R.route(logits, bias, K, **kw)
    assert torch.equal(idx.cpu().long(), ref_idx)
    err = (w.cpu().double() - ref_w).abs()
    assert (err <= weight_tol(logits, ref_idx, ref_w, scale, K)).all(), err.max()
    return ref_idx


SHAPES = [  # T, E, K, groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 1), (3, 7, 7, 1, 1, 1), (257, 33, 5, 3, 2, 2), (64, 256, 8, 8, 4, 2),
    (40, 128, 16, 1, 1, 1), (19, 512, 16, 32, 3, 1), (33, 160, 6, 8, 3, 1), (9, 96, 1, 4, 1, 2),
    (300, 8, 2, 4, 2, 2), (5, 512, 4, 2, 2, 2), (17, 20, 10, 2, 1, 2), (23, 510, 9, 17, 5, 2),
    (31, 200, 8, 1, 1, 1), (8, 32, 16, 32, 16, 1), (11, 384, 8, 8, 4, 2), (6, 100, 7, 4, 3, 2),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,groups,kept,top", SHAPES)
def test_route(M, T, E, K, groups, kept, top, score):
    g = gen(T * 1000 + E)
    for renorm, scale, with_bias in ((True, 2.5, True), (False, 1.0, False), (False, -0.5, True)):
        logits = torch.randn(T, E, generator=g) * 2
        bias = (torch.rand(E, generator=g) - 0.5) * 0.3 if with_bias else None
        check(M, logits, bias, K, score, groups, kept, top, renorm, scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["equal", "ulp", "saturated", "tiny", "bias_ties", "half_out",
                                  "few_left", "all_out", "bias_out", "wide", "huge"])
def test_route_edges(M, kind, score):
    """Scores that 32 bits cannot tell apart, or that are not there."""
    T, E, K = 37, 64, 8
    g = gen(len(kind) * 31)
    logits = torch.randn(T, E, generator=g)
    bias = (torch.rand(E, generator=g) - 0.5) * 0.2
    if kind == "equal":
        logits = torch.full((T, E), 0.75)
        bias = None
    elif kind == "ulp":           # neighbours one step of fp32 apart, shuffled
        base = torch.tensor(1.0)
        steps = [base]
        for _ in range(E - 1):
            steps.append(torch.nextafter(steps[-1], torch.tensor(9.0)))
        steps = torch.stack(steps)
        logits = torch.stack([steps[torch.randperm(E, generator=g)] for _ in range(T)])
        bias = None
    elif kind == "saturated":     # sigmoids that fp32 rounds to 1
        logits = 18 + 6 * torch.rand(T, E, generator=g)
        bias = None
    elif kind == "tiny":          # scores far below fp32's range
        logits = -150 + 3 * torch.randn(T, E, generator=g)
        if score == "softmax":
            logits[:, 0] = 0.0
        bias = None
    elif kind == "bias_ties":     # equal logits and equal biases, and 16 distinct values of each
        logits = torch.randint(0, 4, (T, E), generator=g).float()
        bias = torch.randint(0, 4, (E,), generator=g).float() / 4
    elif kind == "half_out":
        logits[:, torch.randperm(E, generator=g)[:E // 2]] = -math.inf
    elif kind == "few_left":      # fewer experts in service than K
        logits[:, 3:61] = -math.inf
    elif kind == "all_out":       # a row without any expert
        logits[5] = -math.inf
        logits[11] = -math.inf
    elif kind == "bias_out":
        bias[10:40] = -math.inf
    elif kind == "wide":
        logits = logits * 40
    elif kind == "huge":          # fp32's whole range
        logits = torch.sign(logits) * 10 ** (38 * torch.rand(T, E, generator=g))
        if score == "sigmoid":
            logits[:, 7] = math.inf
    for groups, kept, top in ((1, 1, 1), (8, 3, 2), (8, 2, 1)):
        for renorm in (True, False):
            idx = check(M, logits, bias, K, score, groups, kept, top, renorm, 1.5)
            assert ((idx >= 0) & (idx < E)).all()


def test_route_masked_row_has_no_weight(M):
    logits = torch.full((4, 16), -math.inf)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _, idx, w = run(M, logits, None, 3, score=score, renorm=renorm)
            assert (w == 0).all() and torch.equal(idx.cpu(), torch.tensor([[0, 1, 2]] * 4).int())


def test_route_nan_stays_in_range(M):
    logits = torch.randn(50, 48, generator=gen(1))
    logits[::3, ::5] = math.nan
    logits[7] = math.nan
    for groups, kept in ((1, 1), (6, 2)):
        _, idx, _ = run(M, logits, None, 8, groups=groups, topk_groups=kept)
        assert ((idx >= 0) & (idx < 48)).all()
        assert all(len(set(r)) == 8 for r in idx.cpu().tolist())


BACK = [(1, 1, 1), (5, 7, 3), (130, 64, 8), (33, 512, 16), (257, 100, 6)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", BACK)
def test_route_backward(M, T, E, K, score, renorm):
    g = gen(E + K)
    logits = torch.randn(T, E, generator=g) * 2
    if E > 8:
        logits[:, 2] = -math.inf
    d, idx, _ = run(M, logits, None, K, score=score, renorm=renorm, scale=1.7)
    d_w = torch.randn(T, K, generator=g)
    got = torch.full((T, E), float("nan"), device="cuda")
    M.moe_route_backward(d, logits.cuda(), idx, d_w.cuda(), got)
    got = got.cpu().double()
    ref = R.route_backward(logits, idx, d_w, score, renorm, 1.7)
    span = (logits.double().amax(dim=1, keepdim=True) - logits.double())
    span = span[torch.isfinite(span)].max().item()
    tol = R.U32 * (4 * (8 + span) + 2 * K + 48) * 1.7 * d_w.abs().amax(dim=1, keepdim=True)
    assert ((got - ref).abs() <= tol).all()
    # along a direction, against a central difference of the definition: its own
    # error is h^2 f''' / 6 < 1e-9 for h = 1e-5, and the gradient's as above
    v = torch.randn(T, E, generator=g).double()
    i = idx.long().cpu()

    def f(l):
        return (R.weights(l, i, score, renorm, 1.7) * d_w.double()).sum(dim=1)
    h = 1e-5
    l64 = logits.double()
    diff = (f(l64 + h * v) - f(l64 - h * v)) / (2 * h)
    assert ((got * v).sum(dim=1) - diff).abs().max() <= (tol * v.abs()).sum(dim=1).max() + 1e-7


def test_route_backward_repeated_and_bad_indices(M):
    """The same expert twice adds up; an index outside the experts takes no part."""
    T, E, K = 6, 40, 4
    g = gen(9)
    logits = torch.randn(T, E, generator=g)
    d_w = torch.randn(T, K, generator=g)
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    idx[:, 1] = idx[:, 0]
    for score, renorm in (("sigmoid", True), ("softmax", False), ("softmax", True)):
        d = M.make_route(T, E, K, score=score, renorm=renorm)
        got = torch.empty(T, E, device="cuda")
        M.moe_route_backward(d, logits.cuda(), idx.cuda(), d_w.cuda(), got)
        ref = R.route_backward(logits, idx, d_w, score, renorm, 1.0)
        assert (got.cpu().double() - ref).abs().max() <= R.U32 * 200 * d_w.abs().max()
    bad = idx.clone()
    bad[:, 2] = -1
    bad[:, 3] = E
    d = M.make_route(T, E, K, score="sigmoid", renorm=False)
    got = torch.empty(T, E, device="cuda")
    M.moe_route_backward(d, logits.cuda(), bad.cuda(), d_w.cuda(), got)
    ref = R.route_backward(logits, idx[:, :2], d_w[:, :2], "sigmoid", False, 1.0)
    assert (got.cpu().double() - ref).abs().max() <= R.U32 * 200 * d_w.abs().max()


def test_route_leaves_the_rows_behind_alone(M):
    T, E, K = 13, 64, 4
    logits = torch.randn(T, E, generator=gen(2)).cuda()
    idx = torch.full((T + 3, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 3, K), -7.0, device="cuda")
    dl = torch.full((T + 3, E), -7.0, device="cuda")
    d = M.make_route(T, E, K)
    M.moe_route(d, logits, None, idx[:T], w[:T])
    M.moe_route_backward(d, logits, idx[:T], w[:T], dl[:T])
    assert (idx[T:] == -7).all() and (w[T:] == -7).all() and (dl[T:] == -7).all()
    assert (idx[:T] >= 0).all() and torch.isfinite(dl).all()
    e = M.make_route(0, E, K)
    M.moe_route(e, logits[:0], None, idx[:0], w[:0])
    M.moe_route_backward(e, logits[:0], idx[:0], w[:0], dl[:0])


def test_route_many_tokens_repeats_and_streams(M):
    """A large batch twice, on two streams and from a captured graph: the same bits."""
    T, E, K = 5000, 256, 8
    logits = torch.randn(T, E, generator=gen(4)).cuda()
    bias = torch.zeros(E, device="cuda")
    d = M.make_route(T, E, K, groups=8, topk_groups=4, group_top=2, scale=2.5)
    outs = [(torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda"))
            for _ in range(3)]
    M.moe_route(d, logits, bias, *outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.moe_route(d, logits, bias, *outs[1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_route(d, logits, bias, *outs[2])
    graph.replay()
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])
    rows = torch.arange(0, T, 97)
    ref, _ = R.route(logits.cpu()[rows], None, K, groups=8, topk_groups=4, group_top=2)
    assert torch.equal(outs[0][0].cpu()[rows].long(), ref)


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 48), ("bf16", 300), ("f32", 21)])
def test_routed_layer_equals_its_parts(M, dtype, T):
    """moe_layer_forward_routed is the gate's logits, moe_route, and the layer's
    dispatch, experts and combine."""
    wl = mi.Workload("r", "routed", dtype, 256, 32, 4, 256, 256, (T,), 8, bias_uniform=0.2)
    host = mi.draw_layer(wl)
    dev = {k: (v.cuda() if v is not None else None) for k, v in host.items()}
    route = dict(score="sigmoid", groups=4, topk_groups=2, group_top=2, scale=2.5)
    layer = M.MoELayer(dev["w_router"], dev["w1"], dev["w2"], wl.K, dev["ws1"], dev["ws2"],
                       dev["bias"], route=route)
    x = mi.draw_x(wl, T).cuda()
    r = layer.routing_buffers(T)
    y = layer.forward(x, routing=r)
    idx, w = torch.empty_like(r["topk_idx"]), torch.empty_like(r["topk_w"])
    M.moe_route(layer.route_desc(T), r["logits"], dev["bias"], idx, w)
    assert torch.equal(idx, r["topk_idx"]) and torch.equal(w, r["topk_w"])
    ref, _ = R.route(r["logits"].cpu(), host["bias"], wl.K, **route)
    assert torch.equal(idx.cpu().long(), ref)
    # the logits are the ones that the layer's own routing computes
    d, ws = layer.desc(T), layer.workspace(T)
    own = torch.empty_like(r["logits"])
    M.moe_router_topk(d, x, dev["w_router"], dev["bias"], own, idx, w, ws)
    tol = 1e-4 if dtype == "bf16" else 1e-5
    assert (own - r["logits"]).abs().max() <= tol * own.square().mean().sqrt()
    counts, offsets = torch.empty_like(r["counts"]), torch.empty_like(r["offsets"])
    perm, inv = torch.empty_like(r["perm"]), torch.empty_like(r["inv"])
    M.moe_dispatch(d, r["topk_idx"], counts, offsets, perm, inv, ws)
    for a, k in ((counts, "counts"), (offsets, "offsets"), (perm, "perm"), (inv, "inv")):
        assert torch.equal(a, r[k]), k
    rows = torch.empty(T * wl.K, wl.H, device="cuda")
    shared = torch.empty(T, wl.H, device="cuda")
    M.moe_grouped_ffn(d, x, perm, offsets, dev["w1"], dev["w2"], dev["ws1"], dev["ws2"], rows,
                      shared, ws)
    parts = torch.empty_like(y)
    M.moe_combine(d, rows, r["topk_w"], inv, shared, parts)
    assert M.moe_check_status(ws) == 0
    # the layer may split its products' reductions: the hidden layer's rounding to
    # bf16 then differs in places, as between any two orders of its sums
    rms = y.float().square().mean().sqrt()
    assert (parts.float() - y.float()).abs().max() <= (2e-2 if dtype == "bf16" else 1e-5) * rms
    with pytest.raises(ValueError):
        layer.forward(x, gumbel_noise=torch.zeros(T, wl.E, device="cuda"))


def test_routing_gradient_chain(M):
    """combine -> routing weights -> logits, as a training step takes them."""
    T, H, E, K = 24, 128, 32, 4
    g = gen(12)
    wl = mi.Workload("r", "routed", "f32", H, E, K, 128, 0, (T,), 3)
    dev = {k: (v.cuda() if v is not None else None) for k, v in mi.draw_layer(wl).items()}
    layer = M.MoELayer(dev["w_router"], dev["w1"], dev["w2"], K,
                       route=dict(score="sigmoid", groups=4, topk_groups=2, scale=1.3))
    x = mi.draw_x(wl, T).cuda()
    r = layer.routing_buffers(T)
    layer.forward(x, routing=r)
    rows = torch.empty(T * K, H, device="cuda")
    M.moe_grouped_ffn(layer.desc(T), x, r["perm"], r["offsets"], dev["w1"], dev["w2"], None, None,
                      rows, None, layer.workspace(T))
    dy = torch.randn(T, H, generator=g).cuda()
    got = layer.router_backward(dy, rows, r)
    l = r["logits"].double().cpu().requires_grad_(True)
    rows64 = rows.double().cpu().requires_grad_(True)
    w = R.weights(l, r["topk_idx"].long().cpu(), "sigmoid", True, 1.3)
    y = (w[:, :, None] * rows64[r["inv"].long().cpu()].view(T, K, H)).sum(dim=1)
    dl, drows = torch.autograd.grad(y, [l, rows64], dy.double().cpu())
    # d_topk_w sums H products (depth < 64), the weights err by < 64 steps
    size = (rows64.detach()[r["inv"].long().cpu()].view(T, K, H).abs()
            * dy.cpu().double()[:, None].abs()).sum(dim=2).max()
    assert (got["d_logits"].cpu().double() - dl).abs().max() <= 400 * R.U32 * size
    assert (got["d_y_rows"].cpu().double() - drows).abs().max() <= 80 * R.U32 * drows.abs().max()
