"""moe_block_norm, its gradients and moe_combine_backward against the 64-bit
definitions, at the widths, batches, gates and parts where they can go wrong."""
import pytest
import torch

import block_ref as R
import moe_inputs as mi

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module")
def M():
    from _lib import build_and_import
    return build_and_import()


def draw(seed, T, H, dt, kind, post=True, pre=True, block=True):
    g = torch.Generator("cpu").manual_seed(seed)

    def n(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dt).cuda()
    shape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[kind]
    return {"h": n(T, H, std=2.0), "y": n(T, H, std=0.5) if block else None,
            "w_post": n(H) if post and block else None,
            "gate": n(*shape, std=0.7) if shape and block else None,
            "w_pre": n(H) if pre else None, "d_h_out": n(T, H), "d_x": n(T, H) if pre else None}


def forward(M, t, kind, alpha=1.0, into=None):
    T, H = t["h"].shape
    d = M.make_norm(T, H, M.dtype_code(t["h"].dtype), gate=kind, alpha=alpha, eps=EPS)
    out = into or {"h_out": torch.full_like(t["h"], float("nan")) if t["y"] is not None else None,
                   "x": torch.full_like(t["h"], float("nan")) if t["w_pre"] is not None else None}
    M.moe_block_norm(d, t["h"], t["y"], t["w_post"], t["gate"], t["w_pre"], out["h_out"], out["x"])
    return d, out


def check_forward(t, out, kind, alpha):
    """fp32: each norm factor errs by its sum (chains of < 16 + 10 adds, halved by the square
    root), rsqrtf and two products; then one rounding to the type."""
    ref_h, ref_x = R.block_norm(t["h"], t["y"], t["w_post"], t["gate"], kind, t["w_pre"], alpha, EPS)
    half = R.HALF[t["h"].dtype]
    h = t["h"].double()
    size = h.abs()
    if t["y"] is not None:
        size = size + R.block(*(v.double() if v is not None else None for v in
                                (t["y"], t["w_post"], t["gate"])), kind, alpha, EPS).abs()
        err = (out["h_out"].double() - ref_h).abs()
        assert (err <= half * ref_h.abs() + 24 * R.U32 * size).all(), err.max()
    if t["w_pre"] is not None:
        full = ref_h if ref_h is not None else h
        r = 1 / torch.sqrt((full * full).mean(dim=1, keepdim=True) + EPS)
        err = (out["x"].double() - ref_x).abs()
        tol = half * ref_x.abs() + 64 * R.U32 * size * r * t["w_pre"].double().abs()
        assert (err <= tol).all(), err.max()


FORMS = [  # gate, post, pre, block, alpha
    ("none", True, True, True, 1.0), ("channel", True, True, True, 0.5),
    ("token", True, False, True, 0.22), ("full", False, True, True, -1.5),
    ("none", False, False, True, 1.0), ("none", False, True, False, 1.0),
]
SIZES = [("bf16", 1, 8), ("bf16", 3, 128), ("bf16", 77, 1000), ("bf16", 2, 4096), ("bf16", 5, 6152),
         ("bf16", 2, 16384), ("f32", 1, 4), ("f32", 9, 1004), ("f32", 4, 8192), ("f32", 6000, 132),
         ("bf16", 3001, 256)]


@pytest.mark.parametrize("kind,post,pre,block,alpha", FORMS)
@pytest.mark.parametrize("dtype,T,H", SIZES)
def test_block_norm(M, dtype, T, H, kind, post, pre, block, alpha):
    t = draw(T + H, T, H, DT[dtype], kind, post, pre, block)
    _, out = forward(M, t, kind, alpha)
    check_forward(t, out, kind, alpha)


def backward(M, t, h_out, kind, alpha, skip=()):
    T, H = t["h"].shape
    d = M.make_norm(T, H, M.dtype_code(t["h"].dtype), gate=kind, alpha=alpha, eps=EPS)
    nan = float("nan")

    def new(on, shape, dt):
        return torch.full(shape, nan, dtype=dt, device="cuda") if on else None
    dt, f32 = t["h"].dtype, torch.float32
    gate = t["gate"]
    out = {"d_h": new(True, (T, H), dt), "d_y": new(t["y"] is not None, (T, H), dt),
           "d_w_post": new(t["w_post"] is not None, (H,), f32),
           "d_gate": new(gate is not None, tuple(gate.shape) if gate is not None else (),
                         dt if kind == "full" else f32),
           "d_w_pre": new(t["w_pre"] is not None, (H,), f32)}
    for k in skip:
        out[k] = None
    M.moe_block_norm_backward(d, t["d_h_out"], t["d_x"], h_out if t["w_pre"] is not None else None,
                              t["y"], t["w_post"], gate, t["w_pre"], out["d_h"], out["d_y"],
                              out["d_w_post"], out["d_gate"], out["d_w_pre"], M.alloc_workspace(d))
    return {k: v for k, v in out.items() if v is not None}


def check_backward(t, h_out, got, kind, alpha):
    """Each value is a short fp32 expression of sums over the row; its error is bounded by a
    number of steps times the sum of its terms' magnitudes, a column sum's by the same over
    the tokens, plus one rounding for what is stored in the layer's type."""
    ref = R.block_norm_backward(t["d_h_out"], t["d_x"], h_out, t["y"], t["w_post"], t["gate"], kind,
                                t["w_pre"], alpha, EPS)
    half = R.HALF[t["h"].dtype]
    size = {}
    g = t["d_h_out"].double().abs() if t["d_h_out"] is not None else torch.zeros_like(h_out.double())
    if t["w_pre"] is not None:
        v = h_out.double()
        r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
        n, dn = (v * r).abs(), (t["d_x"].double() * t["w_pre"].double()).abs()
        size["d_w_pre"] = (t["d_x"].double().abs() * n).sum(dim=0)
        g = g + r * (dn + n * (dn * n).mean(dim=1, keepdim=True))
    size["d_h"] = g
    if t["y"] is not None:
        gate = R.widen(t["gate"].double().abs() if t["gate"] is not None else None, kind)
        n, r, w = t["y"].double().abs(), 1.0, 1.0
        if t["w_post"] is not None:
            r = 1 / torch.sqrt((n * n).mean(dim=1, keepdim=True) + EPS)
            n, w = n * r, t["w_post"].double().abs()
        g = g * abs(alpha)
        du = g * n * w
        size["d_gate"] = {"channel": du.sum(dim=0), "token": du.sum(dim=1), "full": du,
                          "none": None}[kind]
        size["d_w_post"] = (g * gate * n).sum(dim=0)
        dn = g * gate * w
        size["d_y"] = dn if t["w_post"] is None else r * (dn + n * (dn * n).mean(dim=1, keepdim=True))
    for k, v in got.items():
        stored = half if v.dtype == t["h"].dtype else R.U32
        err = (v.double() - ref[k]).abs()
        steps = 200 + t["h"].shape[0] / 64
        assert (err <= stored * ref[k].abs() + steps * R.U32 * size[k]).all(), (k, err.max())


@pytest.mark.parametrize("kind,post,pre,block,alpha", FORMS)
@pytest.mark.parametrize("dtype,T,H", SIZES)
def test_block_norm_backward(M, dtype, T, H, kind, post, pre, block, alpha):
    t = draw(T + H + 1, T, H, DT[dtype], kind, post, pre, block)
    got = backward(M, t, t["h"], kind, alpha)
    check_backward(t, t["h"], got, kind, alpha)


def test_block_norm_backward_parts(M):
    """Outputs left out do not change the others; without d_h_out it counts as zero."""
    t = draw(5, 40, 512, torch.bfloat16, "channel")
    whole = backward(M, t, t["h"], "channel", 0.5)
    for skip in (("d_h",), ("d_y", "d_w_post"), ("d_gate", "d_w_pre"), ("d_w_post", "d_gate", "d_w_pre")):
        part = backward(M, t, t["h"], "channel", 0.5, skip)
        for k, v in part.items():
            assert torch.equal(v, whole[k]), (skip, k)
    t["d_h_out"] = None
    check_backward(t, t["h"], backward(M, t, t["h"], "channel", 0.5), "channel", 0.5)


def test_block_norm_gradients_against_differences(M):
    """fp32, along random directions: f = <h', a> + <x, b> of the 64-bit definition. The
    central difference with h = 1e-4 errs by h^2 f''' / 6 (< 1e-6 of the values here), the
    fp32 gradient by < 1e-4 of the sums of its terms."""
    T, H, kind, alpha = 6, 64, "full", 0.8
    t = draw(8, T, H, torch.float32, kind)
    h_out, _ = R.block_norm(t["h"], t["y"], t["w_post"], t["gate"], kind, t["w_pre"], alpha, EPS)
    got = backward(M, t, h_out.float(), kind, alpha)
    grads = {"h": "d_h", "y": "d_y", "w_post": "d_w_post", "gate": "d_gate", "w_pre": "d_w_pre"}
    gen = torch.Generator("cpu").manual_seed(1)
    for name, grad in grads.items():
        v = torch.randn(t[name].shape, generator=gen).double().cuda()

        def f(s):
            u = {k: x.double() if x is not None else None for k, x in t.items()}
            u[name] = u[name] + s * v
            a, b = R.block_norm(u["h"], u["y"], u["w_post"], u["gate"], kind, u["w_pre"], alpha, EPS)
            return (a * u["d_h_out"]).sum() + (b * u["d_x"]).sum()
        diff = (f(1e-4) - f(-1e-4)) / 2e-4
        dot = (got[grad].double() * v).sum()
        assert (dot - diff).abs() <= 1e-4 * (got[grad].double().abs() * v.abs()).sum(), name


def test_block_norm_in_place_and_rows_behind(M):
    t = draw(3, 50, 1024, torch.bfloat16, "channel")
    _, want = forward(M, t, "channel", 0.5)
    big = torch.full((53, 1024), 7.0, dtype=torch.bfloat16, device="cuda")
    h = big.clone()
    h[:50] = t["h"]
    y = big.clone()
    y[:50] = t["y"]
    forward(M, dict(t, h=h[:50], y=y[:50]), "channel", 0.5, into={"h_out": h[:50], "x": y[:50]})
    assert torch.equal(h[:50], want["h_out"]) and torch.equal(y[:50], want["x"])
    assert (h[50:] == 7).all() and (y[50:] == 7).all()
    # backward: d_h over d_h_out, d_y over d_x
    d = M.make_norm(50, 1024, M.MOE_BF16, gate="channel", alpha=0.5, eps=EPS)
    ref = backward(M, t, want["h_out"], "channel", 0.5)
    g, dx = t["d_h_out"].clone(), t["d_x"].clone()
    M.moe_block_norm_backward(d, g, dx, want["h_out"], t["y"], t["w_post"], t["gate"], t["w_pre"], g, dx,
                              None, None, None, M.alloc_workspace(d))
    assert torch.equal(g, ref["d_h"]) and torch.equal(dx, ref["d_y"])


def test_block_norm_zero_rows_and_empty_batch(M):
    """A row of zeros: rms is 1 / sqrt(eps), no NaN in either direction."""
    t = draw(4, 4, 256, torch.float32, "token")
    for k in ("h", "y"):
        t[k][1:3] = 0
    t["gate"][2] = 0
    _, out = forward(M, t, "token", 1.0)
    check_forward(t, out, "token", 1.0)
    check_backward(t, out["h_out"], backward(M, t, out["h_out"], "token", 1.0), "token", 1.0)
    e = draw(4, 0, 256, torch.float32, "token")
    forward(M, e, "token", 1.0)
    got = backward(M, e, e["h"], "token", 1.0)
    assert (got["d_w_post"] == 0).all() and (got["d_w_pre"] == 0).all()


def test_block_norm_captured_and_on_two_streams(M):
    """Two captured graphs with one workspace, replayed one after the other, and eager
    calls on another stream give the same bits."""
    t = draw(6, 600, 4096, torch.bfloat16, "channel")
    d, want = forward(M, t, "channel", 0.5)
    ref = backward(M, t, want["h_out"], "channel", 0.5)
    ws = M.alloc_workspace(d)
    outs = [{k: torch.zeros_like(v) for k, v in ref.items()} for _ in range(3)]

    def call(o, stream=None):
        M.moe_block_norm_backward(d, t["d_h_out"], t["d_x"], want["h_out"], t["y"], t["w_post"],
                                  t["gate"], t["w_pre"], o["d_h"], o["d_y"], o["d_w_post"],
                                  o["d_gate"], o["d_w_pre"], ws, stream)
    graphs = []
    for o in outs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(outs[2], side)
    side.synchronize()
    for o in outs:
        for k, v in ref.items():
            assert torch.equal(o[k], v), k


COMBINE = [("f32", 1, 1, 4, 1), ("f32", 37, 3, 132, 7), ("bf16", 5, 16, 128, 40),
           ("bf16", 130, 8, 1024, 32), ("bf16", 2, 2, 4096, 8), ("bf16", 700, 3, 4096, 8),
           ("f32", 3001, 4, 68, 9), ("bf16", 1200, 16, 384, 64)]


@pytest.mark.parametrize("dtype,T,K,H,E", COMBINE)
def test_combine_backward(M, dtype, T, K, H, E):
    g = torch.Generator("cpu").manual_seed(T + H)
    dt = DT[dtype]
    d = M.make_desc(T, H, E, K, 128, 0, M.dtype_code(dt))
    idx = torch.rand(T, E, generator=g).topk(K, dim=1).indices.int().cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    perm, inv = torch.empty(T * K, **i32), torch.empty(T * K, **i32)
    M.moe_dispatch(d, idx, counts, offsets, perm, inv, M.alloc_workspace(d))
    if T > 2:
        inv = inv.clone()
        inv[1] = -1           # a copy that was not placed
        inv[2 * K] = T * K    # an index past the rows
    rows = torch.randn(T * K, H, generator=g).cuda()
    w = torch.rand(T, K, generator=g).cuda()
    dy = torch.randn(T, H, generator=g).to(dt).cuda()
    d_rows = torch.full((T * K, H), 9.0, dtype=dt, device="cuda")
    d_w = torch.full((T, K), float("nan"), device="cuda")
    M.moe_combine_backward(d, dy, rows, w, inv, d_rows, d_w)
    at = inv.long()
    ok = (at >= 0) & (at < T * K)
    token = torch.arange(T * K, device="cuda") // K
    ref = torch.full((T * K, H), 9.0, dtype=torch.float64, device="cuda")
    ref[at[ok]] = (w.double().reshape(-1, 1) * dy.double()[token])[ok]
    # one fp32 product, one rounding
    assert ((d_rows.double() - ref).abs() <= (R.HALF[dt] + 2 * R.U32) * ref.abs()).all()
    prod = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    prod[ok] = rows.double()[at[ok]] * dy.double()[token][ok]
    # chains of H / 256 fp32 products and adds, then 8 + 5 adds
    tol = (H / 256 + 24) * R.U32 * prod.abs().sum(dim=1)
    assert ((d_w.double().reshape(-1) - prod.sum(dim=1)).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moe_block(M, dtype):
    """Pre-norm, routed layer, post-norm with gate and residual, next pre-norm."""
    wl = mi.Workload("b", "block", dtype, 256, 16, 2, 256, 0, (40,), 4)
    dev = {k: (v.cuda() if v is not None else None) for k, v in mi.draw_layer(wl).items()}
    layer = M.MoELayer(dev["w_router"], dev["w1"], dev["w2"], 2, route=dict(groups=4, topk_groups=2))
    t = draw(2, 40, 256, DT[dtype], "channel")
    block = M.MoEBlock(layer, t["w_pre"], t["w_post"], t["gate"], alpha=0.5)
    h_out, x = block(t["h"], next_w_pre=t["w_pre"])
    x0 = block.pre_norm(t["h"])
    check_forward(dict(t, y=None, w_post=None, gate=None), {"h_out": None, "x": x0}, "none", 1.0)
    y = layer(x0)
    check_forward(dict(t, y=y), {"h_out": h_out, "x": x}, "channel", 0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = block(t["h"], stream=side)
    side.synchronize()
    assert torch.equal(other, h_out)
    plain = M.MoEBlock(layer, t["w_pre"])
    check_forward(dict(t, y=y, w_post=None, gate=None, w_pre=None),
                  {"h_out": plain(t["h"], x=x0), "x": None}, "none", 1.0)


def test_offsets_past_32_bits(M):
    """More than 2^31 elements: the last rows are what they are in a small batch."""
    T, H = (1 << 18) + 7, 8200
    g = torch.Generator("cuda").manual_seed(1)
    tail = torch.randn(9, H, generator=g, device="cuda").bfloat16()
    h = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    h[-9:] = tail
    w = torch.randn(H, generator=g, device="cuda").bfloat16()
    x = torch.empty_like(h)
    M.moe_block_norm(M.make_norm(T, H, eps=EPS), h, w_pre=w, x=x)
    small = torch.empty_like(tail)
    M.moe_block_norm(M.make_norm(9, H, eps=EPS), tail, w_pre=w, x=small)
    assert torch.equal(x[-9:], small) and (x[:5] == 0).all()
    del h, x
    T, K, H = 33000, 16, 4096
    d = M.make_desc(T, H, 64, K, 128, 0, M.MOE_BF16)
    rows = torch.zeros((T * K, H), device="cuda")
    rows[-K:] = torch.randn(K, H, generator=g, device="cuda")
    dy = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    dy[-1] = torch.randn(H, generator=g, device="cuda").bfloat16()
    inv = torch.arange(T * K, dtype=torch.int32, device="cuda")
    wk = torch.rand(T, K, generator=g, device="cuda")
    d_rows = torch.empty((T * K, H), dtype=torch.bfloat16, device="cuda")
    d_w = torch.empty((T, K), device="cuda")
    M.moe_combine_backward(d, dy, rows, wk, inv, d_rows, d_w)
    ref = wk[-1].double()[:, None] * dy[-1].double()
    assert ((d_rows[-K:].double() - ref).abs() <= (R.HALF[torch.bfloat16] + 2 * R.U32) * ref.abs()).all()
    prod = rows[-K:].double() * dy[-1].double()
    assert ((d_w[-1].double() - prod.sum(dim=1)).abs() <= 40 * R.U32 * prod.abs().sum(dim=1)).all()
    assert (d_w[:-1] == 0).all()
