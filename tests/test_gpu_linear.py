"""moe_linear and moe_linear_backward against the 64-bit definition: one token to
many, odd sizes, every activation, epilogue part and gradient, and DenseFFN."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def M():
    from _lib import build_and_import
    return build_and_import()


def draw(seed, T, n_in, n_out, dt):
    g = torch.Generator("cuda").manual_seed(seed)

    def n(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)
    return {"x": n(T, n_in), "w": n(n_out, n_in, std=n_in ** -0.5), "bias": n(n_out, std=0.5),
            "residual": n(T, n_out), "dy": n(T, n_out), "pre": n(T, n_out, std=1.5)}


def sum_steps(K, dt):
    """Bound on the error of a K-term fp32 sum over the sum of magnitudes, in steps of 2^-24:
    CUDA cores add 128 products in a chain and then K / 128 such sums; the tensor cores add 16
    products at a time, each add to 2^-22 at worst, and up to 16 splits."""
    return 128 + K / 128 + 8 if dt == torch.float32 else 4 * (K / 16 + 32)


def check_values(got, ref, size, K, dt, extra=0.0):
    tol = R.HALF[got.dtype] * ref.abs() + sum_steps(K, dt) * R.U32 * size + extra
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), (err - tol).max()


def check_forward(t, y, pre, act, with_bias, with_residual):
    bias = t["bias"] if with_bias else None
    residual = t["residual"] if with_residual else None
    ref, z = R.linear(t["x"], t["w"], bias, residual, act)
    size = t["x"].double().abs() @ t["w"].double().abs().t() + 1
    K, dt = t["x"].shape[1], t["x"].dtype
    # activations have slopes below 1.13 and their own fp32 error below 8 steps of 1 + |z|
    check_values(y, ref, 1.13 * size, K, dt, 8 * R.U32 * (1 + z.abs() + ref.abs()))
    if pre is not None:
        check_values(pre, z, size, K, dt)


SIZES = [("bf16", 1, 8, 8), ("bf16", 2, 72, 24), ("bf16", 8, 4104, 520), ("bf16", 5, 1024, 200), ("bf16", 3, 2048, 1032),
         ("bf16", 7, 2056, 2048),
         ("bf16", 9, 512, 264), ("f32", 4, 2052, 68), ("f32", 8, 260, 28), ("f32", 9, 64, 12), ("bf16", 1, 4096, 1000), ("bf16", 3, 1032, 136), ("bf16", 17, 128, 4096),
         ("bf16", 64, 2048, 2056), ("bf16", 128, 520, 256), ("bf16", 129, 264, 72),
         ("bf16", 200, 4096, 512), ("bf16", 300, 1000, 1528), ("bf16", 1000, 136, 776),
         ("bf16", 2500, 256, 4104),
         ("f32", 1, 4, 4), ("f32", 5, 1004, 36), ("f32", 65, 128, 132), ("f32", 200, 516, 260)]


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("dtype,T,n_in,n_out", SIZES)
def test_linear(M, dtype, T, n_in, n_out, act):
    dt = DT[dtype]
    t = draw(T + n_in, T, n_in, n_out, dt)
    d = M.make_linear(T, n_in, n_out, M.dtype_code(dt), act)
    ws = M.alloc_workspace(d)
    for bias, residual, keep in ((True, True, True), (False, False, False), (True, False, True)):
        big = torch.full((T + 2, n_out), float("nan"), dtype=dt, device="cuda")
        pre = torch.full_like(big, float("nan"))
        M.moe_linear(d, t["x"], t["w"], t["bias"] if bias else None,
                     t["residual"] if residual else None, pre[:T] if keep else None, big[:T], ws)
        check_forward(t, big[:T], pre[:T] if keep else None, act, bias, residual)
        assert torch.isnan(big[T:]).all() and torch.isnan(pre[T:]).all()
    # the residual's own buffer as the output
    y = t["residual"].clone()
    M.moe_linear(d, t["x"], t["w"], t["bias"], y, None, y, ws)
    check_forward(t, y, None, act, True, True)
    assert M.moe_check_status(ws) == 0


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("dtype,T,n_in,n_out", SIZES)
def test_linear_backward(M, dtype, T, n_in, n_out, act):
    dt = DT[dtype]
    t = draw(T + n_out, T, n_in, n_out, dt)
    d = M.make_linear(T, n_in, n_out, M.dtype_code(dt), act)
    ws = M.alloc_workspace(d)
    pre = t["pre"] if act != "none" else None
    nan = float("nan")

    def call(dx=True, dw=True, db=True):
        out = {"dx": torch.full((T, n_in), nan, dtype=dt, device="cuda") if dx else None,
               "dw": torch.full((n_out, n_in), nan, dtype=dt, device="cuda") if dw else None,
               "db": torch.full((n_out,), nan, device="cuda") if db else None}
        M.moe_linear_backward(d, t["dy"], t["x"] if dw else None, t["w"] if dx else None, pre,
                              out["dx"], out["dw"], out["db"], ws)
        return out
    got = call()
    dz = R.act_backward(t["dy"], t["pre"], act)
    x, w = t["x"].double(), t["w"].double()
    # dz is rounded once to the operand type, and errs by 16 steps of |dy| (1 + |z|) before
    slack = 0.0 if act == "none" else \
        R.HALF[dt] * dz.abs() + 16 * R.U32 * t["dy"].double().abs() * (1 + t["pre"].double().abs())
    size = dz.abs() + 1e-3
    check_values(got["dx"], dz @ w, size @ w.abs(), n_out, dt,
                 slack @ w.abs() if act != "none" else 0.0)
    check_values(got["dw"], dz.t() @ x, size.t() @ x.abs(), T, dt,
                 slack.t() @ x.abs() if act != "none" else 0.0)
    fine = 0.0 if act == "none" else \
        (16 * R.U32 * t["dy"].double().abs() * (1 + t["pre"].double().abs())).sum(dim=0)
    err = (got["db"].double() - dz.sum(dim=0)).abs()
    # chains of 8 rows, 8 slices, then T / 64 blocks in 8 strided chains
    assert (err <= (24 + T / 512) * R.U32 * dz.abs().sum(dim=0) + fine).all()
    for part in (dict(dx=False), dict(dw=False), dict(db=False), dict(dx=False, dw=False)):
        for k, v in call(**part).items():
            assert v is None or torch.equal(v, got[k]), (part, k)
    assert M.moe_check_status(ws) == 0


def test_linear_gradients_against_differences(M):
    """fp32, along random directions; the central difference with h = 1e-4 errs by
    h^2 f''' / 6, far below the 1e-4 of the sums of magnitudes allowed here."""
    T, n_in, n_out = 7, 20, 24
    t = draw(3, T, n_in, n_out, torch.float32)
    for act in ("gelu", "silu"):
        d = M.make_linear(T, n_in, n_out, M.MOE_F32, act)
        ws = M.alloc_workspace(d)
        y, pre = torch.empty_like(t["dy"]), torch.empty_like(t["dy"])
        M.moe_linear(d, t["x"], t["w"], t["bias"], None, pre, y, ws)
        out = {"x": torch.empty_like(t["x"]), "w": torch.empty_like(t["w"]),
               "bias": torch.empty_like(t["bias"])}
        M.moe_linear_backward(d, t["dy"], t["x"], t["w"], pre, out["x"], out["w"], out["bias"], ws)
        for name, grad in out.items():
            v = torch.randn_like(t[name]).double()

            def f(s):
                u = {k: a.double() for k, a in t.items()}
                u[name] = u[name] + s * v
                return (R.linear(u["x"], u["w"], u["bias"], None, act)[0] * u["dy"]).sum()
            diff = (f(1e-4) - f(-1e-4)) / 2e-4
            dot = (grad.double() * v).sum()
            assert (dot - diff).abs() <= 1e-4 * (grad.double().abs() * v.abs()).sum(), (act, name)


def test_linear_extreme_values(M):
    """Infinities pass through as in the definition; large |z| does not make the
    activations or their gradients NaN."""
    T, n = 4, 64
    for dtype in ("bf16", "f32"):
        dt = DT[dtype]
        x = torch.eye(T, n, device="cuda").to(dt)
        z = torch.linspace(-3e4, 3e4, n * n, device="cuda").view(n, n).to(dt)   # w[o, i] = z
        for act in ("gelu", "silu"):
            d = M.make_linear(T, n, n, M.dtype_code(dt), act)
            ws = M.alloc_workspace(d)
            y, pre = torch.empty(T, n, dtype=dt, device="cuda"), torch.empty(T, n, dtype=dt, device="cuda")
            M.moe_linear(d, x, z, None, None, pre, y, ws)
            assert torch.equal(pre, z[:, :T].t().contiguous())
            ref = R.act(pre.double(), act)
            assert ((y.double() - ref).abs() <= (R.HALF[dt] + 8 * R.U32) * ref.abs() + 1e-30).all()
            db = torch.empty(n, device="cuda")
            M.moe_linear_backward(d, torch.ones_like(y), None, None, pre, None, None, db, ws)
            assert torch.isfinite(db).all()


def test_linear_empty_batch(M):
    for dt in DT.values():
        d = M.make_linear(0, 64, 128, M.dtype_code(dt), "gelu")
        ws = M.alloc_workspace(d)
        e = draw(1, 0, 64, 128, dt)
        M.moe_linear(d, e["x"], e["w"], e["bias"], None, None, e["dy"], ws)
        dw, db = torch.ones_like(e["w"]), torch.ones(128, device="cuda")
        M.moe_linear_backward(d, e["dy"], e["x"], e["w"], e["pre"], torch.empty_like(e["x"]), dw, db, ws)
        assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T,n_in,n_out", [(1, 4096, 512), (40, 2048, 264), (300, 4096, 512)])
def test_linear_same_bits_every_time(M, T, n_in, n_out):
    """Products with reduction splits: repeated, captured twice with one workspace, and on
    another stream, the bits do not change."""
    t = draw(T, T, n_in, n_out, torch.bfloat16)
    d = M.make_linear(T, n_in, n_out, M.MOE_BF16, "gelu")
    ws = M.alloc_workspace(d)

    def call(out, stream=None):
        M.moe_linear(d, t["x"], t["w"], t["bias"], t["residual"], None, out["y"], ws, stream)
        M.moe_linear_backward(d, t["dy"], t["x"], t["w"], t["pre"], out["dx"], out["dw"], out["db"],
                              ws, stream)

    def new():
        return {"y": torch.zeros_like(t["dy"]), "dx": torch.zeros_like(t["x"]),
                "dw": torch.zeros_like(t["w"]), "db": torch.zeros(n_out, device="cuda")}
    ref = new()
    call(ref)
    outs = [new() for _ in range(4)]
    for o in outs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        g.replay()
        g.replay()
    call(outs[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(outs[3], side)
    side.synchronize()
    for o in outs:
        for k, v in ref.items():
            assert torch.equal(o[k], v), k
    assert M.moe_check_status(ws) == 0


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 70), ("bf16", 300), ("f32", 9)])
def test_dense_ffn(M, dtype, T):
    """Two layers with residual, and the chain of their gradients."""
    dt, H, D = DT[dtype], 256, 520
    g = torch.Generator("cuda").manual_seed(T)

    def n(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)
    w1, w2, b1, b2 = n(D, H, std=H ** -0.5), n(H, D, std=D ** -0.5), n(D, std=0.5), n(H, std=0.5)
    x, dy = n(T, H), n(T, H)
    ffn = M.DenseFFN(w1, w2, b1, b2, "silu")
    saved = ffn.saved_buffers(T)
    y = ffn(x, residual=x, saved=saved)
    assert torch.equal(y, ffn(x, residual=x))
    hidden, z = R.linear(x, w1, b1, None, "silu")
    check_values(saved["pre"], z, x.double().abs() @ w1.double().abs().t() + 1, H, dt)
    ref, _ = R.linear(saved["hidden"], w2, b2, x, "none")
    check_values(y, ref, saved["hidden"].double().abs() @ w2.double().abs().t() + 2, D, dt,
                 8 * R.U32 * ref.abs())
    got = ffn.backward(dy, x, saved)
    # d_hidden errs by its sum and a rounding, dz by that times the slope (< 1.1), by its own
    # fp32 error and a rounding; the sums over them carry those errors on
    x64, w64, h64, dy64 = x.double(), w1.double(), saved["hidden"].double(), dy.double()
    dh = dy64 @ w2.double()
    dz = R.act_backward(dh, saved["pre"], "silu")
    e_dh = R.HALF[dt] * dh.abs() + sum_steps(H, dt) * R.U32 * (dy64.abs() @ w2.double().abs())
    fine = 1.1 * e_dh + 16 * R.U32 * dh.abs() * (1 + saved["pre"].double().abs())
    e_dz = fine + R.HALF[dt] * (dz.abs() + fine)
    check_values(got["dx"], dz @ w64, dz.abs() @ w64.abs(), D, dt, e_dz @ w64.abs())
    check_values(got["dw1"], dz.t() @ x64, dz.abs().t() @ x64.abs(), T, dt, e_dz.t() @ x64.abs())
    check_values(got["dw2"], dy64.t() @ h64, dy64.abs().t() @ h64.abs(), T, dt)
    for k, v, e in (("db1", dz, fine), ("db2", dy64, 0 * dy64)):
        err = (got[k].double() - v.sum(dim=0)).abs()
        assert (err <= 32 * R.U32 * v.abs().sum(dim=0) + e.sum(dim=0)).all(), k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = ffn(x, residual=x, stream=side)
    side.synchronize()
    assert torch.equal(on_side, y)


def test_offsets_past_32_bits(M):
    """More than 2^31 elements of x: the last rows are what they are in a small batch."""
    T, n_in, n_out = (1 << 20) + 3, 2056, 40
    t = draw(2, 300, n_in, n_out, torch.bfloat16)
    x = torch.zeros((T, n_in), dtype=torch.bfloat16, device="cuda")
    x[-300:] = t["x"]
    d = M.make_linear(T, n_in, n_out, M.MOE_BF16, "gelu")
    ws = M.alloc_workspace(d)
    y = torch.empty((T, n_out), dtype=torch.bfloat16, device="cuda")
    M.moe_linear(d, x, t["w"], None, None, None, y, ws)
    check_forward(t, y[-300:], None, "gelu", False, False)
    assert (y[:-300] == 0).all()
    dy = torch.zeros_like(y)
    dy[-300:] = t["dy"]
    pre = torch.zeros_like(y)
    pre[-300:] = t["pre"]
    dx, dw = torch.empty_like(x), torch.empty_like(t["w"])
    M.moe_linear_backward(d, dy, x, t["w"], pre, dx, dw, None, ws)
    dz = R.act_backward(t["dy"], t["pre"], "gelu")
    slack = R.HALF[torch.bfloat16] * dz.abs() + \
        16 * R.U32 * t["dy"].double().abs() * (1 + t["pre"].double().abs())
    w64, x64 = t["w"].double(), t["x"].double()
    check_values(dx[-300:], dz @ w64, dz.abs() @ w64.abs(), n_out, torch.bfloat16, slack @ w64.abs())
    # zeros before the last rows add nothing: the sum errs as one of 300 terms
    check_values(dw, dz.t() @ x64, dz.abs().t() @ x64.abs(), 300, torch.bfloat16, slack.t() @ x64.abs())
    assert M.moe_check_status(ws) == 0
