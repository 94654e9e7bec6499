"""Refusals of the block operators, without a GPU: every bad argument is reported
before any launch, by the library or by the binding's own checks."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def M():
    from _lib import build_and_import
    return build_and_import()


@pytest.fixture(scope="module")
def buf():
    keep = ctypes.create_string_buffer(1 << 16)
    return keep, (ctypes.addressof(keep) + 255) & ~255


def ref(d):
    return ctypes.addressof(d)


def test_descriptor_layout_matches_header(M):
    assert ctypes.sizeof(M.MoERouteDesc) == 36 and M.MoERouteDesc.scale.offset == 32
    assert ctypes.sizeof(M.MoENormDesc) == 24 and M.MoENormDesc.alpha.offset == 20
    assert ctypes.sizeof(M.MoELinearDesc) == 20 and M.MoELinearDesc.act.offset == 16


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(K=0), 1), (dict(groups=0), 1), (dict(groups=5), 1),
    (dict(groups=4, topk_groups=5), 1), (dict(groups=4, topk_groups=0), 1), (dict(group_top=3), 1),
    (dict(group_top=0), 1), (dict(groups=64, group_top=2, topk_groups=64), 1),
    (dict(groups=32, topk_groups=1, K=3), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(K=17), 2), (dict(E=514), 2),
    (dict(groups=64, topk_groups=64), 2), (dict(T=1 << 30), 2)])
def test_route_refusals(M, buf, bad, status):
    kw = dict(T=8, E=64, K=4)
    kw.update(bad)
    d = M.make_route(**kw)
    p = buf[1]
    lib = M._binding.lib
    assert lib.moe_route(ref(d), p, None, p, p, None) == status
    assert lib.moe_route_backward(ref(d), p, p, p, p, None) == status


def test_route_pointers(M, buf):
    lib, p = M._binding.lib, buf[1]
    d = M.make_route(8, 64, 4)
    assert lib.moe_route(None, p, None, p, p, None) == 1
    for i in range(3):
        a = [p, p, p]
        for bad in (None, p + 4):
            a[i] = bad
            assert lib.moe_route(ref(d), a[0], None, a[1], a[2], None) == 1
    assert lib.moe_route(ref(d), p, p + 4, p, p, None) == 1
    for i in range(4):
        a = [p] * 4
        a[i] = None
        assert lib.moe_route_backward(ref(d), *a, None) == 1
    for field, value in (("score", 2), ("renorm", 2), ("score", -1)):
        e = M.make_route(8, 64, 4)
        setattr(e, field, value)
        assert lib.moe_route(ref(e), p, None, p, p, None) == 1
    empty = M.make_route(0, 64, 4)
    assert lib.moe_route(ref(empty), None, None, None, None, None) == 0
    with pytest.raises(ValueError):
        M.make_route(8, 64, 4, score="relu")


def test_routed_layer_refusals(M, buf):
    lib, p = M._binding.lib, buf[1]
    d = M.make_desc(8, 256, 16, 2, 512, 0, M.MOE_F32)
    w = M.MoELayerWeights(p, p, p, None, None, None)
    n = M.moe_workspace_size(d)
    for r in (M.make_route(9, 16, 2), M.make_route(8, 32, 2), M.make_route(8, 16, 3),
              M.make_route(8, 16, 2, groups=3)):
        assert lib.moe_layer_forward_routed(ctypes.byref(d), ref(r), ctypes.byref(w), p, p, None, p,
                                            n, None) == 1
    good = M.make_route(8, 16, 2)
    assert lib.moe_layer_forward_routed(ctypes.byref(d), None, ctypes.byref(w), p, p, None, p, n, None) == 1
    assert lib.moe_layer_forward_routed(ctypes.byref(d), ref(good), ctypes.byref(w), p, p, None, p,
                                        n - 1, None) == 3
    assert lib.moe_layer_forward_routed(ctypes.byref(d), ref(good), None, p, p, None, p, n, None) == 1
    assert lib.moe_combine_backward(ctypes.byref(d), p, p, p, None, p, p, None) == 1
    assert lib.moe_combine_backward(ctypes.byref(d), p, p + 4, p, p, p, p, None) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(dtype=3), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(alpha=float("inf")), 1), (dict(H=20), 2),
    (dict(H=16392), 2), (dict(T=(1 << 30) + 1), 2), (dict(H=8196, dtype=0), 2), (dict(H=6, dtype=0), 2)])
def test_norm_refusals(M, buf, bad, status):
    kw = dict(T=8, H=64, dtype=1)
    kw.update(bad)
    d = M.make_norm(**kw)
    lib, p = M._binding.lib, buf[1]
    assert lib.moe_norm_workspace_size(ref(d)) == 0
    assert lib.moe_block_norm(ref(d), p, None, None, None, p, None, p, None) == status
    assert lib.moe_block_norm_backward(ref(d), p, p, p, None, None, None, p, p, None, None, None, None, p,
                                       1 << 16, None) == status


def test_norm_parts(M, buf):
    lib, p = M._binding.lib, buf[1]
    d, g = M.make_norm(2, 64), M.make_norm(2, 64, gate="channel")

    def fwd(desc, h=p, y=None, w_post=None, gate=None, w_pre=None, h_out=None, x=None):
        return lib.moe_block_norm(ref(desc), h, y, w_post, gate, w_pre, h_out, x, None)
    assert fwd(d) == 1                                   # nothing to write
    assert fwd(d, h=None, w_pre=p, x=p) == 1
    assert fwd(d, w_pre=p) == 1 and fwd(d, x=p) == 1     # a norm without its output, or weights
    assert fwd(d, w_post=p, w_pre=p, x=p) == 1           # parts of a block output that is not there
    assert fwd(d, h_out=p, w_pre=p, x=p) == 1
    assert fwd(g, w_pre=p, x=p) == 1
    assert fwd(g, y=p, h_out=p) == 1 and fwd(d, y=p, gate=p, h_out=p) == 1
    assert fwd(d, h=p + 8, w_pre=p, x=p) == 1 and fwd(d, y=p + 2, h_out=p) == 1
    assert fwd(M.make_norm(0, 64), h=None) == 0
    names = "d_h_out d_x h_out y w_post gate w_pre d_h d_y d_w_post d_gate d_w_pre".split()
    n = M.moe_norm_workspace_size(g)

    def bwd(desc, ws=p, size=n, **kw):
        return lib.moe_block_norm_backward(ref(desc), *[kw.get(k) for k in names], ws, size, None)
    ok = dict(d_h_out=p, y=p, d_y=p)
    assert bwd(d, ws=None, **ok) == 3 and bwd(d, size=n - 1, **ok) == 3 and bwd(d, ws=p + 4, **ok) == 3
    for extra in (dict(w_pre=p), dict(w_pre=p, d_x=p), dict(d_x=p), dict(d_w_post=p), dict(d_gate=p),
                  dict(d_w_pre=p), dict(gate=p), dict(d_y=p + 4), dict(y=None), dict(y=None, d_y=None, w_post=p)):
        assert bwd(d, **{**ok, **extra}) == 1, extra
    assert bwd(g, **ok) == 1
    with pytest.raises(ValueError):
        M.make_norm(2, 64, gate="row")


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), 1), (dict(n_in=0), 1), (dict(n_out=-8), 1), (dict(dtype=2), 1), (dict(n_in=12), 2),
    (dict(n_out=20), 2), (dict(n_in=6, dtype=0), 2), (dict(T=(1 << 21) + 1), 2),
    (dict(n_in=(1 << 18) + 8), 2), (dict(n_out=(1 << 18) + 8), 2)])
def test_linear_refusals(M, buf, bad, status):
    kw = dict(T=8, n_in=64, n_out=64, dtype=1)
    kw.update(bad)
    d = M.make_linear(**kw)
    lib, p = M._binding.lib, buf[1]
    assert lib.moe_linear_workspace_size(ref(d)) == 0
    assert lib.moe_linear(ref(d), p, p, None, None, None, p, p, 1 << 16, None) == status
    assert lib.moe_linear_backward(ref(d), p, p, p, None, p, p, p, p, 1 << 16, None) == status


def test_linear_pointers(M, buf):
    lib, p = M._binding.lib, buf[1]
    d, a = M.make_linear(8, 64, 64), M.make_linear(8, 64, 64, act="gelu")
    n = M.moe_linear_workspace_size(a)
    assert 0 < M.moe_linear_workspace_size(d) <= n
    assert lib.moe_linear(ref(d), p, p, None, None, None, p, p, 255, None) == 3
    assert lib.moe_linear(ref(d), p, p, None, None, None, p, None, n, None) == 3
    for i in (0, 1, 5):
        q = [p, p, None, None, None, p]
        for bad in (None, p + 2):
            q[i] = bad
            assert lib.moe_linear(ref(d), *q, p, n, None) == 1
    for i in (2, 3, 4):
        q = [p, p, None, None, None, p]
        q[i] = p + 8
        assert lib.moe_linear(ref(d), *q, p, n, None) == 1
    bwd = lib.moe_linear_backward      # dy, x, w, pre, dx, dw, d_bias
    assert bwd(ref(d), p, None, p, None, p, p, None, p, n, None) == 1      # dw without x
    assert bwd(ref(d), p, p, None, None, p, None, None, p, n, None) == 1   # dx without w
    assert bwd(ref(a), p, p, p, None, p, p, p, p, n, None) == 1            # an activation without pre
    assert bwd(ref(d), p, p, p, p, p, p, p, p, n, None) == 1               # pre without one
    assert bwd(ref(d), None, p, p, None, p, p, p, p, n, None) == 1
    assert bwd(ref(d), p, p, p, None, p + 4, p, p, p, n, None) == 1
    e = M.make_linear(8, 64, 64)
    e.act = 3
    assert lib.moe_linear(ref(e), p, p, None, None, None, p, p, n, None) == 1
    with pytest.raises(ValueError):
        M.make_linear(8, 64, 64, act="tanh")


def test_linear_workspace_covers_every_product(M):
    """Sizes depend on the shape alone, grow with the batch inside one regime of
    reduction splits, and hold dz of the backward pass."""
    for T, i, o in ((1, 4096, 4096), (64, 4096, 14336), (4096, 4096, 14336)):
        plain = M.moe_linear_workspace_size(M.make_linear(T, i, o))
        act = M.moe_linear_workspace_size(M.make_linear(T, i, o, act="silu"))
        assert act - plain >= 2 * T * o
        assert plain == M.moe_linear_workspace_size(M.make_linear(T, i, o))


def test_binding_checks_tensors(M):
    """Types, shapes and layouts that the C ABI cannot see."""
    d = M.make_route(4, 16, 2)
    cpu = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        M.moe_route(d, cpu, None, cpu, cpu)
    arg = M._binding._arg
    with pytest.raises(ValueError, match="missing"):
        arg("x", None, (4, 16), torch.float32)
    with pytest.raises(ValueError, match="expected"):
        arg("x", cpu, (4, 8), torch.float32)
    with pytest.raises(ValueError, match="expected"):
        arg("x", cpu, (4, 16), torch.bfloat16)
    with pytest.raises(ValueError, match="contiguous"):
        arg("x", torch.zeros(16, 4).t(), (4, 16), torch.float32)
    with pytest.raises(ValueError, match="is on"):
        arg("x", cpu, (4, 16), torch.float32, torch.device("meta"))
    assert arg("x", None, (4, 16), torch.float32, optional=True) == 0
