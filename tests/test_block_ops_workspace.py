"""Workspaces that the block operators' calls refuse: the kernels would write past them
or to the host's memory. The refusals come before any launch."""
import pytest
import torch


@pytest.fixture(scope="module")
def M():
    from _lib import build_and_import
    return build_and_import()


def test_workspace_address(M):
    space = M._binding._space
    ws = torch.zeros(512, dtype=torch.uint8)
    assert space(ws, -1) == (ws.data_ptr(), 512)      # -1: what torch calls the host
    with pytest.raises(ValueError, match="is on cpu"):
        space(ws, 0)
    with pytest.raises(ValueError, match="contiguous"):
        space(ws[:1].expand(512), -1)
    with pytest.raises(ValueError, match="missing"):
        space(None, 0)


@pytest.mark.gpu
def test_calls_refuse_a_workspace_elsewhere(M):
    def n(*shape, dtype=torch.float32):
        return torch.ones(shape, dtype=dtype, device="cuda")
    lin, norm = M.make_linear(16, 64, 64, M.MOE_F32), M.make_norm(16, 64, M.MOE_F32)
    moe, route = M.make_desc(16, 128, 16, 2, 128, 0, M.MOE_F32), M.make_route(16, 16, 2)
    weights = M.make_weights(n(16, 128), n(16, 128, 128), n(16, 128, 128))
    x, w, b, y = n(16, 64), n(64, 64), n(64), torch.full((16, 64), -7.0, device="cuda")
    h, out = n(16, 128), torch.full((16, 128), -7.0, device="cuda")

    def calls(of):
        yield lambda: M.moe_linear(lin, x, w, None, None, None, y, of(lin))
        yield lambda: M.moe_linear_backward(lin, x, x, w, None, y, None, None, of(lin))
        yield lambda: M.moe_block_norm_backward(norm, x, x, x, None, None, None, b, y, None, None,
                                                None, None, of(norm))
        yield lambda: M.moe_layer_forward_routed(moe, route, weights, h, out, None, of(moe))
    for call in calls(lambda d: M.alloc_workspace(d, "cpu")):
        with pytest.raises(ValueError):
            call()
    for call in calls(lambda d: M.alloc_workspace(d)[:1].expand(1 << 24)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert (y == -7).all() and (out == -7).all()
    for call in calls(M.alloc_workspace):
        call()
    torch.cuda.synchronize()
    assert (y != -7).all() and (out != -7).all()


def test_descriptor_subclasses_have_a_workspace(M):
    for d in (M.make_desc(4, 128, 16, 2, 128, 0, M.MOE_F32), M.make_norm(4, 64), M.make_linear(4, 64, 64)):
        kind = type("Own", (type(d),), {})
        own = kind(*[getattr(d, name) for name, _ in type(d)._fields_])
        assert M.alloc_workspace(own, "cpu").numel() == M.alloc_workspace(d, "cpu").numel()
