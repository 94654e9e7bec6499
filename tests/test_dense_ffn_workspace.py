"""Whose workspace a DenseFFN call gets: without a GPU by a stand-in for the current
stream, and on one by calls that run at the same time."""
import re
import weakref

import pytest
import torch


@pytest.fixture(scope="module")
def M():
    from _lib import build_and_import
    return build_and_import()


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def now(monkeypatch):
    """The current stream and whether it is being captured."""
    state = {"stream": 0, "capturing": False}
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(state["stream"]))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    return state


def test_a_workspace_for_each_stream_and_capture(M, now):
    ffn = M.DenseFFN(torch.zeros(64, 32), torch.zeros(32, 64))
    a = ffn.workspace(8)
    assert (a[:M._binding.MOE_LINEAR_WS_HEAD] == 0).all()
    assert ffn.workspace(4) is a and ffn.workspace(8) is a
    now["stream"] = 7
    b = ffn.workspace(8)
    assert b.data_ptr() != a.data_ptr() and ffn.workspace(8) is b
    now["capturing"] = True
    c, d = ffn.workspace(8), ffn.workspace(8)
    assert len({t.data_ptr() for t in (a, b, c, d)}) == 4
    assert (c[:M._binding.MOE_LINEAR_WS_HEAD] == 0).all()
    now["capturing"] = False
    assert ffn.workspace(8) is b      # nothing of a capture is kept
    now["stream"] = 0
    assert ffn.workspace(8) is a


def test_an_outgrown_workspace_is_released(M, now):
    ffn = M.DenseFFN(torch.zeros(64, 32), torch.zeros(32, 64))
    old = weakref.ref(ffn.workspace(8))
    need = max(M.moe_linear_workspace_size(d) for d in ffn.descs(500))
    assert ffn.workspace(500).numel() >= need
    assert old() is None
    assert ffn.workspace(8).numel() >= need


def test_the_head_is_the_headers(M):
    import os
    from _lib import ROOT
    with open(os.path.join(ROOT, "include", "moe.h")) as f:
        n = re.search(r"#define MOE_LINEAR_WS_HEAD (\d+)", f.read())
    assert int(n.group(1)) == M._binding.MOE_LINEAR_WS_HEAD


def layer(M, T, H=2048, D=1032):
    """Shapes whose products share tiles between units."""
    g = torch.Generator("cuda").manual_seed(T)

    def n(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    ffn = M.DenseFFN(n(D, H, std=H ** -0.5), n(H, D, std=D ** -0.5), n(D), n(H), "gelu")
    return ffn, [(n(T, H), n(T, H)) for _ in range(2)]


def step(ffn, x, dy, stream=None):
    saved = ffn.saved_buffers(x.shape[0])
    y = ffn(x, residual=x, saved=saved, stream=stream)
    return {"y": y, **saved, **ffn.backward(dy, x, saved, stream)}


def equal(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 300])
def test_two_streams_at_once(M, T):
    ffn, inputs = layer(M, T)
    ref = [step(ffn, *i) for i in inputs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in inputs]
    fresh = layer(M, T)[0]            # both streams' first calls, too
    for f in (fresh, ffn):
        outs = [[], []]
        torch.cuda.synchronize()
        for _ in range(12):
            for s, i, o in zip(sides, inputs, outs):
                with torch.cuda.stream(s):
                    o.append(step(f, *i))
        torch.cuda.synchronize()
        for r, o in zip(ref, outs):
            assert all(equal(r, got) for got in o)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 300])
def test_graphs_beside_one_another_and_eager_calls(M, T):
    """Captured before any eager call, replayed on two streams beside eager calls."""
    ffn, inputs = layer(M, T)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(ffn, *i))
        graphs.append(g)
    ref = [step(ffn, *i) for i in inputs]       # no replay has run yet
    other = layer(M, T)[0]
    want = [step(other, *i) for i in inputs]
    assert all(equal(w, r) for w, r in zip(want, ref))
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in graphs]
    for _ in range(8):
        for s, g in zip(sides, graphs):
            with torch.cuda.stream(s):
                g.replay()
        again = step(ffn, *inputs[0])
    torch.cuda.synchronize()
    assert equal(want[0], again)
    assert all(equal(w, o) for w, o in zip(want, outs))
