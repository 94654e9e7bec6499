"""moe_route where fp32 scores are no help: logits whose 64-bit scores are equal.
Choices equal the 64-bit definition's exactly."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    from _lib import build_and_import
    return build_and_import()


def choice(M, logits, bias, K, **kw):
    """Indices by the kernel and by the definition; weights finite."""
    T, E = logits.shape
    d = M.make_route(T, E, K, **kw)
    idx = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), float("nan"), device="cuda")
    M.moe_route(d, logits.cuda(), bias.cuda() if bias is not None else None, idx, w)
    ref, ref_w = R.route(logits, bias, K, **kw)
    assert torch.isfinite(w).all()
    return idx.cpu().long(), ref, w.cpu().double(), ref_w


def same(M, logits, bias, K, **kw):
    idx, ref, w, ref_w = choice(M, logits, bias, K, **kw)
    assert torch.equal(idx, ref), (idx != ref).nonzero()[:5]
    return w, ref_w


@pytest.mark.parametrize("E", [32, 96, 128])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_equal_64_bit_scores_go_by_index(M, groups, kept, E):
    """Distinct logits whose 64-bit softmax scores are equal (|l| < 1e-18 beside a maximum of
    that size: exp gives 1) are chosen by index, among few of them and among many."""
    g = torch.Generator("cpu").manual_seed(5)
    T, K = 48, 6
    logits = -1 - torch.rand(T, E, generator=g)
    for t in range(T):
        at = torch.randperm(E, generator=g)[:2 + t % 9]
        logits[t, at] = 1e-18 * torch.rand(len(at), generator=g) * (-1.0) ** t
    same(M, logits, None, K, score="softmax", groups=groups, topk_groups=kept)
    same(M, logits, None, K, score="softmax", groups=groups, topk_groups=kept, renorm=False)


def test_scores_that_are_zero_in_64_bits_go_by_index(M):
    """Two experts in service whose scores underflow 64 bits too, behind one that counts."""
    logits = torch.full((6, 8), -float("inf"))
    logits[:, 2] = 1.0
    logits[:3, 0], logits[:3, 5] = -900.0, -800.0
    logits[3:, 0], logits[3:, 5] = -1e30, -2000.0
    same(M, logits, None, 2, score="softmax")
    same(M, logits, None, 3, score="softmax")
