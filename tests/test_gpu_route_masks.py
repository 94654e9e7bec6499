"""moe_route where fp32 scores are no help: finite masks whose softmax scores
underflow beside strong experts, logits whose 64-bit scores are equal, and biases
near the end of fp32's range. Choices equal the 64-bit definition's exactly."""
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


def test_one_strong_expert_in_a_group(M):
    rows = torch.tensor([[10., -200, 5, 4, 0, -1, 0, -1], [0, -1e9, -1e9, -1e9, -0.5, -1, -1.5, -2]])
    for bias in (None, torch.zeros(8)):
        same(M, rows[:1], bias, 1, score="softmax", groups=4, topk_groups=1, group_top=2)
        same(M, rows, bias, 2, score="softmax", groups=2, topk_groups=1, group_top=2)


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("mask", [-95.0, -104.0, -110.0, -1e4, -1e9, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("E,groups,kept,K", [(64, 8, 3, 8), (256, 8, 4, 8), (96, 4, 1, 6), (40, 8, 5, 3),
                                             (512, 2, 1, 16), (64, 1, 1, 8)])
def test_finite_masks(M, E, groups, kept, K, mask, group_top):
    """Groups with one survivor, with several and with none; masked logits equal or apart."""
    g = torch.Generator("cpu").manual_seed(E + K)
    T, size = 61, E // groups
    logits = torch.randn(T, groups, size, generator=g)
    order = torch.rand(T, groups, size, generator=g).argsort(dim=2).argsort(dim=2)
    left = torch.randint(0, 4, (T, groups, 1), generator=g)      # survivors of a group
    left[torch.arange(T), torch.randint(0, groups, (T,), generator=g), 0] = 1
    strong = (left == 1) & (order == 0)
    logits = torch.where(strong, logits + 4, logits)
    apart = torch.rand(T, groups, size, generator=g) * (torch.arange(T) % 2).view(T, 1, 1) * 3
    logits = torch.where(order >= left, torch.full_like(logits, mask) + apart, logits).view(T, E)
    lowest = torch.zeros(E)
    lowest[::2] = -0.5            # the most negative bias, on masked experts among others
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(E), lowest):
            same(M, logits, bias, K, score=score, groups=groups, topk_groups=kept,
                 group_top=min(group_top, size))


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


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (8, 3, 2), (8, 2, 1)])
def test_biases_near_the_end_of_fp32(M, score, groups, kept, top):
    """Finite biases whose sums leave fp32's range."""
    g = torch.Generator("cpu").manual_seed(groups)
    T, E, K = 20, 64, 8
    logits = torch.randn(T, E, generator=g)
    for low, high in ((1.8e38, 3.4e38), (-3.4e38, 3.4e38), (0.0, 3.4e38)):
        bias = (low + (high - low) * torch.rand(E, generator=g, dtype=torch.float64)).float()
        same(M, logits, bias, K, score=score, groups=groups, topk_groups=kept, group_top=top)
    for at in ([0, 5, 10, 35, 60], [1, 4], [4, 1], [9, 62], [17, 40, 41]):
        bias = torch.zeros(E)
        bias[at] = 3.4e38 - 1e37 * torch.arange(len(at))      # a few beyond the others
        for k in (2, K):
            same(M, logits, bias, k, score=score, groups=groups, topk_groups=kept, group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_past_fp32_in_different_places(M, score):
    """Sums past fp32's range at different places of their lanes, the largest not the first."""
    E = 512
    logits = torch.randn(9, E, generator=torch.Generator("cpu").manual_seed(1))
    at = torch.tensor([0, 17, 34, 51, 132, 149, 166, 183])
    bias = torch.zeros(E)
    bias[at] = 2.5e38 + 1e37 * torch.arange(8)
    for k in (1, 2):
        same(M, logits, bias, k, score=score)
        for top in (1, 2):
            same(M, logits, bias, k, score=score, groups=4, topk_groups=1, group_top=top)
            same(M, logits, bias, k, score=score, groups=2, topk_groups=1, group_top=top)
