"""The router's choice where ranks, or the values of groups, lie nearer to each other than fp32 tells apart, and where biases
are negative, large or of either sign (MI355X only)."""
import pytest
import torch

from test_rows_gpu import check_choice, dev, log, qa  # noqa: F401

pytestmark = pytest.mark.gpu


def test_two_groups_below_zero(qa):
    """Both groups' largest ranks are -99.5 in fp32; in 64 bits that of the second is larger."""
    logits = torch.full((1, 8), -3.0)
    logits[0, 0], logits[0, 4] = 0.0, 1.2e-5
    bias = torch.full((8,), -100.0)
    for top in (1, 3):
        check_choice(qa, logits.cuda(), top, top, score="sigmoid", bias=bias.cuda(), groups=2, top_groups=1, best=1)
    assert qa.qr_choose(logits.cuda(), 1, score="sigmoid", bias=bias.cuda(), groups=2)[1].item() == 4


def near(experts, groups, best, level, score, seed, tokens=200):
    """Logits and a bias that put the ``best`` first ranks of every group at ``level``, a number or one for each of them,
    up to the bias's rounding and some 1e-4 of a logit, and all others 0.5 to 2.5 below."""
    gen = torch.Generator().manual_seed(seed)
    base, each = torch.randn(experts, generator=gen), experts // groups
    p = base.double()
    p = torch.sigmoid(p) if score == "sigmoid" else torch.softmax(p, 0)
    at = torch.rand(groups, each, generator=gen).argsort(1)[:, :best] + torch.arange(groups)[:, None] * each
    low = torch.as_tensor(level, dtype=torch.float64).min() - 0.5 - 2 * torch.rand(experts, generator=gen).double()
    rank = low.clone()
    rank[at] = torch.as_tensor(level, dtype=torch.float64).expand(groups, best)
    return base + 1e-4 * torch.randn(tokens, experts, generator=gen), (rank - p).float()


SHAPES = [(256, 8, 4, 2), (256, 8, 4, 1), (200, 10, 4, 2), (70, 5, 2, 1), (64, 16, 7, 2), (512, 2, 1, 2), (640, 20, 7, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("level", [0.3, -3.0, -50.0, -1000.0, -1e6])
@pytest.mark.parametrize("E,groups,top_groups,best", SHAPES)
def test_close_groups(qa, score, level, E, groups, top_groups, best):
    logits, bias = near(E, groups, best, level, score, E + groups)
    check_choice(qa, logits.cuda(), top_groups * best, (score, level, E), score=score, bias=bias.cuda(), groups=groups,
                 top_groups=top_groups, best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [30.0, 1000.0, 3e5])
@pytest.mark.parametrize("E,groups,top_groups", [(16, 8, 4), (256, 8, 4), (200, 10, 4), (32, 16, 8), (512, 2, 1), (640, 20, 7)])
def test_groups_whose_ranks_cancel(qa, score, size, E, groups, top_groups):
    """A group's two first ranks are near +size and -size, their sum is small and as far off in fp32 as they are."""
    logits, bias = near(E, groups, 2, [size, -size], score, E + groups)
    check_choice(qa, logits.cuda(), top_groups, (score, size, E), score=score, bias=bias.cuda(), groups=groups, top_groups=top_groups,
                 best=2)
    # and against groups whose ranks are small themselves: the error is the other group's
    other = near(E, groups, 2, [size, -size], score, E + groups)[1].view(groups, -1)
    plain = near(E, groups, 2, 0.0, score, E + groups)[1].view(groups, -1)
    other[::2] = plain[::2]
    check_choice(qa, logits.cuda(), top_groups, (score, size, E, "mixed"), score=score, bias=other.reshape(-1).cuda(), groups=groups,
                 top_groups=top_groups, best=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups", [(16, 4, 2), (16, 4, 4), (256, 8, 4), (200, 10, 9), (640, 20, 19)])
def test_biases_at_the_end_of_the_range(qa, score, E, groups, top_groups):
    """Two ranks whose sum is past fp32: a mask of the lowest value leaves its experts in, last, and large ones stay apart."""
    gen = torch.Generator().manual_seed(E)
    logits = torch.randn(40, E, generator=gen).cuda()
    each, big = E // groups, torch.finfo(torch.float32).max
    low = torch.randn(groups, each, generator=gen) * 0.1
    low[0] = low[2] = -big                                        # whole groups of it
    mixed = low.clone()
    mixed[1, 1:] = -big                                           # a group of one other
    high = low.clone()
    high[1, :2], high[2, :2], high[3, 0] = torch.tensor([3e38, 1e38]), torch.tensor([3e38, 2e38]), big
    ends = low.clone()
    ends[1, 0], ends[3, :2] = float("inf"), torch.tensor([big, big])
    only = torch.full((groups, each), -big)
    only[0] = -float("inf")                                       # no expert to be had, before groups of the lowest value
    kw = dict(score=score, groups=groups, top_groups=top_groups, best=2)
    for name, bias in (("low", low), ("mixed", mixed), ("high", high), ("ends", ends), ("only", only)):
        for top in (2, min(16, E)):
            check_choice(qa, logits, top, (name, top), bias=bias.reshape(-1).cuda(), **kw)


@pytest.mark.parametrize("E,groups,top_groups,best", [(256, 8, 4, 2), (64, 4, 2, 1), (200, 10, 4, 2), (512, 2, 1, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_a_token_does_not_depend_on_its_neighbours(qa, score, renormalise, E, groups, top_groups, best):
    """Bit for bit the same beside tokens whose choice fp32 leaves open, which are compared again in 64 bits."""
    kw = dict(score=score, groups=groups, top_groups=top_groups, group_best=best, renormalise=renormalise)
    gen = torch.Generator().manual_seed(E)
    logits = torch.randn(400, E, generator=gen) * 2
    close, bias = near(E, groups, best, -3.0, score, E, tokens=400)
    clear = qa.qr_choose(logits.cuda(), 4, bias=bias.cuda(), **kw)
    for first in range(4):
        mixed = logits.clone()
        mixed[first::4] = close[first::4]
        own = torch.arange(400) % 4 != first
        got = qa.qr_choose(mixed.cuda(), 4, bias=bias.cuda(), **kw)
        assert torch.equal(got[0][own], clear[0][own]) and torch.equal(got[1][own], clear[1][own]), first
        moved = qa.qr_choose(mixed.roll(1, 0).cuda(), 4, bias=bias.cuda(), **kw)
        assert torch.equal(moved[0].roll(-1, 0), got[0]) and torch.equal(moved[1].roll(-1, 0), got[1])
    alone = [qa.qr_choose(logits[i:i + 1].cuda(), 4, bias=bias.cuda(), **kw) for i in range(8)]
    assert torch.equal(torch.cat([g for g, _ in alone]), clear[0][:8]) and torch.equal(torch.cat([i for _, i in alone]), clear[1][:8])
