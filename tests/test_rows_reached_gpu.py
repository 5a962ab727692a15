"""Every variant of the kernels of the norm, the 8-bit rows and the router's choice (MI355X only): which of them the cases
reach is checked against the rules, so that no later change of those leaves one untested."""
import pytest
import torch

from rows_reference import DT
from rows_rule import choice, row_shape
from test_rows_gpu import LOGITS, SIZES, check_choice, log, qa, values  # noqa: F401

pytestmark = pytest.mark.gpu


def test_sizes_of_rows_reach_every_shape():
    """The sizes at which the norm and the 8-bit rows are compared with 64 bits."""
    assert {row_shape(*s) for s in SIZES} == {(1, 1), (1, 2), ("long",)} | {(w, c) for w in (4, 16) for c in (1, 2, 3, 4)}


# (groups, experts of a group): lanes hold them in whole runs of 1 to 32, in runs that are not full, and not at all
CHOICES = [(1, e) for e in (2, 16, 17, 32, 40, 64, 72, 128, 200, 256, 300, 512, 513)] \
    + [(2, e) for e in (1, 8, 16, 13, 32, 30, 64, 128, 100, 256, 240, 257)] + [(3, e) for e in (4, 7, 16, 11, 32, 64, 50, 128, 129)] \
    + [(4, e) for e in (2, 8, 9, 32, 64, 128, 70)] + [(7, e) for e in (2, 4, 8, 7, 16, 32, 21, 64, 65)] \
    + [(8, e) for e in (1, 2, 3, 32, 64)] + [(13, e) for e in (2, 3, 4, 5, 8, 16, 11, 32, 33)] + [(16, e) for e in (1, 2, 32)] + [(17, 3), (64, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_choices_reach_every_layout(qa, score, biased):
    reached = set()
    for i, (groups, each) in enumerate(CHOICES):
        experts, dtype = groups * each, sorted(LOGITS)[i % 3]
        best, top_groups = 1 if each < 2 else 1 + i % 2, max(1, groups * 2 // 3)
        top = min(experts, (1, 4, 8, 16)[i % 4])
        v = choice(experts, groups, top)
        log(f"{v} {dtype} {groups} groups of {each}, top {top} of {top_groups}, best {best}")
        reached.add(v)
        gen = torch.Generator().manual_seed(i)
        logits = (torch.randn(21, experts, generator=gen) * 2).to(LOGITS[dtype])
        logits[3, ::2] = -float("inf")
        logits[4] = -float("inf")
        bias = (torch.randn(experts, generator=gen) * 0.3 - 2).cuda() if biased else None
        check_choice(qa, logits.cuda(), top, (groups, each), score=score, bias=bias, groups=groups, top_groups=top_groups, best=best,
                     renormalise=i % 3 != 1)
    layouts = {("rows", run, span) for run in (1, 2, 4, 8, 16, 32) for span in (1, 2, 4, 8, 16)}
    assert {v[:3] for v in reached} == layouts | {("wave",)}
    assert {v[1] for v in reached if len(v) > 1 and v[1] != v[3]} == {4, 8, 16, 32}   # lanes that are not full
    assert choice(64, 1, 17) == ("wave",)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_norm_in_place_in_every_shape(qa, dtype):
    """The sum over the residual or over x, the result over the other one: nobody reads what another lane has written."""
    for rows, k in SIZES:
        x, r, w = values(rows, k, dtype, 1), values(rows, k, dtype, 2), values(1, k, dtype, 3)[0]
        log(f"norm in place {dtype} {rows}x{k} {row_shape(rows, k)}")
        codes, scales, total, y = qa.qr_norm_rows(x, w, residual=r, with_output=True)
        for first in (False, True):
            a, b = x.clone(), r.clone()
            got = qa.qr_norm_rows(a, w, residual=b, total=a if first else b, y=b if first else a)
            assert all(torch.equal(p, q) for p, q in zip(got, (codes, scales, total, y))), (rows, k, first)
