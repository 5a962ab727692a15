"""How far the gates of a router's choice may be off: (d + 60) 2^-24 of a gate, d being how far its logit lies below the one
that its exponential is taken from (MI355X only)."""
import pytest
import torch

from test_rows_gpu import qa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,top,groups", [(8, 2, 1), (256, 8, 1), (256, 8, 8), (512, 16, 1), (1000, 64, 1), (160, 6, 20)])
@pytest.mark.parametrize("spread", [1.0, 12.0])
def test_gates_within_their_bound(qa, score, renormalise, E, top, groups, spread):
    gen = torch.Generator().manual_seed(E + top)
    logits = (torch.randn(600, E, generator=gen) * spread).cuda()
    bias = (torch.randn(E, generator=gen) * 0.2 - 1).cuda()
    for b in (None, bias):
        gates, ids = qa.qr_choose(logits, top, score=score, bias=b, groups=groups, top_groups=groups, group_best=1 + (groups > 1),
                                  renormalise=renormalise, factor=2.5)
        l = logits.double()
        low = l if score == "softmax" else l.clamp(max=0)
        chosen = ids.long()
        if renormalise:
            base = low.gather(1, chosen).amax(1, keepdim=True)
        else:
            base = low.amax(1, keepdim=True) if score == "softmax" else torch.zeros(len(l), 1, device="cuda").double()
        p = torch.exp(low - base) / (1 if score == "softmax" else 1 + torch.exp(-l.abs()))
        total = p.gather(1, chosen).sum(1, keepdim=True) if renormalise else p.sum(1, keepdim=True) if score == "softmax" else 1
        want, d = 2.5 * p.gather(1, chosen) / total, (base - low).gather(1, chosen)
        off = ((gates.double() - want).abs() - (d + 60) * 2.0 ** -24 * want - 2.0 ** -149).amax().item()
        assert off <= 0, (off, b is not None)
        print(f"{score} renormalise={renormalise} {E} top {top}: rms {((gates.double() - want) / want)[want > 2 ** -100].square().mean().sqrt().item():.2e}", flush=True)
