"""Routing plans of any size: their cost on the host, and large ones on an MI355X."""
import numpy as np
import pytest
import torch

from bit_quantized_all_amd import qr_ops


@pytest.mark.parametrize("experts", [1, 64, 256, 1024])
def test_counts_read_by_a_plan_are_bounded(experts):
    """Each workgroup of a large plan reads the counts of all of them, workspace bytes: all together
    stay within 2^30 bytes up to the largest plan there is."""
    L = qr_ops._lib()
    for slots in (4097, 1 << 18, (1 << 20) + 1, 1 << 23, (1 << 27) + 5, 1 << 30):
        ws = L.qr_route_workspace(slots, 1, experts)
        groups = ws // (4 * experts)
        assert ws == groups * 4 * experts and 1 < groups and groups * ws <= 1 << 30, (slots, groups)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,top,experts", [(1 << 19, 2, 1024), ((1 << 20) + 1, 1, 7), (3000017, 3, 200), ((1 << 24) + 3, 1, 1024)])
@pytest.mark.parametrize("dtype", [np.int32, np.int64])
def test_large_plans(tokens, top, experts, dtype):
    import bit_quantized_all_amd as qa
    from test_ops_gpu import plan
    rng = np.random.default_rng(tokens)
    ids = np.minimum(rng.geometric(3 / experts, (tokens, top)) - 1, experts).astype(dtype)   # experts: dropped
    ids[rng.random((tokens, top)) < 0.05] = -1
    got = qa.qr_route(torch.from_numpy(ids).cuda(), experts)
    for g, w, name in zip(got, plan(ids, experts), ("offsets", "rows", "pos")):
        assert np.array_equal(g.cpu().numpy(), w), name
