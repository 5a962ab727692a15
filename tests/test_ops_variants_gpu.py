"""Every variant of the product kernels (MI355X only): which of them the cases reach is checked
against the rule of the choice, so that no later change of it leaves one untested."""
import numpy as np
import pytest
import torch

from product_rule import variant
from test_ops_exact_gpu import FORMATS, MANY, check, exact_packed, linear, signs, sums
from test_ops_gpu import DT, GROUP, extreme_scales, qa, random_packed, weight64  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS = [("row", mr, ks) for mr in (1, 2) for ks in (1, 2, 4)]
# one slice of 2048 values a wave and several; whole blocks and not
ROW_SHAPES = [(1, 300, 8192), (2, 300, 8192), (1, 300, 8229), (2, 90, 16500), (1, 5000, 4229), (2, 5000, 4229), (1, 8300, 2100),
              (2, 8200, 2085), (1, 40, 1), (2, 16, 33), (1, 4100, 4096), (2, 70, 4104)]
FEW_SHAPES = [(5, 66000, 72), (5, 66000, 71), (12, 12300, 1160), (9, 12300, 517), (3, 700, 8200), (7, 333, 8229), (16, 100, 264),
              (100, 5600, 520), (100, 5600, 517), (100, 2600, 4104), (100, 2600, 1031), (40, 64, 8200)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("gated", [False, True])
def test_one_or_two_rows(qa, fmt, dtype, gated):
    reached = set()
    for m, n, k in ROW_SHAPES:
        n = (n + 1) // 2 if gated else n
        v = variant(m, n, k, gated, fmt)
        print(f"{v} {fmt} {dtype} gated={gated} {m}x{n}x{k}", flush=True)
        blocks = -(-k // 128) * 4 if fmt == "asym4" else -(-k // 32)
        reached |= {v, v + ("panels",)} if blocks > 64 * v[2] else {v}
        linear(qa, fmt, dtype, gated, m, n, k)
    assert reached == set(ROWS) | {v + ("panels",) for v in ROWS}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("gated", [False, True])
def test_few_rows(qa, fmt, dtype, gated):
    reached = set()
    for m, n, k in FEW_SHAPES:
        n = (n + 1) // 2 if gated else n
        v = variant(m, n, k, gated, fmt)
        print(f"{v} {fmt} {dtype} gated={gated} {m}x{n}x{k}", flush=True)
        reached.add(v)
        linear(qa, fmt, dtype, gated, m, n, k)
    want = {("few", *v, a) for v in ((2, 8, 1), (2, 4, 2), (1, 4, 1), (1, 4, 4), (1, 2, 4)) for a in (True, False)}
    if not gated:
        want ^= {("few", 1, 2, 4, True), ("few", 1, 1, 4, True)}
    assert reached == want


def groups_of(experts, slots, seed):
    cuts = np.sort(np.random.default_rng(seed).integers(0, slots, experts - 1))
    return np.concatenate([[0], cuts, [slots - slots // 50]]).clip(0, slots - slots // 50).astype(np.int32)


# rows of y, experts, n, k
EXPERT_SHAPES = [(4, 3, 300, 8229), (7, 5, 5000, 520), (11, 3, 90, 8229), (10, 8, 1700, 4229), (64, 9, 700, 1031), (500, 40, 1100, 264),
                 (1600, 3, 4200, 72), (1600, 3, 4200, 71), (3000, 5, 4500, 136), (900, 3, 1500, 2056)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,gated", [("fp16", False), ("bf16", True)])
def test_experts(qa, fmt, dtype, gated):
    """Groups of all sizes, rows of x by number, some numbers out of range; rows of no expert."""
    reached = set()
    for slots, experts, n, k in EXPERT_SHAPES:
        n = (n + 1) // 2 if gated else n
        v = variant(slots, n, k, gated, fmt, experts=experts)
        print(f"{v} {fmt} {dtype} gated={gated} {slots} rows, {experts} experts, {n}x{k}", flush=True)
        reached.add(v[:1] + v[1:3] * (v[0] == "many"))
        wide = n * (2 if gated else 1)
        p = exact_packed(fmt, experts * wide, k, slots + n)
        tokens = max(1, slots // 2)
        x = signs(tokens, k, n)
        rng = np.random.default_rng(k)
        rows = rng.integers(0, tokens, slots).astype(np.int32)
        bad = rng.random(slots) < 0.05
        rows[bad] = rng.choice(np.array([-1, tokens, 2 ** 31 - 1, -(2 ** 31)], np.int32), bad.sum())
        off = groups_of(experts, slots, slots)
        xd, w = x.to(DT[dtype]).cuda(), torch.from_numpy(p.reshape(-1)).cuda()
        args = (fmt, xd, w, n, torch.from_numpy(off).cuda())
        y = qa.qr_experts(*args, rows=torch.from_numpy(rows).cuda(), gated=gated)
        assert torch.equal(y, qa.qr_experts(*args, rows=torch.from_numpy(rows).cuda(), gated=gated))
        gone = torch.from_numpy(bad).cuda()
        assert (y[gone] == 0).all() and (y[off[-1]:] == 0).all()
        kp = -(-k // GROUP[fmt]) * GROUP[fmt]
        for e in {0, experts // 2, experts - 1}:
            lo, hi = int(off[e]), int(off[e + 1])
            here = np.arange(lo, hi)[~bad[lo:hi]]
            if here.size:
                # the expert's rows from the tile that holds the first of them
                first = e * wide * kp
                values = torch.from_numpy(code_values(fmt, p, first, wide, k)).cuda()
                h = torch.mm(x[torch.from_numpy(rows[here]).long()].double().cuda(), values.t().contiguous())
                check(y[torch.from_numpy(here).cuda()], h, n, gated, dtype, (v, fmt, dtype, gated, e))
        nothing = qa.qr_experts(fmt, xd[:0], w, n, args[-1], rows=torch.from_numpy(rows).cuda(), gated=gated)
        assert (nothing == 0).all()
    assert reached == {("row",), ("few",), ("many", 64, 128), ("many", 128, 256)}


def code_values(fmt, packed, first, rows, k):
    """Rows of a weight that begin at padded value ``first``, in fp64."""
    kp = -(-k // GROUP[fmt]) * GROUP[fmt]
    tile = first // 2048
    part = packed[tile:-(-(first + rows * kp) // 2048)]
    total = part.shape[0] * 2048
    flat = weight64(fmt, part, 1, total, "fp16")[1].reshape(-1)
    return flat[first - tile * 2048:][:rows * kp].reshape(rows, kp)[:, :k]


TILES = {("many", 64, 128, True): (300, 9000), ("many", 64, 128, False): (300, 9000), ("many", 256, 128, True): (1300, 4500),
         ("many", 128, 256, True): (2050, 4500)}
assert list(TILES) == MANY


def shape_of(tile, k):
    m, n = TILES[tile]
    k += 0 if tile[3] else 3
    assert variant(m, n, k, False, "int4") == tile
    return m, n, k


@pytest.mark.parametrize("tile", MANY)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", sorted(DT))
def test_many_rows_extreme_scales(qa, fmt, dtype, tile):
    """Each value of W alone, for scales from the smallest subnormal to the largest: its own rounding."""
    m, n, k = shape_of(tile, 96)
    p = extreme_scales(fmt, n, k, 11)
    w = torch.from_numpy(weight64(fmt, p, n, k, dtype)[1]).to(DT[dtype]).cuda()
    cols = torch.from_numpy(np.random.default_rng(5).integers(0, k, m)).cuda()
    x = torch.zeros(m, k, dtype=DT[dtype], device="cuda")
    x[torch.arange(m, device="cuda"), cols] = 1
    y = qa.qr_linear(fmt, x, torch.from_numpy(p.reshape(-1)).cuda(), n)
    assert torch.equal(y, w[:, cols].t())


@pytest.mark.parametrize("rows,tile", [(9000, (64, 128)), (24700, (256, 128)), (33000, (128, 256))])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", sorted(DT))
def test_many_rows_read_the_codec_s_weights(qa, fmt, dtype, rows, tile):
    """Unit vectors read out what qr_decode returns, bit for bit."""
    k = 256
    assert variant(k, rows, k, False, fmt)[:3] == ("many", *tile)
    w = (torch.randn(rows, k, generator=torch.Generator().manual_seed(3)) * 0.1).to(DT[dtype]).cuda()
    p = qa.qr_encode_weight(fmt, w)
    y = qa.qr_linear(fmt, torch.eye(k, dtype=DT[dtype], device="cuda"), p, rows)
    n = -(-rows * k // 2048) * 2048
    assert torch.equal(y.t(), qa.qr_decode(fmt, p, n, DT[dtype])[:rows * k].view(rows, k))


@pytest.mark.parametrize("tile", MANY)
@pytest.mark.parametrize("fmt,dtype", [("int4", "bf16"), ("asym4", "fp16"), ("fp4", "bf16")])
def test_many_rows_as_parts_of_matrices(qa, fmt, dtype, tile):
    """x and y inside larger matrices, what lies around them not finite and kept; rows of x that are
    not finite stay the only ones; equal calls have equal results."""
    m, n, k = shape_of(tile, 136)
    p = exact_packed(fmt, n, k, 7)
    w = torch.from_numpy(p.reshape(-1)).cuda()
    off = 8 if tile[3] else 1
    big = torch.full((m, k + (24 if tile[3] else 6)), float("nan"), dtype=DT[dtype], device="cuda")
    x = big[:, off:off + k]
    assert (big.stride(0) % 8 == 0) == tile[3] or not tile[3]
    values = signs(m, k, 3)
    x.copy_(values.to(DT[dtype]))
    out = torch.full((m + 2, n + 5), 7.0, dtype=DT[dtype], device="cuda")
    y = out[1:-1, 3:3 + n]
    qa.qr_linear(fmt, x, w, n, y=y)
    check(y, sums(fmt, p, n, k, values), n, False, dtype, (tile, fmt, dtype))
    rest = out.clone()
    rest[1:-1, 3:3 + n] = 7.0
    assert (rest == 7.0).all()
    clean = y.clone()
    for _ in range(3):
        y.zero_()
        qa.qr_linear(fmt, x, w, n, y=y)
        assert torch.equal(y, clean)
    x[1, k // 2], x[m - 1, k - 1] = float("nan"), float("inf")
    qa.qr_linear(fmt, x, w, n, y=y)
    assert torch.equal(y[2:-1], clean[2:-1]) and torch.equal(y[0], clean[0]) and y[1].isnan().all()
    last = torch.from_numpy(weight64(fmt, p, n, k, dtype)[1][:, k - 1]).cuda()
    row = y[-1]
    assert (row[last > 0] == float("inf")).all() and (row[last < 0] == float("-inf")).all() and row[last == 0].isnan().all()
