"""The operators over 4-bit weights against plain computations in 64 bits (MI355X only).

Tolerances follow from the operators' definitions.  A product multiplies by the
weights code value times scale, and with many rows by these rounded to the
call's dtype; it has to agree with one or the other throughout.  What remains
is the fp32 sum of k products (k 2^-23 of the sum of their magnitudes, which
also covers truncating adders; a format with a zero point may sum codes and
zero points apart, whose magnitudes are up to 15 and 15 steps), and one rounding
of the result (2^-11 of it for fp16, 2^-8 for bf16, half the smallest subnormal
below the normal range).  silu(g) * u passes the errors of g and u on with the
magnitudes of its derivatives, |silu'| <= 1.1, and adds its own evaluation
(|g| + 8 units of 2^-23).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}
GROUP = {"int4": 32, "asym4": 128, "fp4": 32}
TILE = {"int4": 1152, "asym4": 1072, "fp4": 1152}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


@pytest.fixture(scope="module")
def qa():
    import bit_quantized_all_amd as qa
    qa.lib()
    assert torch.cuda.is_available()
    return qa


def log(*a):
    print(*a, flush=True)


def random_packed(fmt, rows, k, seed, scale=0.05):
    """Packed bytes with every code and scales over several binades (zeros among
    them), as tiles on the host."""
    rng = np.random.default_rng(seed)
    kp = -(-k // GROUP[fmt]) * GROUP[fmt]
    tiles = -(-rows * kp // 2048)
    p = rng.integers(0, 256, (tiles, TILE[fmt]), dtype=np.uint8)
    groups = 2048 // GROUP[fmt]
    s = (scale * np.exp(rng.uniform(-3, 1, (tiles, groups)))).astype(np.float16)
    s[rng.random(s.shape) < 0.02] = 0
    p[:, 1024:1024 + 2 * groups] = s.view(np.uint8).reshape(tiles, -1)
    if fmt == "asym4":
        p[:, 1056:] = rng.integers(0, 16, (tiles, 16), dtype=np.uint8)
    return p


def weight64(fmt, packed, rows, k, dtype):
    """[rows, k] weight of packed tiles in fp64: rounded to the dtype, exact, and
    the magnitudes that the codes and the zero points have summed apart."""
    kp = -(-k // GROUP[fmt]) * GROUP[fmt]
    code = np.stack([packed[:, :1024] & 15, packed[:, :1024] >> 4], 2).reshape(-1, 2048)
    groups = 2048 // GROUP[fmt]
    s = np.ascontiguousarray(packed[:, 1024:1024 + 2 * groups]).view(np.float16).astype(np.float64)
    if fmt == "fp4":
        v = E2M1[code]
    elif fmt == "int4":
        v = code.astype(np.float64) - 8
    else:
        v = code.astype(np.float64) - np.repeat(packed[:, 1056:].astype(np.float64), 128, 1)
    def matrix(v):
        return (v * np.repeat(s, GROUP[fmt], 1)).reshape(-1)[:rows * kp].reshape(rows, kp)[:, :k]

    w = matrix(v)
    # value * scale has at most 15 significant bits: exact in fp32
    rounded = torch.from_numpy(w.astype(np.float32)).to(DT[dtype]).double().numpy()
    return rounded, w, np.abs(w) if fmt == "fp4" else matrix(code + (code - v))


def check_product(got, x, weights, n, gated, dtype, what):
    """got, x: device tensors; weights: what weight64() gives, of the rows in question."""
    x64, y = x.double().cpu().numpy(), got.double().cpu().numpy()
    rounded, exact, apart = weights
    found = [wrong(y, x64, w, mag, n, gated, dtype) for w, mag in ((rounded, np.abs(rounded)), (exact, apart))]
    assert any(not bad.any() for bad, _ in found), (what, [(np.argwhere(bad)[:4].tolist(), y[bad][:4], want[bad][:4],
                                                            int(bad.sum())) for bad, want in found])


def wrong(y, x64, w, mag, n, gated, dtype):
    """Which values of y are not silu(x w') etc. within the tolerance, and what is right."""
    k = x64.shape[1]
    h = x64 @ w.T
    err = k * 2.0 ** -23 * (np.abs(x64) @ mag.T)
    if gated:
        g, u, eg, eu = h[:, :n], h[:, n:], err[:, :n], err[:, n:]
        silu = g / (1 + np.exp(-np.clip(g, -700, 700)))
        want = silu * u
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + (np.abs(g) + 8) * 2.0 ** -23 * np.abs(want)
    else:
        want = h
    tol = err + HALF_ULP[dtype] * (np.abs(want) + err) + TINY[dtype]
    return ~(np.abs(y - want) <= tol), want


def activations(m, k, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k))
    x[rng.random((m, k)) < 0.01] *= 20
    return torch.from_numpy(x).to(DT[dtype]).cuda()


SHAPES = [(1, 1, 1), (1, 16, 32), (2, 17, 33), (3, 5, 127), (1, 256, 4096), (4, 70, 1000), (16, 64, 128), (17, 48, 160),
          (33, 100, 257), (5, 130, 2049), (64, 40, 96), (70, 64, 1000), (128, 256, 512), (257, 515, 640), (200, 33, 8191),
          (512, 384, 1024), (1030, 300, 392)]


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("gated", [False, True])
def test_linear(qa, fmt, dtype, gated):
    for m, n, k in SHAPES:
        log(f"linear {fmt} {dtype} gated={gated} {m}x{n}x{k}")
        wide = n * (2 if gated else 1)
        p = random_packed(fmt, wide, k, seed=m + n + k)
        x = activations(m, k, dtype, seed=m * n + k)
        assert qa.qr_weight_bytes(fmt, wide, k) == p.size
        y = qa.qr_linear(fmt, x, torch.from_numpy(p.reshape(-1)).cuda(), n, gated=gated)
        assert y.shape == (m, n) and y.dtype == DT[dtype]
        check_product(y, x, weight64(fmt, p, wide, k, dtype), n, gated, dtype, (fmt, dtype, gated, m, n, k))


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("m,n,k,gated", [(1300, 4500, 200, False), (1290, 2305, 136, True), (2050, 3001, 72, False)])
def test_linear_many_rows_and_columns(qa, fmt, dtype, m, n, k, gated):
    wide = n * (2 if gated else 1)
    p = random_packed(fmt, wide, k, seed=m)
    x = activations(m, k, dtype, seed=n)
    y = qa.qr_linear(fmt, x, torch.from_numpy(p.reshape(-1)).cuda(), n, gated=gated)
    check_product(y, x, weight64(fmt, p, wide, k, dtype), n, gated, dtype, (fmt, dtype, gated, m, n, k))


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("dtype,m,n,k,gated", [("bf16", 2050, 4500, 328, False), ("fp16", 4100, 2305, 136, True),
                                               ("fp16", 2305, 4200, 64, False), ("bf16", 1025, 5003, 456, False)])
def test_linear_many_tiles(qa, fmt, dtype, m, n, k, gated):
    """Above and below one large tile a CU; odd and even numbers of stages, whole and not."""
    wide = n * (2 if gated else 1)
    p = random_packed(fmt, wide, k, seed=m)
    x = activations(m, k, dtype, seed=n)
    y = qa.qr_linear(fmt, x, torch.from_numpy(p.reshape(-1)).cuda(), n, gated=gated)
    check_product(y, x, weight64(fmt, p, wide, k, dtype), n, gated, dtype, (fmt, dtype, gated, m, n, k))


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("dtype,gated", [("fp16", True), ("bf16", False)])
@pytest.mark.parametrize("m,n,k", [(12, 12300, 1160), (9, 12300, 1165), (5, 66000, 264), (5, 66000, 259), (30, 66000, 72),
                                   (30, 66000, 71), (20, 9000, 1288), (100, 2600, 1031), (3, 700, 4136), (7, 333, 2049)])
def test_linear_few_rows_many_columns(qa, fmt, dtype, gated, m, n, k):
    if gated:
        n = (n + 1) // 2
    wide = n * (2 if gated else 1)
    p = random_packed(fmt, wide, k, seed=m)
    x = activations(m, k, dtype, seed=n)
    y = qa.qr_linear(fmt, x, torch.from_numpy(p.reshape(-1)).cuda(), n, gated=gated)
    check_product(y, x, weight64(fmt, p, wide, k, dtype), n, gated, dtype, (fmt, dtype, gated, m, n, k))


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("dtype", sorted(DT))
def test_weights_are_the_codec_s(qa, fmt, dtype):
    """A packed weight is qr_encode's, and a unit vector reads out what qr_decode returns."""
    k, rows = 256, 64
    w = (torch.randn(rows, k, generator=torch.Generator().manual_seed(3)) * 0.1).to(DT[dtype]).cuda()
    p = qa.qr_encode_weight(fmt, w)
    assert torch.equal(p, qa.qr_encode(fmt, w.reshape(-1)))
    y = qa.qr_linear(fmt, torch.eye(k, dtype=DT[dtype], device="cuda"), p, rows)
    assert torch.equal(y.t(), qa.qr_decode(fmt, p, rows * k, DT[dtype]).view(rows, k))


@pytest.mark.parametrize("fmt", sorted(GROUP))
def test_encode_weight_pads_rows(qa, fmt):
    w = torch.randn(3, 5, 70, generator=torch.Generator().manual_seed(4)).half().cuda()
    kp = -(-70 // GROUP[fmt]) * GROUP[fmt]
    flat = torch.zeros(-(-15 * kp // 2048) * 2048, dtype=torch.float16, device="cuda")
    flat[:15 * kp].view(15, kp)[:, :70] = w.view(15, 70)
    assert torch.equal(qa.qr_encode_weight(fmt, w), qa.qr_encode(fmt, flat))


def extreme_scales(fmt, rows, k, seed):
    """Scales from the smallest subnormal to the largest finite fp16."""
    p = random_packed(fmt, rows, k, seed)
    groups = 2048 // GROUP[fmt]
    s = np.random.default_rng(seed).choice(np.array([0x0001, 0x0003, 0x03ff, 0x0400, 0x3c01, 0x7bff], np.uint16),
                                           (p.shape[0], groups))
    p[:, 1024:1024 + 2 * groups] = s.view(np.uint8).reshape(p.shape[0], -1)
    return p


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("m", [1, 40, 300])
def test_extreme_scales(qa, fmt, dtype, m):
    """Each value of W alone (one-hot rows of x): exact for every scale that leaves it finite."""
    n, k = 48, 384
    p = extreme_scales(fmt, n, k, 11)
    w = weight64(fmt, p, n, k, dtype)[0]
    cols = np.random.default_rng(5).integers(0, k, m)
    x = torch.zeros(m, k, dtype=DT[dtype])
    x[np.arange(m), cols] = 1
    y = qa.qr_linear(fmt, x.cuda(), torch.from_numpy(p.reshape(-1)).cuda(), n).double().cpu().numpy()
    # an infinite weight (fp16 overflow) times the other zeros of x is NaN throughout its column
    fine = np.isfinite(w).all(1)
    assert np.array_equal(y[:, fine], w[:, cols].T[:, fine])


@pytest.mark.parametrize("m", [1, 20, 300])
@pytest.mark.parametrize("k", [256, 250])
def test_strides_and_alignment(qa, m, k):
    """x and y as parts of larger matrices, from odd addresses; what lies around y stays."""
    n = 90
    p = random_packed("int4", n, k, 7)
    w = torch.from_numpy(p.reshape(-1)).cuda()
    for off, ldx, ldy in ((0, k + 8, n + 6), (1, k + 3, n + 1), (3, k + 1, n + 5)):
        big = torch.randn(m, ldx + off, generator=torch.Generator().manual_seed(off)).half().cuda()
        big[:, :off] = float("nan")
        big[:, off + k:] = float("nan")
        out = torch.full((m + 2, ldy + off), 7.0, dtype=torch.float16, device="cuda")
        x, y = big[:, off:off + k], out[1:-1, off:off + n]
        qa.qr_linear("int4", x, w, n, y=y)
        check_product(y, x, weight64("int4", p, n, k, "fp16"), n, False, "fp16", (m, k, off))
        rest = out.clone()
        rest[1:-1, off:off + n] = 7.0
        assert (rest == 7.0).all()


@pytest.mark.parametrize("m,n,k", [(5, 64, 333), (40, 64, 333), (300, 64, 333), (5, 66000, 72), (30, 66000, 72), (12, 12300, 600),
                                   (1300, 4500, 72), (2, 50, 4096)])
def test_not_finite_values_stay_in_their_row(qa, m, n, k):
    p = random_packed("asym4", n, k, 9)
    w = torch.from_numpy(p.reshape(-1)).cuda()
    x = activations(m, k, "bf16", 2)
    clean = qa.qr_linear("asym4", x, w, n)
    x[1, 17], x[m // 3 * 2, k - 1] = float("nan"), float("inf")
    y = qa.qr_linear("asym4", x, w, n)
    keep = [i for i in range(m) if i not in (1, m // 3 * 2)]
    assert torch.equal(y[keep], clean[keep])
    assert y[1].isnan().all()
    if m < 3:
        return
    # infinity times each weight that is not zero
    last = torch.from_numpy(weight64("asym4", p, n, k, "bf16")[0][:, k - 1]).cuda()
    row = y[m // 3 * 2]
    assert (row[last > 0] == float("inf")).all() and (row[last < 0] == float("-inf")).all() and row[last == 0].isnan().all()


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("dtype,gated", [("fp16", False), ("bf16", True)])
@pytest.mark.parametrize("k,off", [(200, 0), (136, 8), (203, 0), (71, 1), (64, 3)])
def test_linear_middle(qa, fmt, dtype, gated, k, off):
    """More small tiles than CUs, and few large ones; x that may pass to LDS directly and x
    that may not, as part of a larger matrix, with rows that are not finite."""
    m, n = 700, 3300 if not gated else 1601
    wide = n * (2 if gated else 1)
    p = random_packed(fmt, wide, k, seed=k)
    w = torch.from_numpy(p.reshape(-1)).cuda()
    big = torch.full((m, k + 24 + off), float("nan"), dtype=DT[dtype], device="cuda")
    out = torch.full((m + 2, n + 3), 7.0, dtype=DT[dtype], device="cuda")
    x, y = big[:, off:off + k], out[1:-1, 1:1 + n]
    x.copy_(activations(m, k, dtype, seed=off))
    qa.qr_linear(fmt, x, w, n, gated=gated, y=y)
    check_product(y, x, weight64(fmt, p, wide, k, dtype), n, gated, dtype, (fmt, dtype, gated, k, off))
    rest = out.clone()
    rest[1:-1, 1:1 + n] = 7.0
    assert (rest == 7.0).all()
    clean = y.clone()
    x[1, k // 2], x[m - 1, k - 1] = float("nan"), float("inf")
    qa.qr_linear(fmt, x, w, n, gated=gated, y=y)
    assert torch.equal(y[2:-1], clean[2:-1]) and torch.equal(y[0], clean[0])
    assert y[1].isnan().all() and not y[-1].isfinite().all()


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def check_experts(qa, fmt, dtype, gated, sizes, n, k, tail, gather, seed):
    experts, rng = len(sizes), np.random.default_rng(seed)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    slots = int(offsets[-1]) + tail
    wide = n * (2 if gated else 1)
    p = random_packed(fmt, experts * wide, k, seed)
    w = weight64(fmt, p, experts * wide, k, dtype)
    tokens = max(1, slots // 2) if gather else slots
    x = activations(tokens, k, dtype, seed)
    rows = rng.integers(0, tokens, slots).astype(np.int32) if gather else None
    y = torch.full((slots, n), float("nan"), dtype=DT[dtype], device="cuda")
    qa.qr_experts(fmt, x, torch.from_numpy(p.reshape(-1)).cuda(), n, torch.from_numpy(offsets).cuda(),
                  rows=None if rows is None else torch.from_numpy(rows).cuda(), gated=gated, y=y)
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            xe = x[torch.from_numpy(rows[lo:hi]).long().cuda()] if gather else x[lo:hi]
            check_product(y[lo:hi], xe, [v[e * wide:(e + 1) * wide] for v in w], n, gated, dtype, (fmt, dtype, gated, e, n, k))
    assert (y[offsets[-1]:] == 0).all()


GROUPS = [[1], [0, 3, 0], [5, 0, 1, 70, 0, 16], [1] * 70, [0] * 65 + [9], [300, 2, 0, 40], [17, 16, 15, 33, 64, 65, 128, 129]]


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("gated", [False, True])
def test_experts(qa, fmt, dtype, gated):
    for i, sizes in enumerate(GROUPS):
        for n, k, tail, gather in ((33, 160, 0, True), (70, 129, 19, False), (64, 256, 3, True)):
            log(f"experts {fmt} {dtype} gated={gated} {sizes[:8]} n={n} k={k} tail={tail} gather={gather}")
            check_experts(qa, fmt, dtype, gated, sizes, n, k, tail, gather, seed=i)


@pytest.mark.parametrize("fmt", sorted(GROUP))
def test_experts_many_rows(qa, fmt):
    check_experts(qa, fmt, "bf16", True, [700, 0, 1, 513, 256], 272, 544, 300, True, seed=3)
    check_experts(qa, fmt, "fp16", False, [700, 0, 1, 513, 256], 1001, 333, 300, True, seed=4)
    check_experts(qa, fmt, "bf16", True, [700, 0, 1, 513, 256], 2500, 88, 300, True, seed=5)
    check_experts(qa, fmt, "fp16", False, [700, 0, 1, 513, 256], 5003, 104, 300, False, seed=6)


@pytest.mark.parametrize("fmt", sorted(GROUP))
@pytest.mark.parametrize("gated", [False, True])
def test_experts_many_small_groups(qa, fmt, gated):
    rng = np.random.default_rng(7)
    sizes = [int(v) for v in rng.poisson(8, 64)]
    check_experts(qa, fmt, "bf16", gated, sizes, 1100, 136, 5, True, seed=7)
    check_experts(qa, fmt, "fp16", gated, [3 * v for v in sizes[:40]], 2601, 77, 9, True, seed=8)
    check_experts(qa, fmt, "fp16", gated, [20, 0, 31, 5], 700, 1033, 0, False, seed=9)


def test_experts_all_rows_dropped(qa):
    p = random_packed("int4", 4 * 32, 64, 1)
    y = torch.full((50, 32), float("nan"), dtype=torch.float16, device="cuda")
    qa.qr_experts("int4", activations(50, 64, "fp16", 1), torch.from_numpy(p.reshape(-1)).cuda(), 32,
                  torch.zeros(5, dtype=torch.int32, device="cuda"), y=y)
    assert (y == 0).all()


@pytest.mark.parametrize("size", [4, 400])
def test_experts_numbers_out_of_range(qa, size):
    """Row numbers outside x give rows of zeros; offsets out of order or range stay inside the buffers."""
    n, k, experts = 40, 96, 3
    p = random_packed("fp4", experts * n, k, 5)
    w = torch.from_numpy(p.reshape(-1)).cuda()
    x = activations(7, k, "fp16", 6)
    slots = 3 * size
    rows = torch.arange(slots, dtype=torch.int32, device="cuda") % 7
    offsets = torch.tensor([0, size, 2 * size, 3 * size], dtype=torch.int32, device="cuda")
    want = qa.qr_experts("fp4", x, w, n, offsets, rows=rows)
    bad = rows.clone()
    bad[1], bad[size], bad[-1] = -1, 7, 2 ** 31 - 1
    y = qa.qr_experts("fp4", x, w, n, offsets, rows=bad)
    gone = torch.zeros(slots, dtype=torch.bool, device="cuda")
    gone[1] = gone[size] = gone[-1] = True
    assert (y[gone] == 0).all() and torch.equal(y[~gone], want[~gone])
    nothing = qa.qr_experts("fp4", x[:0], w, n, offsets, rows=rows)
    assert (nothing == 0).all()
    out = torch.full((slots + 2, n), 7.0, dtype=torch.float16, device="cuda")
    for o in ([-5, size, size - 3, 2 ** 31 - 1], [2 ** 31 - 1] * 4, [-(2 ** 31)] * 4, [3, 2, 1, 0]):
        qa.qr_experts("fp4", x, w, n, torch.tensor(o, dtype=torch.int32, device="cuda"), rows=rows, y=out[1:-1])
        assert (out[0] == 7).all() and (out[-1] == 7).all()


def test_experts_beyond_32_bit_offsets(qa):
    """A weight of more than 2^32 bytes, and rows of y more than 2^32 bytes apart."""
    experts, n, k, fmt = 260, 4096, 8192, "int4"
    kept = (0, 131, 259)
    one = n * k // 2048 * TILE[fmt]
    w = torch.empty(experts * one, dtype=torch.uint8, device="cuda")
    parts = {}
    for e in kept:
        parts[e] = random_packed(fmt, n, k, e)
        w[e * one:(e + 1) * one] = torch.from_numpy(parts[e].reshape(-1)).cuda()
    offsets = torch.zeros(experts + 1, dtype=torch.int32)
    for e in kept:
        offsets[e + 1:] += 2
    x = activations(6, k, "fp16", 8)
    ld = 3 << 28
    y = torch.empty(5 * ld + n, dtype=torch.float16, device="cuda").as_strided((6, n), (ld, 1))
    qa.qr_experts(fmt, x, w, n, offsets.cuda(), y=y)
    for i, e in enumerate(kept):
        check_product(y[2 * i:2 * i + 2].contiguous(), x[2 * i:2 * i + 2], weight64(fmt, parts[e], n, k, "fp16"), n,
                      False, "fp16", e)


# ---------------------------------------------------------------------------
# routing plan and combination
# ---------------------------------------------------------------------------

def plan(ids, experts):
    flat = ids.reshape(-1).astype(np.int64)
    kept = (flat >= 0) & (flat < experts)
    order = np.argsort(np.where(kept, flat, experts), kind="stable")[:kept.sum()]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=experts))])
    rows = np.full(flat.size, -1)
    rows[:order.size] = order // ids.shape[1]
    pos = np.full(flat.size, -1)
    pos[order] = np.arange(order.size)
    return offsets, rows, pos.reshape(ids.shape)


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("tokens,top,experts", [(0, 2, 8), (1, 1, 1), (1, 2, 8), (7, 3, 5), (64, 8, 64), (65, 1, 1024),
                                                (1000, 4, 40), (1024, 8, 7), (1025, 8, 256), (4097, 2, 3), (9000, 5, 129),
                                                (32768, 8, 256), (100001, 1, 1000), (8192, 64, 64)])
def test_route(qa, dtype, tokens, top, experts):
    log(f"route {tokens} {top} {experts} {dtype}")
    rng = np.random.default_rng(tokens + experts)
    for kind in ("even", "skewed", "dropped", "one", "none"):
        if kind == "even":
            ids = rng.integers(0, experts, (tokens, top))
        elif kind == "skewed":
            ids = np.minimum(rng.geometric(0.3, (tokens, top)) - 1, experts - 1)
        elif kind == "dropped":
            ids = rng.integers(-2, experts + 2, (tokens, top))
            ids[rng.random((tokens, top)) < 0.1] = 2 ** 31 - 1
        elif kind == "one":
            ids = np.full((tokens, top), experts - 1)
        else:
            ids = np.full((tokens, top), -(2 ** 31))
        ids = ids.astype(dtype)
        if dtype is np.int64 and kind == "dropped":
            ids[rng.random((tokens, top)) < 0.05] = 1 << 32
        got = qa.qr_route(torch.from_numpy(ids).cuda(), experts)
        for g, w, name in zip(got, plan(ids, experts), ("offsets", "rows", "pos")):
            assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w), (kind, name)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("tokens,top,n", [(1, 1, 1), (3, 2, 7), (5, 8, 8), (64, 8, 2048), (33, 3, 1001), (1000, 5, 96),
                                          (2, 64, 4100), (700, 1, 20)])
def test_combine(qa, dtype, tokens, top, n):
    rng = np.random.default_rng(tokens + n)
    slots = tokens * top
    pos = rng.permutation(slots).astype(np.int32).reshape(tokens, top)
    pos[rng.random((tokens, top)) < 0.2] = -1
    pos[rng.random((tokens, top)) < 0.1] = slots
    pos[0] = -1
    gates = rng.standard_normal((tokens, top)).astype(np.float32)
    gates[pos < 0] = np.nan   # a dropped slot's gate is not looked at
    y = torch.from_numpy(rng.standard_normal((slots, n))).to(DT[dtype]).cuda()
    for off in (0, 1):
        ys = torch.empty(slots, n + off, dtype=DT[dtype], device="cuda")[:, off:]
        ys.copy_(y)
        big = torch.full((tokens + 2, n + off), 7.0, dtype=DT[dtype], device="cuda")
        out = big[1:-1, off:]
        assert qa.qr_combine(ys, torch.from_numpy(pos).cuda(), torch.from_numpy(gates).cuda(), out=out) is out
        y64 = y.double().cpu().numpy()
        want, mag = np.zeros((tokens, n)), np.zeros((tokens, n))
        for j in range(top):
            here = (pos[:, j] >= 0) & (pos[:, j] < slots)
            term = gates[here, j].astype(np.float64)[:, None] * y64[pos[here, j]]
            want[here] += term
            mag[here] += np.abs(term)
        err = top * 2.0 ** -23 * mag
        tol = err + HALF_ULP[dtype] * (np.abs(want) + err) + TINY[dtype]
        got = out.double().cpu().numpy()
        assert (np.abs(got - want) <= tol).all()
        assert (got[0] == 0).all()
        assert (big[0] == 7).all() and (big[-1] == 7).all() and (big[:, :off] == 7).all()


def test_combine_spreads_what_is_not_finite_by_row_only(qa):
    y = torch.ones(4, 16, dtype=torch.float16, device="cuda")
    y[2] = float("inf")
    pos = torch.tensor([[0, 1], [2, 3], [3, -1]], dtype=torch.int32, device="cuda")
    out = qa.qr_combine(y, pos, torch.full((3, 2), 0.5, device="cuda"))
    assert (out[0] == 1).all() and out[1].isinf().all() and (out[2] == 0.5).all()


def test_combine_beyond_32_bit_offsets(qa):
    ld, n = 3 << 28, 100
    y = torch.empty(5 * ld + n, dtype=torch.float16, device="cuda").as_strided((6, n), (ld, 1))
    y.copy_(torch.arange(6, device="cuda").half()[:, None].expand(6, n))
    out = torch.empty(2 * ld + n, dtype=torch.float16, device="cuda").as_strided((3, n), (ld, 1))
    pos = torch.tensor([[5, 0], [4, 1], [3, 2]], dtype=torch.int32, device="cuda")
    qa.qr_combine(y, pos, torch.tensor([[1.0, 2.0]] * 3, device="cuda"), out=out)
    assert torch.equal(out[:, 7].cpu(), torch.tensor([5.0, 6.0, 7.0]).half())


# ---------------------------------------------------------------------------
# together: streams, graphs, repeated calls
# ---------------------------------------------------------------------------

def layer(qa, x, ids, gates, w1, w2, fmt, inner, experts, stream=None):
    offsets, rows, pos = qa.qr_route(ids, experts, stream=stream)
    h = qa.qr_experts(fmt, x, w1, inner, offsets, rows=rows, gated=True, stream=stream)
    y = qa.qr_experts(fmt, h, w2, x.shape[1], offsets, stream=stream)
    return qa.qr_combine(y, pos, gates, stream=stream)


def layer_inputs(qa, tokens, k, inner, experts, top, fmt, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, k, generator=gen).half().cuda()
    w1 = qa.qr_encode_weight(fmt, (torch.randn(experts, 2 * inner, k, generator=gen) / k ** 0.5).half().cuda())
    w2 = qa.qr_encode_weight(fmt, (torch.randn(experts, k, inner, generator=gen) / inner ** 0.5).half().cuda())
    gates, ids = torch.softmax(torch.randn(tokens, experts, generator=gen), 1).topk(top, 1)
    ids[tokens // 2] = -1
    return x, ids.cuda(), gates.contiguous().cuda(), w1, w2


@pytest.mark.parametrize("tokens", [3, 50, 900])
def test_repeated_calls_give_the_same_bits(qa, tokens):
    a = layer_inputs(qa, tokens, 512, 192, 9, 3, "asym4", tokens)
    first = layer(qa, *a, "asym4", 192, 9)
    assert (first[tokens // 2] == 0).all() and first.isfinite().all()
    for _ in range(5):
        assert torch.equal(layer(qa, *a, "asym4", 192, 9), first)


@pytest.mark.parametrize("tokens", [4, 3000])
def test_other_stream(qa, tokens):
    """Calls on a stream of their own, whose results the current stream waits for."""
    a = layer_inputs(qa, tokens, 256, 128, 8, 4, "int4", 1)
    want = layer(qa, *a, "int4", 128, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        got = layer(qa, *a, "int4", 128, 8, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, want)
        del got
    with torch.cuda.stream(s):
        got = layer(qa, *a, "int4", 128, 8)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("tokens", [4, 3000])
def test_in_a_graph(qa, tokens):
    x, ids, gates, w1, w2 = layer_inputs(qa, tokens, 256, 128, 8, 4, "fp4", 2)
    xs, ids2 = [x.clone(), x.flip(0).contiguous()], ids.flip(0).contiguous()
    want = [layer(qa, xs[0], ids, gates, w1, w2, "fp4", 128, 8), layer(qa, xs[1], ids2, gates, w1, w2, "fp4", 128, 8)]
    static_x, static_ids = x.clone(), ids.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(qa, static_x, static_ids, gates, w1, w2, "fp4", 128, 8)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(qa, static_x, static_ids, gates, w1, w2, "fp4", 128, 8)
    for i in (0, 1, 1, 0, 1):
        static_x.copy_(xs[i])
        static_ids.copy_((ids, ids2)[i])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        eager = layer(qa, xs[1 - i], (ids2, ids)[i], gates, w1, w2, "fp4", 128, 8)
        assert torch.equal(eager, want[1 - i])


def test_no_rows(qa):
    p = torch.from_numpy(random_packed("int4", 32, 64, 1).reshape(-1)).cuda()
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    assert qa.qr_linear("int4", x, p, 32).shape == (0, 32)
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    offsets, rows, pos = qa.qr_route(ids, 1)
    assert (offsets == 0).all()
    y = qa.qr_experts("int4", x, p, 32, offsets, rows=rows)
    assert y.shape == (0, 32)
    assert qa.qr_combine(y, pos, torch.empty(0, 2, device="cuda")).shape == (0, 32)
    # tokens but nothing to combine
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    assert (qa.qr_combine(y, none, torch.ones(3, 2, device="cuda")) == 0).all()


def test_refusals(qa):
    p = torch.from_numpy(random_packed("int4", 32, 64, 1).reshape(-1)).cuda()
    x = activations(4, 64, "fp16", 1)
    ok = dict(fmt="int4", x=x, w=p, n=32)
    for change in (dict(fmt="int3"), dict(fmt="int8"), dict(fmt="int5"), dict(x=x.float()), dict(x=x[0]), dict(x=x.cpu()),
                   dict(x=x.t()), dict(x=x[:1].expand(4, 64)), dict(n=0), dict(n=3000), dict(w=p[:-1]), dict(w=p.cpu()),
                   dict(x=x[:, :0]), dict(gated=True, n=2000), dict(y=torch.empty(3, 32, dtype=x.dtype, device="cuda")),
                   dict(y=torch.empty(4, 31, dtype=x.dtype, device="cuda")), dict(y=torch.empty(4, 32, device="cuda"))):
        with pytest.raises(ValueError):
            qa.qr_linear(**{**ok, **change})
    with pytest.raises(qa.QRError):
        qa.qr_linear("int4", x, p[1:].contiguous()[:0].new_empty(p.numel() + 16)[1:p.numel() + 1], 32)
    buf = torch.zeros(4, 96, dtype=torch.float16, device="cuda")
    with pytest.raises(qa.QRError) as e:
        qa.qr_linear("int4", buf[:, :64], p, 32, y=buf[:, 32:64])
    assert e.value.status == qa.QR_ERR_ALIAS
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for change in (dict(offsets=off.long()), dict(offsets=off[:1]), dict(rows=torch.zeros(4, device="cuda")),
                   dict(rows=torch.zeros(4, dtype=torch.int32)), dict(offsets=torch.zeros(9, dtype=torch.int32,
                                                                                         device="cuda"), n=32000)):
        with pytest.raises(ValueError):
            qa.qr_experts(**{**ok, "offsets": off, **change})
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for bad in (dict(ids=ids.float()), dict(ids=ids[0]), dict(ids=ids.cpu()), dict(ids=ids.t()), dict(experts=0),
                dict(ids=ids[:, :0]), dict(pos=ids.long()), dict(rows=ids[0])):
        with pytest.raises(ValueError):
            qa.qr_route(**{**dict(ids=ids, experts=4), **bad})
    with pytest.raises(qa.QRError):
        qa.qr_route(ids, 1025)
    with pytest.raises(qa.QRError) as e:
        qa.qr_route(ids, 4, pos=ids)
    assert e.value.status == qa.QR_ERR_ALIAS
    gates = torch.ones(4, 2, device="cuda")
    for bad in (dict(y=x.float()), dict(y=x[0]), dict(pos=ids.long()), dict(gates=gates.half()), dict(gates=gates[:2]),
                dict(out=x[:3]), dict(out=x.bfloat16()), dict(gates=gates.t())):
        with pytest.raises(ValueError):
            qa.qr_combine(**{**dict(y=x, pos=ids, gates=gates), **bad})
    with pytest.raises(qa.QRError) as e:
        qa.qr_combine(x, ids, gates, out=x)
    assert e.value.status == qa.QR_ERR_ALIAS


@pytest.mark.parametrize("fmt", sorted(GROUP))
def test_example_layer(qa, fmt):
    """The tensor-parallel layer of examples/, against the same layer in fp32.  Quantized
    weights differ by up to half a step: a block of 32 normal values has a step of its
    largest value (near 2.3 standard deviations) / 8, a group of 128 (2 x 2.6) / 15, that
    is 0.29 and 0.35, uniform errors of 0.08 and 0.10 of a value; FP4's steps are 0.5 to 2 of
    its largest value / 6, near 0.12.  Two layers of them, and the 8-bit wire, stay
    under twice the larger of these."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tensor_parallel_moe.py")
    spec = importlib.util.spec_from_file_location("tensor_parallel_moe", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    err = ex.main(["--fmt", fmt, "--tokens", "64", "--ranks", "2", "--width", "512", "--inner", "256", "--experts", "6"])
    assert err < 0.25
    x, gate_up, down, ids, gates = ex.make(32, 512, 256, 6, 2, torch.float16, "cuda", seed=1)
    whole, halves = [ex.Rank(fmt, gate_up, down, 0, 256)], [ex.Rank(fmt, gate_up, down, 0, 128),
                                                            ex.Rank(fmt, gate_up, down, 128, 256)]
    one, two = ex.layer(whole, x, ids, gates, 6).float(), ex.layer(halves, x, ids, gates, 6).float()
    # the same weights in two parts: what differs is the 8-bit wire (a step of 1/128 of a block's
    # largest value on each rank and on the sum) and fp16 roundings
    assert ((one - two).norm() / one.norm()).item() < 0.03
