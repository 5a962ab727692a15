"""The norm, the 8-bit rows, their products and the router's choice against plain computations in 64
bits (MI355X only).  Where the tolerances come from stands in rows_reference.py."""
import numpy as np
import pytest
import torch

import rows_reference as R
from rows_reference import DT, HALF_ULP, TINY, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qa():
    import bit_quantized_all_amd as qa
    qa.lib()
    assert torch.cuda.is_available()
    return qa


def log(*a):
    print(*a, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def values(rows, k, dtype, seed, size=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, k)) * size
    x[rng.random((rows, k)) < 0.01] *= 20
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def strided(x, off, pad=3):
    """The same values as columns ``off`` on of a wider matrix."""
    big = torch.full((x.shape[0], x.shape[1] + off + pad), 7.0, dtype=x.dtype, device=x.device)
    big[:, off:off + x.shape[1]] = x
    return big[:, off:off + x.shape[1]]


# ---------------------------------------------------------------------------
# 8-bit rows
# ---------------------------------------------------------------------------

SIZES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 127), (4, 128), (7, 129), (3, 500), (2, 1000), (6, 2048), (5, 2049), (3, 4096),
         (2, 4104), (3, 5003), (2, 8192), (2, 8195), (1, 16384), (2, 16391), (1, 32768), (1, 33001), (1, 130944), (300, 70), (700, 300), (600, 513),
         (530, 1030), (520, 4095), (515, 4100), (514, 7000), (513, 7169), (513, 20000)]


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("off", [0, 1])
def test_encode_and_decode_rows(qa, dtype, off):
    for rows, k in SIZES:
        log(f"rows {dtype} {rows}x{k} off {off}")
        x = strided(values(rows, k, dtype, rows + k), off) if off else values(rows, k, dtype, rows + k)
        codes, scales = qa.qr_encode_rows(x)
        assert codes.shape == (rows, R.padded(k)) and codes.dtype == torch.int8 and scales.shape == (rows,)
        assert codes.numel() == qa.qr_row_bytes(rows, k)
        top = f64(x).astype(np.float32)
        assert np.array_equal(scales.cpu().numpy(), np.abs(top).max(1) / np.float32(127)), (rows, k)
        R.check_rows(codes, scales, f64(x), 0.0, k, (dtype, rows, k))
        out = torch.full((rows, k + off + 2), 7.0, dtype=DT[dtype], device="cuda")
        y = qa.qr_decode_rows(codes, scales, k, DT[dtype], y=out[:, off:off + k])
        want = (codes[:, :k].cpu().float() * scales.cpu()[:, None]).to(DT[dtype])   # one rounding of fp32, one of the dtype
        assert torch.equal(y.cpu(), want), (rows, k)
        assert (out[:, :off] == 7).all() and (out[:, off + k:] == 7).all()


@pytest.mark.parametrize("dtype", sorted(DT))
def test_rows_at_the_ends_of_the_range(qa, dtype):
    """Zeros, subnormals, the largest values, and rows with a NaN or an infinity, beside ordinary ones."""
    big, small = torch.finfo(DT[dtype]).max, torch.finfo(DT[dtype]).smallest_normal
    for k in (5, 128, 4099):
        x = values(9, k, dtype, k)
        x[0] = 0
        x[1] = 0
        x[1, k // 2] = small / 8
        x[2] *= small
        x[3, k - 1] = big
        x[4] = -big
        x[5, 0] = float("nan")
        x[6, k - 1] = float("inf")
        x[7, k // 2] = -float("inf")
        codes, scales = qa.qr_encode_rows(x)
        s = scales.cpu()
        assert s[0] == 0 and not codes[0].any() and s[1] > 0 and abs(int(codes[1, k // 2])) == 127
        assert s[5:8].isnan().all() and not codes[5:8].any()
        fine = [0, 1, 2, 3, 4, 8]
        R.check_rows(codes[fine], scales[fine], f64(x)[fine], 0.0, k, (dtype, k))
        y = qa.qr_decode_rows(codes, scales, k, DT[dtype])
        assert y[5:8].isnan().all() and not y[0].any()
        assert torch.isfinite(y[fine]).all()


def test_rows_of_more_dimensions_and_views(qa):
    x = values(6 * 33, 200, "bf16", 1).view(6, 33, 200)
    codes, scales = qa.qr_encode_rows(x)
    want, ws = qa.qr_encode_rows(x.view(-1, 200))
    assert codes.shape == (6, 33, 256) and torch.equal(codes.view(-1, 256), want) and torch.equal(scales.view(-1), ws)
    t = x.transpose(0, 1)
    codes, scales = qa.qr_encode_rows(t)
    want, ws = qa.qr_encode_rows(t.contiguous())
    assert torch.equal(codes, want) and torch.equal(scales, ws)
    assert qa.qr_decode_rows(codes, scales, 200, torch.bfloat16).shape == (33, 6, 200)
    empty, none = qa.qr_encode_rows(x[:0].view(0, 200))
    assert empty.shape == (0, 256) and none.shape == (0,)
    assert qa.qr_decode_rows(empty, none, 200, torch.float16).shape == (0, 200)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("off", [0, 1])
def test_norm(qa, dtype, residual, off):
    for rows, k in SIZES:
        log(f"norm {dtype} {rows}x{k} residual={residual} off {off}")
        x, w = values(rows, k, dtype, rows + k), values(1, k, dtype, k)[0]
        r = values(rows, k, dtype, rows * k, 3.0) if residual else None
        h = f64(x) + (f64(r) if residual else 0)
        want, rel = R.norm(h, f64(w), 1e-5)
        tol = rel * np.abs(want) + HALF_ULP[dtype] * np.abs(want) * (1 + rel) + TINY[dtype]
        if off:
            x, r = strided(x, off), None if r is None else strided(r, off + 1)
        y, total = qa.qr_norm(x, w, 1e-5, residual=r)
        assert (np.abs(f64(y) - want) <= tol).all(), (rows, k)
        assert total is None if not residual else torch.equal(total, (x.float() + r.float()).to(DT[dtype])), (rows, k)
        codes, scales, total8, none = qa.qr_norm_rows(x, w, 1e-5, residual=r)
        assert none is None and (total8 is None or torch.equal(total8, total))
        R.check_rows(codes, scales, want, rel, k, (dtype, rows, k))
        c2, s2, _, y2 = qa.qr_norm_rows(x, w, 1e-5, residual=r, with_output=True)
        assert torch.equal(c2, codes) and torch.equal(s2, scales) and torch.equal(y2, y), (rows, k)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("k", [64, 4096, 5003, 33001])
def test_norm_in_place(qa, dtype, k):
    x, r, w = values(5, k, dtype, 1), values(5, k, dtype, 2), values(1, k, dtype, 3)[0]
    y, total = qa.qr_norm(x, w, residual=r)
    codes, scales, _, _ = qa.qr_norm_rows(x, w, residual=r)
    a, b = x.clone(), r.clone()
    qa.qr_norm(a, w, residual=b, total=b, y=a)
    assert torch.equal(a, y) and torch.equal(b, total)
    a, b = x.clone(), r.clone()
    qa.qr_norm(a, w, residual=b, total=a, y=b)
    assert torch.equal(b, y) and torch.equal(a, total)
    a, b = x.clone(), r.clone()
    c, s, _, _ = qa.qr_norm_rows(a, w, residual=b, total=b)
    assert torch.equal(c, codes) and torch.equal(s, scales) and torch.equal(b, total) and torch.equal(a, x)
    a = x.clone()
    qa.qr_norm(a, w, y=a)
    assert torch.equal(a, qa.qr_norm(x, w)[0])


def test_norm_of_rows_whose_squares_leave_the_range(qa):
    """bf16 has fp32's range and its squares do not: 2^120 and 2^-120 have their norm, beside ordinary rows."""
    for k in (3, 1000, 40000):
        w = values(1, k, "bf16", 3)[0]
        x = torch.cat([values(1, k, "bf16", i, s) for i, s in enumerate([1.0, 2.0 ** 118, 2.0 ** 64, 2.0 ** -60, 2.0 ** -118])]
                      + [torch.full((1, k), v, dtype=torch.bfloat16, device="cuda") for v in (torch.finfo(torch.bfloat16).max, 2.0 ** -130)])
        for eps in (0.0, 1e-6, 2.0 ** -130):
            want, rel = R.norm(f64(x), f64(w), float(np.float32(eps)))
            y, _ = qa.qr_norm(x, w, eps)
            tol = rel * np.abs(want) + HALF_ULP["bf16"] * np.abs(want) * (1 + rel) + TINY["bf16"]
            assert (np.abs(f64(y) - want) <= tol).all(), (k, eps)
            codes, scales, _, _ = qa.qr_norm_rows(x, w, eps)
            R.check_rows(codes, scales, want, rel, k, (k, eps))


def test_norm_of_rows_that_are_not_finite(qa):
    x, w = values(6, 700, "bf16", 1), values(1, 700, "bf16", 2)[0]
    want = qa.qr_norm(x, w)[0]
    codes, scales, _, _ = qa.qr_norm_rows(x, w)
    x[1, 5] = float("nan")
    x[3, 699] = float("inf")
    x[4] = 0
    y = qa.qr_norm(x, w)[0]
    assert y[1].isnan().all() and y[3, 699].isnan() and not y[4].any()
    c, s, _, _ = qa.qr_norm_rows(x, w)
    assert s[[1, 3]].isnan().all() and not c[[1, 3]].any() and not c[4].any() and s[4] == 0
    for i in (0, 2, 5):
        assert torch.equal(y[i], want[i]) and torch.equal(c[i], codes[i]) and s[i] == scales[i]


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

SHAPES = [(1, 1, 1), (1, 16, 32), (2, 17, 33), (3, 5, 127), (1, 256, 4096), (4, 70, 1000), (16, 64, 128), (17, 48, 160),
          (33, 100, 257), (5, 130, 2049), (64, 40, 96), (70, 64, 1000), (128, 256, 512), (257, 515, 640), (200, 33, 8191),
          (512, 384, 1024), (1030, 300, 392), (1, 2, 16384), (1, 4097, 128), (9, 33, 130944)]


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("gated", [False, True])
def test_linear8(qa, dtype, gated):
    for m, n, k in SHAPES:
        log(f"linear8 {dtype} gated={gated} {m}x{n}x{k}")
        x, xs = R.random_rows(m, k, m + k, full=True)
        w, ws = R.random_rows(n * (2 if gated else 1), k, n + k, full=True)
        y = qa.qr_linear8(dev(x), dev(xs), dev(w), dev(ws), DT[dtype], gated=gated)
        assert y.shape == (m, n) and y.dtype == DT[dtype]
        R.check_product(y, x, xs, w, ws, gated, dtype, (dtype, gated, m, n, k))


def product_on_gpu(qa, m, n, k, gated, dtype, seed):
    """A large product against sums in fp64 on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    wide, kp = n * (2 if gated else 1), R.padded(k)
    x = torch.zeros(m, kp, dtype=torch.int8, device="cuda")
    w = torch.zeros(wide, kp, dtype=torch.int8, device="cuda")
    x[:, :k] = torch.randint(-127, 128, (m, k), generator=gen, device="cuda")
    w[:, :k] = torch.randint(-127, 128, (wide, k), generator=gen, device="cuda")
    xs = torch.rand(m, generator=gen, device="cuda") * 0.01
    ws = torch.rand(wide, generator=gen, device="cuda") * 0.001
    y = qa.qr_linear8(x, xs, w, ws, DT[dtype], gated=gated)
    h = torch.mm(x.double(), w.double().t().contiguous()) * xs.double()[:, None] * ws.double()
    err, want = 3.01 * 2.0 ** -24 * h.abs(), h
    if gated:
        g, u, eg, eu = h[:, :n], h[:, n:], err[:, :n], err[:, n:]
        silu = g * torch.sigmoid(g)
        want = silu * u
        err = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (g.abs() + 8) * 2.0 ** -23 * want.abs()
    tol = err + HALF_ULP[dtype] * (want.abs() + err) + TINY[dtype]
    assert ((y.double() - want).abs() <= tol).all(), (m, n, k, gated, dtype)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype,m,n,k", [("bf16", 2050, 4500, 328), ("fp16", 4100, 2305, 136), ("fp16", 2305, 4200, 64),
                                         ("bf16", 1025, 5003, 456), ("bf16", 130, 8200, 1031), ("fp16", 20, 66000, 264),
                                         ("bf16", 300, 300, 20000), ("fp16", 4096, 4096, 384), ("bf16", 4097, 4097, 640),
                                         ("bf16", 1000, 2000, 2688), ("fp16", 65, 9000, 1288), ("bf16", 40, 640, 70000)])
def test_linear8_large(qa, gated, dtype, m, n, k):
    product_on_gpu(qa, m, n, k, gated, dtype, m + n)


def test_linear8_writes_only_its_columns(qa):
    for m, n, k in [(1, 5, 70), (3, 37, 128), (20, 61, 300), (130, 259, 256), (1400, 1301, 128)]:
        x, xs = R.random_rows(m, k, 1)
        w, ws = R.random_rows(n, k, 2)
        out = torch.full((m + 2, n + 5), 7.0, dtype=torch.float16, device="cuda")
        y = qa.qr_linear8(dev(x), dev(xs), dev(w), dev(ws), torch.float16, y=out[1:-1, 3:3 + n])
        R.check_product(y, x, xs, w, ws, False, "fp16", (m, n, k))
        assert (out[0] == 7).all() and (out[-1] == 7).all() and (out[:, :3] == 7).all() and (out[:, 3 + n:] == 7).all()


@pytest.mark.parametrize("m", [1, 20, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_scales_below_the_normal_range(qa, m, gated):
    """Scales of rows of the smallest values: exact powers of two, some below fp32's normal range, whose products with
    the sums are all above it."""
    n, k = 40, 640
    x, _ = R.random_rows(m, k, 1)
    w, _ = R.random_rows(n * (2 if gated else 1), k, 2)
    for a, b in ((-140, 20), (20, -140), (-110, 0), (0, -110), (-126, 8), (70, -149), (100, -140), (64, -130)):
        xs, ws = np.full(m, 2.0 ** a, np.float32), np.full(w.shape[0], 2.0 ** b, np.float32)
        if gated:
            with np.errstate(over="ignore"):  # (2^140 is infinite)
                ws[n:] = np.float32(2.0 ** -a) if a < 0 else 1.0  # up rows' products ordinary, the gates' the smallest
        y = qa.qr_linear8(dev(x), dev(xs), dev(w), dev(ws), torch.bfloat16, gated=gated)
        R.check_product(y, x, xs, w, ws, gated, "bf16", (m, a, b))


@pytest.mark.parametrize("m", [1, 20, 300])
def test_scales_at_the_ends_of_the_range(qa, m):
    """Largest and smallest scales whose result is in range: nothing on the way leaves it."""
    n, k = 40, 640
    x, _ = R.random_rows(m, k, 1)
    w, _ = R.random_rows(n, k, 2)
    for a, b in ((2.6e36, 1e-10), (1e-10, 2.6e36), (2.0 ** -100, 2.0 ** 60), (2.0 ** 60, 2.0 ** -100), (2.6e36, 0.0), (0.0, 2.6e36)):
        xs, ws = np.full(m, a, np.float32), np.full(n, b, np.float32)
        y = qa.qr_linear8(dev(x), dev(xs), dev(w), dev(ws), torch.bfloat16)
        R.check_product(y, x, xs, w, ws, False, "bf16", (m, a, b))
    xs, ws = np.full(m, 0.01, np.float32), np.full(n, 0.01, np.float32)
    xs[m // 2], ws[3] = np.nan, np.nan
    y = qa.qr_linear8(dev(x), dev(xs), dev(w), dev(ws), torch.bfloat16)
    fine = torch.ones(m, n, dtype=torch.bool)
    fine[m // 2], fine[:, 3] = False, False
    assert torch.equal(~y.isnan().cpu(), fine)


def groups_of(rows, experts, seed):
    rng = np.random.default_rng(seed)
    return np.sort(rng.integers(0, rows + 1, experts + 1)).astype(np.int32)


@pytest.mark.parametrize("dtype,gated", [("fp16", False), ("bf16", True), ("bf16", False)])
@pytest.mark.parametrize("slots,experts,n,k", [(1, 1, 5, 70), (7, 3, 33, 128), (40, 70, 20, 200), (300, 5, 130, 384), (1000, 9, 64, 131),
                                               (2000, 3, 600, 256), (513, 1, 40, 1000), (3000, 40, 260, 130), (5000, 4, 1100, 200)])
def test_experts8(qa, dtype, gated, slots, experts, n, k):
    rng = np.random.default_rng(slots)
    wide, tokens = n * (2 if gated else 1), max(1, slots // 3)
    x, xs = R.random_rows(tokens, k, slots)
    w, ws = R.random_rows(experts * wide, k, n)
    offsets = groups_of(slots, experts, slots + n)
    offsets[0] = 0
    rows = rng.integers(-2, tokens + 2, slots).astype(np.int32)
    out = torch.full((slots + 2, n), float("nan"), dtype=DT[dtype], device="cuda")
    y = qa.qr_experts8(dev(x), dev(xs), dev(w).view(experts, wide, -1), dev(ws).view(experts, wide), dev(offsets), DT[dtype],
                       rows=dev(rows), gated=gated, y=out[1:-1])
    assert out[0].isnan().all() and out[-1].isnan().all()
    real = (rows >= 0) & (rows < tokens)
    for e in range(experts):
        at = np.arange(offsets[e], offsets[e + 1])
        at = at[real[at]]
        if at.size:
            R.check_product(y[torch.from_numpy(at).cuda()], x[rows[at]], xs[rows[at]], w[e * wide:(e + 1) * wide],
                            ws[e * wide:(e + 1) * wide], gated, dtype, (dtype, gated, slots, experts, e))
    none = ~real | (np.arange(slots) >= offsets[-1])
    assert not y[torch.from_numpy(none).cuda()].any()


def test_experts8_without_row_numbers_and_without_tokens(qa):
    x, xs = R.random_rows(50, 130, 1)
    w, ws = R.random_rows(3 * 20, 130, 2)
    off = np.array([0, 10, 10, 45], np.int32)
    args = dev(w).view(3, 20, -1), dev(ws).view(3, 20), dev(off), torch.float16
    y = qa.qr_experts8(dev(x), dev(xs), *args)
    same = qa.qr_experts8(dev(x), dev(xs), *args, rows=torch.arange(50, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, same) and not y[45:].any()
    assert np.array_equal(y[:45].any(1).cpu().numpy(), xs[:45] > 0)
    none = qa.qr_experts8(dev(x)[:0], dev(xs)[:0], *args, rows=torch.zeros(50, dtype=torch.int32, device="cuda"))
    assert not none.any()
    assert qa.qr_experts8(dev(x)[:0], dev(xs)[:0], *args).shape == (0, 20)
    assert qa.qr_linear8(dev(x)[:0], dev(xs)[:0], dev(w), dev(ws), torch.float16).shape == (0, 60)


ORDERS = [[0, 1000, 0, 1600], [0, 1500, 0, 1500], [0, 0, 1600, 3], [7, 3, 900, 100], [1600, 0, 5, 0], [-4, 2000, 10, 1600]]


@pytest.mark.parametrize("scale,n", [(200, 40), (16, 40), (1, 40), (1, 2100)])
def test_experts8_offsets_out_of_order(qa, scale, n):
    """Offsets count as the largest up to them: every row from the first on is written, by one group."""
    k, slots = 64, 1600 // scale
    x, xs = R.random_rows(slots, k, 5)
    w, ws = R.random_rows(3 * n, k, 3)
    for o in ORDERS:
        o = [v // scale for v in o]
        y = torch.full((2, slots + 2, n), float("nan"), dtype=torch.bfloat16, device="cuda")
        for i, offsets in enumerate((o, np.maximum.accumulate(np.clip(o, 0, slots)))):
            qa.qr_experts8(dev(x), dev(xs), dev(w).view(3, n, -1), dev(ws).view(3, n), dev(np.array(offsets, np.int32)),
                           torch.bfloat16, y=y[i, 1:-1])
        first = min(max(o[0], 0), slots)
        assert torch.equal(y[0, 1 + first:-1], y[1, 1 + first:-1]) and not y[0, 1 + first:-1].isnan().any()
        assert y[0, :1 + first].isnan().all() and y[0, -1].isnan().all()


# ---------------------------------------------------------------------------
# choice
# ---------------------------------------------------------------------------

LOGITS = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def check_choice(qa, logits, top, what, **kw):
    gates, ids = qa.qr_choose(logits, top, **{("group_best" if k == "best" else k): v for k, v in kw.items()})
    ref = dict(kw, bias=None if kw.get("bias") is None else kw["bias"].double().cpu().numpy())
    want, wid, rel = R.choice(f64(logits), top, **ref)
    assert gates.shape == ids.shape == (logits.shape[0], top) and gates.dtype == torch.float32 and ids.dtype == torch.int32
    bad = (ids.cpu().numpy() != wid).any(1)
    assert not bad.any(), (what, np.argwhere(bad)[:3].tolist(), ids.cpu().numpy()[bad][:2], wid[bad][:2])
    off = ~(np.abs(f64(gates) - want) <= rel * np.abs(want) + 2.0 ** -140)
    assert not off.any(), (what, np.argwhere(off)[:4].tolist(), f64(gates)[off][:4], want[off][:4], wid[off][:4])


@pytest.mark.parametrize("dtype", sorted(LOGITS))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_choose(qa, dtype, score, biased):
    for i, (tokens, experts, top, groups, top_groups, best) in enumerate([
            (1, 1, 1, 1, 1, 1), (5, 2, 2, 1, 1, 1), (40, 7, 3, 1, 1, 1), (64, 64, 8, 1, 1, 1), (30, 65, 8, 1, 1, 1), (9, 130, 64, 1, 1, 1),
            (33, 256, 8, 8, 4, 2), (33, 256, 8, 8, 4, 1), (20, 160, 6, 8, 3, 1), (10, 1024, 10, 64, 5, 2), (7, 1000, 64, 4, 2, 2),
            (25, 72, 5, 3, 2, 2), (12, 128, 4, 64, 3, 1), (12, 512, 8, 16, 1, 2), (300, 48, 4, 6, 6, 2), (3, 1023, 7, 1, 1, 1),
            (21, 70, 6, 10, 3, 2), (11, 35, 4, 5, 2, 2), (400, 100, 7, 4, 2, 1), (13, 320, 8, 5, 2, 2), (9, 39, 3, 13, 4, 2), (50, 496, 16, 16, 9, 1),
            (18, 160, 12, 8, 3, 2), (6, 60, 16, 2, 1, 1)]):
        gen = torch.Generator().manual_seed(100 + i)
        logits = (torch.randn(tokens, experts, generator=gen) * 2).to(LOGITS[dtype]).cuda()
        bias = (torch.randn(experts, generator=gen) * 0.2).cuda() if biased else None
        log(f"choose {dtype} {score} bias={biased} {tokens}x{experts} top {top} of {top_groups}/{groups} best {best}")
        check_choice(qa, logits, top, (i, dtype, score), score=score, bias=bias, groups=groups, top_groups=top_groups, best=best,
                     renormalise=i % 3 != 0, factor=1.0 if i % 2 else 2.5)
        wide = torch.zeros(tokens, experts + 3, dtype=LOGITS[dtype], device="cuda")
        wide[:, 1:1 + experts] = logits
        check_choice(qa, wide[:, 1:1 + experts], top, (i, "strided"), score=score, bias=bias, groups=groups, top_groups=top_groups,
                     best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,top_groups,best", [(1, 1, 1), (8, 3, 2), (8, 2, 1), (5, 3, 2), (10, 4, 1)])
def test_choose_masks_ties_and_extremes(qa, score, biased, groups, top_groups, best):
    """Rows without any expert, with fewer than top, of equal logits, and of values at the ends of the range."""
    E, top = 64 if 64 % groups == 0 else 70, 6
    inf = float("inf")
    gen = torch.Generator().manual_seed(3)
    l = torch.randn(16, E, generator=gen)
    l[0] = -inf
    l[1] = float("nan")
    l[2] = -inf
    l[2, [5, 60, 61]] = torch.tensor([0.5, -1.0, 2.0])
    l[3] = 0.25                                     # all equal
    l[4] = (l[4] * 2).round() / 2                   # many ties
    l[5] = torch.finfo(torch.float32).min           # masked by the type's lowest value, all of it
    l[6, 10:] = torch.finfo(torch.float32).min
    l[7, 3] = inf
    l[7, 9] = float("nan")
    l[8] = -200.0
    l[8, 7] = -300.0
    l[9, ::2] = -inf
    l[10, :8] = -inf
    l[11, 1:] = -inf
    l[12] = l[12] * 30
    l[13] = torch.finfo(torch.float32).max
    l[14, 20] = 3e38
    bias = torch.randn(E, generator=gen) * 0.1 if biased else None
    kw = dict(score=score, groups=groups, top_groups=top_groups, best=best)
    # score and bias are equal in 64 bits or apart by more than their rounding
    check_choice(qa, l.cuda(), top, score, bias=None if bias is None else bias.cuda(), **kw)
    if biased:
        zero = torch.zeros(E)
        check_choice(qa, l.cuda(), top, "zero bias", bias=zero.cuda(), **kw)
        zero[[3, 7]] = float("nan")
        zero[12] = -inf
        zero[20] = 5.0
        check_choice(qa, l.cuda(), top, "bias out", bias=zero.cuda(), **kw)
    gates, ids = qa.qr_choose(l[:3].cuda(), top, **{"group_best" if k == "best" else k: v for k, v in kw.items()})
    assert (ids[:2] == -1).all() and not gates[:2].any()


@pytest.mark.parametrize("E,choices", [(256, ((1, 1, 1), (8, 4, 2), (8, 4, 1))), (200, ((1, 1, 1), (10, 4, 2), (5, 2, 1), (4, 2, 2)))])
def test_choose_close_ranks(qa, E, choices):
    """Ranks that fp32 cannot tell apart are in the order of 64 bits."""
    tokens = 200
    gen = torch.Generator().manual_seed(5)
    l = torch.randn(tokens, E, generator=gen)
    p = torch.sigmoid(l[0].double())
    l[:] = l[0]
    l[1:] += torch.randint(-2, 3, (tokens - 1, E), generator=gen) * 2.0 ** -23
    bias = (0.7 - p).float()                       # score + bias is 0.7 up to the bias's rounding
    for groups, top_groups, best in choices:
        check_choice(qa, l.cuda(), 8, "close", score="sigmoid", bias=bias.cuda(), groups=groups, top_groups=top_groups, best=best)
    s = torch.softmax(l[0].double(), 0)
    check_choice(qa, l.cuda(), 8, "close softmax", score="softmax", bias=(0.01 - s).float().cuda())


# ---------------------------------------------------------------------------
# together, on streams and in graphs
# ---------------------------------------------------------------------------

def layer(qa, x, res, weights):
    norm_w, router, w1, s1, w2, s2, bias = weights
    E = w1.shape[0]
    codes, scales, total, y = qa.qr_norm_rows(x, norm_w, residual=res, with_output=True)
    gates, ids = qa.qr_choose((y.float() @ router).contiguous(), 2, score="sigmoid", bias=bias, groups=2, top_groups=1, group_best=2)
    offsets, rows, pos = qa.qr_route(ids, E)
    h = qa.qr_experts8(codes, scales, w1, s1, offsets, x.dtype, rows=rows, gated=True)
    hc, hs = qa.qr_encode_rows(h)
    return qa.qr_combine(qa.qr_experts8(hc, hs, w2, s2, offsets, x.dtype), pos, gates), total, ids


def layer_weights(qa, width, inner, E, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    w1 = (torch.randn(E, 2 * inner, width, generator=gen) / width ** 0.5).to(dtype).cuda()
    w2 = (torch.randn(E, width, inner, generator=gen) / inner ** 0.5).to(dtype).cuda()
    norm_w = (1 + 0.1 * torch.randn(width, generator=gen)).to(dtype).cuda()
    router = torch.randn(width, E, generator=gen).cuda() / width ** 0.5
    bias = (torch.randn(E, generator=gen) * 0.05).cuda()
    return (norm_w, router, *qa.qr_encode_rows(w1), *qa.qr_encode_rows(w2), bias), w1, w2


@pytest.mark.parametrize("tokens", [1, 5, 96, 700])
def test_layer(qa, tokens):
    """Norm, choice, plan, products and sums as a layer uses them, against the layer in fp64 with the same experts."""
    width, inner, E = 512, 200, 8
    weights, w1, w2 = layer_weights(qa, width, inner, E, torch.bfloat16, 1)
    x, res = values(tokens, width, "bf16", 2), values(tokens, width, "bf16", 3)
    out, total, ids = layer(qa, x, res, weights)
    h = f64(x) + f64(res)
    y, _ = R.norm(h, f64(weights[0]), 1e-6)
    logits = (torch.from_numpy(y).to(torch.bfloat16).float() @ weights[1].cpu()).numpy()
    gates, wid, _ = R.choice(logits, 2, score="sigmoid", bias=weights[-1].double().cpu().numpy(), groups=2, top_groups=1, best=2)
    same = (ids.cpu().numpy() == wid).all(1)
    assert same.mean() > 0.95                       # logits are summed in another order, and y has been rounded
    want = np.zeros((tokens, width))
    a, b = f64(w1), f64(w2)
    for t in range(tokens):
        for j in range(2):
            e = wid[t, j]
            g, u = np.split(a[e] @ y[t], 2)
            want[t] += gates[t, j] * (b[e] @ (g / (1 + np.exp(-g)) * u))
    err = np.linalg.norm(f64(out)[same] - want[same]) / np.linalg.norm(want[same])
    # four times 8 bits (steps of max / 127, at most 20 times the root mean square: 2 % each, and outliers) and bf16
    assert err < 0.08, err
    assert torch.equal(total, (x.float() + res.float()).bfloat16())


def test_layer_on_another_stream_and_in_a_graph(qa):
    width, inner, E, tokens = 512, 256, 8, 64
    weights, _, _ = layer_weights(qa, width, inner, E, torch.float16, 4)
    inputs = [(values(tokens, width, "fp16", 10 + i), values(tokens, width, "fp16", 20 + i)) for i in range(4)]

    def call(x, res):
        codes, scales, total, _ = qa.qr_norm_rows(x, weights[0], residual=res)
        y = qa.qr_norm(x, weights[0], residual=res)[0]
        logits = y[:, :E]                            # no library product inside a graph
        gates, ids = qa.qr_choose(logits, 2, bias=weights[-1], groups=2, top_groups=2, group_best=2)
        offsets, rows, pos = qa.qr_route(ids, E)
        h = qa.qr_experts8(codes, scales, weights[2], weights[3], offsets, x.dtype, rows=rows, gated=True)
        hc, hs = qa.qr_encode_rows(h)
        return qa.qr_combine(qa.qr_experts8(hc, hs, weights[4], weights[5], offsets, x.dtype), pos, gates), total, gates, ids
    want = [call(*i) for i in inputs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [call(*i) for i in inputs]
    s.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    x, res = (t.clone() for t in inputs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(x, res)
    for k in (1, 2, 3, 0, 2):
        x.copy_(inputs[k][0])
        res.copy_(inputs[k][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[k])), k
        call(*inputs[k])                             # eager work between the replays


def test_given_stream(qa):
    x, w = values(300, 512, "bf16", 1), values(1, 512, "bf16", 2)[0]
    codes, scales = qa.qr_encode_rows(x)
    wc, ws = qa.qr_encode_rows(values(300, 512, "bf16", 3))
    logits = x[:, :64].float().contiguous()
    calls = [lambda s: qa.qr_encode_rows(x, stream=s), lambda s: qa.qr_decode_rows(codes, scales, 512, torch.bfloat16, stream=s),
             lambda s: qa.qr_norm(x, w, stream=s)[0], lambda s: qa.qr_norm_rows(x, w, residual=x, stream=s)[:3],
             lambda s: qa.qr_linear8(codes, scales, wc, ws, torch.bfloat16, stream=s), lambda s: qa.qr_choose(logits, 4, stream=s)]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [c(s) for c in calls]
    s.synchronize()
    for a, b in zip(want, got):
        a, b = (v if isinstance(v, tuple) else (v,) for v in (a, b))
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_gradients_are_not_lost_in_silence(qa):
    x, w = values(4, 64, "bf16", 1), values(1, 64, "bf16", 2)[0]
    for a, b, r in ((x.clone().requires_grad_(), w, None), (x, w.clone().requires_grad_(), None), (x, w, x.clone().requires_grad_())):
        for call in (lambda: qa.qr_norm(a, b, residual=r), lambda: qa.qr_norm_rows(a, b, residual=r)):
            with pytest.raises(ValueError, match="gradient"):
                call()
            with torch.no_grad():
                call()
    logits = torch.randn(4, 8, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        qa.qr_choose(logits, 2)
    with torch.no_grad():
        assert not qa.qr_choose(logits, 2)[0].requires_grad
    with pytest.raises(ValueError, match="gradient"):
        qa.qr_choose(logits.detach(), 2, bias=logits[0].detach().requires_grad_())
    p = torch.nn.Parameter(torch.randn(8, 64, device="cuda").half())
    assert not qa.qr_encode_rows(p)[1].requires_grad
    codes, scales = qa.qr_encode_rows(x)
    learned = scales.clone().requires_grad_()
    offsets = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: qa.qr_decode_rows(codes, learned, 64, torch.bfloat16),
                 lambda: qa.qr_linear8(codes, learned, codes, scales, torch.bfloat16),
                 lambda: qa.qr_linear8(codes, scales, codes, learned, torch.bfloat16),
                 lambda: qa.qr_experts8(codes, scales, codes[None], learned[None], offsets, torch.bfloat16)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()
