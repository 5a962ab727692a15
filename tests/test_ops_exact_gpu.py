"""Products whose sums are exact, so that nothing but the one rounding of the result is left to
compare, at any depth and whichever kernel a call reaches (MI355X only).

x holds -1, 0 and 1, at most 250 of them not zero in a row.  Scales are fp16 values of one
binade [2^-6, 2^-5), all 11 bits of them in use, or zero.  Every weight, and every partial sum in whatever
order, is then a multiple of 2^-16, and below 250 * 30 * 2^-5 < 2^8 in magnitude, the codes' and the zero points'
sums apart too (FP4, whose values are halves: multiples of 2^-17 below 250 * 6 * 2^-5 < 2^7).  These are fewer
than 2^24 steps, so fp32 holds all of them, and y has to be the sum rounded once to the dtype, bit for bit.  A
product that rounds its weights first, or leaves one out, differs.
"""
import numpy as np
import pytest
import torch

from product_rule import variant
from test_ops_gpu import DT, GROUP, HALF_ULP, TINY, qa, random_packed, weight64  # noqa: F401

pytestmark = pytest.mark.gpu

FORMATS = sorted(GROUP)


def exact_packed(fmt, rows, k, seed):
    p = random_packed(fmt, rows, k, seed)
    groups = 2048 // GROUP[fmt]
    rng = np.random.default_rng(seed + 1)
    s = ((1024 + rng.integers(0, 1024, (p.shape[0], groups))) * 2.0 ** -16).astype(np.float16)
    s[rng.random(s.shape) < 0.02] = 0
    p[:, 1024:1024 + 2 * groups] = s.view(np.uint8).reshape(p.shape[0], -1)
    return p


def signs(m, k, seed):
    rng = np.random.default_rng(seed)
    x = np.where(rng.random((m, k)) < min(1.0, 200 / k), rng.choice([-1.0, 1.0], (m, k)), 0.0)
    x[np.cumsum(x != 0, axis=1) > 250] = 0
    x[:, k - 1] = np.where(np.arange(m) % 2, 1.0, -1.0)   # the last value always counts
    return torch.from_numpy(x)


def sums(fmt, packed, rows, k, x):
    """x W^T in fp64 on the GPU, exact; checks that fp32 holds every partial sum."""
    _, w, apart = weight64(fmt, packed, rows, k, "fp16")
    w, apart, x = torch.from_numpy(w).cuda(), torch.from_numpy(apart).cuda(), x.double().cuda()
    assert torch.mm(x.abs(), apart.t().contiguous()).max() < (2.0 ** 7 if fmt == "fp4" else 2.0 ** 8)
    return torch.mm(x, w.t().contiguous())


def check(y, h, n, gated, dtype, what):
    if not gated:
        assert torch.equal(y, h.to(DT[dtype])), what
        return
    g, u = h[:, :n], h[:, n:]
    want = g / (1 + torch.exp(-g)) * u
    tol = ((g.abs() + 8) * 2.0 ** -23 + HALF_ULP[dtype]) * want.abs() * (1 + 2.0 ** -8) + TINY[dtype]
    assert ((y.double() - want).abs() <= tol).all(), what


def linear(qa, fmt, dtype, gated, m, n, k, off=0):
    """One product against its exact sums; ``off``: x begins that many values into rows of k + off."""
    wide = n * (2 if gated else 1)
    p = exact_packed(fmt, wide, k, m + n + k)
    x = signs(m, k, m * k + n)
    big = torch.zeros(m, k + off, dtype=DT[dtype], device="cuda")
    big[:, off:] = x.to(DT[dtype])
    y = qa.qr_linear(fmt, big[:, off:], torch.from_numpy(p.reshape(-1)).cuda(), n, gated=gated)
    check(y, sums(fmt, p, wide, k, x), n, gated, dtype, (fmt, dtype, gated, m, n, k, off))


MANY = [("many", 64, 128, True), ("many", 64, 128, False), ("many", 256, 128, True), ("many", 128, 256, True)]
MANY_SHAPES = [(700, 3300, 200), (130, 16500, 64), (2100, 1100, 8200), (700, 3300, 203), (2100, 1100, 8205),
               (1300, 4500, 72), (1024, 8192, 456), (2050, 4500, 328), (2305, 8200, 136)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("gated", [False, True])
def test_many_rows_use_the_weight_as_it_is(qa, fmt, dtype, gated):
    """The weight is not rounded to the dtype before it is multiplied, in any of the tiles."""
    reached = set()
    for m, n, k in MANY_SHAPES:
        n = (n + 1) // 2 if gated else n
        print(f"exact {fmt} {dtype} gated={gated} {m}x{n}x{k}", flush=True)
        reached.add(variant(m, n, k, gated, fmt))
        linear(qa, fmt, dtype, gated, m, n, k)
    assert reached == set(MANY)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(6, 512, 256), (5, 96, 70)])
def test_weight_packed_on_another_stream(qa, fmt, shape):
    """A weight that has to be copied, packed on a stream that the weight's own does not wait for."""
    w = torch.randn(*shape, generator=torch.Generator().manual_seed(1)).half().cuda()
    for view in (w.transpose(1, 2), w[:, 8:72], w.flip(0).transpose(0, 1)):
        want = qa.qr_encode_weight(fmt, view)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = qa.qr_encode_weight(fmt, view, stream=s)
        other = torch.zeros(view.numel(), dtype=w.dtype, device="cuda")   # memory that a copy may have been freed to
        s.synchronize()
        assert torch.equal(got, want) and not other.any()


ORDERS = [[0, 1000, 0, 1600], [0, 1500, 0, 1500], [0, 0, 1600, 3], [7, 3, 900, 100], [1600, 0, 5, 0], [-4, 2000, 10, 1600]]


@pytest.mark.parametrize("fmt,dtype,gated", [("int4", "fp16", False), ("asym4", "bf16", True)])
@pytest.mark.parametrize("scale,n,kind", [(200, 40, "row"), (16, 40, "few"), (1, 40, "few"), (1, 4200, "many")])
def test_offsets_out_of_order(qa, fmt, dtype, gated, scale, n, kind):
    """Offsets count as the largest up to them: every row from the first on is written, by one group."""
    k, slots = 64, 1600 // scale
    wide = n * (2 if gated else 1)
    rng = np.random.default_rng(n)
    orders = [([v // scale for v in o], 3) for o in ORDERS]
    orders += [(rng.integers(-slots // 4, slots * 5 // 4, 71 if scale == 1 else 68).tolist(), 70 if scale == 1 else 67)]
    for o, experts in orders:
        if experts == 3:
            assert variant(slots, n, k, gated, fmt, experts=3)[0] == kind
        w = torch.from_numpy(exact_packed(fmt, experts * wide, k, 3).reshape(-1)).cuda()
        x = signs(slots, k, 5).to(DT[dtype]).cuda()
        y = torch.full((2, slots + 2, n), float("nan"), dtype=DT[dtype], device="cuda")
        for i, offsets in enumerate((o, np.maximum.accumulate(np.clip(o, 0, slots)))):
            qa.qr_experts(fmt, x, w, n, torch.tensor(np.array(offsets), dtype=torch.int32).cuda(), gated=gated, y=y[i, 1:-1])
        first = min(max(o[0], 0), slots)
        print(f"offsets {o[:8]} of {slots} rows, {kind}", flush=True)
        assert torch.equal(y[0, 1 + first:-1], y[1, 1 + first:-1]) and not y[0, 1 + first:-1].isnan().any()
        assert y[0, :1 + first].isnan().all() and y[0, -1].isnan().all()


LARGE_SHAPES = [(1, 300, 4200), (2, 300, 4200), (1, 5000, 200), (2, 400, 8229), (5, 64, 333), (12, 12300, 136), (9, 12300, 331),
                (30, 9000, 72), (40, 64, 1032), (30, 66000, 71), (700, 3300, 200), (700, 3300, 203), (1300, 4500, 72), (2050, 4500, 72)]


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_near_the_end_of_the_range(qa, fmt):
    """bf16 x of the type's lowest value, 255 * 2^120 in magnitude: alone among others, in a whole block and throughout
    a row.  The sums of codes times x leave the range of fp32, the products x W and their sums do not."""
    low = torch.finfo(torch.bfloat16).min
    for m, n, k in LARGE_SHAPES:
        p = exact_packed(fmt, n, k, m + n + k)
        groups = 2048 // GROUP[fmt]
        s = np.ascontiguousarray(p[:, 1024:1024 + 2 * groups]).view(np.float16) * np.float16(2.0 ** -6)   # [2^-12, 2^-11)
        p[:, 1024:1024 + 2 * groups] = s.view(np.uint8).reshape(p.shape[0], -1)
        x = torch.randn(m, k, generator=torch.Generator().manual_seed(k)).to(torch.bfloat16).cuda()
        x[0, k // 2] = low
        if m > 1:
            x[m - 1, :] = low
        if m > 2:
            x[m // 2, :32] = -low
            x[m // 2 + 1, k - 33:] = low
        print(f"range {fmt} {m}x{n}x{k} {variant(m, n, k, False, fmt)}", flush=True)
        y = qa.qr_linear(fmt, x, torch.from_numpy(p.reshape(-1)).cuda(), n).double()
        _, w, apart = weight64(fmt, p, n, k, "bf16")
        w, apart = torch.from_numpy(w).cuda(), torch.from_numpy(apart).cuda()
        want = torch.mm(x.double(), w.t().contiguous())
        err = k * 2.0 ** -23 * torch.mm(x.double().abs(), apart.t().contiguous())
        # columns whose sum itself, or sum of magnitudes in fp32, leaves the range are not looked at
        inside = (want.abs() + err < 2.0 ** 127) & (torch.mm(x.double().abs(), w.abs().t().contiguous()) < 2.0 ** 127)
        tol = err + HALF_ULP["bf16"] * (want.abs() + err) + TINY["bf16"]
        assert ((y - want).abs() <= tol)[inside].all() and inside.double().mean() >= 0.5, (fmt, m, n, k)
        assert inside[0].all()


def test_gradients_are_not_lost_in_silence(qa):
    w = qa.qr_encode_weight("int4", torch.nn.Parameter(torch.randn(32, 64, device="cuda").half()))
    x = torch.randn(4, 64, device="cuda").half()
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    offsets, rows, pos = qa.qr_route(ids, 1)
    gates = torch.ones(4, 2, device="cuda")
    want = qa.qr_linear("int4", x, w, 32)
    y = qa.qr_experts("int4", x, w, 32, offsets, rows=rows)
    out = qa.qr_combine(y, pos, gates)
    xg, yg, gg = (t.clone().requires_grad_() for t in (x, y, gates))
    for call in (lambda: qa.qr_linear("int4", xg, w, 32), lambda: qa.qr_linear("int4", xg * 1, w, 32, gated=False),
                 lambda: qa.qr_experts("int4", xg, w, 32, offsets, rows=rows), lambda: qa.qr_combine(yg, pos, gates),
                 lambda: qa.qr_combine(y, pos, gg)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            assert not call().requires_grad
    assert torch.equal(qa.qr_linear("int4", xg.detach(), w, 32), want)
    with torch.inference_mode():
        assert torch.equal(qa.qr_combine(yg, pos, gg), out)


def test_columns_of_one_matrix(qa):
    """x and y beside each other in the rows of one buffer, either one first, and one row of y between two of x."""
    n, k = 40, 64
    p = exact_packed("int4", n, k, 1)
    w = torch.from_numpy(p.reshape(-1)).cuda()
    for m in (1, 2, 20, 700):
        x = signs(m, k, m)
        want = sums("int4", p, n, k, x).half()
        for first, second in ((0, k), (n, 0), (3, k + 3)):
            buf = torch.full((m, n + k + 3), 7.0, dtype=torch.float16, device="cuda")
            buf[:, first:first + k] = x.half()
            y = buf[:, second:second + n]
            qa.qr_linear("int4", buf[:, first:first + k], w, n, y=y)
            assert torch.equal(y, want) and torch.equal(buf[:, first:first + k], x.half().cuda())
    x = signs(2, k, 5)
    buf = torch.full((2, n + k), 7.0, dtype=torch.float16, device="cuda")
    buf[:, :k] = x.half()
    ids = torch.tensor([1], dtype=torch.int32, device="cuda")
    qa.qr_experts("int4", buf[:, :k], w, n, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), rows=ids, y=buf[:1, k:])
    assert torch.equal(buf[:1, k:], sums("int4", p, n, k, x)[1:].half()) and (buf[1, k:] == 7).all()
    y = torch.randn(6, 80, device="cuda").half()
    pos = torch.tensor([[3, 1], [0, 5], [2, 4], [-1, 0], [1, 1], [5, 5]], dtype=torch.int32, device="cuda")
    gates = torch.rand(6, 2, device="cuda")
    want = qa.qr_combine(y[:, :40], pos, gates)
    assert torch.equal(qa.qr_combine(y[:, :40], pos, gates, out=y[:, 40:]), want)
