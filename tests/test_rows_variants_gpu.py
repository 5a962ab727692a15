"""Every variant of the 8-bit products' kernels (MI355X only): which of them the cases reach is checked against the
rule of the choice, so that no later change of it leaves one untested.  Sums are whole numbers and y is rounded once, so
the tolerances of rows_reference.py hold at any depth."""
import numpy as np
import pytest
import torch

import rows_reference as R
from rows_reference import DT, HALF_ULP, TINY
from rows_rule import variant
from test_rows_gpu import dev, qa  # noqa: F401

pytestmark = pytest.mark.gpu

FEW = {("fragments", mf, nf, kw) for mf, nf in ((1, 1), (1, 2), (1, 4), (2, 1), (2, 2), (2, 4), (4, 4)) for kw in (4, 8)}
DENSE_FEW = FEW - {("fragments", 4, 4, 4)} | {("fragments", 3, 4, 8)}
TILES = {("tiles", 128, 128), ("tiles", 128, 256), ("tiles", 256, 256)}
# rows of x, columns of y (rows of the weight), k: one run of 128 a wave and several, whole and not
SHAPES = [(7, 300, 1100), (16, 5200, 130), (9, 5700, 1290), (3, 10400, 264), (16, 11300, 2050), (16, 90000, 129), (20, 3000, 1100),
          (64, 2000, 130), (40, 5000, 2100), (64, 4000, 640), (64, 6100, 900), (300, 1250, 1000), (120, 4700, 140), (40, 16000, 1153),
          (130, 5100, 1300), (250, 4100, 700), (48, 30000, 131), (200, 5200, 257), (600, 2200, 390), (500, 4000, 128), (520, 8000, 129),
          (1000, 7900, 260), (2100, 4400, 513), (4000, 4100, 384), (4099, 4099, 131), (2050, 9000, 200), (8200, 2100, 130), (33, 2576, 260), (33, 5164, 140),
          (33, 10320, 131), (33, 15016, 384), (50, 11264, 270)]


def weights(wide, k, seed):
    q, s = R.random_rows(wide, k, seed)
    return dev(q), dev(s)


def check(y, x, xs, w, ws, gated, dtype, what):
    """Sums in fp64 on the GPU."""
    h = torch.mm(x.double(), w.double().t().contiguous()) * xs.double()[:, None] * ws.double()
    err, want = 3.01 * 2.0 ** -24 * h.abs(), h
    if gated:
        n = h.shape[1] // 2
        g, u, eg, eu = h[:, :n], h[:, n:], err[:, :n], err[:, n:]
        silu = g * torch.sigmoid(g)
        want = silu * u
        err = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (g.abs() + 8) * 2.0 ** -23 * want.abs()
    tol = err + HALF_ULP[dtype] * (want.abs() + err) + TINY[dtype]
    over = y.isinf() & (y.double() * want > 0) & (want.abs() + err + TINY[dtype] >= R.OVER[dtype])
    bad = ~(((y.double() - want).abs() <= tol) | over)
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), y[bad][:4], want[bad][:4], int(bad.sum()))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("gated", [False, True])
def test_dense(qa, dtype, gated):
    reached = set()
    for m, n, k in SHAPES:
        for n in (n, n - 3) if m % 2 else (n,):
            n = (n + 1) // 2 if gated else n
            v = variant(m, n, gated)
            print(f"{v} {dtype} gated={gated} {m}x{n}x{k}", flush=True)
            reached.add(v)
            x, xs = weights(m, k, m + k)
            w, ws = weights(n * (2 if gated else 1), k, n + k)
            check(qa.qr_linear8(x, xs, w, ws, DT[dtype], gated=gated), x, xs, w, ws, gated, dtype, (v, m, n, k))
    assert reached == {v for v in DENSE_FEW | TILES if not gated or v[2] > 1}


# rows of y, experts, n, k
GROUPS = [(7, 5, 700, 1100), (40, 3, 1600, 390), (51, 3, 1360, 140), (100, 9, 2600, 257), (64, 9, 6000, 130), (60, 3, 800, 1300), (130, 4, 1200, 270),
          (400, 9, 300, 131), (1000, 30, 260, 520), (900, 3, 1500, 2056), (500, 40, 1100, 264), (1600, 3, 4200, 200), (3000, 40, 2100, 128),
          (6000, 5, 4500, 136), (2500, 6, 700, 513), (9000, 3, 3000, 384), (20000, 70, 1100, 130), (52, 3, 1355, 1030), (2, 1, 2566, 260),
          (2, 1, 5644, 390), (1, 1, 10250, 140), (17, 1, 5272, 131), (18, 1, 10332, 270), (18, 1, 15856, 520), (54, 1, 9346, 130)]


@pytest.mark.parametrize("dtype,gated", [("fp16", False), ("bf16", True), ("bf16", False)])
def test_groups(qa, dtype, gated):
    reached = set()
    for slots, experts, n, k in GROUPS:
        n = (n + 1) // 2 if gated else n
        wide, tokens = n * (2 if gated else 1), slots // 2 + 1
        v = variant(slots, n, gated, experts)
        print(f"{v} {dtype} gated={gated} {slots} rows of {experts} x {n} x {k}", flush=True)
        reached.add(v)
        rng = np.random.default_rng(slots)
        cuts = np.sort(rng.integers(0, slots, experts - 1))
        off = np.concatenate([[0], cuts, [slots - slots // 50]]).clip(0, slots - slots // 50).astype(np.int32)
        x, xs = weights(tokens, k, slots)
        w, ws = weights(experts * wide, k, n)
        rows = torch.from_numpy(rng.integers(0, tokens, slots).astype(np.int32)).cuda()
        rows[::37] = -1
        rows[5::41] = tokens
        y = qa.qr_experts8(x, xs, w.view(experts, wide, -1), ws.view(experts, wide), dev(off), DT[dtype], rows=rows, gated=gated)
        real = (rows >= 0) & (rows < tokens)
        for e in range(experts):
            at = torch.arange(off[e], off[e + 1], device="cuda")
            at = at[real[at]]
            if at.numel():
                t = rows[at].long()
                check(y[at], x[t], xs[t], w[e * wide:(e + 1) * wide], ws[e * wide:(e + 1) * wide], gated, dtype, (v, slots, e))
        none = ~real
        none[off[-1]:] = True
        assert not y[none].any()
    assert reached == {v for v in FEW | TILES if not gated or v[2] > 1}
