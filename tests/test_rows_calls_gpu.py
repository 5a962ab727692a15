"""Calls of the norm, the 8-bit rows, their products and the router's choice in the company of others: made of several
launches, on several threads and streams at once, into parts of larger matrices, and on more than 2^32 bytes (MI355X only)."""
import threading

import numpy as np
import pytest
import torch

import rows_reference as R
from rows_reference import DT
from rows_rule import variant
from test_ops_launches import libraries  # noqa: F401
from test_rows_gpu import check_choice, dev, qa, strided, values  # noqa: F401
from test_rows_variants_gpu import check, weights

pytestmark = pytest.mark.gpu


def same(a, b):
    a, b = (v if isinstance(v, (tuple, list)) else (v,) for v in (a, b))
    return len(a) == len(b) and all(p is q is None or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("rows,k", [(3000, 40), (700, 700), (600, 3000), (40, 7000), (129, 1000), (5, 40000), (300, 40000)])
def test_rows_and_norm_of_several_launches(libraries, rows, k):
    """The library built with launches of at most 2^15 threads."""
    qa, small = libraries
    x, r, w = values(rows, k, "bf16", 1), values(rows, k, "bf16", 2), values(1, k, "bf16", 3)[0]
    codes, scales = qa.qr_encode_rows(x)

    def calls():
        return (*qa.qr_encode_rows(x), qa.qr_decode_rows(codes, scales, k, torch.bfloat16), *qa.qr_norm(x, w, residual=r),
                *qa.qr_norm_rows(x, w, residual=r, with_output=True), qa.qr_norm(x, w)[0])
    assert same(calls(), small(calls))


@pytest.mark.parametrize("tokens,experts,top,groups", [(5000, 64, 4, 1), (3001, 256, 8, 8), (700, 1000, 20, 1), (2500, 7, 2, 1), (4000, 160, 6, 8), (3333, 35, 3, 5)])
def test_choice_of_several_launches(libraries, tokens, experts, top, groups):
    qa, small = libraries
    gen = torch.Generator().manual_seed(tokens)
    logits, bias = torch.randn(tokens, experts, generator=gen).cuda(), (torch.randn(experts, generator=gen) * 0.1).cuda()

    def call():
        return (*qa.qr_choose(logits, top, score="sigmoid", bias=bias, groups=groups, top_groups=max(1, groups // 2)),
                *qa.qr_choose(logits.bfloat16(), top))
    assert same(call(), small(call))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,n,k,experts", [(1, 3000, 96, 1), (7, 5000, 200, 3), (50, 11000, 264, 1), (900, 300, 71, 9), (1300, 9000, 130, 1),
                                              (4100, 4100, 128, 1), (5000, 4500, 72, 3), (9000, 3000, 140, 3)])
def test_products_of_several_launches(libraries, gated, rows, n, k, experts):
    qa, small = libraries
    wide = n * (2 if gated else 1)
    x, xs = weights(rows, k, k)
    w, ws = weights(experts * wide, k, n)
    if experts == 1:
        def call():
            return qa.qr_linear8(x, xs, w, ws, torch.float16, gated=gated)
    else:
        off = dev(np.sort(np.random.default_rng(1).integers(0, rows + 1, experts + 1)).astype(np.int32))
        off[0] = 0

        def call():
            return qa.qr_experts8(x, xs, w.view(experts, wide, -1), ws.view(experts, wide), off, torch.float16, gated=gated)
    assert same(call(), small(call))


def test_calls_on_several_threads_and_streams(qa):
    """Each thread has inputs, a stream and results of its own; none of the calls keeps anything between them."""
    def work(seed):
        n = 100 + 37 * seed
        x, r, w = values(n, 1000, "bf16", seed), values(n, 1000, "bf16", seed + 50), values(1, 1000, "bf16", seed + 90)[0]
        q, s = weights(2 * 600, 1000, seed)
        logits = x[:, :64].float().contiguous()

        def call():
            codes, scales, total, _ = qa.qr_norm_rows(x, w, residual=r)
            gates, ids = qa.qr_choose(logits, 4, score="sigmoid", bias=logits[0], groups=8, top_groups=3, group_best=2)
            y = qa.qr_linear8(codes, scales, q, s, torch.bfloat16, gated=True)
            offsets, rows, pos = qa.qr_route(ids, 64)
            return codes, scales, total, gates, ids, y, *qa.qr_encode_rows(y), offsets, rows, pos
        return call
    calls = [work(i) for i in range(4)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [calls[i]() for _ in range(20)]
        stream.synchronize()
        wrong.extend((i, j) for j, g in enumerate(got) if not same(g, want[i]))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_columns_of_one_matrix(qa):
    """Inputs and outputs beside each other in the rows of one buffer."""
    for m, k in ((1, 200), (5, 333), (600, 70), (3, 33000)):
        x, r, w = values(m, k, "fp16", 1), values(m, k, "fp16", 2), values(1, k, "fp16", 3)[0]
        y, total = qa.qr_norm(x, w, residual=r)
        codes, scales = qa.qr_encode_rows(x)
        buf = torch.full((m, 4 * k + 7), 5.0, dtype=torch.float16, device="cuda")
        a, b, c, d = (buf[:, i * k + 2 * i:(i + 1) * k + 2 * i] for i in range(4))
        a.copy_(x)
        b.copy_(r)
        qa.qr_norm(a, w, residual=b, y=c, total=d)
        assert torch.equal(c, y) and torch.equal(d, total) and torch.equal(a, x) and torch.equal(b, r)
        assert same(qa.qr_encode_rows(a), (codes, scales))
        qa.qr_decode_rows(codes, scales, k, torch.float16, y=d)
        assert torch.equal(d, qa.qr_decode_rows(codes, scales, k, torch.float16)) and torch.equal(c, y)
        gaps = torch.cat([buf[:, (i + 1) * k + 2 * i:(i + 1) * k + 2 * i + 2] for i in range(3)] + [buf[:, 4 * k + 6:]], 1)
        assert (gaps == 5).all()
        if m > 1:                                   # rows that overlap by a value
            from bit_quantized_all_amd.qr import QRError
            with pytest.raises(QRError):
                qa.qr_norm(a, w, residual=b, y=buf[:, 1:1 + k])


def test_given_outputs(qa):
    x, w = values(40, 300, "bf16", 1), values(1, 300, "bf16", 2)[0]
    codes, scales = qa.qr_encode_rows(x)
    c, s = torch.full_like(codes, 99), torch.full_like(scales, 9.0)
    qa.qr_encode_rows(x, codes=c, scales=s)
    assert torch.equal(c, codes) and torch.equal(s, scales)      # the padding too
    c.fill_(99)
    out = qa.qr_norm_rows(x, w, codes=c, scales=s)
    assert out[0] is c and out[1] is s and same(out[:2], qa.qr_norm_rows(x, w)[:2])
    logits = torch.randn(40, 16, device="cuda")
    gates, ids = torch.empty(40, 3, device="cuda"), torch.empty(40, 3, dtype=torch.int32, device="cuda")
    assert qa.qr_choose(logits, 3, gates=gates, ids=ids)[0] is gates and same((gates, ids), qa.qr_choose(logits, 3))
    for bad in (lambda: qa.qr_encode_rows(x, codes=c[:, :128]), lambda: qa.qr_encode_rows(x, scales=s[:3]), lambda: qa.qr_norm(x, w, y=x.half()),
                lambda: qa.qr_norm(x, w[:5]), lambda: qa.qr_norm(x, w, total=x), lambda: qa.qr_norm(x, w, eps=-1.0), lambda: qa.qr_norm(x, w.half()),
                lambda: qa.qr_norm(x, w, residual=x[:3]), lambda: qa.qr_norm(x.t(), w), lambda: qa.qr_decode_rows(codes, scales, 200, torch.bfloat16),
                lambda: qa.qr_linear8(codes, scales, codes[:, :128].contiguous(), scales, torch.bfloat16),
                lambda: qa.qr_linear8(codes, scales[:5], codes, scales, torch.bfloat16),
                lambda: qa.qr_linear8(codes, scales, codes[:3], scales[:3], torch.bfloat16, gated=True),
                lambda: qa.qr_linear8(codes.short(), scales, codes, scales, torch.bfloat16),
                lambda: qa.qr_linear8(codes, scales.double(), codes, scales, torch.bfloat16),
                lambda: qa.qr_linear8(codes, scales, codes, scales, torch.float32), lambda: qa.qr_linear8(codes, scales.cpu(), codes, scales, torch.bfloat16),
                lambda: qa.qr_experts8(codes, scales, codes, scales, ids, torch.bfloat16), lambda: qa.qr_choose(logits, 0),
                lambda: qa.qr_choose(logits, 3, score="max"), lambda: qa.qr_choose(logits, 3, bias=logits[0].half()), lambda: qa.qr_choose(logits.long(), 3),
                lambda: qa.qr_choose(logits[:, ::2], 3)):
        with pytest.raises(ValueError):
            bad()


def test_no_rows(qa):
    x, w = values(1, 300, "bf16", 1)[:0], values(1, 300, "bf16", 2)[0]
    assert [t.shape for t in qa.qr_norm(x, w, residual=x)] == [(0, 300), (0, 300)]
    codes, scales, _, _ = qa.qr_norm_rows(x, w)
    assert codes.shape == (0, 384) and scales.shape == (0,)
    gates, ids = qa.qr_choose(torch.empty(0, 16, device="cuda"), 3)
    assert gates.shape == ids.shape == (0, 3)


@pytest.mark.parametrize("top,experts", [(16, 16), (17, 40), (64, 64), (16, 512), (3, 513), (1, 1024)])
def test_choices_of_many(qa, top, experts):
    gen = torch.Generator().manual_seed(top)
    for tokens in (1, 3, 5, 17, 70):
        logits = (torch.randn(tokens, experts, generator=gen) * 3).cuda()
        check_choice(qa, logits, top, (tokens, top, experts))
        check_choice(qa, logits.half(), top, (tokens, top, experts), score="sigmoid", bias=logits[0] * 0.05)


def test_ties_and_signed_zeros(qa):
    """Equal logits of either sign go by their number, over lanes and within them."""
    gen = torch.Generator().manual_seed(1)
    for experts in (5, 16, 64, 200, 512):
        logits = torch.randint(-2, 3, (50, experts), generator=gen).float().cuda()
        logits *= torch.where(torch.rand(50, experts, generator=gen).cuda() < 0.5, -1.0, 1.0)
        top = min(8, experts)
        for dt in (torch.float32, torch.bfloat16, torch.float16):
            check_choice(qa, logits.to(dt), top, (experts, dt))
            check_choice(qa, logits.to(dt), top, (experts, dt), score="sigmoid", bias=torch.zeros(experts, device="cuda"))


def test_rows_of_more_than_4_gib(qa):
    """Offsets past 2^32 bytes, of values and of codes."""
    rows, k = 40000, 65536
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    some = [0, 1, 16383, 16384, 32767, 32768, rows - 1]
    codes, scales = qa.qr_encode_rows(x)
    part, ps = qa.qr_encode_rows(x[some].contiguous())
    assert torch.equal(codes[some], part) and torch.equal(scales[some], ps)
    w = values(1, k, "bf16", 1)[0]
    want = qa.qr_norm(x[some].contiguous(), w)[0]
    y = qa.qr_decode_rows(codes, scales, k, torch.bfloat16)
    assert torch.equal(y[some], qa.qr_decode_rows(part, ps, k, torch.bfloat16))
    qa.qr_norm(x, w, y=y)
    assert torch.equal(y[some], want)


@pytest.mark.parametrize("rows,n,gated", [(40000, 70, False), (40000, 900, True)])
def test_products_of_more_than_4_gib(qa, rows, n, gated):
    k = 130944
    x = torch.randint(-127, 128, (rows, k), dtype=torch.int8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    xs = torch.rand(rows, device="cuda") * 1e-3
    w, ws = weights(n * (2 if gated else 1), k, 3)
    some = torch.tensor([0, 1, 16401, 16402, 32803, 32804, rows - 1], device="cuda")
    print(variant(rows, n, gated), flush=True)
    y = qa.qr_linear8(x, xs, w, ws, torch.bfloat16, gated=gated)
    check(y[some], x[some], xs[some], w, ws, gated, "bf16", (rows, n))
    ids = torch.randint(0, rows, (3000,), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    ids[:some.numel()] = some
    y = qa.qr_experts8(x, xs, w.view(1, *w.shape), ws.view(1, -1), torch.tensor([0, 3000], dtype=torch.int32, device="cuda"), torch.bfloat16, rows=ids,
                       gated=gated)
    check(y[:64], x[ids[:64].long()], xs[ids[:64].long()], w, ws, gated, "bf16", (rows, n, "rows"))


def test_weights_of_more_than_4_gib(qa):
    experts, n, k, tokens = 50, 700, 130944, 300
    w = torch.randint(-127, 128, (experts, n, k), dtype=torch.int8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    ws = torch.rand(experts, n, device="cuda") * 1e-3
    x, xs = weights(tokens, k, 2)
    off = torch.arange(0, tokens + 1, tokens // experts, dtype=torch.int32, device="cuda")
    y = qa.qr_experts8(x, xs, w, ws, off, torch.bfloat16)
    big = qa.qr_experts8(x, xs, w, ws, torch.tensor([0] * experts + [tokens], dtype=torch.int32, device="cuda"), torch.bfloat16)
    for e in (0, 23, 24, 46, 47, experts - 1):
        at = slice(int(off[e]), int(off[e + 1]))
        check(y[at], x[at], xs[at], w[e], ws[e], False, "bf16", e)
    check(big[::29], x[::29], xs[::29], w[-1], ws[-1], False, "bf16", "last expert")


@pytest.mark.parametrize("fmt,bound", [("rows8", 0.055), ("int4", 0.25)])
def test_example_runs(fmt, bound):
    """The layer over simulated ranks against the same layer in fp32.  8-bit rows, relative to root mean squares: a row of
    2048 normal values has a step of its largest, near 3.5, over 127, and uniform errors of 0.8 %, in x and in the weights:
    1.1 % of the first product, 1.6 % of its gate times up; those products reach 8 to 10, errors of 1.8 to 2.3 %; with the
    second weight's 0.8 % and the 8-bit wire's 0.5 % twice 2.7 %, and twice that as the bound.  4 bits: as where the layer
    over them is tested."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tensor_parallel_moe.py")
    spec = importlib.util.spec_from_file_location("tensor_parallel_moe", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(["--tokens", "64", "--ranks", "2", "--fmt", fmt]) < bound
