"""Calls whose threads exceed one launch: the launches they are made of, counted on the host, and
small calls made of many launches on an MI355X."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = "/opt/rocm"
HIPCC = os.path.join(ROCM, "bin", "hipcc")


@pytest.mark.timeout(600)
def test_combine_of_any_documented_size_is_launched(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("ROCm compilers are not installed")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "bit_quantized_all_amd", "csrc")]
    exe = str(tmp_path / "count")
    cmd = [HIPCC, "--offload-arch=gfx950", "-std=c++17", "-O1", *inc, "-x", "hip",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           os.path.join(ROOT, "bit_quantized_all_amd", "csrc", "qr_ops.hip"),
           os.path.join(ROOT, "tests", "c_abi", "ops_count_launches.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    rows = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
    assert len(rows) == 7
    for tokens, n, status, launches, threads, largest in rows:
        pieces = tokens * -(-n // 8)          # a thread each, of 8 columns
        assert status == 0 and largest < 1 << 32, (tokens, n)
        # all of them, less than twice as many, and no more launches than these threads need, and one
        assert pieces <= threads < 2 * pieces + 2048 and launches <= threads // (1 << 31) + 1, (tokens, n, launches, threads)


@pytest.fixture
def libraries(monkeypatch):
    """Calls of the library as it is, and of one built with launches of at most 2^15 threads."""
    import bit_quantized_all_amd as qa
    from bit_quantized_all_amd import build, qr

    qa.lib()
    whole = qr._lib

    def small(call):
        with monkeypatch.context() as m:
            m.setattr(qr, "LIB_PATH", build.SMALL_GRID_LIB)
            m.setattr(qr, "_lib", None)
            qr.lib()
            assert qr._lib is not whole
            return call()
    return qa, small


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype,gated", [("int4", torch.float16, False), ("asym4", torch.bfloat16, True),
                                             ("fp4", torch.bfloat16, False)])
@pytest.mark.parametrize("rows,n,k,experts", [(1, 3000, 96, 1), (2, 700, 4200, 1), (7, 500, 200, 3), (50, 1100, 264, 1),
                                              (900, 300, 71, 9), (1300, 4500, 72, 1), (700, 3300, 203, 1),
                                              (2050, 4500, 72, 1), (3000, 2300, 64, 5)])
def test_products_of_several_launches(libraries, fmt, dtype, gated, rows, n, k, experts):
    from test_ops_gpu import random_packed
    qa, small = libraries
    wide = n * (2 if gated else 1)
    w = torch.from_numpy(random_packed(fmt, experts * wide, k, n).reshape(-1)).cuda()
    x = torch.randn(rows, k, generator=torch.Generator().manual_seed(k)).to(dtype).cuda()
    if experts == 1:
        def call():
            return qa.qr_linear(fmt, x, w, n, gated=gated)
    else:
        off = torch.tensor([0] + sorted((torch.randperm(rows, generator=torch.Generator().manual_seed(1))[:experts])
                                        .tolist()), dtype=torch.int32).cuda()

        def call():
            return qa.qr_experts(fmt, x, w, n, off, gated=gated)
    assert torch.equal(call(), small(call))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,top,n", [(1000, 2, 96), (77, 3, 4100), (5, 1, 60000), (4099, 2, 7)])
def test_combinations_of_several_launches(libraries, tokens, top, n):
    qa, small = libraries
    gen = torch.Generator().manual_seed(n)
    y = torch.randn(tokens, n, generator=gen).half().cuda()
    pos = torch.randint(-1, tokens + 1, (tokens, top), generator=gen, dtype=torch.int32).cuda()
    gates = torch.rand(tokens, top, generator=gen).cuda()

    def call():
        return qa.qr_combine(y, pos, gates)
    assert torch.equal(call(), small(call))
