"""The C ABI of include/qr_ops.h on the host: exports, sizes and every refusal,
which come before any HIP call (no valid call is made here)."""
import os
import re
import shutil
import subprocess

import pytest
import torch

import bit_quantized_all_amd as qa
from bit_quantized_all_amd import qr, qr_ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qr_ops.h")
# Fake, never-dereferenced device addresses, far apart
X, W, Y, O, R, P, S = (0x700000000000 + (i << 40) for i in range(7))


@pytest.fixture(scope="module")
def L():
    return qr_ops._lib()


def test_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qr_\w+)\s*\(", text)))
    assert names == ["qr_combine", "qr_experts", "qr_linear", "qr_route", "qr_route_workspace", "qr_weight_bytes"]
    for name in names:
        assert hasattr(L, name) and hasattr(qa, name) or name == "qr_route_workspace", name


@pytest.mark.parametrize("lang,std", [("c", "-std=c99"), ("c++", "-std=c++11")])
def test_header_compiles_strictly(tmp_path, lang, std):
    cc = "gcc" if lang == "c" else "g++"
    if shutil.which(cc) is None:
        pytest.skip(f"{cc} is not installed")
    src = tmp_path / ("h.c" if lang == "c" else "h.cpp")
    src.write_text('#include "qr_ops.h"\nint main(void) { return (int)(sizeof(&qr_linear) + QR_MAX_TOP) * 0; }\n')
    r = subprocess.run([cc, std, "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-fsyntax-only", str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_weight_bytes(L):
    assert L.qr_weight_bytes(4, 64, 32) == 1152                   # one tile
    assert L.qr_weight_bytes(4, 65, 32) == 2 * 1152
    assert L.qr_weight_bytes(36, 64, 1) == 1152                   # a row of one value takes a block
    assert L.qr_weight_bytes(36, 3, 33) == 1152
    assert L.qr_weight_bytes(20, 16, 128) == 1072
    assert L.qr_weight_bytes(20, 16, 129) == 2 * 1072             # padded to whole groups
    assert L.qr_weight_bytes(4, 4096, 4096) == 8192 * 1152
    for fmt in (0, 3, 8, 24, 5):
        assert L.qr_weight_bytes(fmt, 64, 32) == 0
    assert L.qr_weight_bytes(4, 0, 32) == 0 and L.qr_weight_bytes(4, 1, 0) == 0
    assert L.qr_weight_bytes(4, 1, (1 << 22) + 1) == 0
    assert L.qr_weight_bytes(4, 1 << 63, 1 << 22) == 0            # no overflow on the way
    assert L.qr_weight_bytes(4, 1 << 19, 1 << 22) == (1 << 30) * 1152
    assert L.qr_weight_bytes(4, (1 << 19) + 1, 1 << 22) == 0
    assert L.qr_packed_bytes(4, 4096 * 4096) == L.qr_weight_bytes(4, 4096, 4096)


def linear(L, fmt=4, dt=0, gated=0, x=X, ldx=64, w=W, y=Y, ldy=32, m=8, n=32, k=64):
    return L.qr_linear(fmt, dt, gated, x, ldx, w, y, ldy, m, n, k, None)


def test_linear_refusals(L):
    for fmt in (0, 3, 8, 24, 7):
        assert linear(L, fmt=fmt, n=0, x=0) == qr.QR_ERR_UNSUPPORTED
    assert linear(L, dt=2) == linear(L, dt=-1) == qr.QR_ERR_UNSUPPORTED
    for bad in (dict(n=0), dict(n=(1 << 24) + 1, ldy=1 << 25), dict(k=0), dict(k=(1 << 22) + 1, ldx=1 << 23), dict(ldx=63),
                dict(ldy=31), dict(m=(1 << 30) + 1), dict(ldx=(1 << 32) + 1), dict(ldy=1 << 63), dict(m=1 << 63)):
        assert linear(L, **{**dict(x=0), **bad}) == qr.QR_ERR_SIZE, bad
    # sizes are checked for a call without rows too; pointers are not
    assert linear(L, m=0, n=0) == qr.QR_ERR_SIZE
    assert linear(L, m=0, x=0, w=0, y=0) == qr.QR_OK
    assert linear(L, x=0) == linear(L, w=0) == linear(L, y=0) == qr.QR_ERR_ARG
    assert linear(L, x=X + 1) == linear(L, y=Y + 1) == linear(L, w=W + 8) == qr.QR_ERR_ALIGN
    assert linear(L, y=X + 2 * 8 * 64 - 2) == qr.QR_ERR_ALIAS     # y begins in the last value of x
    assert linear(L, x=Y + 2 * (7 * 40 + 32) - 2, ldy=40) == qr.QR_ERR_ALIAS
    assert linear(L, y=W + 1150) == qr.QR_ERR_ALIAS
    assert linear(L, w=W, y=W + 1152 + 1150, n=65, ldy=65) == qr.QR_ERR_ALIAS
    assert linear(L, gated=1, y=W + 1152 + 1150, n=33, ldy=33, k=32, ldx=64) == qr.QR_ERR_ALIAS


def experts(L, fmt=20, dt=1, gated=0, x=X, ldx=128, tokens=8, w=W, off=O, rows=R, y=Y, ldy=32, slots=16, n_exp=4, n=32,
            k=128):
    return L.qr_experts(fmt, dt, gated, x, ldx, tokens, w, off, rows, y, ldy, slots, n_exp, n, k, None)


def test_experts_refusals(L):
    assert experts(L, fmt=24) == experts(L, dt=5) == qr.QR_ERR_UNSUPPORTED
    for bad in (dict(n_exp=0), dict(n_exp=1025), dict(rows=0, tokens=15), dict(slots=(1 << 30) + 1), dict(n=0), dict(ldx=127),
                dict(tokens=(1 << 30) + 1), dict(n_exp=1024, n=1 << 24, k=1 << 22, ldx=1 << 22, ldy=1 << 24)):
        assert experts(L, **bad) == qr.QR_ERR_SIZE, bad
    assert experts(L, slots=0, x=0, w=0, off=0, rows=0, y=0) == qr.QR_OK
    assert experts(L, off=0) == experts(L, x=0) == experts(L, w=0) == experts(L, y=0) == qr.QR_ERR_ARG
    assert experts(L, off=O + 2) == experts(L, rows=R + 2) == qr.QR_ERR_ALIGN
    assert experts(L, y=O + 16) == experts(L, y=R + 60) == experts(L, y=X + 2046) == qr.QR_ERR_ALIAS
    assert experts(L, y=W + 8 * 1072 - 2) == qr.QR_ERR_ALIAS      # 4 experts of 32 x 128 values: 8 tiles


def route(L, ids=X, idb=4, off=O, rows=R, pos=P, tokens=16, top=2, n_exp=4, ws=S):
    return L.qr_route(ids, idb, off, rows, pos, tokens, top, n_exp, ws, None)


def test_route_refusals(L):
    assert L.qr_route_workspace(64, 8, 64) == 0
    assert L.qr_route_workspace(32768, 8, 256) % (256 * 4) == 0 and L.qr_route_workspace(32768, 8, 256) > 0
    assert L.qr_route_workspace(1 << 63, 8, 64) == 0
    assert route(L, idb=2) == route(L, idb=0) == qr.QR_ERR_UNSUPPORTED
    for bad in (dict(top=0), dict(top=65), dict(n_exp=0), dict(n_exp=1025), dict(tokens=(1 << 29) + 1), dict(tokens=1 << 63)):
        assert route(L, **bad) == qr.QR_ERR_SIZE, bad
    assert route(L, ids=0) == route(L, off=0) == route(L, rows=0) == route(L, pos=0) == qr.QR_ERR_ARG
    assert route(L, tokens=32768, ws=0) == qr.QR_ERR_ARG
    assert route(L, ids=X + 4, idb=8) == route(L, off=O + 1) == route(L, rows=R + 2) == route(L, pos=P + 3) == qr.QR_ERR_ALIGN
    assert route(L, tokens=32768, ws=S + 2) == qr.QR_ERR_ALIGN
    assert route(L, pos=X + 4 * 31) == route(L, rows=O + 16) == route(L, pos=R - 4) == qr.QR_ERR_ALIAS
    assert route(L, tokens=32768, ws=R + 8) == qr.QR_ERR_ALIAS


def combine(L, dt=0, y=Y, ldy=64, slots=16, pos=P, gates=R, out=X, ldo=64, tokens=8, top=2, n=64):
    return L.qr_combine(dt, y, ldy, slots, pos, gates, out, ldo, tokens, top, n, None)


def test_combine_refusals(L):
    assert combine(L, dt=2) == qr.QR_ERR_UNSUPPORTED
    for bad in (dict(n=0), dict(top=0), dict(top=65), dict(ldy=63), dict(ldo=63), dict(tokens=1 << 30), dict(slots=1 << 31),
                dict(n=(1 << 24) + 1, ldy=1 << 25, ldo=1 << 25), dict(ldo=1 << 33)):
        assert combine(L, **bad) == qr.QR_ERR_SIZE, bad
    assert combine(L, tokens=0, y=0, pos=0, gates=0, out=0) == qr.QR_OK
    assert combine(L, y=0) == combine(L, pos=0) == combine(L, gates=0) == combine(L, out=0) == qr.QR_ERR_ARG
    assert combine(L, y=Y + 1) == combine(L, out=X + 1) == combine(L, pos=P + 2) == combine(L, gates=R + 1) == qr.QR_ERR_ALIGN
    assert combine(L, out=Y + 2 * 16 * 64 - 2) == combine(L, out=P + 60) == combine(L, out=R + 60) == qr.QR_ERR_ALIAS


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.float16)
    w = torch.zeros(1152, dtype=torch.uint8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: qa.qr_linear("int4", x, w, 32), lambda: qa.qr_route(ids, 4),
                 lambda: qa.qr_experts("int4", x, w, 32, torch.tensor([0, 4], dtype=torch.int32)),
                 lambda: qa.qr_combine(x, ids, torch.ones(4, 2)), lambda: qa.qr_encode_weight("int4", x),
                 lambda: qa.qr_encode_weight("int3", x), lambda: qa.qr_weight_bytes("int4", 0, 1)):
        with pytest.raises(ValueError):
            call()


def test_missing_library_fails_loudly(monkeypatch):
    monkeypatch.setattr(qr, "_lib", None)
    monkeypatch.setattr(qr, "LIB_PATH", os.path.join(ROOT, "no_such_dir", "libqr.so"))
    with pytest.raises(RuntimeError, match="missing"):
        qr_ops._lib()
