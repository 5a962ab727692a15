"""The C ABI of include/qr_rows.h on the host: exports, sizes and every refusal, which come before
any HIP call (no valid call is made here), and the binding's own."""
import os
import re
import shutil
import subprocess

import pytest
import torch

import bit_quantized_all_amd as qa
from bit_quantized_all_amd import qr, qr_rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qr_rows.h")
# Fake, never-dereferenced device addresses, far apart
X, R, W, T, Y, C, S, V, O, I = (0x700000000000 + (i << 40) for i in range(10))
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return qr_rows._lib()


def test_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qr_\w+)\s*\(", text)))
    assert names == ["qr_choose", "qr_decode_rows", "qr_encode_rows", "qr_experts8", "qr_linear8", "qr_norm", "qr_row_bytes"]
    for name in names:
        assert hasattr(L, name) and hasattr(qa, name), name


@pytest.mark.parametrize("lang,std", [("c", "-std=c99"), ("c++", "-std=c++11")])
def test_header_compiles_strictly(tmp_path, lang, std):
    cc = "gcc" if lang == "c" else "g++"
    if shutil.which(cc) is None:
        pytest.skip(f"{cc} is not installed")
    src = tmp_path / ("h.c" if lang == "c" else "h.cpp")
    src.write_text('#include "qr_rows.h"\nint main(void) { qr_dtype d = QR_FP32; return (int)(sizeof(&qr_norm) + QR_MAX_ROW_K + d) * 0; }\n')
    r = subprocess.run([cc, std, "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-fsyntax-only", str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_row_bytes(L):
    assert L.qr_row_bytes(1, 1) == 128 and L.qr_row_bytes(3, 128) == 384 and L.qr_row_bytes(3, 129) == 768
    assert L.qr_row_bytes(1 << 30, 130944) == (1 << 30) * 130944 and L.qr_row_bytes(1 << 40, 1) == 1 << 47
    assert L.qr_row_bytes(0, 8) == L.qr_row_bytes(1, 0) == L.qr_row_bytes(1, 130945) == L.qr_row_bytes((1 << 40) + 1, 1) == 0
    assert L.qr_row_bytes(1 << 63, 64) == L.qr_row_bytes(4, 1 << 63) == 0
    assert qr_rows.MAX_ROW_K * 128 * 128 < 1 << 31 and qr_rows.MAX_ROW_K % 128 == 0


def encode(L, dt=0, x=X, ldx=64, c=C, s=S, rows=8, k=64):
    return L.qr_encode_rows(dt, x, ldx, c, s, rows, k, None)


def decode(L, dt=0, c=C, s=S, y=Y, ldy=64, rows=8, k=64):
    return L.qr_decode_rows(dt, c, s, y, ldy, rows, k, None)


def test_codec_refusals(L):
    for dt in (2, 3, -1):
        assert encode(L, dt=dt, k=0) == decode(L, dt=dt, k=0) == qr.QR_ERR_UNSUPPORTED
    for bad in (dict(k=0), dict(k=130945, ldx=1 << 20), dict(ldx=63), dict(ldx=(1 << 32) + 1), dict(rows=(1 << 30) + 1), dict(rows=1 << 63)):
        assert encode(L, **{**dict(x=0), **bad}) == qr.QR_ERR_SIZE, bad
        assert decode(L, **{("ldy" if key == "ldx" else key): v for key, v in bad.items()}) == qr.QR_ERR_SIZE, bad
    assert encode(L, rows=0, k=0) == qr.QR_ERR_SIZE
    assert encode(L, rows=0, x=0, c=0, s=0) == decode(L, rows=0, c=0, s=0, y=0) == qr.QR_OK
    assert encode(L, x=0) == encode(L, c=0) == encode(L, s=0) == decode(L, c=0) == decode(L, s=0) == decode(L, y=0) == qr.QR_ERR_ARG
    assert encode(L, x=X + 1) == encode(L, c=C + 8) == encode(L, s=S + 2) == qr.QR_ERR_ALIGN
    assert decode(L, y=Y + 1) == decode(L, c=C + 8) == decode(L, s=S + 2) == qr.QR_ERR_ALIGN
    assert encode(L, c=X + 16 * 63) == encode(L, s=X + 1020) == encode(L, s=C + 1020) == qr.QR_ERR_ALIAS
    assert decode(L, y=C + 1022) == decode(L, y=S + 30) == decode(L, s=Y + 1020) == qr.QR_ERR_ALIAS


def norm(L, dt=0, x=X, ldx=64, r=R, ldr=64, w=W, eps=1e-6, t=T, ldt=64, y=Y, ldy=64, c=C, s=S, rows=8, k=64):
    return L.qr_norm(dt, x, ldx, r, ldr, w, eps, t, ldt, y, ldy, c, s, rows, k, None)


def test_norm_refusals(L):
    assert norm(L, dt=2) == norm(L, dt=7, k=0) == qr.QR_ERR_UNSUPPORTED
    for bad in (dict(k=0), dict(k=130945, ldx=1 << 20, ldr=1 << 20, ldt=1 << 20, ldy=1 << 20), dict(ldx=63), dict(ldr=63), dict(ldt=63),
                dict(ldy=63), dict(ldt=(1 << 32) + 1), dict(rows=(1 << 30) + 1)):
        assert norm(L, **{**dict(x=0), **bad}) == qr.QR_ERR_SIZE, bad
    # strides of matrices that are not there are not looked at
    assert norm(L, rows=0, r=0, ldr=0, t=0, ldt=0, y=0, ldy=0) == qr.QR_OK
    assert norm(L, rows=0, x=0, r=0, w=0, t=0, y=0, c=0, s=0) == qr.QR_OK
    for bad in (dict(eps=-1e-9), dict(eps=NAN), dict(r=0), dict(c=0), dict(s=0), dict(x=0), dict(w=0), dict(y=0, c=0, s=0)):
        assert norm(L, **bad) == qr.QR_ERR_ARG, bad
    for bad in (dict(x=X + 1), dict(r=R + 1), dict(w=W + 1), dict(t=T + 1), dict(y=Y + 1), dict(c=C + 8), dict(s=S + 2)):
        assert norm(L, **bad) == qr.QR_ERR_ALIGN, bad
    for bad in (dict(t=X + 2), dict(t=R + 2), dict(y=X + 2), dict(y=R - 2), dict(t=Y), dict(t=X, y=X), dict(t=X, ldt=65), dict(y=R, ldy=70),
                dict(w=T + 2), dict(w=Y + 1022), dict(c=X), dict(c=R + 1008), dict(c=T), dict(c=Y), dict(s=X), dict(s=T + 4), dict(s=Y + 8),
                dict(s=C + 1020), dict(c=W - 1024 + 16), dict(s=W + 124), dict(s=R + 1020)):
        assert norm(L, **bad) == qr.QR_ERR_ALIAS, bad


def linear8(L, dt=0, gated=0, x=X, xs=S, w=W, ws=V, y=Y, ldy=32, m=8, n=32, k=64):
    return L.qr_linear8(dt, gated, x, xs, w, ws, y, ldy, m, n, k, None)


def experts8(L, dt=1, gated=0, x=X, xs=S, tokens=8, w=W, ws=V, off=O, rows=I, y=Y, ldy=32, slots=16, n_exp=4, n=32, k=128):
    return L.qr_experts8(dt, gated, x, xs, tokens, w, ws, off, rows, y, ldy, slots, n_exp, n, k, None)


def test_product_refusals(L):
    assert linear8(L, dt=2) == linear8(L, dt=-1, n=0) == experts8(L, dt=2) == qr.QR_ERR_UNSUPPORTED
    for bad in (dict(n=0), dict(n=(1 << 24) + 1, ldy=1 << 25), dict(k=0), dict(k=130945), dict(ldy=31), dict(ldy=(1 << 32) + 1),
                dict(m=(1 << 30) + 1), dict(m=1 << 63)):
        assert linear8(L, **{**dict(x=0), **bad}) == qr.QR_ERR_SIZE, bad
    for bad in (dict(n_exp=0), dict(n_exp=1025), dict(rows=0, tokens=15), dict(slots=(1 << 30) + 1), dict(tokens=(1 << 30) + 1), dict(n=0)):
        assert experts8(L, **bad) == qr.QR_ERR_SIZE, bad
    assert linear8(L, m=0, n=0) == qr.QR_ERR_SIZE
    assert linear8(L, m=0, x=0, xs=0, w=0, ws=0, y=0) == experts8(L, slots=0, x=0, xs=0, w=0, ws=0, off=0, rows=0, y=0) == qr.QR_OK
    for bad in (dict(x=0), dict(xs=0), dict(w=0), dict(ws=0), dict(y=0)):
        assert linear8(L, **bad) == experts8(L, **bad) == qr.QR_ERR_ARG, bad
    assert experts8(L, off=0) == qr.QR_ERR_ARG
    for bad in (dict(x=X + 8), dict(xs=S + 2), dict(w=W + 4), dict(ws=V + 1), dict(y=Y + 1)):
        assert linear8(L, **bad) == experts8(L, **bad) == qr.QR_ERR_ALIGN, bad
    assert experts8(L, off=O + 2) == experts8(L, rows=I + 2) == qr.QR_ERR_ALIGN
    for bad in (dict(y=X + 1022), dict(y=S + 30), dict(y=W + 32 * 128 - 2), dict(y=V + 126)):
        assert linear8(L, **bad) == qr.QR_ERR_ALIAS, bad
    assert linear8(L, gated=1, y=W + 64 * 128 - 2) == linear8(L, gated=1, y=V + 4 * 64 - 2) == qr.QR_ERR_ALIAS
    assert experts8(L, y=W + 4 * 32 * 128 - 2) == experts8(L, y=O + 18) == experts8(L, y=I + 62) == qr.QR_ERR_ALIAS


def choose(L, dt=2, score=0, l=X, ldl=64, bias=V, groups=8, tg=4, best=2, ren=1, factor=1.0, gates=S, ids=I, tokens=16, experts=64, top=8):
    return L.qr_choose(dt, score, l, ldl, bias, groups, tg, best, ren, factor, gates, ids, tokens, experts, top, None)


def test_choose_refusals(L):
    assert choose(L, dt=3) == choose(L, dt=-1) == choose(L, score=2) == choose(L, score=-1, experts=0) == qr.QR_ERR_UNSUPPORTED
    for bad in (dict(experts=0), dict(experts=1025, ldl=2000, groups=1, tg=1), dict(top=0), dict(top=65), dict(experts=4, top=5, groups=1, tg=1),
                dict(ldl=63), dict(ldl=(1 << 32) + 1), dict(groups=0), dict(groups=7), dict(groups=128, experts=256, ldl=256), dict(tg=0),
                dict(tg=9), dict(best=0), dict(best=3), dict(groups=64, tg=8, best=2), dict(tokens=(1 << 27) + 1), dict(tokens=1 << 63)):
        assert choose(L, **{**dict(l=0), **bad}) == qr.QR_ERR_SIZE, bad
    assert choose(L, factor=NAN) == choose(L, factor=INF) == choose(L, factor=-INF) == qr.QR_ERR_ARG
    assert choose(L, tokens=0, l=0, gates=0, ids=0, bias=0) == qr.QR_OK
    assert choose(L, l=0) == choose(L, gates=0) == choose(L, ids=0) == qr.QR_ERR_ARG
    for bad in (dict(l=X + 2), dict(dt=1, l=X + 1), dict(bias=V + 2), dict(gates=S + 1), dict(ids=I + 2)):
        assert choose(L, **bad) == qr.QR_ERR_ALIGN, bad
    for bad in (dict(ids=S + 508), dict(gates=X + 4 * 16 * 64 - 4), dict(ids=X - 508), dict(gates=V + 252), dict(ids=V)):
        assert choose(L, **bad) == qr.QR_ERR_ALIAS, bad


def test_binding_refuses_host_tensors_and_other_shapes():
    x = torch.zeros(4, 64, dtype=torch.float16)
    c, s = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)
    off = torch.tensor([0, 4], dtype=torch.int32)
    for call in (lambda: qa.qr_encode_rows(x), lambda: qa.qr_encode_rows(x[0]), lambda: qa.qr_decode_rows(c, s, 64, torch.float16),
                 lambda: qa.qr_decode_rows(c, s, 64, torch.float32), lambda: qa.qr_norm(x, x[0]), lambda: qa.qr_norm_rows(x, x[0]),
                 lambda: qa.qr_linear8(c, s, c, s, torch.float16), lambda: qa.qr_experts8(c, s, c.view(1, 4, 128), s.view(1, 4), off, torch.float16),
                 lambda: qa.qr_choose(x, 2), lambda: qa.qr_row_bytes(0, 1), lambda: qa.qr_row_bytes(1, 130945)):
        with pytest.raises(ValueError):
            call()


def test_missing_library_fails_loudly(monkeypatch):
    monkeypatch.setattr(qr, "_lib", None)
    monkeypatch.setattr(qr, "LIB_PATH", os.path.join(ROOT, "no_such_dir", "libqr.so"))
    with pytest.raises(RuntimeError, match="missing"):
        qr_rows._lib()
