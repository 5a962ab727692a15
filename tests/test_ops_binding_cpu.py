"""What the binding of the layer operators does around a call, on the host (no call is made)."""
import pytest
import torch

import bit_quantized_all_amd as qa
from bit_quantized_all_amd import qr_ops


@pytest.mark.parametrize("fmt,shape,dims", [("int4", (3, 64, 32), (1, 2)), ("int4", (4, 24, 70), (1, 2)),
                                            ("asym4", (16, 128), (0, 1)), ("fp4", (2, 5, 32), (0, 1))])
def test_encode_weight_copies_on_the_given_stream(monkeypatch, fmt, shape, dims):
    """Whatever a weight that is not contiguous needs in copies is made, and its memory taken, where
    the call's stream is current: the packing reads it there."""
    import contextlib

    from torch.utils._python_dispatch import TorchDispatchMode

    inside, work, encoded = [], [], []

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        yield
        inside.pop()

    class Record(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if not func.is_view:
                work.append((str(func), list(inside)))
            return func(*args, **(kwargs or {}))

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(qr_ops, "qr_encode", lambda fid, flat, packed, st: encoded.append((flat, st)))
    w = torch.randn(*shape).half().transpose(*dims)
    want = w.contiguous()
    k = w.shape[-1]
    packed = torch.empty(qa.qr_weight_bytes(fmt, w.numel() // k, k), dtype=torch.uint8)
    with Record():
        qa.qr_encode_weight(fmt, w, packed, stream="s")
    assert work and all(at == ["s"] for _, at in work), work
    flat, st = encoded[0]
    kp = -(-k // qr_ops.WEIGHT_FORMATS[qr_ops._fmt(fmt)]) * qr_ops.WEIGHT_FORMATS[qr_ops._fmt(fmt)]
    assert st == "s" and torch.equal(flat[:w.numel() // k * kp].view(-1, kp)[:, :k], want.view(-1, k))


def test_outputs_that_share_a_value_with_an_input_are_refused():
    """Matrices beside each other in rows of one stride share none (on a GPU: test_ops_exact_gpu.py);
    these do, by one value at least.  Fake, never-dereferenced addresses; no call is launched."""
    from bit_quantized_all_amd import qr
    L = qr_ops._lib()
    X, W = 0x700000000000, 0x710000000000

    def linear(y, m=8, k=64, n=32, ldx=96, ldy=96):
        return L.qr_linear(4, 0, 0, X, ldx, W, y, ldy, m, n, k, None)
    for y in (X + 2 * 63, X + 2 * 65, X - 2 * 31, X - 2 * 33, X + 2 * (96 + 63), X - 2 * 96 * 3 + 2, X + 2 * (7 * 96 + 63)):
        assert linear(y) == qr.QR_ERR_ALIAS, hex(y)
    assert linear(X + 2 * 64, ldy=95) == linear(X + 2 * 64, n=33) == qr.QR_ERR_ALIAS
    assert linear(X + 2 * 64, ldx=80, ldy=80, n=17) == qr.QR_ERR_ALIAS
    # two rows of x and one of y between them, and over the second's first value
    R, O, P = 0x720000000000, 0x730000000000, 0x740000000000
    assert L.qr_experts(4, 0, 0, X, 96, 2, W, O, R, X + 2 * 65, 32, 1, 1, 32, 64, None) == qr.QR_ERR_ALIAS
    assert L.qr_combine(0, X, 96, 8, P, R, X + 2 * 47, 96, 8, 2, 48, None) == qr.QR_ERR_ALIAS
    assert L.qr_combine(0, X, 96, 8, P, R, X + 2 * 48, 97, 8, 2, 48, None) == qr.QR_ERR_ALIAS
