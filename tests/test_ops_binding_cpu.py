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
