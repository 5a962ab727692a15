"""MI355X (gfx950) block-quantization codec and compressed-domain reduction.

The kernels live in ``csrc/`` and are built into ``libqr.so``; ``qr`` is the
ctypes binding of the C ABI declared in ``include/qr.h``, ``qr_ops`` that of the
layer operators over 4-bit weights declared in ``include/qr_ops.h``, ``qr_rows`` that
of the norm, the router's choice and the operators over 8-bit rows declared in
``include/qr_rows.h``.
"""
from .qr import (FORMATS, MAX_RANKS, QR_ERR_ALIAS, QR_ERR_ALIGN, QR_ERR_ARG, QR_ERR_HIP,  # noqa: F401
                 QR_ERR_SIZE, QR_ERR_UNSUPPORTED, QR_OK, QRError, TILE_VALUES, lib, qr_decode, qr_encode,
                 qr_packed_bytes, qr_reduce_compressed, qr_reduce_compressed_mixed, qr_status_string)
from .qr_ops import (qr_combine, qr_encode_weight, qr_experts, qr_linear, qr_route,  # noqa: F401
                     qr_weight_bytes)
from .qr_rows import (qr_choose, qr_decode_rows, qr_encode_rows, qr_experts8, qr_linear8,  # noqa: F401
                      qr_norm, qr_norm_rows, qr_row_bytes)
