"""Which kernel a call of the operators over 8-bit rows reaches: the rules of ``launch_dtype`` and ``launch_few`` in
``csrc/qr_product8.hip`` and of ``row_shape`` and ``qr_choose`` in ``csrc/qr_rows.hip``, written out once more so that
the tests can say (and check) which variant each of their cases runs.

``variant``, of ``qr_linear8`` or ``qr_experts8``:
    ("fragments", MF, NF, KW)     16 MF rows of x by 16 NF of the weight, KW waves along k
    ("tiles", rows, columns)      tiles of rows of x by rows of the weight
``row_shape``, of ``qr_encode_rows`` or ``qr_norm``:
    (waves, chunks)               a row in the registers of so many waves, chunks of 8 values a lane
    ("long",)                     a row that is read again for each step
``choice``, of ``qr_choose``:
    ("rows", run, span, per)      16 lanes a token: registers of a lane, lanes of a group and experts of a lane
    ("wave",)                     a wave a token
"""
import math

from product_rule import CUS, row_tiles


def fragments(slots, e, dense, n, halves, mf, nf):
    groups = row_tiles(slots, e, dense, 16 * mf) * -(-n * halves // (16 * nf))
    return ("fragments", mf, nf, 8 if groups <= 320 else 4)


def few(slots, e, dense, n, gated, rows):
    halves = 2 if gated else 1
    area = row_tiles(slots, e, dense, 16) * -(-n // 16) * halves

    def pick(mf, nf):
        return fragments(slots, e, dense, n, halves, mf, nf)
    if rows <= 16:
        return pick(1, 4) if area >= 704 else pick(1, 2) if gated or area >= 352 else pick(1, 1)
    if area >= 2816:
        return ("fragments", 3, 4, 8) if dense and -(-slots // 48) == -(-slots // 64) else pick(4, 4)
    return pick(2, 4) if area >= 1408 else pick(2, 2) if gated or area >= 512 else pick(2, 1)


def variant(slots, n, gated, experts=None):
    """``experts`` None: qr_linear8."""
    dense = experts is None
    e = 1 if dense else experts
    rows = -(-slots // e)
    if rows <= 16:
        return few(slots, e, dense, n, gated, rows)

    def cost(bm, bn, first, more):
        cols = -(-n * (2 if gated else 1) // bn)
        tiles = cols * -(-slots // bm) if dense else cols * e * max(1.0, slots / e / bm + 0.7)
        rounds = math.ceil(tiles / CUS)
        return first if rounds <= 1 else more * rounds
    costs = [(cost(64, 64, 570, 500), 0), (cost(128, 128, 620, 620), 1), (cost(128, 256, 1000, 1000), 2), (cost(256, 256, 1440, 1440), 3)]
    which = min(costs)[1]
    return few(slots, e, dense, n, gated, rows) if which == 0 else ("tiles", *((128, 128), (128, 256), (256, 256))[which - 1])


def row_shape(rows, k):
    if rows <= 512:
        waves = 1 if k <= 512 else 4 if k <= 2048 else 16
    else:
        waves = 1 if k <= 1024 else 4 if k <= 7168 else 16
    chunks = -(-k // (512 * waves))
    return (waves, chunks) if chunks <= 4 else ("long",)


def choice(experts, groups, top):
    each, span, run = experts // groups, 16, 1
    while groups * span > 16 and span > 1:
        span //= 2
    held = -(-each // span)
    while run < held:
        run *= 2
    if top > 16 or run > 32 or groups * span > 16:
        return ("wave",)
    return ("rows", run, span, run if groups == 1 else held)
