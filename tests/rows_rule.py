"""Which product kernel a call of ``qr_linear8`` or ``qr_experts8`` reaches: the rule of ``launch_dtype`` and
``launch_few`` in ``csrc/qr_product8.hip``, written out once more so that the tests can say (and check) which
variant each of their cases runs.

    ("fragments", MF, NF, KW)     16 MF rows of x by 16 NF of the weight, KW waves along k
    ("tiles", rows, columns)      tiles of rows of x by rows of the weight
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
