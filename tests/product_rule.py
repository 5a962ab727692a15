"""Which product kernel a call of ``qr_linear`` or ``qr_experts`` reaches: the rule of
``launch_product`` in ``csrc/qr_product.hip``, written out once more so that the tests can
say (and check) which variant each of their cases runs.

    ("row", MR, KS)                     one or two rows, KS waves along k
    ("few", MF, NW, KW, aligned)        few rows
    ("many", rows, columns, aligned)    tiles of rows x columns of the weight's rows
"""

CUS = 256


def row_tiles(slots, experts, dense, bm):
    if dense:
        return -(-slots // bm)
    groups = min(experts + 1, slots)
    return groups + (slots - groups) // bm


def variant(slots, n, k, gated, fmt, experts=None, aligned=None, xrows=None):
    """``experts`` None: qr_linear.  ``aligned``: whether x and its rows begin on 16 bytes (by
    default a matrix of its own: if k is a multiple of 8)."""
    dense = experts is None
    e = 1 if dense else experts
    halves = 2 if gated else 1
    blocks = -(-k // 128) * 4 if fmt == "asym4" else -(-k // 32)
    rows = -(-slots // e)
    most = slots if dense else slots // 4
    if most <= 2:
        mr = 1 if most <= 1 else 2
        groups = row_tiles(slots, e, dense, mr) * n * halves // 32
        if blocks <= 64 or groups >= CUS:
            return ("row", mr, 1)
        return ("row", mr, 2 if blocks <= 128 or groups >= CUS // 2 else 4)
    if aligned is None:
        aligned = k % 8 == 0
    tiles = row_tiles(slots, e, dense, 64) * -(-n * halves // 128)
    if rows <= 64 or tiles <= CUS:
        quads = row_tiles(slots, e, dense, 16) * -(-n // 64) * halves
        if rows > 16 and quads > CUS:
            return ("few", 2, 8, 1, aligned) if quads >= 600 else ("few", 2, 4, 2, aligned)
        if quads >= 1024:
            return ("few", 1, 4, 1, aligned)
        if quads >= 192:
            return ("few", 1, 4, 4, aligned)
        return ("few", 1, 1, 4, aligned) if aligned and not gated else ("few", 1, 2, 4, aligned)
    if not aligned:
        return ("many", 64, 128, False)
    large = row_tiles(slots, e, dense, 128) * -(-n * halves // 256)
    if large >= 192 if dense else large >= 420 and rows >= 192:
        return ("many", 256, 128, True) if dense and large <= CUS else ("many", 128, 256, True)
    return ("many", 64, 128, True)
