"""Which kernel a call takes, by the rules of the library's sources written out
again: the tests assert that their sizes reach the kernels that they are for,
and test_mxfp4_rules.py that these rules are still the sources'."""
import math

LARGE_DELTA, LARGE_SPREAD = 1 << 20, 20
DENSE_SPREAD, DENSE_EXTRA = 10, 1 << 19


def apply_way(elems, nnz):
    """How mxfp4_apply_many takes nnz entries into elems values: "dense" (the
    apply's kernels, then the whole list quantised), or steps of 1024 or 256."""
    if nnz >= elems // DENSE_SPREAD + DENSE_EXTRA:
        return "dense"
    return "1024" if nnz >= LARGE_DELTA and nnz >= elems // LARGE_SPREAD else "256"


# bm, bn, full, each, held of the product's tiles
TILES = ((256, 256, 8.5, 0.0, 1), (128, 128, 2.9, 1.2, 2), (64, 64, 1.0, 0.9, 4))
CUS, TURN_BLOCKS = 256, 32
ROWS_M, ROWS_READ = 32, 16384


def _up(a, b):
    return -(-a // b)


def _turn_us(tile, tiles):
    _, _, full, each, held = tile
    per_cu = tiles / CUS
    rounds = math.ceil(per_cu / held)
    return each * rounds + full * (rounds if held == 1 else max(per_cu, 1.0))


def cut_of(m, n, k):
    """(tile side or "rows", shares of k, tile side of the last round or 0)."""
    if m <= ROWS_M and _up(m, 16) * n <= ROWS_READ:
        return "rows", 1, 0
    turns = _up(_up(k, 32), TURN_BLOCKS)
    best, least = None, math.inf
    for t, tile in enumerate(TILES):
        tiles = _up(m, tile[0]) * _up(n, tile[1])
        for shares in (1, 2, 4, 8):
            if shares > turns:
                break
            us = _up(turns, shares) * _turn_us(tile, tiles * shares)
            if shares > 1:
                us += 3.0 + shares * float(m) * float(n) * 8.0 / 4e6
            if us < least:
                best, least = (tile[0], shares, 0), us
    tiles = _up(m, 256) * _up(n, 256)
    last = tiles % CUS
    if tiles > CUS and last > 0:
        for t in (1, 2):
            us = turns * (_turn_us(TILES[0], tiles - last) + _turn_us(TILES[t], last << 2 * t)) + 3.0
            if us < least:
                best, least = (256, 1, TILES[t][0]), us
    return best


# A shape (m, n, k) for every cut, ragged in each of its sides, with shares that
# the last one does not fill, and where there are such, shares that are empty.
CUTS = {
    (4, 81, 1686): ("rows", 1, 0),
    (29, 7001, 2077): ("rows", 1, 0),
    (122, 341, 1068): (64, 1, 0),
    (62, 7023, 8625): (64, 2, 0),
    (587, 5, 6317): (64, 4, 0),
    (111, 102, 5925): (64, 4, 0),  # three of four shares have work
    (119, 37, 30298): (64, 8, 0),
    (117, 33, 12158): (64, 8, 0),  # six of eight
    (216, 13813, 1313): (128, 1, 0),
    (4034, 620, 19265): (128, 2, 0),
    (3885, 220, 27282): (128, 4, 0),
    (1579, 379, 21707): (128, 8, 0),
    (4100, 84, 14159): (128, 8, 0),  # seven of eight
    (437, 28911, 109): (256, 1, 0),
    (4081, 4090, 2079): (256, 1, 0),  # one whole round
    (1820, 10739, 150): (256, 1, 128),
    (2885, 7755, 1523): (256, 1, 128),
    (3213, 16123, 381): (256, 1, 64),
    (511, 13282, 22927): (256, 2, 0),
    (526, 4643, 30530): (256, 4, 0),
    (6725, 183, 31512): (256, 8, 0),
    (161, 7497, 26859): (256, 8, 0),  # seven of eight
}
