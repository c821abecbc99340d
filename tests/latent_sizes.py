"""Sizes of the latent attention tests, and the forms that calls of them take."""

# Sequences whose last tokens' rows are not finite and that some of the call's tokens do
# not see: new tokens, lengths, heads, page size, pages of the table (None: as many as the
# longest needs), rows of a workgroup.  Tiles of one step, of several, and so many that
# the last steps are another workgroup's.
UNSEEN = [
    ([9], [9], 10, 16, None, 32),
    ([9, 2], [75, 33], 10, 64, None, 32),
    ([9, 4], [1500, 33], 7, 8, None, 32),
    ([12], [2100], 5, 64, None, 32),
    ([20], [24], 20, 64, 512, 64),
    ([20, 6], [20, 8], 20, 16, 2048, 64),
    ([20], [330], 20, 8, 4096, 64),
    ([20], [1500], 20, 16, 2048, 64),
    ([20], [1500], 20, 64, 512, 64),
    ([3] * 70, [3 + 5 * b for b in range(70)], 12, 16, 1024, 64),  # more sequences than lanes
]

# Sequences far shorter than their table: the larger tile at few rows.  As above.
SHORT = [
    ([20], [60], 20, 64, 512, 64),
    ([7, 0, 30, 1], [70, 5, 1000, 600], 20, 8, 4096, 64),
    ([40], [300], 12, 16, 4096, 64),
    ([1, 19], [1, 19], 20, 32, 1024, 64),
    ([32], [40], 100, 64, 4096, 64),
    ([9], [9], 100, 64, 4096, 32),   # fewer than 32 tiles: the width does not count
    ([5, 2], [400, 2], 65, 64, 4096, 32),
]

# Caches of many rows.
LONG = [([1], [100000], 4, 64, None, 32), ([1, 1], [100000, 31], 2, 1024, None, 32), ([7], [20001], 20, 8, 8192, 64)]

# Prompts whose last keys are not finite: new tokens, keys, heads, whether the keys are
# shared among workgroups.
UNSEEN_KEYS = [([50], [50], 3, False), ([50], [2000], 3, True), ([130, 7], [700, 530], 2, True), ([40, 300], [40, 300], 4, False)]


def capacity(lens, page, width):
    return (max(-(-n // page) for n in lens) if width is None else width) * page


def rows_of(lib, counts, lens, H, page, width, e4m3):
    """Rows of a workgroup in the absorbed form."""
    return lib.skg_latent_rows(len(counts), sum(counts), H, capacity(lens, page, width), 1 if e4m3 else 0)


def parts_of(lib, counts, keys, H):
    return lib.skg_latent_parts(len(counts), sum(counts), sum(keys), H)
