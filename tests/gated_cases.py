"""Sizes (groups, rows, n, k, rows of each expert or None) at which every kernel of the gated product runs, B stored
either way: those whose shapes belong to few rows of many columns, and tiles of 256."""
SIZES = [(0, 3, 8200, 1100), (0, 1, 8193, 130), (0, 39, 2501, 1099), (0, 20, 8200, 600), (0, 60, 7000, 1100), (0, 33, 7001, 72),
         (0, 27, 2504, 136), (40, 120, 500, 600), (40, 300, 500, 1100), (0, 5, 100, 2300), (0, 12, 13000, 600), (0, 31, 13000, 520),
         (0, 30, 100, 1100), (0, 200, 100, 70), (0, 900, 1100, 130), (0, 1090, 2050, 130), (0, 2049, 2200, 1100)]


def shares(groups, rows):
    """Uneven rows of each expert, some of them without any."""
    if not groups:
        return None
    counts = [(5 * e * e + 3 * e) % 7 for e in range(groups)]
    counts[1] = 0
    scale = rows / sum(counts)
    return [int(c * scale) for c in counts]
