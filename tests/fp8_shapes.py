"""Sizes at which vnm_fp8_linear takes each of its tilings on 152 SMs: the rule's answer, T, R, K
and whether a CTA (or pair) takes more than one tile."""

# (tokens of a tile, splits of K): 8 the few-token kernel, 0 pairs of CTAs
SHAPES = [
    ((8, 1), 1, 4095, 1000, False), ((8, 1), 8, 11008, 4096, False),
    ((16, 1), 16, 20000, 300, False), ((16, 1), 12, 39700, 200, True),
    ((16, 2), 16, 11008, 4096, False), ((16, 4), 16, 4096, 4096, False), ((16, 4), 9, 3001, 1000, False),
    ((16, 8), 11, 129, 5001, False), ((16, 8), 13, 300, 8192, False),
    ((32, 1), 32, 11008, 4096, False), ((32, 1), 24, 39200, 300, True),
    ((32, 2), 25, 6000, 700, False), ((32, 4), 32, 4096, 4096, False), ((32, 4), 31, 5000, 1000, False),
    ((32, 8), 100, 260, 6001, False),
    ((64, 1), 60, 11007, 1000, False), ((64, 1), 36, 39990, 300, True),
    ((64, 2), 61, 5999, 700, False), ((64, 4), 64, 4096, 4096, False), ((64, 4), 130, 1000, 4100, False),
    ((64, 8), 419, 120, 5818, False),
    ((128, 1), 100, 11008, 4096, False), ((128, 1), 69, 19676, 1170, True),
    ((128, 2), 777, 1000, 1041, False), ((128, 2), 256, 4096, 4096, False),
    ((128, 4), 128, 4096, 4096, False), ((128, 4), 333, 1000, 1000, False),
    ((128, 8), 2008, 120, 3370, False),
    ((0, 1), 600, 2050, 300, False), ((0, 1), 2500, 2600, 1041, True),
]

# one K block a tile, several tiles a CTA: with a scale a row of W only
ONE_BLOCK = [((16, 1), 10, 39601, 100, True), ((32, 1), 19, 39201, 90, True)]


def several_tiles(plan, T, R, sm_count):
    """Whether a CTA or pair takes more than one tile of an unsplit product."""
    tile, splits = plan
    if tile == 0:
        return -(-T // 256) * -(-R // 256) > sm_count // 2
    return tile != 8 and splits == 1 and -(-R // 128) * -(-T // tile) > sm_count * (2 if tile <= 64 else 1)
