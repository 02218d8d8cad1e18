"""Calls of ft_kv_attend that take each number of teams, by the rule of csrc/kv_rules.h: name -> (format, head size, KV heads,
query heads of each, page, lengths, teams)."""

_ragged = [2000, 1, 0, 1700, 33, 1999, 64, 1024, 500, 1311, 2047, 3]

CALLS = {
    # two teams to a compute unit: rows of 64 bytes from 16 items on, of 128 bytes from 192 on
    "e4m3_64_16_items": ("e4m3", 64, 4, 3, 32, [4000, 3001, 2500, 5003], 512),
    "e4m3_64_one_long_request": ("e4m3", 64, 16, 2, 64, [20011], 512),
    "e4m3_64_wide_groups": ("e4m3", 64, 4, 12, 16, [4000, 3001, 2500, 5003], 512),
    "bf16_64_192_items": ("bf16", 64, 8, 2, 16, [2000, 1700, 33, 1999, 64, 1024, 500, 1311, 2047, 3] * 2 + [9, 90, 900, 2001], 512),
    "bf16_64_wide_groups": ("bf16", 64, 16, 9, 16, _ragged + [4097], 512),
    "e4m3_128_192_items": ("e4m3", 128, 8, 2, 32, [2000, 1700, 33, 1999, 64, 1024, 500, 1311, 2047, 3] * 2 + [9, 90, 900, 2001], 512),
    "bf16_64_more_items_than_teams": ("bf16", 64, 12, 1, 16, (_ragged + [17]) * 4, 512),
    # one team, below those numbers
    "e4m3_64_15_items": ("e4m3", 64, 3, 3, 32, [4000, 3001, 2500, 5003, 3024], 256),
    "bf16_64_190_items": ("bf16", 64, 10, 2, 16, [2000, 1700, 33, 1999, 64, 1024, 500, 1311, 2047, 3] + [9, 90, 900, 2001, 41, 1500, 77, 1030, 640], 256),
    "e4m3_128_190_items": ("e4m3", 128, 10, 2, 32, [2000, 1700, 33, 1999, 64, 1024, 500, 1311, 2047, 3] + [9, 90, 900, 2001, 41, 1500, 77, 1030, 640], 256),
    # the launch has room for two, by its table and number of requests, and few of them hold anything
    "bf16_64_few_busy": ("bf16", 64, 8, 2, 16, [0] * 11 + [20011] + [0] * 11 + [5], 256),
    "e4m3_64_few_busy": ("e4m3", 64, 2, 2, 16, [0] * 9 + [30011, 0, 2, 0, 40], 256),
    "bf16_64_short_items": ("bf16", 64, 8, 2, 16, [40] * 24 + [1025], 200),
    # rows of 256 bytes and more: one team at most, with more items than that too
    "bf16_128_clamped": ("bf16", 128, 8, 2, 16, [2000, 1, 1700, 33, 1999, 64, 1024, 500, 1311, 2047] * 4, 256),
    "bf16_128_clamped_wide_groups": ("bf16", 128, 8, 10, 16, [2000, 1, 1700, 33, 1999, 64, 1024, 500, 1311, 2047] * 4, 256),
    "e4m3_256_clamped": ("e4m3", 256, 6, 2, 32, [2000, 1, 1700, 33, 1999, 64, 1024, 500, 1311, 2047] * 5, 256),
    "bf16_256_clamped": ("bf16", 256, 6, 2, 32, [2000, 1, 1700, 33, 1999, 64, 1024, 500, 1311, 2047] * 5, 256),
}


def width(P, lens):
    """Table entries of a request: more than whole items have."""
    return max(-(-max(lens) // P), 1) + 1 + 1024 // P
