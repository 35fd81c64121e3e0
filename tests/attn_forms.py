"""Attention calls for each way the library cuts up its work: the call, and the
plan it is there for, (column blocks per wave, key-value heads per block,
splits, waves share the keys), of the walks over keys (forward and dq, one plan
where they have the same) and of the walk over query rows (dk, dv)."""

def ragged(sets, low, high, long=0, length=0):
    """Lengths that step through [low, high], every 9th set empty, `long` sets of `length` among them."""
    n = [0 if i % 9 == 5 else low + (i * 7919) % (high - low + 1) for i in range(sets)]
    for i in range(long):
        n[(i + 1) * sets // (long + 1)] = length + i
    return n


# name, dtype, query lengths, key lengths (None: the same rows), hq, hk, d, cap, bias, plan over keys (or those of forward and dq), plan over rows
FORMS = [
    # one head after the other in a block: the last group whole and not, sets of one tile, of several whose coordinates
    # stay in LDS and of more than four that are read again, shared heads
    ("heads_4", "bf16", ragged(1150, 1, 40, 3, 300), None, 4, 4, 32, 0.0, True, (1, 4, 1, False), (1, 4, 1, False)),
    ("heads_4_of_6", "f16", ragged(1100, 1, 36, 2, 290), None, 6, 6, 24, 5.0, True, (1, 4, 1, False), (1, 4, 1, False)),
    ("heads_2_of_3", "f16", ragged(1100, 1, 40, 2, 270), None, 6, 3, 48, 0.0, True, (1, 2, 1, False), (1, 2, 1, False)),
    ("heads_2_shared", "bf16", ragged(1060, 1, 36, 2, 200), ragged(1060, 1, 45, 2, 259), 6, 2, 40, 4.0, False, (1, 2, 1, False), (1, 2, 1, False)),
    # two column blocks a wave: split walks, and heads that share a key head (in even and in changing places of a tile)
    ("two_split", "bf16", [2048], None, 16, 16, 32, 0.0, True, (2, 1, 2, False), (2, 1, 2, False)),
    ("two_split_64", "f16", [2200], None, 16, 16, 64, 7.0, False, (2, 1, 2, False), (2, 1, 2, False)),
    ("two_shared", "bf16", [1061], None, 64, 32, 64, 6.0, True, (2, 1, 1, False), (2, 1, 2, False)),
    ("two_shared_odd", "f16", [1024], None, 96, 32, 32, 0.0, True, (2, 1, 1, False), (2, 1, 3, False)),
    # one column block and split walks, either way; waves that share the keys, split
    ("one_split", "f16", [40], [2100], 4, 2, 128, 0.0, True, (1, 1, 8, False), (1, 1, 1, False)),
    ("rows_split", "bf16", [2000], [40], 4, 2, 32, 3.0, True, (1, 1, 1, False), (1, 1, 15, False)),
    ("share_forward", "f16", [2, 1, 0, 3], [90, 17, 30, 60], 4, 2, 24, 0.0, True, ((1, 1, 1, True), (1, 1, 1, False)), (1, 1, 1, False)),
    ("share_dq", "bf16", ragged(40, 1, 9), ragged(40, 100, 300), 6, 3, 64, 5.0, True, ((1, 1, 1, False), (1, 1, 1, True)), (1, 1, 1, False)),
    ("short_sets", "f16", ragged(700, 1, 14), None, 4, 4, 64, 0.0, True, (1, 2, 1, False), (1, 2, 1, False)),
    ("share_split", "bf16", [3, 2], [2600, 700], 4, 2, 64, 0.0, True, (1, 1, 6, True), (1, 1, 1, False)),
]
