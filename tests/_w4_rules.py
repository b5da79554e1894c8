"""A copy of the launch rules of the 4-bit products (csrc/w4_launch.hip) and of
the depths of their rings (csrc/w4_kernel.hpp), from which the tests tell
which kernel a shape reaches and how often its rings are filled again.
tests/test_w4_rules.py holds the copy's constants against the sources."""
from dataclasses import dataclass

SPLIT8, SPLIT4, STREAM_SETS, STREAM_BYTES, STREAM_WORKGROUPS = 256, 768, 1536, 64 * 1024, 2048
WAVES, LDS_BYTES, STREAM_DEPTH = 8, 156 * 1024, 3


@dataclass
class Plan:
    tokens: int        # of a tile
    rows: int          # 16-row operands of a wave
    steps: int         # of 128 columns in a block
    streamed: bool
    split: int         # waves that share rows
    blocks: int        # of the wave with the most, over all its row sets
    per_set: int       # of these, of one row set
    depth: int         # blocks of the ring
    period: int        # blocks that a copy of scales serves


def cdiv(a, b):
    return -(-a // b)


def plan(m, n, k, group, zeros, experts=None):
    """m tokens, or pairs with `experts`."""
    routed = experts is not None
    tiles = max(experts, m // 16) if routed else cdiv(m, 16)
    sets16 = cdiv(n, 16)
    if m <= experts // 8 if routed else m == 1:
        tx, r, u = 1, 1, 2
    elif m <= (experts if routed else 4):
        tx, r, u = 4, 1, 2
    elif not routed and sets16 * cdiv(m, 4) <= SPLIT8:
        tx, r, u = 4, 1, 2
    elif not routed and sets16 * cdiv(m, 8) <= SPLIT8:
        tx, r, u = 8, 1, 2
    else:
        tx, r, u = 16, 1 if sets16 * tiles <= SPLIT8 else 2, 1
    if routed:
        tiles = m if tx < 16 else tiles
    else:
        tiles = cdiv(m, tx)
    row_sets = cdiv(n, 16 * r)
    sets, blocks = row_sets * tiles, cdiv(k, 128 * u)
    groups = u * (128 // group)  # of a block
    period = 1 if groups >= 4 else 4 // groups
    if (tx < 8 or r > 1) and sets >= STREAM_SETS and cdiv(blocks * 256 * u, 1024) * 1024 * tx <= STREAM_BYTES:
        reps = max(1, sets // (WAVES * STREAM_WORKGROUPS))
        return Plan(tx, r, u, True, 1, blocks * min(reps, cdiv(row_sets, WAVES)), blocks, STREAM_DEPTH, period)
    log2 = 3 if sets <= SPLIT8 else 2 if sets <= SPLIT4 else 1 if sets < STREAM_SETS else 0
    while 1 << log2 > max(1, blocks):
        log2 -= 1
    block = (u * r + (tx * u + 3) // 4) * 1024
    slot = max(1, groups // 4) * r * 256 * (2 if zeros else 1)
    depth = 5
    while depth > 2 and (depth * block + (cdiv(depth, period) + (period > 1)) * slot) * WAVES > LDS_BYTES:
        depth -= 1
    mine = cdiv(blocks, 1 << log2)
    return Plan(tx, r, u, False, 1 << log2, mine, mine, depth, period)
