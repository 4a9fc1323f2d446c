"""The split of chunk attention's work, on the formulas of chunk_attention_tc.cu: tiles of four tokens laid on a line of
units, equal ranges of it, and where the combine finds the parts of a tile that lies in several."""
import bisect
import random

import pytest

TILE, UNIT = 4, 128  # kChunkTileTokens, keys of a unit
CHARGES = 3, 4       # kChunkPieceUnits, kChunkPieceUnitsQuantised


def floor_sum(m):
    q = m >> 5
    return (16 * q * (q - 1) + q * ((m & 31) + 1)) % 2 ** 32


def full_tiles_cost(i, a, charge):
    z = (a + UNIT - 1) >> 2
    return (floor_sum(i + z) - floor_sum(z)) % 2 ** 32 + i * charge


def units_of(keys):
    return -(-keys // UNIT)


def sequence_cost(length, n, charge):
    return full_tiles_cost(-(-n // TILE) - 1, length - n, charge) + units_of(length) + charge if n else 0


def pieces(lens, rows, lo, hi, charge):
    """(sequence, tile, first unit, end, units, line position of the tile) of a range, as next_piece finds them."""
    n = [min(rows[b + 1] - rows[b], lens[b]) for b in range(len(lens))]
    cost = [0]
    for b in range(len(lens)):
        cost.append(cost[-1] + sequence_cost(lens[b], n[b], charge))
    b, x = -1, lo
    while x < hi:
        if b < 0 or x >= cost[b + 1]:
            b = bisect.bisect_right(cost[:-1], x) - 1
            a, first = lens[b] - n[b], cost[b]
            i0, i1 = 0, -(-n[b] // TILE) - 1
            if x == first:
                i1 = 0
            while i0 < i1:
                mid = (i0 + i1 + 1) >> 1
                if first + full_tiles_cost(mid, a, charge) <= x:
                    i0 = mid
                else:
                    i1 = mid - 1
            i, first = i0, first + full_tiles_cost(i0, a, charge)
        else:
            i, first = i + 1, x
        tokens = min(TILE, n[b] - TILE * i)
        units = units_of(a + TILE * i + tokens)
        u0, u1 = max(0, x - first - charge), min(units, hi - first - charge)
        x = first + charge + units
        if u0 < u1:
            yield b, i, u0, u1, units, first


@pytest.mark.parametrize("a", [0, 1, 2, 3, 4, 124, 125, 126, 127, 128, 129, 1000, 4093, 1 << 24])
@pytest.mark.parametrize("charge", CHARGES)
def test_closed_form_of_full_tiles(a, charge):
    total = 0
    for i in range(200):
        assert full_tiles_cost(i, a, charge) == total
        total += units_of(a + TILE * (i + 1)) + charge


@pytest.mark.parametrize("seed", range(60))
def test_every_unit_once_and_parts_where_the_combine_looks(seed):
    charge = CHARGES[seed % 2]
    rng = random.Random(seed)
    B, pairs = rng.choice([1, 2, 5, 40]), rng.choice([1, 2, 7, 76])
    new = [rng.choice([0, 1, 1, 2, 3, 4, 5, rng.randint(1, 300)]) for _ in range(B)]
    lens = [max(0, x + rng.choice([-2, 0, 0, 1, 127, 128, rng.randint(0, 3000)])) for x in new]
    rows = [sum(new[:b]) for b in range(B + 1)]
    n = [min(x, y) for x, y in zip(new, lens)]
    total = sum(sequence_cost(x, y, charge) for x, y in zip(lens, n))
    W = min(pairs, max(total, 1))
    bounds = [w * total // W for w in range(W + 1)]
    held, slots = {}, {}
    for w in range(W):
        got = list(pieces(lens, rows, bounds[w], bounds[w + 1], charge))
        for k, (b, i, u0, u1, units, first) in enumerate(got):
            assert 0 <= u0 < u1 <= units
            for u in range(u0, u1):
                assert (b, i, u) not in held
                held[b, i, u] = w
            if not (u0 == 0 and u1 == units):  # a partial result: at most two, in slots of their own
                slot = 2 * w + (u0 == 0)
                assert slot not in slots
                slots[slot] = (b, i)
                assert k in (0, len(got) - 1)
        # what publish_parts leaves for the combine
        if bounds[w] < bounds[w + 1]:
            tail = list(pieces(lens, rows, bounds[w + 1] - 1, bounds[w + 1], charge))
            if tail and tail[0][3] < tail[0][4] and bounds[w] <= tail[0][5] + charge:
                b, i, _, _, units, first = tail[0]
                end = ((first + charge + units - 1 + 1) * W - 1) // total  # pair_of_unit
                slots["parts", b, i] = [2 * (w + k) + (k == 0) for k in range(end - w + 1)]
    want = {(b, i, u) for b in range(B) for i in range(-(-n[b] // TILE))
            for u in range(units_of(lens[b] - n[b] + min(TILE * (i + 1), n[b])))}
    assert set(held) == want
    split = {}
    for slot, tile in slots.items():
        if isinstance(slot, int):
            split.setdefault(tile, []).append(slot)
    assert {k[1:] for k in slots if not isinstance(k, int)} == set(split)
    for tile, mine in split.items():
        assert sorted(mine) == sorted(slots["parts", *tile])
