"""The plan of chunk attention, compiled for the host from the kernel's own source (csrc/chunk_plan.hpp) and followed for all pairs
of CTAs, against row tiles counted one by one: pieces in the line's order, and with a tile's rest last."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from decode_attention_mfa_gb300 import build as mfa_build

HERE = os.path.dirname(os.path.abspath(__file__))
UNIT = 128


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(mfa_build._nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", mfa_build.CSRC, "-I", cuda, "-isystem", "/usr/local/cuda/include",
                    os.path.join(HERE, "chunk_plan_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.sequence_units.restype = ctypes.c_longlong
    return lib


def follow(lib, lens, rows, pairs, charge, l2_units, turn, room=200000):
    ints = lambda a: (ctypes.c_int * len(a))(*a)  # noqa: E731
    out, parts, m = np.zeros((room, 12), np.int32), np.zeros((pairs, 4), np.int32), ctypes.c_int()
    n = lib.plan(len(lens), ints(lens), ints(rows), pairs, charge, l2_units, int(turn), out.ctypes.data_as(ctypes.c_void_p), room,
                 parts.ctypes.data_as(ctypes.c_void_p), ctypes.byref(m))
    assert n >= 0
    return [tuple(int(v) for v in x) for x in out[:n]], [tuple(int(v) for v in x) for x in parts[:m.value]]


def tiles_of(lens, rows, tile):
    """(first row, tokens, positions that the first and the last of them see) of every tile, in order, by (sequence, tile)."""
    found = {}
    for b, length in enumerate(lens):
        n = min(rows[b + 1] - rows[b], length)
        for i in range(-(-n // tile)):
            tokens = min(tile, n - tile * i)
            before = length - n + tile * i
            found[b, i] = (rows[b + 1] - n + tile * i, tokens, before + 1, before + tokens)
    return found


def check(lib, lens, rows, pairs, charge, l2_units, turn):
    tiles = tiles_of(lens, rows, lib.tile_tokens())
    pieces, parts = follow(lib, lens, rows, pairs, charge, l2_units, turn)
    held, slots, turned = set(), {}, 0
    at = {k: n for n, k in enumerate(tiles)}  # the line's order
    for w in {x[0] for x in pieces}:
        mine = [x for x in pieces if x[0] == w]
        order = [(at[x[1], x[2]], x[3]) for x in mine]
        if mine[-1][11]:
            turned += 1
            assert turn and mine[-1][3] > 0 and mine[-1][4] == mine[-1][5]
            if len(mine) > 1:  # (else what follows it on the range is a tile's charge alone)
                assert order[-1] < order[0] and mine[0][3] == 0
            order = order[-1:] + order[:-1]
        assert order == sorted(order) and not any(x[11] for x in mine[:-1])
        partial = [x for x in mine if x[10] >= 0]
        assert len(partial) <= 2 and len({x[10] for x in partial}) == len(partial)
    for w, b, i, u0, u1, units, row, tokens, seen0, seen, slot, last in pieces:
        assert (row, tokens, seen0, seen) == tiles[b, i] and units == -(-seen // UNIT) and 0 <= u0 < u1 <= units
        for u in range(u0, u1):
            assert (b, i, u) not in held
            held.add((b, i, u))
        assert (slot >= 0) == (u1 - u0 < units)
        if slot >= 0:
            assert 0 <= slot < 2 * pairs and slot not in slots
            slots[slot] = (row, tokens)
    assert held == {(b, i, u) for (b, i), (_, _, _, seen) in tiles.items() for u in range(-(-seen // UNIT))}
    # what the combine reads: for every tile in parts the slots that hold them, its beginning's first
    read = {}
    for row, tokens, w, k in parts:
        assert k >= 2
        for j in range(k):
            slot = lib.slot(w + j, int(j == 0))
            assert slot not in read
            read[slot] = (row, tokens)
    assert read == slots
    return turned


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("seed", range(80))
def test_every_unit_once_and_every_part_read(lib, seed, turn):
    rng = random.Random(seed)
    charge = lib.charge(seed % 2)
    B, pairs = rng.choice([1, 2, 5, 40, 300]), rng.choice([1, 2, 7, 76, lib.most_pairs()])
    new = [rng.choice([0, 1, 1, 2, 3, 4, 5, rng.randint(1, 300 if B < 40 else 20)]) for _ in range(B)]
    lens = [max(0, x + rng.choice([-2, 0, 0, 1, 127, 128, rng.randint(0, 3000)])) for x in new]
    lead = rng.choice([0, 5])
    rows = [lead + sum(new[:b]) for b in range(B + 1)]
    check(lib, lens, rows, pairs, charge, rng.choice([0, 20, 200, 10 ** 9]), turn)


@pytest.mark.parametrize("new,held,charge,l2_units,turns", [
    # the sequences hold 110, 164, 164 and 473 units together
    ([2048], [12000], 3, 100, True), ([1000, 1000], [9000, 10000], 3, 100, True), ([256] * 4, [5000] * 4, 4, 100, True),
    ([700, 3, 40, 1], [9000, 30000, 20000, 700], 4, 200, True),
    ([2048], [12000], 3, 640, False),                   # the pages fit L2
    ([4, 3, 1], [30000, 30000, 30000], 3, 100, False),  # a tile each: no other pair goes through the same pages
])
def test_a_rest_comes_last_where_pages_are_more_than_l2_holds(lib, new, held, charge, l2_units, turns):
    rows = [sum(new[:b]) for b in range(len(new) + 1)]
    turned = check(lib, [n + h for n, h in zip(new, held)], rows, 76, charge, l2_units, True)
    assert (turned > 0) == turns
    check(lib, [n + h for n, h in zip(new, held)], rows, 76, charge, l2_units, False)


@pytest.mark.parametrize("a", [0, 1, 2, 3, 4, 124, 125, 126, 127, 128, 129, 1000, 4093, 1 << 24, (1 << 30) - 900])
def test_units_of_a_sequence(lib, a):
    """Its closed form against a sum over its tiles, up to the longest that a call takes."""
    for quantised in (0, 1):
        charge = lib.charge(quantised)
        total = 0
        for n in range(1, 900):
            if n % 4 == 1:
                before = total  # of full tiles
            total = before + -(-(a + n) // UNIT) + charge
            assert lib.sequence_units(a + n, n, charge) == total


def test_lines_as_long_as_a_call_takes(lib):
    """Few tiles of 2^23 units: (tokens / 4 + batch) * (pages / 2 + 4) just below 2^31."""
    for quantised in (0, 1):
        charge = lib.charge(quantised)
        lens = [1 << 30] * 100 + [(1 << 30) - 1] * 100
        rows = list(range(0, 201))
        units = (1 << 23) + charge
        assert 250 * units < 2 ** 31
        for turn in (False, True):
            pieces, parts = follow(lib, lens, rows, 76, charge, 640, turn)
            assert sum(x[4] - x[3] for x in pieces) == 200 << 23
            by = {}
            for x in pieces:
                by.setdefault(x[1], []).append((x[3], x[4]))
            for b, spans in by.items():
                spans.sort()
                assert spans[0][0] == 0 and spans[-1][1] == 1 << 23 and all(p[1] == q[0] for p, q in zip(spans, spans[1:]))
            assert len(by) == 200 and sum(k for *_, k in parts) == sum(x[10] >= 0 for x in pieces)
