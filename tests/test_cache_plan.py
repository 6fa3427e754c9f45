"""How the workgroups of the cached attention share its work, and the division of
a slot into page and place, on the host."""
import ctypes
import random

import numpy as np
import pytest

import all_reduce_amd as ar

SZ, U32, I32, I64 = ctypes.c_size_t, ctypes.c_uint32, ctypes.c_int32, ctypes.c_int64


def pieces_of(lengths, capacity, window, step, units, grid, block):
    lib = ar.library()
    fn = lib.ar_cache_attention_share
    fn.restype = SZ
    fn.argtypes = [ctypes.POINTER(I32), SZ, SZ, SZ, U32, U32, U32, U32, ctypes.c_void_p, SZ]
    most = len(lengths) * units + 2
    out = np.zeros((most, 12), dtype=np.uint64)
    n = fn((I32 * len(lengths))(*lengths), len(lengths), capacity, window, step, units, grid, block,
           out.ctypes.data, most)
    assert n <= most
    return out[:n].astype(np.int64).tolist()


def check_plan(lengths, capacity, window, step, units, grid):
    """Every token of every unit is in one piece; a unit's pieces meet in slots and
    counters of their own, in the numbers that the workgroups wait for; equal shares."""
    covered, partial, sizes = {}, {}, []
    slots = set()
    for block in range(grid):
        pieces = pieces_of(lengths, capacity, window, step, units, grid, block)
        sizes.append(sum(p[3] - p[2] for p in pieces))
        for unit, seq, s0, s1, steps, t0, t1, slot, gc, gn, uc, groups in pieces:
            assert 0 <= unit < units and 0 <= seq < len(lengths) and 0 <= s0 < s1 <= steps
            covered.setdefault((unit, seq), []).append((s0, s1, t0, t1))
            if s0 == 0 and s1 == steps:
                continue
            assert slot < 2 * grid and gc < 4 * grid and uc < 4 * grid
            assert slot not in slots
            slots.add(slot)
            partial.setdefault((unit, seq), []).append((gc, gn, uc, groups))
    assert set(covered) == {(u, s) for u in range(units) for s in range(len(lengths))}
    for (unit, seq), got in covered.items():
        n = lengths[seq]
        first = end = 0
        if 0 <= n <= capacity:
            end, first = n, max(0, n - window) if window else 0
        got.sort()
        at, t = 0, first
        for s0, s1, t0, t1 in got:
            assert s0 == at and t0 == t and t1 - t0 <= (s1 - s0) * step
            at, t = s1, t1
        assert at == max(1, -(-(end - first) // step)) and t == end
    used = {}
    for key, got in partial.items():
        unit_counter = {(uc, groups) for _, _, uc, groups in got}
        assert len(unit_counter) == 1
        members = {}
        for gc, gn, _, _ in got:
            members.setdefault(gc, []).append(gn)
        for gc, sizes_of in members.items():
            assert all(x == len(sizes_of) for x in sizes_of), (key, gc, sizes_of)
        uc, groups = unit_counter.pop()
        assert groups == len(members)
        for c in (*members, uc):
            assert used.setdefault(c, key) == key, "two units share a counter"
        assert len({*members, uc}) == len(members) + 1
    busy = [x for x in sizes if x]
    assert max(busy) - min(busy) <= 1
    assert len(busy) == grid or max(busy) == 1


PLANS = [
    ([0], 128, 0, 128, 1, 8), ([1], 128, 0, 128, 1, 512), ([5000], 1 << 20, 0, 128, 1, 512),
    ([131072], 1 << 20, 0, 128, 8, 512), ([70001] * 3, 1 << 17, 0, 64, 1, 256), ([0] * 700, 1024, 0, 128, 3, 512),
    ([-1, 5, 2000, 1025, 0, 1024], 1024, 0, 128, 2, 16), ([2 ** 31 - 1], 2 ** 31 - 1, 0, 128, 1, 512),
    ([2 ** 31 - 1, 7], 2 ** 31 - 1, 129, 128, 5, 64), ([100000, 3], 1 << 17, 50000, 128, 4, 512),
]


@pytest.mark.parametrize("lengths,capacity,window,step,units,grid", PLANS, ids=[str(i) for i in range(len(PLANS))])
def test_shares(lengths, capacity, window, step, units, grid):
    check_plan(lengths, capacity, window, step, units, grid)


def test_drawn_shares():
    rng = random.Random(4)
    for _ in range(150):
        seqs = rng.choice([1, 1, 2, 3, 9, 40, 130])
        longest = rng.choice([1, 130, 2000, 30000])
        lengths = [int(longest * rng.random() ** 2) for _ in range(seqs)]
        lengths[rng.randrange(seqs)] = longest
        check_plan(lengths, 32768, rng.choice([0, 0, 1, 100, 5000]), rng.choice([64, 128]), rng.choice([1, 2, 8, 24]),
                   rng.choice([8, 16, 64, 256, 512]))


def test_places():
    fn = ar.library().ar_cache_place
    fn.argtypes = [SZ, SZ, I64, ctypes.POINTER(U32)]
    at = (U32 * 2)()
    rng = random.Random(5)
    most = 2 ** 31 - 1
    sizes = [*range(1, 70), 100, 127, 128, 129, 255, 256, 1000, 1023, 1024, 1 << 16, 65537, (1 << 30) - 1, 1 << 30,
             (1 << 30) + 1, most]
    for page in sizes:
        pages = most // page
        near = [0, 1, page - 1, page, page + 1, 2 * page - 1, (pages - 1) * page, pages * page - 1]
        for slot in [*near, *(rng.randrange(pages * page) for _ in range(300))]:
            if slot >= pages * page:
                continue
            assert fn(pages, page, slot, at) == 1
            assert (at[0], at[1]) == divmod(slot, page), (page, slot)
        for slot in (-1, -2 ** 40, pages * page, 2 ** 31, 2 ** 32 + 1, 2 ** 63 - 1):
            assert fn(pages, page, slot, at) == 0
