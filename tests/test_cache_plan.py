"""How the workgroups of the cached attention share its work, and the division of
a slot into page and place, on the host."""
import ctypes
import random

import numpy as np
import pytest

import all_reduce_amd as ar

SZ, U32, I32, I64 = ctypes.c_size_t, ctypes.c_uint32, ctypes.c_int32, ctypes.c_int64


def pieces_of(lengths, capacity, window, queries, tokens, ranks, heads, group, grid, block, team):
    lib = ar.library()
    fn = lib.ar_cache_attention_share
    fn.restype = SZ
    fn.argtypes = [ctypes.POINTER(I32), SZ, SZ, SZ, U32, U32, U32, U32, U32, U32, U32, U32, ctypes.POINTER(U32), ctypes.c_void_p,
                   SZ]
    teams = (U32 * 5)()
    most = 1 << 16
    out = np.zeros((most, 13), dtype=np.uint32)
    n = fn(lengths, len(lengths), capacity, window, queries, tokens, ranks, heads, group, grid, block, team, teams,
           out.ctypes.data, most)
    assert n <= most
    return list(teams), out[:n].astype(np.int64).tolist()


def check_plan(lengths, capacity, window, tokens, ranks, heads, group, grid, queries):
    """Every token of every unit is in one piece; a unit's pieces meet in slots and
    counters of their own, in the numbers that the teams wait for; equal shares."""
    covered, partial, sizes, slots = {}, {}, [], set()
    array = (I32 * len(lengths))(*lengths)
    (waves, side, tiles, a_pass, step), _ = pieces_of(array, capacity, window, queries, tokens, ranks, heads, group, grid, 0, 0)
    assert waves in (1, 4) and side <= waves and a_pass == waves // side << tokens and step >= a_pass and step % a_pass == 0
    wide = 1 << queries
    assert (tiles - 1) * side * wide < group <= tiles * side * wide
    teams = grid * 4 // waves
    for block in range(grid):
        for team in range(4 // waves):
            _, pieces = pieces_of(array, capacity, window, queries, tokens, ranks, heads, group, grid, block, team)
            sizes.append(sum(p[4] - p[3] for p in pieces))
            for rank, seq, unit, s0, s1, steps, t0, t1, slot, gc, gn, uc, groups in pieces:
                assert 0 <= rank < ranks and 0 <= seq < len(lengths) and 0 <= unit < tiles * heads and 0 <= s0 < s1 <= steps
                covered.setdefault((rank, seq, unit), []).append((s0, s1, t0, t1))
                if s0 == 0 and s1 == steps:
                    continue
                assert slot < 2 * teams and gc < 4 * teams and uc < 4 * teams
                assert slot not in slots
                slots.add(slot)
                partial.setdefault((rank, seq, unit), []).append((gc, gn, uc, groups))
    assert len(covered) == ranks * heads * len(lengths) * tiles
    for (_, seq, _), got in covered.items():
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
            assert len(sizes_of) <= 32
        uc, groups = unit_counter.pop()
        assert groups == len(members)
        for c in (*members, uc):
            assert used.setdefault(c, key) == key, "two units share a counter"
        assert len({*members, uc}) == len(members) + 1
    busy = [x for x in sizes if x]
    assert max(busy) - min(busy) <= 1
    assert len(busy) == teams or max(busy) == 1
    return waves, side


PLANS = [
    ([0], 128, 0, 5, 1, 1, 1, 8), ([1], 128, 0, 5, 1, 1, 8, 512), ([5000], 1 << 20, 0, 5, 1, 1, 16, 512),
    ([131072], 1 << 20, 0, 5, 8, 1, 17, 512), ([70001] * 3, 1 << 17, 0, 4, 1, 1, 33, 256),
    ([0] * 700, 1024, 0, 5, 1, 3, 64, 512), ([-1, 5, 2000, 1025, 0, 1024], 1024, 0, 5, 2, 1, 65, 16),
    ([2 ** 31 - 1], 2 ** 31 - 1, 0, 5, 1, 1, 8, 512), ([2 ** 31 - 1, 7], 2 ** 31 - 1, 129, 5, 1, 5, 200, 64),
    ([2 ** 31 - 1] * 9, 2 ** 31 - 1, 0, 5, 8, 4, 16, 512), ([3, 2 ** 31 - 1, 0], 2 ** 31 - 1, 0, 4, 2, 250, 64, 256),
    ([100000, 3], 1 << 17, 50000, 5, 2, 2, 8, 512), ([20] * 700 + [32768], 1 << 16, 0, 5, 1, 2, 8, 512),
    ([2 ** 31 - 1] + [1] * 600, 2 ** 31 - 1, 0, 5, 1, 2, 8, 512), ([2 ** 31 - 1, 3], 2 ** 50, 0, 5, 1, 2, 8, 512),
    ([2 ** 31 - 1, 100], 2 ** 50, 2 ** 40, 4, 32, 16, 4, 256), ([2 ** 31 - 1] * 3, 2 ** 62, 0, 5, 16, 8, 64, 512),
]


@pytest.mark.parametrize("lengths,capacity,window,tokens,ranks,heads,group,grid", PLANS,
                         ids=[str(i) for i in range(len(PLANS))])
def test_shares(lengths, capacity, window, tokens, ranks, heads, group, grid):
    for queries in (4, 5):
        check_plan(lengths, capacity, window, tokens, ranks, heads, group, grid, queries)


def test_drawn_shares():
    rng = random.Random(4)
    seen = set()
    for _ in range(200):
        seqs = rng.choice([1, 1, 2, 3, 9, 40, 130])
        longest = rng.choice([1, 130, 600, 2000, 30000])
        lengths = [int(longest * rng.random() ** 2) for _ in range(seqs)]
        lengths[rng.randrange(seqs)] = longest
        seen.add(check_plan(lengths, 32768, rng.choice([0, 0, 1, 100, 5000]), rng.choice([4, 5]),
                            rng.choice([1, 2, 8]), rng.choice([1, 1, 3]), rng.choice([1, 8, 16, 17, 40, 100]),
                            rng.choice([8, 16, 64, 256]), rng.choice([4, 5])))
    assert seen == {(1, 1), (4, 1), (4, 2), (4, 4)}


def test_steps_of_extreme_calls():
    """As many units as a call may have, of the longest sequences: steps are counted in
    31 bits and shifts stay below 32."""
    array = (I32 * 65536)(*[2 ** 31 - 1] * 65536)
    (waves, _, tiles, _, step), pieces = pieces_of(array, 2 ** 31 - 1, 0, 4, 5, 32, 8, 1, 512, 511, 0)
    units = 65536 * 32 * 8 * tiles
    steps = -(-(2 ** 31 - 1) // step)
    assert units == 2 ** 24 and units * steps < 2 ** 31 and step <= 2 ** 30 and waves == 4
    assert pieces[-1][:5] == [31, 65535, 7, pieces[-1][3], steps]


@pytest.mark.parametrize("tokens,length", [(4, 0), (4, 16), (4, 60), (4, 100), (4, 2 ** 31 - 1), (5, 1), (5, 100), (5, 200), (5, 2 ** 31 - 1)])
def test_longest_steps(tokens, length):
    """The same number of units for waves of 16 and 32 tokens, and for single waves, whose steps
    are the longest."""
    array = (I32 * 65536)(*[length] * 65536)
    (waves, _, tiles, _, step), pieces = pieces_of(array, 2 ** 31 - 1, 0, 4, tokens, 32, 8, 1, 512, 511, 3 if length <= 200 else 0)
    units = 65536 * 32 * 8 * tiles
    steps = max(1, -(-length // step))
    assert units == 2 ** 24 and units * steps < 2 ** 31 and step <= 2 ** 30
    assert waves == (4 if length > 200 else 1)
    if (tokens, length) in ((4, 100), (5, 200)):
        assert step == 2 ** 30
    assert pieces[-1][:3] == [31, 65535, 7] and pieces[-1][4:6] == [steps, steps]
    assert pieces[-1][7] == length


def test_parts():
    """What a group's and a unit's last team reads: every team's slot once, then the
    slot of every group's first."""
    fn = ar.library().ar_cache_attention_part
    fn.restype = U32
    fn.argtypes = [U32] * 5
    for w0, w1 in ((0, 1), (3, 5), (15, 16), (0, 511), (7, 40), (16, 31), (31, 32), (5, 2047), (3, 18), (3, 19), (9, 72), (9, 73), (0, 255), (0, 256)):
        def slot(w):
            return 2 * w + (w == w0)
        starts = []
        n = w1 - w0 + 1
        each = 16 if n <= 16 else 8 if n <= 64 else 16 if n <= 256 else 32
        for b in range(w0, w1 + 1, each):
            members = list(range(b, min(w1, b + each - 1) + 1))
            starts.append(members[0])
            for w in members:
                assert [fn(w0, w1, w, 1, i) for i in range(len(members))] == [slot(m) for m in members]
        for w in (w0, w1, (w0 + w1) // 2):
            assert [fn(w0, w1, w, 2, i) for i in range(len(starts))] == [slot(m) for m in starts]


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


def streams(lengths, ranks, heads, group, token_bytes, queries=4, tokens=5, grid=512, window=0, capacity=2 ** 31 - 1):
    fn = ar.library().ar_cache_attention_streams
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.POINTER(I32), SZ, SZ, SZ] + [U32] * 7
    return fn((I32 * len(lengths))(*lengths), len(lengths), capacity, window, queries, tokens, ranks, heads, group, grid,
              token_bytes)


def test_streamed_loads_go_by_the_cache_that_is_read():
    """Loads past the caches from 128 MiB of keys and values on, whatever the length of a step
    is: 512 bytes a token are heads of 128 in 16 bits."""
    assert not streams([67] * 256, 8, 1, 8, 512)       # 67 MiB
    assert not streams([33] * 256, 8, 1, 8, 512)
    assert not streams([200] * 128, 8, 1, 8, 512)      # 100 MiB
    assert not streams([1] * 4096, 8, 1, 8, 512)       # 16 MiB, in tiles of 32 tokens 512
    assert streams([8192] * 64, 8, 1, 8, 512)
    assert not streams([8192] * 64, 8, 1, 8, 512, window=127)
    assert streams([8192] * 64, 8, 1, 8, 512, window=1024)
    assert streams([131072], 8, 1, 8, 256) and not streams([131072], 1, 1, 8, 256)
    assert streams([2 ** 31 - 1], 1, 1, 1, 32) and streams([2 ** 31 - 1] + [1] * 600, 1, 1, 1, 512)
    assert not streams([5] * 65536, 1, 1, 1, 32)
    # waves or units that read the same tokens for other query heads
    assert streams([8192] * 64, 8, 1, 32, 512, queries=5) and not streams([8192] * 64, 8, 1, 33, 512, queries=5)
    assert streams([250] * 600, 8, 1, 16, 512) and not streams([250] * 600, 8, 1, 17, 512)


def test_drawn_streamed_loads():
    """Tokens decide, on both sides of 128 MiB, for every choice of teams and steps."""
    rng = random.Random(6)
    seen = set()
    for _ in range(400):
        seqs, ranks, heads, tokens = rng.choice([1, 3, 20, 64, 65, 300, 2000]), rng.choice([1, 2, 8]), rng.choice([1, 4]), \
            rng.choice([4, 5])
        token_bytes = rng.choice([32, 256, 512, 1024, 2048])
        limit = (1 << 27) / (token_bytes * ranks * heads)  # tokens
        share = [rng.random() ** 2 + 0.01 for _ in range(seqs)]
        share = [x / sum(share) for x in share]
        lengths = [min(2 ** 21, max(1, int(x * limit * rng.choice([0.5, 0.9, 1.1, 2.0])))) for x in share]
        want = sum(lengths) * ranks * heads * token_bytes >= 1 << 27
        assert streams(lengths, ranks, heads, 8, token_bytes, tokens=tokens, grid=rng.choice([64, 256, 512])) == want
        seen.add((want, seqs * ranks * heads > 512))
    assert len(seen) == 4
