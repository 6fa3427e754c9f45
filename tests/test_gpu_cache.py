"""The operators of ar_cache.h on the GPU against their definitions in 64 bits
(tests/cache_ref.py, with the bounds derived there): writing the paged cache,
reading it back, attention of one new token a sequence, and the half layer they
make with the operators around the all-reduce."""
import pytest
import torch

import all_reduce_amd as ar
import block_ref
import cache_ref as ref
from gpu_util import note

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": E4M3}


@pytest.fixture(scope="module")
def comm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = ar.Comm(device="cuda:0", max_ranks=32, max_ll_bytes_per_rank=1 << 16)
    yield c
    c.close()


def draw(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def raw(t):
    """Bit patterns, so that NaN equals itself."""
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def pages_of(pools):
    scales = dict(key_scales=[p.key_scales for p in pools], value_scales=[p.value_scales for p in pools]) \
        if pools[0].eight else {}
    return dict(key_pages=[p.keys for p in pools], value_pages=[p.values for p in pools], **scales)


# ---- writing and reading back ------------------------------------------------
COPIES = [
    # ranks, tokens, heads, dim, places of a page, dtype, cache, order: every group of
    # lanes whole and not, one token to several workgroups, more than 64 MiB
    (1, 1, 1, 16, 1, "bf16", "bf16", "head"), (2, 3, 1, 64, 16, "fp16", "e4m3", "head"),
    (3, 17, 2, 80, 7, "fp16", "fp16", "token"), (1, 33, 3, 128, 64, "bf16", "e4m3", "token"),
    (8, 64, 1, 128, 64, "bf16", "e4m3", "head"), (2, 100, 5, 48, 20, "fp32", "e4m3", "pair"),
    (1, 50, 2, 256, 16, "fp32", "fp32", "pair"), (4, 29, 3, 192, 32, "bf16", "e4m3", "pair"),
    (2, 40, 1, 240, 3, "fp32", "e4m3", "head"), (32, 2, 2, 112, 8, "bf16", "bf16", "head"),
    (2, 1000, 4, 96, 128, "fp16", "e4m3", "token"), (1, 300, 8, 32, 1, "fp32", "fp32", "token"),
    (2, 9000, 4, 256, 256, "bf16", "bf16", "head"), (3, 20000, 3, 80, 50, "fp32", "e4m3", "pair"),
    (1, 777, 2, 144, 33, "bf16", "e4m3", "head"), (5, 257, 1, 208, 64, "fp16", "fp16", "pair"),
]


def copy_case(ranks, tokens, heads, dim, page, dtype, cache, order, seed=1):
    """(rows with a wider stride [ranks, tokens, 3 heads, dim] with keys and values as
    parts of them, slots with some that are none, pools)."""
    pages = -(-tokens * 5 // (4 * page)) + 1
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(seed))[:tokens]
    slots[5::7] = -1
    slots[6::29] = pages * page
    slots[9::31] = -2 ** 40
    slots[11::37] = 2 ** 40
    pools = [ref.Pool(pages, heads, page, dim, DT[cache], order) for _ in range(ranks)]
    return slots, pools


@pytest.mark.parametrize("ranks,tokens,heads,dim,page,dtype,cache,order", COPIES)
def test_write_and_read(comm, ranks, tokens, heads, dim, page, dtype, cache, order):
    note(f"cache write R={ranks} {tokens}x{heads}x{dim} page {page} {dtype} {cache} {order}")
    slots, pools = copy_case(ranks, tokens, heads, dim, page, dtype, cache, order)
    before = [p.snapshot() for p in pools]
    x = draw((ranks, tokens, 3 * heads * dim), tokens + dim, DT[dtype], 2.0)
    x *= torch.linspace(0.1, 3, tokens)[None, :, None].to(DT[dtype])
    rows = x.cuda()
    keys, values = ([r[:, a * heads * dim:(a + 1) * heads * dim].unflatten(1, (heads, dim)) for r in rows]
                    for a in (1, 2))
    comm.cache_write(keys, values, slots.cuda(), **pages_of(pools))
    torch.cuda.synchronize()
    assert torch.equal(raw(rows.cpu()), raw(x)), "the rows changed"
    size = pools[0].keys.shape[0] * page
    there = ((slots >= 0) & (slots < size)).nonzero()[:, 0]
    at = (slots[there] // page, slots[there] % page)
    for r, pool in enumerate(pools):
        assert pool.edges()
        for which, t, s in (("key", keys, pool.key_scales), ("value", values, pool.value_scales)):
            y = t[r].cpu()[there]
            got = pool.bytes(which)[at[0].cuda(), :, at[1].cuda()].cpu()
            if pool.eight:
                want, tol, scale, scale_tol = ref.quantise(y)
                block_ref.assert_within(s[at[0].cuda(), :, at[1].cuda()], scale, scale_tol, f"{which} scales")
                block_ref.assert_within(got.view(E4M3).float(), want, tol, f"{which} values")
            else:
                assert torch.equal(raw(got), raw(y)), which
        # the places of no token are as they were
        after = pool.snapshot()
        for which, s in (("key", pool.key_scales), ("value", pool.value_scales)):
            pool.bytes(which)[at[0].cuda(), :, at[1].cuda()] = 0
            if s is not None:
                s[at[0].cuda(), :, at[1].cuda()] = 0
        for a, b in zip(pool.raw, before[r]):
            changed = a != b
            assert not bool((changed & (a != 0)).any()), "a place of no token was written"
        for a, b in zip(pool.raw, after):
            a.copy_(b)

    # and back, into parts of the same rows; twice the same slot
    slots[there[-1]] = slots[there[0]]
    note("cache read")
    to = torch.full((ranks, tokens, 2 * heads * dim * DT[dtype].itemsize), ref.POISON, dtype=torch.uint8,
                    device="cuda:0").view(DT[dtype])
    out_k, out_v = ([r[:, a * heads * dim:(a + 1) * heads * dim].unflatten(1, (heads, dim)) for r in to]
                    for a in (0, 1))
    frozen = [p.snapshot() for p in pools]
    cached = pages_of(pools)
    comm.cache_read(slots.cuda(), cached["key_pages"], cached["value_pages"], out_k, out_v,
                    cached.get("key_scales"), cached.get("value_scales"))
    torch.cuda.synchronize()
    at = (slots[there] // page, slots[there] % page)
    gone = torch.ones(tokens, dtype=torch.bool)
    gone[there] = False
    for r, pool in enumerate(pools):
        assert all(torch.equal(a, b) for a, b in zip(pool.raw, frozen[r])), "the cache changed"
        for which, t, s in (("key", out_k, pool.key_scales), ("value", out_v, pool.value_scales)):
            x = pool.bytes(which)[at[0].cuda(), :, at[1].cuda()].cpu()
            if pool.eight:  # one product in binary32, one rounding
                x = (x.view(E4M3).float() * s[at[0].cuda(), :, at[1].cuda()].cpu().unsqueeze(-1)).to(DT[dtype])
            assert torch.equal(raw(t[r].cpu()[there]), raw(x)), which
        assert bool((raw(to[r].cpu()[gone]).view(torch.uint8) == ref.POISON).all()), "a row of no slot was written"


class PairPool(ref.Pool):
    """Keys and values next to each other inside each head or token of a page."""

    def __init__(self, pages, heads, page_tokens, dim, dtype, inside):
        super().__init__(pages, heads, page_tokens, dim, dtype, "pair")
        both = self.raw[0][256:-256].view(dtype)
        if inside == "head":
            both = both.view(pages, heads, 2, page_tokens, dim)
            self.keys, self.values = both[:, :, 0], both[:, :, 1]
        elif inside == "token":
            both = both.view(pages, page_tokens, 2, heads, dim).transpose(1, 3)
            self.keys, self.values = both[:, :, 0], both[:, :, 1]
        else:  # a token's head
            both = both.view(pages, page_tokens, heads, 2, dim).transpose(1, 2)
            self.keys, self.values = both[:, :, :, 0], both[:, :, :, 1]


@pytest.mark.parametrize("inside", ["head", "token", "token's head"])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "e4m3")])
def test_pairs_inside_heads_and_tokens(comm, inside, dtype, cache):
    note(f"cache with pairs inside a {inside} {dtype} {cache}")
    heads, dim, page, group = 3, 80, 7, 4
    a = Attend(2, [300, 41, 0, 1], heads, group, dim, page, dtype, cache)
    for r, pool in enumerate(a.pools):
        a.pools[r] = PairPool(*pool.keys.shape, DT[cache], inside)
        ref.fill(a.pools[r], a.table, a.lengths, 50 + r)
    comm.cache_attention(**a.args())
    a.check()
    # new tokens in, and back
    slots = torch.randperm(a.pools[0].keys.shape[0] * page, generator=torch.Generator().manual_seed(3))[:100]
    x = draw((2, 2, 100, heads, dim), 5, DT[dtype]).cuda()
    back = torch.empty_like(x)
    cached = pages_of(a.pools)
    at = (slots // page).cuda(), (slots % page).cuda()
    for p in a.pools:
        p.raw[0][256:-256] = ref.POISON
    comm.cache_write(list(x[0]), list(x[1]), slots.cuda(), **cached)
    comm.cache_read(slots.cuda(), cached["key_pages"], cached["value_pages"], list(back[0]), list(back[1]),
                    cached.get("key_scales"), cached.get("value_scales"))
    torch.cuda.synchronize()
    for r, p in enumerate(a.pools):
        assert p.edges()
        for i, which in enumerate(("key", "value")):
            if p.eight:
                want, tol, scale, scale_tol = ref.quantise(x[i, r].cpu())
                s = p.key_scales if which == "key" else p.value_scales
                block_ref.assert_within(s[at[0], :, at[1]], scale, scale_tol, "scales")
                block_ref.assert_within(p.bytes(which)[at[0], :, at[1]].view(E4M3).float(), want, tol, "values")
                stored = p.bytes(which)[at[0], :, at[1]].view(E4M3).float() * s[at[0], :, at[1]].unsqueeze(-1)
                assert torch.equal(raw(back[i, r]), raw(stored.to(DT[dtype])))
            else:
                assert torch.equal(raw(back[i, r]), raw(x[i, r])) and torch.equal(raw(p.bytes(which)[at[0], :, at[1]]), raw(x[i, r]))
            p.bytes(which)[at[0], :, at[1]] = torch.full((), ref.POISON, dtype=torch.uint8, device="cuda:0") if p.eight else \
                torch.full((p.dtype.itemsize,), ref.POISON, dtype=torch.uint8, device="cuda:0").view(p.dtype)
        assert bool((p.raw[0] == ref.POISON).all()), "a place of no token was written"


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_write_special_values(comm, dtype):
    """A token of zeros, with an infinity, with a NaN, of tiny and of the largest
    values: each changes its own scale alone."""
    note(f"cache write special {dtype}")
    x = draw((6, 2, 64), 3, DT[dtype])
    x[0, 0] = 0
    x[1, 1, 7] = float("inf")
    x[2, 0, 63] = float("nan")
    x[3, 1] *= 2.0 ** -14
    x[4, 0, 5] = torch.finfo(DT[dtype]).max
    pool = ref.Pool(2, 2, 4, 64, E4M3)
    rows = x.cuda()
    comm.cache_write([rows], [rows], torch.tensor([7, 0, 2, 4, 1, 6]).cuda(), **pages_of([pool]))
    torch.cuda.synchronize()
    page, place = torch.tensor([1, 0, 0, 1, 0, 1]), torch.tensor([3, 0, 2, 0, 1, 2])
    for values, scales in ((pool.bytes("key"), pool.key_scales), (pool.bytes("value"), pool.value_scales)):
        q = values.cpu()[page, :, place].view(E4M3).float()
        s = scales.cpu()[page, :, place]
        assert s[0, 0] == 2.0 ** -126 and (q[0, 0] == 0).all()
        assert s[1, 1] == float("inf") and q[1, 1, 7].isnan() and (q[1, 1, :7] == 0).all()
        assert s[2, 0].isnan() and q[2, 0].isnan().all()
        fine = torch.ones((6, 2), dtype=torch.bool)
        fine[1, 1] = fine[2, 0] = False
        want, tol, scale, scale_tol = ref.quantise(x[fine])
        block_ref.assert_within(s[fine], scale, scale_tol, "scales")
        block_ref.assert_within(q[fine], want, tol, "values")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_written_8_bit_values_are_quotients(comm, dtype):
    """Scales and values have the bits of binary32 divisions, ties among them: max / 448 and
    y / s, rounded to nearest even.  (A product with a reciprocal, rounded, takes one value in
    1000 to the other side of a tie.)"""
    note(f"cache write, quotients {dtype}")
    x = draw((20000, 2, 64), 11, DT[dtype]) * torch.rand((20000, 2, 1), generator=torch.Generator().manual_seed(3)).add(0.1).to(DT[dtype])
    pool = ref.Pool(20000, 2, 1, 64, E4M3)
    rows = x.cuda()
    comm.cache_write([rows], [rows], torch.arange(20000, device="cuda:0"), **pages_of([pool]))
    torch.cuda.synchronize()
    y = x.float()
    scale = y.abs().amax(-1) / torch.full((20000, 2), 448.0)
    want = (y / scale.unsqueeze(-1).expand_as(y)).to(E4M3)
    for which, s in (("key", pool.key_scales), ("value", pool.value_scales)):
        assert torch.equal(raw(s[:, :, 0].cpu()), raw(scale))
        assert torch.equal(pool.bytes(which)[:, :, 0].cpu(), raw(want))


def test_write_of_no_tokens_and_one_row(comm):
    note("cache write of no tokens; a row of one token")
    pool = ref.Pool(1, 1, 1, 32, torch.bfloat16)
    before = pool.snapshot()
    none = torch.empty((0, 1, 32), dtype=torch.bfloat16, device="cuda:0")
    comm.cache_write([none], [none], torch.empty(0, dtype=torch.int64, device="cuda:0"), **pages_of([pool]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pool.raw, before))
    x = draw((3, 1, 32), 5, torch.bfloat16).cuda()
    comm.cache_write([x[1:2]], [x[2:3]], torch.zeros(1, dtype=torch.int64, device="cuda:0"), **pages_of([pool]))
    torch.cuda.synchronize()
    assert torch.equal(pool.keys[0, 0], x[1]) and torch.equal(pool.values[0, 0], x[2]) and pool.edges()


def test_slots_given_twice(comm):
    """Every element and scale is one of the tokens'."""
    note("cache write, the same slot twice")
    x = draw((64, 1, 128), 6, torch.bfloat16).cuda()
    pool = ref.Pool(2, 1, 16, 128, torch.bfloat16)
    comm.cache_write([x], [x], torch.full((64,), 17, device="cuda:0"), **pages_of([pool]))
    torch.cuda.synchronize()
    assert bool((x[:, 0] == pool.keys[1, 0, 1]).any(0).all()) and pool.edges()
    pool.keys[1, 0, 1].view(torch.uint8).fill_(ref.POISON)
    pool.values[1, 0, 1].view(torch.uint8).fill_(ref.POISON)
    assert all(bool((r == ref.POISON).all()) for r in pool.raw)


# ---- attention ----------------------------------------------------------------
class Attend:
    """A batch on the GPU: pools, table, lengths, queries and poisoned outputs with
    rows behind the last sequence."""

    def __init__(self, ranks, lengths, heads, group, dim, page, dtype, cache=None, order="head", out=None,
                 seed=1, nan=True, spread=1.0, query=1.0):
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        self.table, pages = ref.table_of(lengths, page, seed)
        self.dtype, self.heads, self.group, self.dim, self.page = DT[dtype], heads, group, dim, page
        self.pools = [ref.Pool(pages, heads, page, dim, DT[cache or dtype], order, nan) for _ in range(ranks)]
        for r, pool in enumerate(self.pools):
            ref.fill(pool, self.table, self.lengths, seed * 100 + r, spread)
        seqs = len(lengths)
        self.q = draw((ranks, seqs, heads * group + 2, dim), seed + 7, self.dtype, 1.5 * query)
        self.rows = self.q.cuda()
        self.queries = [r[:, 1:-1] for r in self.rows]  # parts of wider rows
        self.eight = out == "e4m3"
        self.poison = torch.full((ranks, (seqs + 2) * heads * group * dim * 4), ref.POISON, dtype=torch.uint8,
                                 device="cuda:0")
        n = seqs * heads * group
        to = E4M3 if self.eight else self.dtype
        self.out_bytes = n * dim * to.itemsize
        self.out = [b[:self.out_bytes].view(to).view(seqs, heads * group, dim) for b in self.poison]
        self.out_scales = [torch.empty((heads * group * dim // 128, seqs), device="cuda:0") for _ in range(ranks)] \
            if self.eight else None
        self.lse = [torch.empty((seqs, heads * group), device="cuda:0") for _ in range(ranks)]
        self.on = self.table.cuda(), self.lengths.cuda()

    def args(self, **more):
        cached = pages_of(self.pools)
        return dict(queries=self.queries, key_pages=cached["key_pages"], value_pages=cached["value_pages"],
                    page_table=self.on[0], lengths=self.on[1], out=self.out, key_scales=cached.get("key_scales"),
                    value_scales=cached.get("value_scales"), out_scales=self.out_scales, lse=self.lse, **more)

    def want(self, r, i, kv, scale, window=0):
        """ref.attention of a sequence and key-value head, or None if it is empty."""
        n = int(self.lengths[i])
        first = max(0, n - window) if window else 0
        if n == 0:
            return None
        t = torch.arange(first, n)
        page, place = self.table[i].long()[t // self.page], t % self.page
        k, v = (self.pools[r].rows(w, page.cuda(), place.cuda())[:, kv] for w in ("key", "value"))
        q = self.q[r, i, 1 + kv * self.group:1 + (kv + 1) * self.group].double()
        return ref.attention(q, k, v, scale, self.dtype, self.pools[r].eight)

    def check(self, scale=None, window=0, ranks=None, seqs=None, what="attention"):
        torch.cuda.synchronize()
        scale = self.dim ** -0.5 if scale is None else scale
        assert all(p.edges() for p in self.pools)
        assert bool((self.poison[:, self.out_bytes:] == ref.POISON).all()), "rows behind the last sequence"
        for r in range(len(self.pools)) if ranks is None else ranks:
            for i in range(len(self.lengths)) if seqs is None else seqs:
                for kv in range(self.heads):
                    h = slice(kv * self.group, (kv + 1) * self.group)
                    got, lse = self.out[r][i, h], self.lse[r][i, h]
                    w = self.want(r, i, kv, scale, window)
                    if w is None:
                        assert bool((got.float() == 0).all()) and bool((lse == -torch.inf).all()), (r, i)
                        if self.eight:
                            per = self.group * self.dim // 128
                            assert bool((self.out_scales[r][kv * per:(kv + 1) * per, i] == 2.0 ** -126).all())
                        continue
                    y, tol, l, l_tol = w
                    name = f"{what} rank {r} sequence {i} ({int(self.lengths[i])}) head {kv}"
                    block_ref.assert_within(lse, l, l_tol, name + " lse")
                    if self.eight:
                        flat = slice(kv * self.group * self.dim // 128, (kv + 1) * self.group * self.dim // 128)
                        t, t_tol, s, s_tol = block_ref.quantised(y.reshape(1, -1), tol.reshape(1, -1))
                        block_ref.assert_within(self.out_scales[r][flat, i:i + 1], s, s_tol, name + " scales")
                        block_ref.assert_within(got.float().reshape(1, -1), t, t_tol, name)
                    else:
                        block_ref.assert_within(got, y, ref.round_up(y, tol, self.dtype), name)


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257]

ATTENDS = [
    # ranks, lengths, kv heads, group, dim, places of a page, dtype, cache, order, out, window
    (1, [1], 1, 1, 16, 1, "bf16", None, "head", None, 0),
    (1, [5], 1, 1, 64, 16, "fp32", None, "head", None, 0),
    (2, EDGES, 1, 8, 128, 64, "bf16", None, "head", None, 0),
    (1, EDGES, 2, 4, 128, 16, "fp16", None, "token", None, 0),
    (1, EDGES, 1, 3, 80, 20, "fp32", None, "pair", None, 0),
    (2, EDGES, 1, 8, 128, 64, "bf16", "e4m3", "head", "e4m3", 0),
    (1, EDGES, 3, 2, 128, 7, "fp16", "e4m3", "token", None, 0),
    (1, EDGES, 1, 5, 256, 32, "fp32", "e4m3", "head", "e4m3", 0),
    (1, EDGES, 1, 16, 256, 48, "bf16", None, "head", "e4m3", 0),
    (1, EDGES, 1, 17, 64, 8, "bf16", None, "head", None, 0),
    (1, EDGES, 2, 33, 96, 1, "fp16", "e4m3", "token", None, 0),
    (1, EDGES, 1, 40, 128, 5, "fp16", None, "pair", "e4m3", 0),
    (1, EDGES, 1, 64, 256, 16, "bf16", "e4m3", "head", None, 0),
    (1, EDGES, 8, 1, 32, 16, "fp32", None, "head", None, 0),
    (1, EDGES, 1, 24, 48, 3, "fp32", "e4m3", "pair", None, 0),
    (1, EDGES, 1, 6, 240, 10, "fp32", None, "token", None, 0),
    (2, EDGES, 1, 8, 128, 16, "bf16", None, "head", None, 1),
    (1, EDGES, 1, 8, 128, 16, "bf16", "e4m3", "head", None, 33),
    (1, EDGES, 2, 4, 112, 12, "fp16", None, "token", None, 100),
    (1, EDGES, 1, 2, 192, 64, "fp32", None, "head", None, 64),
    (3, [1000, 37, 0, 4097, 1, 999, 2048], 2, 4, 128, 64, "bf16", None, "head", None, 0),
    (2, [5000, 3, 700], 1, 8, 128, 100, "bf16", "e4m3", "token", "e4m3", 0),
    (1, [3001, 2999], 2, 7, 80, 20, "fp16", None, "token", None, 0),
    (1, [9000], 1, 1, 64, 16, "fp32", None, "head", None, 0),
    (1, [6000, 6001], 1, 20, 256, 64, "bf16", None, "pair", None, 0),
    (1, [12000, 100], 1, 8, 128, 64, "fp16", "e4m3", "head", None, 5000),
    (32, [300, 20], 1, 2, 64, 16, "bf16", None, "head", None, 0),
    (1, [2500], 2, 3, 256, 64, "fp32", None, "head", "e4m3", 0),
    (1, [2500], 2, 3, 128, 64, "fp32", "e4m3", "head", None, 0),
    # many query heads to a key-value head: waves that take the same tokens, several tiles
    (1, [5000, 7], 1, 65, 128, 64, "bf16", None, "head", "e4m3", 0),
    (1, [3000, 1, 0, 900], 2, 100, 64, 16, "fp16", "e4m3", "token", None, 700),
    (2, [2000, 40], 1, 48, 256, 16, "fp32", None, "head", None, 0),
    (1, [7000], 1, 32, 128, 64, "bf16", "e4m3", "pair", "e4m3", 0),
    (1, [150, 3], 1, 300, 64, 16, "fp16", None, "head", None, 0),
    (1, [700, 0, 41], 1, 100, 256, 16, "fp32", None, "head", None, 0),
    (1, [70], 1, 4096, 32, 16, "bf16", "e4m3", "head", None, 0),
    (1, [7, 0], 4096, 1, 16, 16, "bf16", None, "token", None, 0),
    # a page that holds the whole sequence, and a table that holds far more
    (1, [3333], 1, 4, 64, 100000, "bf16", None, "head", None, 0),
    (1, [40, 700], 2, 4, 32, 3, "bf16", "e4m3", "head", None, 2 ** 40),
    (1, [64] * 64, 2, 8, 64, 16, "bf16", None, "head", None, 0),
    (1, [65] * 65, 2, 8, 64, 16, "bf16", None, "head", None, 0),
]


@pytest.mark.parametrize("ranks,lengths,heads,group,dim,page,dtype,cache,order,out,window", ATTENDS,
                         ids=[f"{i}" for i in range(len(ATTENDS))])
def test_attention(comm, ranks, lengths, heads, group, dim, page, dtype, cache, order, out, window):
    note(f"attention R={ranks} {lengths} {heads}x{group}x{dim} page {page} {dtype} {cache} {order} {out} {window}")
    a = Attend(ranks, lengths, heads, group, dim, page, dtype, cache, order, out)
    comm.cache_attention(**a.args(window=window))
    a.check(window=window)


# Heads that leave lanes without a part of the row, in every type and number of queries a wave.
NARROWER = [(dtype, cache, dim, group, order)
            for dtype, cache in (("bf16", None), ("fp16", None), ("fp32", None), ("bf16", "e4m3"), ("fp16", "e4m3"), ("fp32", "e4m3"))
            for dim, group, order in ((144, 3, "head"), (176, 16, "token"), (208, 20, "pair"), (240, 40, "head"),
                                      (240, 8, "token"), (144, 32, "head"), (112, 24, "token"), (16, 18, "head"),
                                      (48, 5, "pair"))]


@pytest.mark.parametrize("dtype,cache,dim,group,order", NARROWER)
def test_attention_of_heads_between(comm, dtype, cache, dim, group, order):
    note(f"attention of heads of {dim}, {group} {dtype} {cache} {order}")
    for lengths, heads, window in ((EDGES, 1, 0), ([5000, 37, 1200], 2, 0), ([3000, 400], 1, 777)):
        a = Attend(1, lengths, heads, group, dim, 20, dtype, cache, order)
        comm.cache_attention(**a.args(window=window))
        a.check(window=window)


@pytest.mark.parametrize("seqs,longest,ranks,group,dim", [
    (70, 300, 2, 4, 64), (300, 90, 1, 4, 64), (1500, 20, 1, 4, 64), (5000, 6, 1, 4, 64), (60, 200, 12, 3, 128),
    (600, 300, 1, 20, 64), (700, 40, 2, 70, 64), (400, 50, 2, 1, 256), (64, 100, 16, 16, 80), (65536, 1, 1, 1, 16)])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32")])
def test_attention_of_many_sequences(comm, seqs, longest, ranks, group, dim, dtype, cache):
    """Short ones, and among them one that is far longer."""
    gen = torch.Generator().manual_seed(seqs)
    n = (longest * torch.rand(seqs, generator=gen) ** 3 * 1.2).int().tolist()
    n[seqs // 3] = longest * 20
    note(f"attention of {seqs} sequences to {longest}, R={ranks} {group} x {dim} {dtype} {cache}")
    a = Attend(ranks, n, 1, group, dim, 16, dtype, cache)
    comm.cache_attention(**a.args())
    a.check(seqs=sorted({0, 1, seqs // 3, seqs - 1, *torch.randint(seqs, (40 // ranks + 2,), generator=gen).tolist()}))


@pytest.mark.parametrize("ranks,seqs,tokens,heads,group,dim,dtype,cache", [
    # teams of four waves
    (4, 30, 3001, 1, 8, 128, "bf16", None), (8, 30, 3001, 1, 8, 128, "fp16", "e4m3"), (1, 40, 3303, 4, 5, 80, "fp16", None),
    (2, 30, 5501, 1, 20, 128, "bf16", None), (2, 70, 1201, 1, 16, 256, "bf16", None), (2, 70, 3001, 1, 7, 208, "bf16", "e4m3"),
    (1, 20, 4001, 2, 3, 128, "fp32", None), (1, 17, 5003, 1, 2, 256, "fp32", None), (4, 30, 5501, 2, 24, 64, "fp32", "e4m3"),
    (4, 30, 6001, 1, 9, 64, "bf16", None),
    # waves alone
    (8, 400, 100, 1, 8, 128, "bf16", None), (8, 300, 250, 2, 20, 128, "bf16", "e4m3"), (2, 700, 120, 2, 1, 128, "fp32", None),
])
def test_attention_of_more_than_the_caches_hold(comm, ranks, seqs, tokens, heads, group, dim, dtype, cache):
    """More than 128 MiB of keys and values, which are loaded past the caches."""
    gen = torch.Generator().manual_seed(tokens)
    n = (tokens - (0.2 * tokens * torch.rand(seqs, generator=gen)).int()).tolist()
    a = Attend(ranks, n, heads, group, dim, 64, dtype, cache)
    bytes_ = 2 * ranks * sum(n) * heads * dim * DT[cache or dtype].itemsize
    note(f"attention of {bytes_ >> 20} MiB R={ranks} {seqs} x {tokens} {heads} x {group} x {dim} {dtype} {cache}")
    assert bytes_ >= 1 << 27
    comm.cache_attention(**a.args())
    a.check(ranks=[0, ranks - 1], seqs=sorted({0, seqs - 1, seqs // 2}))


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("fp16", None), ("fp32", None), ("bf16", "e4m3"),
                                         ("fp32", "e4m3")])
def test_attention_of_a_long_sequence(comm, dtype, cache):
    """Every compute unit on one sequence, and on a long and some short ones."""
    for lengths in ([70001], [33333, 5, 400, 20000]):
        note(f"attention of long sequences {lengths} {dtype} {cache}")
        a = Attend(1, lengths, 1, 8, 128, 64, dtype, cache)
        comm.cache_attention(**a.args())
        a.check()


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("fp16", None), ("fp32", None), ("bf16", "e4m3")])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 8.0])
def test_attention_scales(comm, dtype, cache, scale):
    """Flat, sharp (one token has all the weight) and negative scores."""
    note(f"attention scale {scale} {dtype} {cache}")
    a = Attend(1, [700, 40, 1], 1, 4, 128, 16, dtype, cache, query=2.0)
    comm.cache_attention(**a.args(scale=scale))
    a.check(scale=scale)


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("fp16", None), ("fp32", None), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
@pytest.mark.parametrize("group", [4, 20])
def test_scales_of_8_bit_outputs_are_binary32(comm, dtype, cache, group):
    """Two tokens, the second with scores -q and values of 1, the first with scores and
    values of 0: every output is w / (1 + w), w = e^-q.  In steps U = 2^-24: q times log2 e
    2 |q| log2 e (the constant's and the product's rounding; |q| at most 1.5), which makes
    3.1 of w, the exponential 2, the parts of w 1, three cut additions of them 6, the sum
    of weights 1, the division 1, the scale 2: together at most 17 of 20."""
    note(f"scales of 8-bit outputs {dtype} {cache} {group}")
    a = Attend(1, [2] * 32, 1, group, 128, 16, dtype, cache, out="e4m3")
    q = draw((32, group), 3).sigmoid().add(0.5).to(a.dtype)
    a.rows.zero_()
    a.queries[0][:, :, 0] = q.cuda()
    pool, page = a.pools[0], a.table[:, 0].cuda().long()
    if cache == "e4m3":
        pool.key_scales[page] = 1.0
        pool.value_scales[page] = 1.0
    for which, first, second in (("keys", 0.0, -1.0), ("values", 0.0, 1.0)):
        t = getattr(pool, which)
        t = t.view(torch.uint8) if cache == "e4m3" else t
        for place, value in ((0, first), (1, second)):
            to = torch.full((32, 1, 128), value, device="cuda:0").to(DT[cache or dtype])
            t[page, :, place] = to.view(torch.uint8) if cache == "e4m3" else to
    comm.cache_attention(**a.args(scale=1.0))
    torch.cuda.synchronize()
    w = torch.exp(-q.double())
    want = (w / (1 + w) / 448).t().contiguous()
    off = (a.out_scales[0].double().cpu() - want).abs() / want
    assert bool((off <= 20 * 2.0 ** -24).all()), float(off.max() * 2 ** 24)
    assert bool((a.out[0].float() == 448).all())


@pytest.mark.parametrize("dtype,cache,out", [("bf16", None, None), ("fp16", None, None), ("fp32", None, None), ("bf16", None, "e4m3"),
                                             ("bf16", "e4m3", None), ("fp16", "e4m3", None), ("fp32", "e4m3", None)])
@pytest.mark.parametrize("group", [4, 20])
def test_weights_are_binary32(comm, dtype, cache, out, group):
    """Three tokens whose values cancel the first 16 bits of a weight: two of score 0 with
    values -a and -b, one of score -q with value 1, w = e^-q, a the rounding of w to the
    cache's bits (8, or 11), b that of w - a: every output is (w - a - b) / (2 + w).
    In steps U = 2^-24 of 1: q times log2 e and its factor 2 |q| (|q| at most 0.65), the shift of
    8 of float16 6, the exponential 2, the parts of a weight 2, its product with a scale 2, three
    instructions' sums of magnitudes up to 2, cut inside and at their end, 24: together at
    most 38 of 40.  (Two parts of 8 bits would be up to 64 off.)"""
    note(f"weights are binary32 {dtype} {cache} {out} {group}")
    a = Attend(1, [3] * 64, 1, group, 128, 16, dtype, cache, out=out)
    q = (0.05 + 0.6 * torch.rand(64, generator=torch.Generator().manual_seed(4))).to(a.dtype)
    a.rows.zero_()
    a.queries[0][:, :, 0] = q[:, None].cuda()
    w = torch.exp(-q.double())
    bits = torch.float16 if dtype == "fp16" else torch.bfloat16
    first = w.to(bits)
    second = (w - first.double()).to(bits)
    pool, page = a.pools[0], a.table[:, 0].cuda().long()
    keys = torch.zeros((64, 3, 128))
    keys[:, 2] = -1.0
    values = torch.stack([-first.float(), -second.float(), torch.ones(64)], 1)
    for place in range(3):
        if cache == "e4m3":
            for which, x in (("key", keys[:, place].sign()), ("value", values[:, place, None].sign().expand(64, 128))):
                pool.bytes(which)[page, 0, place] = x.to(E4M3).view(torch.uint8).cuda()
            pool.key_scales[page, 0, place] = 1.0
            pool.value_scales[page, 0, place] = values[:, place].abs().cuda()
        else:
            pool.keys[page, 0, place] = keys[:, place].to(pool.dtype).cuda()
            pool.values[page, 0, place] = values[:, place, None].to(pool.dtype).cuda().expand(64, 128)
    comm.cache_attention(**a.args(scale=1.0))
    torch.cuda.synchronize()
    want = ((w - first.double() - second.double()) / (2 + w))[:, None]
    off = 40 * 2.0 ** -24 / (2 + w)[:, None] + torch.zeros((64, group * 128))
    got = a.out[0].cpu().flatten(1)
    if out == "e4m3":  # one value a block: the largest, which is 448 scales
        got = got.double().sign() * 448 * a.out_scales[0].cpu().double().t().repeat_interleave(128, 1)
        off = off + 2.0 ** -24 * want.abs()
    else:
        off = off + block_ref.HALF_STEP[a.dtype] * (want.abs() + off) + block_ref.HALF_LEAST[a.dtype]
    bad = (got.double() - want).abs() > off
    worst = float(((got.double() - want).abs() * (2 + w)[:, None]).max() * 2 ** 24)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, the most {worst:.1f} steps"


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("fp16", None), ("fp32", None), ("bf16", "e4m3"),
                                         ("fp32", "e4m3")])
def test_scores_that_grow(comm, dtype, cache):
    """The largest score comes last, or first: every step moves the maximum, or none."""
    for sign in (1, -1):
        note(f"attention, growing scores {sign} {dtype} {cache}")
        a = Attend(1, [1500, 90], 1, 4, 64, 16, dtype, cache)
        for i, n in enumerate(a.lengths.tolist()):
            t = torch.arange(n)
            page, place = a.table[i].long()[t // 16].cuda(), (t % 16).cuda()
            size = (t.double() / 40 if sign > 0 else (n - t).double() / 40).cuda()
            if cache == "e4m3":
                a.pools[0].key_scales[page, 0, place] = (0.001 * (1 + size)).float()
            else:
                x = a.pools[0].keys[page, :, place].double() * 0.05 * (1 + size)[:, None, None]
                a.pools[0].keys[page, :, place] = x.to(DT[dtype])
        comm.cache_attention(**a.args())
        a.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_attention_special_values(comm, dtype):
    """Scores of minus infinity have no weight; a row of nothing else, an infinite
    score and a NaN give NaN; a value's infinity takes its own column alone (infinity,
    or NaN where a part of its weight is 0); the sequences and heads next to them
    keep their values."""
    note(f"attention special values {dtype}")
    a = Attend(1, [300, 300, 300, 300, 300, 300], 1, 2, 64, 16, dtype)
    inf = float("inf")
    q = a.rows[0]
    q[:, 1:3, 0] = 1.0
    a.q = a.rows.cpu()

    def at(i, t):
        return int(a.table[i, t // 16]), 0, t % 16

    pool = a.pools[0]
    for t in (0, 5, 31, 64, 299):
        pool.keys[at(0, t)][0] = -inf          # masked by its own score
    for t in range(300):
        pool.keys[at(1, t)][0] = -inf          # nothing is left
    pool.keys[at(2, 130)][0] = inf
    pool.values[at(3, 77)][9] = inf
    pool.keys[at(4, 299)][3] = float("nan")
    comm.cache_attention(**a.args())
    torch.cuda.synchronize()
    out, lse = a.out[0].cpu(), a.lse[0].cpu()
    for i in (1, 2, 4):
        assert out[i].isnan().all(), i
    assert lse[4].isnan().all() and (lse[1] == -inf).all()
    assert not out[3][:, 9].isfinite().any()
    fine = [d for d in range(64) if d != 9]
    y, tol, l, l_tol = a.want(0, 3, 0, 0.125)
    block_ref.assert_within(out[3][:, fine], y[:, fine], ref.round_up(y, tol, DT[dtype])[:, fine], "beside an infinity")
    a.check(seqs=[5])
    # the first: as if those tokens were not there
    n = [t for t in range(300) if t not in (0, 5, 31, 64, 299)]
    t = torch.tensor(n)
    page, place = a.table[0].long()[t // 16].cuda(), (t % 16).cuda()
    k, v = (pool.rows(w, page, place)[:, 0] for w in ("key", "value"))
    y, tol, l, l_tol = ref.attention(a.q[0, 0, 1:3].double(), k, v, 0.125, DT[dtype], False)
    block_ref.assert_within(out[0], y, ref.round_up(y, tol, DT[dtype]), "scores of minus infinity")
    block_ref.assert_within(lse[0], l, l_tol, "their lse")


@pytest.mark.parametrize("dtype,cache,group", [("bf16", None, 4), ("fp16", None, 20), ("fp32", None, 4), ("bf16", "e4m3", 8),
                                               ("fp32", "e4m3", 3)])
def test_scores_of_plus_infinity(comm, dtype, cache, group):
    """They make NaN of their query head's output and an infinity of its log-sum, NaN beside a
    NaN score, in any piece of a joined sequence; where the same token's score is minus infinity
    it has no weight."""
    note(f"attention, scores of plus infinity {dtype} {cache} {group}")
    inf = float("inf")
    a = Attend(1, [1, 300, 9000, 9000, 50], 1, group, 64, 16, dtype, cache)
    sign = torch.where(torch.arange(group) % 3 == 1, -1.0, 1.0).to(a.dtype)
    a.rows[0][:, 1:1 + group, 0] = sign.cuda()
    if cache == "e4m3":
        a.rows[0][:, 1:1 + group, 1:] = 0.0
    a.q = a.rows.cpu()
    pool = a.pools[0]

    def at(i, t):
        return int(a.table[i, t // 16]), 0, t % 16

    def set_key(i, t, value):
        if cache == "e4m3":  # a one times the scale (a zero times infinity is NaN, so there only one dim has a query)
            pool.bytes("key")[(*at(i, t), 0)] = torch.tensor(1.0).to(E4M3).view(torch.uint8).cuda()
            pool.key_scales[at(i, t)] = value
        else:
            pool.keys[(*at(i, t), 0)] = value

    infinite = {0: 0, 1: 130, 2: 8999, 3: 17}
    for i, t in infinite.items():
        set_key(i, t, inf)
    set_key(3, 6000, float("nan"))
    comm.cache_attention(**a.args())
    torch.cuda.synchronize()
    out, lse = a.out[0].cpu(), a.lse[0].cpu()
    up = sign > 0
    for i in (0, 1, 2):
        assert out[i][up].isnan().all() and (lse[i][up] == inf).all(), (i, lse[i])
    assert out[0][~up].isnan().all() and (lse[0][~up] == -inf).all()
    assert out[3].isnan().all() and lse[3].isnan().all()
    for i in (1, 2):
        t = torch.tensor([t for t in range(int(a.lengths[i])) if t != infinite[i]])
        page, place = a.table[i].long()[t // 16].cuda(), (t % 16).cuda()
        k, v = (pool.rows(w, page, place)[:, 0] for w in ("key", "value"))
        y, tol, l, l_tol = ref.attention(a.q[0, i, 1:1 + group].double(), k, v, 0.125, a.dtype, cache == "e4m3")
        block_ref.assert_within(out[i][~up], y[~up], ref.round_up(y, tol, a.dtype)[~up], "beside a score of infinity")
        block_ref.assert_within(lse[i][~up], l[~up], l_tol[~up], "their lse")
    a.check(seqs=[4])


@pytest.mark.parametrize("query", [1.0, 4.0])
@pytest.mark.parametrize("dtype,cache,out,group,dim", [
    ("bf16", None, None, 4, 64), ("fp16", None, None, 4, 128), ("fp32", None, None, 4, 64), ("bf16", None, "e4m3", 20, 128),
    ("fp16", None, None, 40, 80), ("bf16", "e4m3", None, 5, 80), ("fp16", "e4m3", None, 20, 208), ("fp32", "e4m3", None, 3, 16),
    ("bf16", "e4m3", None, 4, 128), ("fp16", "e4m3", "e4m3", 8, 128), ("fp32", "e4m3", None, 20, 64)])
def test_infinite_values(comm, dtype, cache, out, group, dim, query):
    """An infinity among the values makes its column one, whatever its weight, in a sequence
    of one token as in a joined one; two of both signs and a NaN make it NaN; the other columns
    keep their values.  (8 bits: a value of zero times a scale of infinity is NaN.)"""
    note(f"attention, infinite values {dtype} {cache} {out} {group} x {dim} {query}")
    inf = float("inf")
    a = Attend(1, [1, 300, 9000, 40], 1, group, dim, 16, dtype, cache, out=out, query=query)
    pool = a.pools[0]

    def put(i, t, column, value):
        at = int(a.table[i, t // 16]), 0, t % 16
        if cache == "e4m3":
            pool.value_scales[at] = value
        else:
            pool.values[at][column] = value

    put(0, 0, 3, inf)
    put(1, 77, 9, -inf)
    put(2, 0, dim - 1, inf)
    if cache == "e4m3":
        put(2, 8000, 0, inf)
    else:
        put(1, 5, 10, inf)
        put(1, 20, 11, inf)
        put(1, 250, 11, -inf)
        put(1, 299, 12, float("nan"))
        put(1, 100, 13, inf)
        put(1, 101, 13, inf)
        put(2, 8999, 0, -inf)
    comm.cache_attention(**a.args())
    a.check()
    y = a.out[0][0].float() if out is None else a.out_scales[0][:, 0]
    assert y.isinf().any()


@pytest.mark.parametrize("dtype,cache,lowest", [
    ("bf16", None, None), ("fp16", None, None), ("fp32", None, None), ("bf16", None, torch.finfo(torch.bfloat16).min),
    ("fp16", None, torch.finfo(torch.float16).min), ("fp32", None, torch.finfo(torch.float32).min / 2), ("bf16", "e4m3", None)])
def test_whole_tiles_of_minus_infinity(comm, dtype, cache, lowest):
    """Long runs of tokens without weight before, between and behind those with it:
    scores of minus infinity, or of the type's lowest values."""
    note(f"attention, long runs of minus infinity {dtype} {cache} {lowest}")
    a = Attend(1, [6000], 1, 4, 64, 16, dtype, cache)
    a.rows[0][:, 1:5, 0] = 1.0
    a.q = a.rows.cpu()
    t = torch.arange(6000)
    keep = (t % 1500 >= 700) & (t % 1500 < 760)
    page, place = a.table[0].long()[t // 16], t % 16
    gone = ~keep
    where = page[gone].cuda(), 0, place[gone].cuda()
    if cache == "e4m3":  # (a scale of -infinity would make NaN of the zeros beside the one)
        a.pools[0].bytes("key")[where] = torch.zeros(64).to(E4M3).view(torch.uint8).cuda()
        a.pools[0].bytes("key")[(*where, 0)] = torch.tensor(1.0).to(E4M3).view(torch.uint8).cuda()
        a.pools[0].key_scales[where] = -2.0 ** 100
    else:
        a.pools[0].keys[(*where, 0)] = lowest if lowest is not None else -torch.inf
    comm.cache_attention(**a.args())
    torch.cuda.synchronize()
    k, v = (a.pools[0].rows(w, page[keep].cuda(), place[keep].cuda())[:, 0] for w in ("key", "value"))
    y, tol, l, l_tol = ref.attention(a.q[0, 0, 1:5].double(), k, v, 0.125, DT[dtype], cache == "e4m3")
    block_ref.assert_within(a.out[0][0], y, ref.round_up(y, tol, DT[dtype]), "runs of minus infinity")
    block_ref.assert_within(a.lse[0][0], l, l_tol, "their lse")


@pytest.mark.parametrize("dtype,cache,out", [("bf16", None, None), ("fp32", None, None), ("fp16", "e4m3", None),
                                             ("bf16", "e4m3", "e4m3")])
def test_bad_pages_and_lengths(comm, dtype, cache, out):
    """They make their own sequence NaN and no other's; what lies past a length, and
    before a window, is never looked at."""
    note(f"attention, bad pages and lengths {dtype} {cache} {out}")
    lengths = [100, 400, 257, 1000, 64, 90, 300]
    for window in (0, 50):
        a = Attend(1, lengths, 1, 4, 128, 16, dtype, cache, out=out)
        pages = a.pools[0].keys.shape[0]
        table, n = a.table.clone(), a.lengths.clone()
        table[0, 6] = pages           # holds tokens 96 .. 99
        table[1, 24] = -1             # 384 .. 399
        table[3, 62] = 2 ** 31 - 1    # 992 .. 999
        n[4], n[5] = -1, table.shape[1] * 16 + 1
        table[2, 17:] = -5            # past its length
        if window:
            table[2, :12] = pages + 7     # before its window: 207 .. 256
            table[6, :15] = -(2 ** 31)    # 250 .. 299
        a.on = table.cuda(), n.cuda()
        comm.cache_attention(**a.args(window=window))
        torch.cuda.synchronize()
        for i in (0, 1, 3, 4, 5):
            if out == "e4m3":
                assert a.out_scales[0][:, i].isnan().all() and a.out[0][i].float().isnan().all(), i
            else:
                assert a.out[0][i].isnan().all(), i
            assert a.lse[0][i].isnan().all(), i
        a.check(window=window, seqs=[2, 6])


def test_padded_batch_and_growing_lengths_in_a_graph(comm):
    """A captured call over fixed buffers: lengths, table and queries change between
    the replays, empty sequences among them; every replay has an eager call's bits."""
    note("attention in a graph")
    full = [700, 20, 1300, 64, 0, 5]
    a = Attend(2, full, 1, 8, 128, 16, "bf16", "e4m3", out="e4m3")
    b = [t.clone() for t in (*a.out, *a.out_scales, *a.lse)]
    call = comm.prepare_cache_attention(**a.args())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        captured = comm.prepare_cache_attention(**a.args(stream=side))
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured()
    for lengths in ([0] * 6, [1, 0, 0, 1, 0, 0], [32, 20, 128, 64, 0, 5], full, [699, 19, 1299, 63, 0, 4], [0] * 6, full):
        a.lengths = torch.tensor(lengths, dtype=torch.int32)
        a.on[1].copy_(a.lengths)
        a.rows.copy_(draw(a.rows.shape, sum(lengths), torch.bfloat16))
        a.q = a.rows.cpu()
        torch.cuda.synchronize()
        for t in (*a.out, *a.out_scales, *a.lse):
            raw(t).fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for t, x in zip((*a.out, *a.out_scales, *a.lse), b):
            raw(x).copy_(raw(t))
            raw(t).fill_(9)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        for t, x in zip((*a.out, *a.out_scales, *a.lse), b):
            assert torch.equal(raw(t), raw(x)), lengths
        a.check(what=f"replay {lengths}")


def test_the_convenience_in_a_graph(comm):
    """Its workspace is the graph's own."""
    note("attention convenience captured")
    a = Attend(1, [3000, 4], 1, 8, 128, 16, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        comm.cache_attention(**a.args())
    for _ in range(3):
        raw(a.out[0]).fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        junk = torch.full((1 << 22,), 7, device="cuda:0")
        del junk
        a.check()


def test_calls_on_two_streams_at_once(comm):
    """Prepared apart, each with its own workspace; joined sequences in both."""
    note("attention on two streams at once")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [Attend(1, [20000, 3], 1, 8, 128, 64, "bf16", "e4m3", seed=s) for s in (1, 2)]
    torch.cuda.synchronize()
    calls = [comm.prepare_cache_attention(**a.args(stream=s)) for a, s in zip(both, streams)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c in calls:
            c()
    torch.cuda.synchronize()
    for a in both:
        a.check()


def test_one_workspace_for_calls_in_order(comm):
    """Calls of other sizes, types and dims share it one after the other; the same
    call again has the same bits."""
    note("attention, one workspace in order")
    work = comm.cache_workspace(256, 64)
    batch = [Attend(1, [80000], 1, 8, 128, 64, "bf16"), Attend(2, [5, 900, 9000], 2, 3, 256, 16, "fp32", "e4m3"),
             Attend(1, [700] * 40, 1, 20, 64, 16, "fp16"), Attend(1, [1 + i % 60 for i in range(1100)], 1, 2, 64, 16, "bf16"),
             Attend(1, [9000], 1, 40, 64, 16, "bf16", "e4m3")]
    calls = [comm.prepare_cache_attention(**a.args(workspace=work)) for a in batch]
    seen = None
    for _ in range(3):
        for c in calls:
            c()
        torch.cuda.synchronize()
        now = [raw(t).clone() for a in batch for t in (*a.out, *a.lse)]
        assert seen is None or all(torch.equal(x, y) for x, y in zip(seen, now))
        seen = now
    for a in batch:
        a.check(seqs=range(0, len(a.lengths), 1 + len(a.lengths) // 40))


def test_a_workspace_serves_fewer_of_either(comm):
    """Its size never falls as dim or group grows, and a call of a smaller dim runs in one that
    was made for a larger."""
    note("attention, workspaces of larger dims")
    sizes = [[ar.arCacheAttentionWorkspace(dim, group, comm.handle) for group in (1, 2, 7, 8, 16, 17, 32, 33, 64, 4096)]
             for dim in range(16, 257, 16)]
    assert all(r == 0 for row in sizes for r, _ in row)
    for row in sizes:
        assert all(a <= b for (_, a), (_, b) in zip(row, row[1:]))
    for row, following in zip(sizes, sizes[1:]):
        assert all(a <= b for (_, a), (_, b) in zip(row, following))
    for group in (8, 40):
        work = comm.cache_workspace(256, group)
        for dim in (64, 80, 128):
            a = Attend(1, [9000, 5], 1, group, dim, 16, "bf16")
            comm.cache_attention(**a.args(workspace=work))
            a.check()


@pytest.mark.parametrize("dtype,cache,group,dim", [("bf16", None, 8, 128), ("fp32", "e4m3", 40, 64), ("fp16", None, 3, 256)])
def test_only_the_first_bytes_of_a_workspace_are_zero(comm, dtype, cache, group, dim):
    """The rest is NaN: partial sums are read where a team of the same call has written."""
    note(f"attention, a workspace of NaN behind its zeros {dtype} {cache} {group} x {dim}")
    work = torch.full((ar.arCacheAttentionWorkspace(dim, group, comm.handle)[1],), 0xFF, dtype=torch.uint8, device="cuda:0")
    work[:ar.AR_CACHE_WORKSPACE_ZEROS] = 0
    for lengths in ([70000], [5, 900, 9000, 0, 33], [200] * 300, [9000]):
        a = Attend(1, lengths, 1, group, dim, 16, dtype, cache)
        comm.cache_attention(**a.args(workspace=work))
        a.check(seqs=range(0, len(lengths), 1 + len(lengths) // 10))
        assert not work[:ar.AR_CACHE_WORKSPACE_ZEROS].any()


def test_shared_pages(comm):
    """Sequences with a common prefix in the same pages, keys that are the values too."""
    note("attention over shared pages")
    a = Attend(1, [500, 480, 64], 1, 8, 64, 16, "bf16")
    a.table[1, :20] = a.table[0, :20]
    a.table[2] = a.table[0, :a.table.shape[1]]
    a.on = a.table.cuda(), a.lengths.cuda()
    a.pools[0].values = a.pools[0].keys
    comm.cache_attention(**a.args())
    a.check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_offsets_past_32_bits(comm, cache):
    """A pool of more than 2^32 bytes (and 2^31 elements): its first and last pages."""
    note(f"cache past 32 bits {cache}")
    pages, page, heads, dim = 40000, 256, 2, 256
    n = pages * page * heads * dim
    pools = []
    eight = cache == "e4m3"

    class Large:
        pass

    p = Large()
    p.eight, p.dtype = eight, DT[cache]
    p.keys, p.values = (torch.empty((pages, heads, page, dim), dtype=DT[cache], device="cuda:0") for _ in range(2))
    p.key_scales = p.value_scales = None
    if eight:
        p.key_scales, p.value_scales = (torch.empty((pages, heads, page), device="cuda:0") for _ in range(2))
    p.bytes = lambda which: ref.Pool.bytes(p, which)
    p.rows = lambda *a: ref.Pool.rows(p, *a)
    p.edges = lambda: True
    assert n > 2 ** 32
    pools.append(p)
    tokens = 2 * page + 40
    order = torch.tensor([pages - 1, 0, pages // 2 + 3])
    a = Attend(1, [tokens], heads, 4, dim, page, "bf16", cache if eight else None)
    a.table = torch.cat([order, torch.tensor([-1])]).int()[None]
    a.on = a.table.cuda(), a.lengths.cuda()
    a.pools = pools
    t = torch.arange(tokens)
    slots = order[t // page] * page + t % page
    x = draw((2, tokens, heads, dim), 3, torch.bfloat16).cuda()
    cached = pages_of(pools)
    comm.cache_write([x[0]], [x[1]], slots.cuda(), **cached)
    back = torch.empty_like(x)
    comm.cache_read(slots.cuda(), cached["key_pages"], cached["value_pages"], [back[0]], [back[1]],
                    cached.get("key_scales"), cached.get("value_scales"))
    comm.cache_attention(**a.args())
    torch.cuda.synchronize()
    for i, which in ((0, "key"), (1, "value")):
        stored = p.rows(which, order[t // page].cuda(), (t % page).cuda())
        if eight:
            off = (stored - x[i].double().cpu()).abs().amax() / x[i].double().abs().amax().cpu()
            assert off < 0.04
        else:
            assert torch.equal(raw(back[i]), raw(x[i]))
        assert (back[i].double().cpu() - stored).abs().amax() <= 2.0 ** -8 * stored.abs().amax()
    a.check()


def test_refusals_with_a_device(comm):
    """What only a communicator shows: the workspace's size, the tensors' device."""
    note("attention refusals")
    a = Attend(1, [5], 1, 1, 64, 16, "bf16")
    with pytest.raises(ar.ArError, match="InvalidArgument"):
        comm.cache_attention(**a.args(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda:0")))
    for change in (dict(lengths=a.on[1].long()), dict(page_table=a.on[0][0]), dict(lengths=a.on[1].cpu()),
                   dict(queries=[a.queries[0].float()]), dict(out=[a.out[0][:, :, ::2]]),
                   dict(value_pages=[a.pools[0].values[:, :, :8]]), dict(key_scales=[a.lse[0]]),
                   dict(lse=[a.lse[0].double()]), dict(window=-1)):
        with pytest.raises(ValueError):
            comm.cache_attention(**dict(a.args(), **change))
    with pytest.raises(ar.ArError, match="Unsupported"):
        eight = torch.empty((1, 1, 64), dtype=E4M3, device="cuda:0")
        comm.cache_attention(**dict(a.args(), out=[eight], out_scales=[torch.empty((1, 1), device="cuda:0")]))


def test_refusals_of_no_heads(comm):
    """They are the library's, not a division by zero."""
    note("attention of no heads")
    a = Attend(1, [5], 2, 1, 64, 16, "bf16")
    none = [t[:, :0] for t in (a.queries[0], a.pools[0].keys, a.pools[0].values)]
    with pytest.raises(ar.ArError, match="Unsupported"):
        comm.cache_attention(**dict(a.args(), key_pages=[none[1]], value_pages=[none[2]]))
    with pytest.raises(ar.ArError, match="Unsupported"):
        comm.cache_attention(**dict(a.args(), queries=[none[0]], out=[a.out[0][:, :0].contiguous()], lse=None))


# ---- the attention half of a layer ---------------------------------------------
@pytest.mark.parametrize("tokens,cache", [(1, "e4m3"), (5, "bf16"), (64, "e4m3")])
def test_attention_half_of_a_layer(comm, tokens, cache):
    """Norm, QKV product, cache write, attention with an 8-bit output and the output
    product with its all-reduce: each operator on what the one before left, checked
    at the end against the same chain in 64 bits over the operators' own
    intermediate values."""
    note(f"attention half of a layer, {tokens} tokens, {cache}")
    ranks, hidden, heads, group, dim, page = 2, 512, 1, 4, 128, 16
    wide = (group + 2) * heads * dim
    bf16 = torch.bfloat16

    def bufs(rows, cols, dtype):
        return list(torch.empty((ranks, rows, cols), dtype=dtype, device="cuda:0").unbind(0))

    x = [draw((tokens, hidden), r, bf16).cuda() for r in range(ranks)]
    q8, qs = bufs(tokens, hidden, E4M3), bufs(ar.scale_blocks(hidden), tokens, torch.float32)
    w1 = [draw((wide, hidden), 10 + r, scale=110.0).clamp(-448, 448).to(E4M3).cuda() for r in range(ranks)]
    s1 = [torch.full((ar.scale_blocks(wide), ar.scale_blocks(hidden)), 1 / (110 * hidden ** 0.5), device="cuda:0")] * ranks
    w2 = [draw((hidden, group * heads * dim), 20 + r, scale=110.0).clamp(-448, 448).to(E4M3).cuda() for r in range(ranks)]
    s2 = [torch.full((ar.scale_blocks(hidden), group * heads), 1e-3, device="cuda:0")] * ranks
    qkv, out = bufs(tokens, wide, bf16), bufs(tokens, hidden, bf16)
    lengths = [1 + 13 * i % 90 for i in range(tokens)]
    table, pages = ref.table_of(lengths, page, 3)
    n = torch.tensor(lengths)
    pools = [ref.Pool(pages, heads, page, dim, DT[cache]) for _ in range(ranks)]
    for r, pool in enumerate(pools):
        ref.fill(pool, table, n - 1, 30 + r)
    slots = table.long()[torch.arange(tokens), (n - 1) // page] * page + (n - 1) % page
    rows = [t.unflatten(1, ((group + 2) * heads, dim)) for t in qkv]
    keys, values = ([t[:, a * heads:(a + 1) * heads] for t in rows] for a in (group, group + 1))
    queries = [t[:, :group * heads] for t in rows]
    att = [t.view(tokens, group * heads, dim) for t in bufs(tokens, group * heads * dim, E4M3)]
    att_s, lse = bufs(group * heads, tokens, torch.float32), bufs(tokens, group * heads, torch.float32)
    cached = pages_of(pools)
    comm.all_reduce_norm(x, torch.ones(hidden, dtype=bf16, device="cuda:0"), 1e-5, out=q8, scales=qs)
    comm.matmul_scaled(q8, qs, w1, s1, qkv)
    comm.cache_write(keys, values, slots.cuda(), **cached)
    comm.cache_attention(queries, cached["key_pages"], cached["value_pages"], table.cuda(), n.int().cuda(), att,
                         cached.get("key_scales"), cached.get("value_scales"), out_scales=att_s, lse=lse)
    comm.matmul_scaled([t.view(tokens, -1) for t in att], att_s, w2, s2, out, reduce=True)
    torch.cuda.synchronize()
    total, total_tol = 0.0, 0.0
    for r in range(ranks):
        for i in range(tokens):
            t = torch.arange(lengths[i])
            at = table[i].long()[t // page].cuda(), (t % page).cuda()
            k, v = (pools[r].rows(w, *at)[:, 0] for w in ("key", "value"))
            y, tol, _, _ = ref.attention(queries[r][i].double().cpu(), k, v, dim ** -0.5, bf16, cache == "e4m3")
            t, t_tol, s, s_tol = block_ref.quantised(y.reshape(1, -1), tol.reshape(1, -1))
            block_ref.assert_within(att_s[r][:, i:i + 1], s, s_tol, f"scales of {r}, {i}")
            block_ref.assert_within(att[r][i].float().reshape(1, -1), t, t_tol, f"attention of {r}, {i}")
        c, tol, step = block_ref.matmul(att[r].view(tokens, -1).cpu().float(), att_s[r].cpu(), w2[r].cpu().float(),
                                        s2[r].cpu(), bf16)
        total, total_tol = total + c, total_tol + tol + ranks * group * step
    for t in out:
        block_ref.assert_within(t, total, block_ref.rounded(total, total_tol, bf16), "the layer's output")
