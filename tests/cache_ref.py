"""The operators of ar_cache.h in 64 bits on the CPU, with bounds on how far a
binary32 computation may be from them (the steps of block_ref.py), and pools to
run them on."""
from __future__ import annotations

import torch

from block_ref import E4M3, HALF_LEAST, HALF_STEP, SCALE_MIN, U

POISON = 0xA5


def quantise(y):
    """y [..., dim]: (values before their rounding, their tolerance, scales [...],
    their tolerance)."""
    y = y.double()
    scale = (y.abs().amax(-1) / 448).clamp_min(SCALE_MIN)
    t = y / scale.unsqueeze(-1)
    # the scale's rounding and the quotient's two (its reciprocal has two parts)
    off = 3 * U * t.abs()
    return t, off + HALF_STEP[E4M3] * (t.abs() + off) + HALF_LEAST[E4M3], scale, U * scale


def attention(q, k, v, scale, dtype, eight):
    """One sequence of one key-value head: q [group, dim], k and v [tokens, dim] in
    64 bits: (out, its tolerance before a rounding, lse, its tolerance).

    With e_t the error of a score: a dot product of dim terms, in some order and at
    worst cut instead of rounded (2 U a step of the sum of magnitudes), its factors,
    and the difference to the shift of the exponent (both in base 2).  exp turns it
    into a relative error, to which the exponential's and the rescalings' own come,
    the parts in which a weight enters the product with the values (two of bfloat16
    hold 16 bits of it, two of float16 22, three of bfloat16 and float32 24) and the
    sum over the tokens: steps of 16 or 32, shared by four waves, and the joins."""
    n, dim = k.shape
    x = scale * (q @ k.t().contiguous())
    size = abs(scale) * (q.abs() @ k.abs().t().contiguous())
    top = x.abs().amax(-1, keepdim=True)
    e = (dim + 8) * 2 * U * size + 12 * U * (x.abs() + top) + 16 * U
    parts = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -16 if eight else 2.0 ** -21,
             torch.float32: 2.0 ** -23}[dtype]
    c = parts + (n / 16 + 128) * 2 * U
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total
    rel = (p * (e + c)).sum(-1, keepdim=True)
    out = p @ v
    # float16 weights below 2^-24 of the largest lose bits that others have
    least = 2.0 ** -30 * v.abs().sum(0) if dtype == torch.float16 and not eight else 0.0
    tol = (p * (e + c + 4 * U)) @ v.abs() + out.abs() * rel + least / total
    lse = (m + total.log()).squeeze(-1)
    lse_tol = rel.squeeze(-1) + 6 * U * (lse.abs() + top.squeeze(-1)) + 4 * U
    return out, 1.01 * tol, lse, 1.01 * lse_tol


def round_up(want, tol, dtype):
    return tol + HALF_STEP[dtype] * (want.abs() + tol) + HALF_LEAST[dtype]


class Pool:
    """A cache of one rank on the GPU with every byte poisoned, the places of no
    token among them (as bfloat16, float16, float32 and e4m3 the poison is finite;
    `nan`: it is a NaN in all of them).  `order`: "head", "token", or "pair" (keys
    and values of a page next to each other in one allocation)."""

    def __init__(self, pages, heads, page_tokens, dim, dtype, order="head", nan=False, device="cuda:0"):
        self.dtype, self.eight = dtype, dtype == E4M3
        self.poison = 0xFF if nan else POISON
        es = torch.empty((), dtype=dtype).element_size()
        n = pages * heads * page_tokens * dim * es

        def raw(n):
            return torch.full((n + 512,), self.poison, dtype=torch.uint8, device=device)

        if order == "pair":
            self.raw = [raw(2 * n)]
            both = self.raw[0][256:256 + 2 * n].view(dtype).view(pages, 2, heads, page_tokens, dim)
            self.keys, self.values = both[:, 0], both[:, 1]
        else:
            self.raw = [raw(n), raw(n)]
            both = [r[256:256 + n].view(dtype) for r in self.raw]
            if order == "head":
                both = [b.view(pages, heads, page_tokens, dim) for b in both]
            else:
                both = [b.view(pages, page_tokens, heads, dim).transpose(1, 2) for b in both]
            self.keys, self.values = both
        self.key_scales = self.value_scales = None
        if self.eight:
            m = pages * heads * page_tokens * 4
            more = [raw(m), raw(m)]
            self.key_scales, self.value_scales = (
                r[256:256 + m].view(torch.float32).view(pages, heads, page_tokens) for r in more)
            self.raw += more

    def snapshot(self):
        return [r.clone() for r in self.raw]

    def edges(self):
        return all(bool((r[:256] == self.poison).all()) and bool((r[-256:] == self.poison).all())
                   for r in self.raw)

    def rows(self, which, page, place):
        """What the places stand for, in 64 bits on the CPU: [..., heads, dim]."""
        x = self.bytes(which)[page, :, place].view(self.dtype).double().cpu()
        if self.eight:
            s = self.key_scales if which == "key" else self.value_scales
            x = x * s[page, :, place].double().cpu().unsqueeze(-1)
        return x

    def bytes(self, which):
        t = self.keys if which == "key" else self.values
        return t.view(torch.uint8) if self.eight else t


def fill(pool, table, lengths, seed, spread=1.0):
    """Random keys and values at the places of the sequences' tokens; nothing else
    is touched."""
    gen = torch.Generator("cuda").manual_seed(seed)
    n = lengths.tolist()
    page_tokens = pool.keys.shape[2]
    for i, count in enumerate(n):
        if count <= 0:
            continue
        t = torch.arange(count, device=pool.keys.device)
        page, place = table[i].to(pool.keys.device).long()[t // page_tokens], t % page_tokens
        shape = (count, pool.keys.shape[1], pool.keys.shape[3])
        for which in ("key", "value"):
            x = torch.randn(shape, generator=gen, device="cuda").to(pool.keys.device) * spread
            if pool.eight:
                scales = pool.key_scales if which == "key" else pool.value_scales
                s = torch.rand(shape[:2], generator=gen, device="cuda").to(pool.keys.device) * 0.01 + 0.005
                scales[page, :, place] = s
                x = (x * 110).clamp(-448, 448).to(E4M3).view(torch.uint8)
            else:
                x = x.to(pool.dtype)
            pool.bytes(which)[page, :, place] = x


def table_of(lengths, page_tokens, seed, spare=2, extra=3):
    """(page table with -1 where a sequence has no page, pages of the pool): pages
    in random order."""
    used = [-(-max(n, 0) // page_tokens) for n in lengths]
    table = torch.full((len(lengths), max(used + [0]) + spare), -1, dtype=torch.int32)
    order = torch.randperm(sum(used) + extra, generator=torch.Generator().manual_seed(seed)).int()
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    return table, sum(used) + extra
