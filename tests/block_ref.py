"""The operators of ar_block.h in 64 bits on the CPU, with bounds on how far a
binary32 computation with one rounding per output may be from them.

Every bound is the sum of what each step may lose: a binary32 operation half a
unit in the last place (2^-24 of its result), a sum of n terms n of those of
the sum of magnitudes, an output's rounding half a step of its type."""
from __future__ import annotations

import torch

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U, E4M3: 2.0 ** -4}
# half of the smallest subnormal: the rounding of values too small for a relative bound
HALF_LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150,
              E4M3: 2.0 ** -10}
SCALE_MIN = 2.0 ** -126


def blocks(cols):
    return -(-cols // 128)


def assert_within(got, want, tol, what):
    """Finite values within `tol` of `want`; NaN and infinities in the same
    places, and infinities where the value is past the type's largest (half a
    step above it rounds to infinity)."""
    largest = torch.finfo(got.dtype).max
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = (got == want) | (got.isnan() & want.isnan())
    same |= got.isinf() & (got.sign() == want.sign()) & (want.abs() + tol > largest)
    bad = ~same & ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(x[0].item() for x in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: "
                             f"{got[i]} against {want[i]}, allowed {tol[i] if tol.dim() else tol}")


def rounded(want, tol, dtype):
    """The tolerance after a rounding to dtype of a value within tol of want."""
    return tol + HALF_STEP[dtype] * (want.abs() + tol) + HALF_LEAST[dtype]


def quantised(y, tol):
    """(values before their rounding, their tolerance, scales, their tolerance) of
    y within tol; scales laid out [blocks, rows]."""
    rows, cols = y.shape
    pad = torch.zeros((rows, blocks(cols) * 128), dtype=torch.float64)
    pad[:, :cols] = y.abs()
    top = pad.view(rows, -1, 128).amax(-1)
    pad.zero_()
    pad[:, :cols] = tol
    slack = pad.view(rows, -1, 128).amax(-1)
    scale = torch.where(top / 448 < SCALE_MIN, torch.tensor(SCALE_MIN, dtype=torch.float64), top / 448)
    scale_tol = slack / 448 + U * scale
    at = torch.arange(cols) // 128
    s, st = scale[:, at], scale_tol[:, at]
    t = y / s
    # the reciprocal and the product round once each; a scale too small by st
    off = tol / s + t.abs() * (st / s * 1.01 + 3 * U)
    return t, off + HALF_STEP[E4M3] * (t.abs() + off) + HALF_LEAST[E4M3], scale.t(), scale_tol.t()


def norm(x, residual, weight, eps):
    """x [R, rows, cols]: (h, tol of h, y, tol of y), before any rounding of outputs."""
    x = x.double()
    ranks, _, cols = x.shape
    h, size = x.sum(0), x.abs().sum(0)
    if residual is not None:
        h, size = h + residual.double(), size + residual.double().abs()
    h_tol = (ranks + 1) * U * size
    ms = h.square().mean(-1, keepdim=True)
    # the sum of squares: at most 32 a lane, 6 steps across a wave, 16 waves,
    # the mean and eps; the errors of h by the triangle inequality
    length = h.norm(dim=-1, keepdim=True)
    off = h_tol.norm(dim=-1, keepdim=True) / length.clamp_min(1e-300)
    ms_rel = (2 * off + off * off) + 64 * U
    inv = 1 / (ms + eps).sqrt()
    y = h * inv * weight.double()
    y_tol = h_tol * inv * weight.double().abs() + y.abs() * (ms_rel + 6 * U)
    return h, h_tol, y, y_tol


def gate(x, act):
    """x [rows, cols] or [rows, 2 cols]: (y, tol of y)."""
    x = x.double()
    if act == "none":
        return x, torch.zeros_like(x)
    g, u = x.chunk(2, -1)
    y = g * torch.sigmoid(g) * u
    # the exponent is off by 2 |g| units (its product with log2 e), the
    # exponential by 2, the sum, quotient and product by 1 or 2 each
    return y, y.abs() * (2 * g.abs() + 10) * U


def matmul(a, sa, b, sb, dtype, columns=None):
    """One rank's product in 64 bits, its tolerance before the rounding to dtype
    and what one more addition may lose.  ``columns``: b holds these output
    columns alone, and sb the row of scales of each.

    A float32 output: sums of 128 products and of the blocks in binary32, in
    some order and at worst cut instead of rounded (2 U a step of the sum of
    magnitudes).  A 16-bit output: the 8-bit matrix instruction adds groups of
    eight consecutive products, in which each of the other seven loses less
    than 2^-13 of the largest (it is cut at 2^-13 of the largest one's leading
    bit); the largest of a group is at most the largest activation times the
    largest weight of the group."""
    k, n = a.shape[1], b.shape[0]
    at = torch.arange(k) // 128
    a = a.double() * sa.double()[at].t()
    rows = torch.arange(n) // 128 if columns is None else torch.arange(n)
    b = b.double() * sb.double()[rows][:, at]
    size = a.abs() @ b.abs().t().contiguous()
    tol = (128 + blocks(k) + 24) * 2 * U * size
    if dtype != torch.float32:
        top = [x.abs().view(x.shape[0], -1, 8).amax(-1) for x in (a, b)]
        tol = tol + 7 * 2.0 ** -13 * (top[0] @ top[1].t().contiguous())
    return a @ b.t().contiguous(), tol, 2 * U * size
