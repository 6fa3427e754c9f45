"""Every kernel of the block-scaled product, by the sizes that take it: exact
sums to the bit, values of any size within derived bounds, and NaN that keep to
their row, column or block."""
import pytest
import torch

import block_ref as ref
from block_shapes import KERNELS
from gpu_util import note
from test_gpu_block import E4M3, Planes, comm, same  # noqa: F401  (comm is a fixture)

pytestmark = pytest.mark.gpu

CASES = [(kernel, form, dtype, shape) for kernel, form, bits, shapes in KERNELS
         for dtype in ((torch.bfloat16, torch.float16) if bits == 16 else (torch.float32,))
         for shape in shapes]
IDS = [f"{'x'.join(map(str, k))}-{f}-{str(d)[6:]}-{'x'.join(map(str, s))}" for k, f, d, s in CASES]
by_kernel = pytest.mark.parametrize("kernel,form,dtype,shape", CASES, ids=IDS)


def run(comm, a, sa, b, sb, dtype, form):
    planes = [Planes(t.shape[0], *t.shape[1:], t.dtype).fill(t) for t in (a, sa, b, sb)]
    out = Planes(a.shape[0], a.shape[1], b.shape[1], dtype)
    comm.matmul_scaled(*[p.ranks for p in planes], out.ranks, reduce=form != "each")
    torch.cuda.synchronize()
    assert out.untouched()
    return out.ranks


def whole(shape, most, gen):
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").float()


def powers(shape, gen):
    """Scales 2^-6 .. 2^-4."""
    return torch.randint(-6, -3, shape, generator=gen, device="cuda").float().exp2()


def scaled(x, s, rows):
    """8-bit values times their scales, in 64 bits; `rows`: s is of blocks of rows."""
    at = torch.arange(x.shape[1], device="cuda") // 128
    s = s.double()
    s = s[torch.arange(x.shape[0], device="cuda") // 128] if rows else s.t().contiguous()
    return x.double() * s[:, at]


@by_kernel
def test_exact_sums(comm, kernel, form, dtype, shape):
    """Whole numbers up to 7 with scales that are powers of two: every sum is a
    multiple of 2^-12 below 2^12 (49 products of 2^-8 a term, at most 21000
    terms), which binary32 holds, so each output is the exact sum's rounding."""
    ranks, rows, n, k = shape
    assert 49 * 16 * k * ranks < 1 << 24
    note(f"exact {kernel} {form} {dtype} {shape}")
    g = torch.Generator("cuda").manual_seed(rows + n + k)
    a, b = whole((ranks, rows, k), 7, g).to(E4M3), whole((ranks, n, k), 7, g).to(E4M3)
    sa, sb = powers((ranks, ref.blocks(k), rows), g), powers((ranks, ref.blocks(n), ref.blocks(k)), g)
    out = run(comm, a, sa, b, sb, dtype, form)
    want = [torch.mm(scaled(a[r].float(), sa[r], False), scaled(b[r].float(), sb[r], True).t().contiguous())
            for r in range(ranks)]
    if form != "each":
        want = [sum(want)] * ranks
    for r in range(ranks):
        assert (want[r].float().double() == want[r]).all()
        off = out[r] != want[r].to(dtype)
        assert not off.any(), f"rank {r}: {int(off.sum())} of {off.numel()}, first {off.nonzero()[0].tolist()}"


@by_kernel
def test_special_values(comm, kernel, form, dtype, shape):
    """A NaN in a row's last activation takes that row, one in a column's first
    weight that column, one in a scale of activations its row and one in a
    scale of weights its 128 columns; the others keep every bit.  In a sum it
    takes them of all outputs."""
    ranks, rows, n, k = shape
    note(f"special {kernel} {form} {dtype} {shape}")
    g = torch.Generator("cuda").manual_seed(rows + n + k + 1)
    a, b = whole((ranks, rows, k), 100, g), whole((ranks, n, k), 100, g)
    sa = torch.rand((ranks, ref.blocks(k), rows), generator=g, device="cuda") * 1e-3
    sb = torch.rand((ranks, ref.blocks(n), ref.blocks(k)), generator=g, device="cuda") * 1e-3
    clean = [t.clone() for t in run(comm, a.to(E4M3), sa, b.to(E4M3), sb, dtype, form)]
    hit = torch.zeros((ranks, rows, n), dtype=torch.bool, device="cuda")
    nan, last = float("nan"), ranks - 1
    if rows > 2:
        a[last, rows - 2, k - 1] = nan
        hit[last, rows - 2] = True
        sa[0, ref.blocks(k) - 1, 0] = nan
        hit[0, 0] = True
    b[last, n - 1, 0] = nan
    hit[last, :, n - 1] = True
    if n > 256:
        sb[0, 1, ref.blocks(k) - 1] = nan
        hit[0, :, 128:256] = True
    if form != "each":
        hit[:] = hit.any(0)
    for r, out in enumerate(run(comm, a.to(E4M3), sa, b.to(E4M3), sb, dtype, form)):
        assert out[hit[r]].isnan().all(), f"rank {r}"
        assert same([out[~hit[r]]], [clean[r][~hit[r]]]), f"rank {r}"


@by_kernel
def test_values(comm, kernel, form, dtype, shape):
    """Values and scales of every size, within the bounds of tests/block_ref.py
    (its formulas, here computed where the values are)."""
    ranks, rows, n, k = shape
    note(f"values {kernel} {form} {dtype} {shape}")
    g = torch.Generator("cuda").manual_seed(rows + n + k + 2)

    def draw(*s):
        return torch.randn(s, generator=g, device="cuda")

    a, b = [draw(ranks, r, k).mul_(110).clamp_(-448, 448).to(E4M3) for r in (rows, n)]
    sa = draw(ranks, ref.blocks(k), rows).mul_(0.5).exp_().mul_(0.01)
    sb = draw(ranks, ref.blocks(n), ref.blocks(k)).mul_(0.3).exp_().mul_(2e-4)
    out = run(comm, a, sa, b, sb, dtype, form)
    sums, tols = [], []
    for r in range(ranks):
        x, w = scaled(a[r].float(), sa[r], False), scaled(b[r].float(), sb[r], True).t().contiguous()
        size = torch.mm(x.abs(), w.abs())
        tol = (128 + ref.blocks(k) + 24) * 2 * ref.U * size
        if dtype != torch.float32:
            tops = [t.abs().reshape(t.shape[0], -1, 8).amax(-1) for t in (x, w.t())]
            tol = tol + 7 * 2.0 ** -13 * torch.mm(tops[0], tops[1].t().contiguous())
        sums.append(torch.mm(x, w))
        tols.append(tol + (ranks * ref.blocks(k) * 2 * ref.U * size if form != "each" else 0))
    if form != "each":
        sums, tols = [sum(sums)] * ranks, [sum(tols)] * ranks
    for r in range(ranks):
        tol = ref.rounded(sums[r], tols[r], dtype)
        off = ~((out[r].double() - sums[r]).abs() <= tol)
        assert not off.any(), f"rank {r}: {int(off.sum())} of {off.numel()}, first {off.nonzero()[0].tolist()}"
