"""The operators of ar_block.h where a plain binary32 computation of the same
formula is exact or the range of a type ends: ties of the 8-bit rounding, rows
and gates far from 1, and the kernels that only large calls take."""
import pytest
import torch

import all_reduce_amd as ar
import block_ref as ref
from gpu_util import note
from test_gpu_block import (DT, E4M3, Planes, check_eight, check_norm, comm,  # noqa: F401  (a fixture)
                            draw, run_norm)

pytestmark = pytest.mark.gpu


# ---- quantisation --------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(2000, 1024), (1, 8192), (9000, 2056)])
def test_quantisation_is_the_quotient(comm, rows, cols, dtype):
    """Without an activation nothing is rounded before the scale: both it and the
    8-bit values are those of binary32 divisions, to the bit.  (The quotient is
    off by one bit of binary32 where it lies within 2^-46 of a tie between two of
    them: of these sizes none is expected to, and of 18 million none that is also
    next to a tie between two 8-bit values.)"""
    x = draw((rows, cols), rows + cols, DT[dtype], 3.0)
    note(f"quotient {rows}x{cols} {dtype}")
    src = Planes(1, rows, cols, DT[dtype]).fill([x])
    out, scales = Planes(1, rows, cols, E4M3), Planes(1, ref.blocks(cols), rows, torch.float32)
    comm.gate_quant(src.ranks, out.ranks, scales.ranks, act="none")
    torch.cuda.synchronize()
    assert src.untouched() and out.untouched() and scales.untouched()
    y = torch.nn.functional.pad(x.float(), (0, -cols % 128)).unflatten(1, (-1, 128))
    s = (y.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    assert torch.equal(scales.ranks[0].cpu(), s.t())
    q = (y / s.unsqueeze(-1)).flatten(1)[:, :cols].to(E4M3)
    off = out.ranks[0].cpu().float() != q.float()
    assert not off.any(), f"{int(off.sum())} of {off.numel()} values"


@pytest.mark.parametrize("dtype,size", [("bf16", 6e37), ("fp32", 6e37), ("bf16", 1e-36), ("bf16", 1e-39),
                                        ("fp32", 1e-36), ("fp32", 1e-43), ("fp16", 1e-7), ("fp16", 1e4)])
def test_quantisation_at_the_ends_of_a_type(comm, dtype, size):
    """The largest scales, and values that the smallest one holds as few steps."""
    x = (draw((300, 520), 92).clamp(-5, 5) * size).to(DT[dtype])
    note(f"quantisation {dtype} {size}")
    src = Planes(1, 300, 520, DT[dtype]).fill([x])
    out, scales = Planes(1, 300, 520, E4M3), Planes(1, 5, 300, torch.float32)
    comm.gate_quant(src.ranks, out.ranks, scales.ranks, act="none")
    torch.cuda.synchronize()
    assert src.untouched() and out.untouched() and scales.untouched()
    check_eight(out.ranks[0], scales.ranks[0], x.double(), torch.zeros_like(x, dtype=torch.float64), "ends")


# ---- norm ------------------------------------------------------------------------
@pytest.mark.parametrize("quant", [False, True], ids=["same", "eight"])
@pytest.mark.parametrize("dtype,sizes", [("bf16", (1e-38, 1e-30, 1e-15, 1.0, 1e15, 1e25, 1e37)),
                                         ("fp32", (1e-41, 1e-30, 1e-15, 1.0, 1e15, 1e25, 1e37)),
                                         ("fp16", (1e-7, 1e-5, 1.0, 3e3))])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("ranks,cols", [(1, 700), (3, 8192), (2, 24577)])
def test_norm_of_rows_of_any_size(comm, ranks, cols, eps, dtype, sizes, quant):
    """Rows whose squares would leave binary32 above or below, and the type's
    smallest values, have the norm of the definition."""
    x = draw((ranks, len(sizes), cols), 81) * torch.tensor(sizes).view(1, -1, 1)
    x = x.to(DT[dtype])
    w = (draw((cols,), 82) * 0.2 + 1).to(DT[dtype])
    kept, out, scales = run_norm(comm, x, None, w, eps, quant, True)
    h, h_tol, y, y_tol = ref.norm(x, None, w, eps)
    # a quotient and a product below 2^-126 round to a multiple of 2^-149
    y_tol = y_tol + 2.0 ** -150 * (1 + w.double().abs())
    for r in range(ranks):
        ref.assert_within(kept[r], h, ref.rounded(h, h_tol, x.dtype), f"h rank {r}")
        if quant:
            check_eight(out[r], scales[r], y, y_tol, f"rank {r}")
        else:
            ref.assert_within(out[r], y, ref.rounded(y, y_tol, x.dtype), f"out rank {r}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_of_one_large_value(comm, dtype):
    """One value of 2^100 in a row of ones: sqrt(cols) there, and what is left of
    the others is small and not zero."""
    x = torch.ones((1, 2, 512), dtype=DT[dtype])
    x[0, 1, 77] = 2.0 ** 100
    _, out, _ = run_norm(comm, x, None, torch.ones(512, dtype=DT[dtype]), 0.0, False, False)
    # 2^100 / sqrt(2^200 / 512) and 1 / sqrt(2^200 / 512), correctly rounded
    far = torch.tensor(512.0, dtype=torch.float64).sqrt()
    want = torch.full((512,), 2.0 ** -100, dtype=torch.float64) * far
    want[77] = far
    assert torch.equal(out[0][0].cpu().float(), torch.ones(512))
    # the root and the quotient round once each, the output once
    tol = want * (4 * ref.U) + want * ref.HALF_STEP[DT[dtype]]
    ref.assert_within(out[0][1], want, tol, "large")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("eps", [1e-42, 3e38])
def test_norm_with_eps_at_the_ends(comm, dtype, eps):
    """The smallest and the largest eps: rows of zeros stay zero, others are
    divided by the root of the sum."""
    x = draw((2, 3, 300), 86, DT[dtype])
    x[:, 1] = 0
    w = (draw((300,), 87) * 0.2 + 1).to(DT[dtype])
    eps = torch.tensor(eps).item()  # as binary32
    _, out, _ = run_norm(comm, x, None, w, eps, False, False)
    _, _, y, y_tol = ref.norm(x, None, w, eps)
    y_tol = y_tol + 2.0 ** -150 * (1 + w.double().abs())
    for t in out:
        assert (t[1] == 0).all()
        ref.assert_within(t[[0, 2]], y[[0, 2]], ref.rounded(y, y_tol, DT[dtype])[[0, 2]], "eps")


def test_norm_rounds_as_often_as_the_division(comm):
    """float32 rows of 64 values alike but for their signs: their sum of squares
    and its mean are exact, so an output has the rounding of eps added (halved
    by the root), of the inverse root, of its product with h and of the weight's
    product: 3.5 units of 2^-24 (and 2^-45, with which the root is computed)."""
    g = torch.Generator("cpu").manual_seed(83)
    size = torch.randint(1 << 10, 1 << 11, (4000, 1), generator=g).float()  # squares of 22 bits
    x = (size * (torch.randint(0, 2, (4000, 64), generator=g) * 2 - 1)).unsqueeze(0)
    w = draw((64,), 84) * 0.2 + 1
    eps = 0.3
    _, out, _ = run_norm(comm, x, None, w, eps, False, False)
    d = x[0].double()
    y = d / (d.square().mean(-1, keepdim=True) + torch.tensor(eps).double()).sqrt() * w.double()
    ref.assert_within(out[0], y, y.abs() * (3.5 * ref.U + 2.0 ** -40), "float32")


# ---- gate ------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_gate_far_below_zero(comm, dtype):
    """Gates whose exponential is below the type's range times an `up` that
    brings the product back into it, each row a block of its own; among them
    both sides of every border, and the 8-bit values and scales of the
    definition."""
    gates = [-60.0, -79.9, -80.0, -80.25, -87.0, -87.5, -88.0, -88.75, -90.0, -100.0, -104.0,
             -110.0, -125.5, -150.0, -170.0, -174.5, -190.0, -199.0, -210.0, -399.0, -401.0, -6e4]
    ups = [1.0, -1.0, 1e4, -6e4] + ([1e30, -3e38, 1e-20] if dtype != "fp16" else [])
    rows = [(g, u) for g in gates for u in ups]
    x = torch.zeros((1, len(rows), 256))
    for i, (g, u) in enumerate(rows):
        x[0, i, :128] = torch.linspace(g, g * 1.01, 128)
        x[0, i, 128:] = torch.linspace(u, u * 0.25, 128)
    x = x.to(DT[dtype])
    note(f"gate far below zero {dtype}")
    src = Planes(1, len(rows), 256, DT[dtype]).fill(x)
    out, scales = Planes(1, len(rows), 128, E4M3), Planes(1, 1, len(rows), torch.float32)
    comm.gate_quant(src.ranks, out.ranks, scales.ranks)
    torch.cuda.synchronize()
    assert src.untouched() and out.untouched() and scales.untouched()
    y, tol = ref.gate(x[0], "silu")
    # results below 2^-126 round to multiples of 2^-149, once or (with the
    # product before it) twice
    check_eight(out.ranks[0], scales.ranks[0], y, tol + 2.0 ** -149, "far")


def test_gate_infinities(comm):
    """Plus infinity passes through, minus infinity divides by an infinity."""
    inf = float("inf")
    x = torch.ones((1, 3, 256))
    x[0, 0, 5], x[0, 1, 5], x[0, 2, 128 + 5] = inf, -inf, inf
    x[0, 2, 5] = -100.0
    src, out = x.cuda(), torch.empty((3, 128), dtype=E4M3, device="cuda:0")
    scales = torch.empty((1, 3), device="cuda:0")
    comm.gate_quant([src[0]], [out], [scales])
    torch.cuda.synchronize()
    s, q = scales[0].cpu(), out.float().cpu()
    assert s[0] == inf and s[1].isnan() and s[2] == inf
    assert q[0, 5].isnan() and q[1].isnan().all() and q[2, 5].isnan()
    keep = torch.arange(128) != 5
    assert (q[0][keep] == 0).all() and (q[2][keep] == 0).all()


# ---- product ---------------------------------------------------------------------
def test_matmul_of_more_tiles_than_a_launch(comm):
    """Two ranks of 2^30 columns that share their weights: each has a launch."""
    n, k = 1 << 30, 16
    note(f"matmul 2 x (1 x {n} x {k})")
    g = torch.Generator("cuda").manual_seed(9)
    b = torch.empty((n, k), dtype=torch.uint8, device="cuda:0")
    for part in b.split(1 << 26):
        part.random_(0, 0x7F, generator=g)  # 0 .. 448
    b = b.view(E4M3)
    sb = torch.rand((n // 128, 1), generator=g, device="cuda:0").add_(0.5)
    a = [draw((1, k), 90 + r, scale=50.0).to(E4M3).cuda() for r in range(2)]
    sa = [torch.full((1, 1), 0.5 + r, device="cuda:0") for r in range(2)]
    out = [torch.full((1, n), float("nan"), dtype=torch.bfloat16, device="cuda:0") for _ in range(2)]
    comm.matmul_scaled(a, sa, [b, b], [sb, sb], out)
    torch.cuda.synchronize()
    at = torch.cat([torch.tensor([0, 127, 128, n // 2 - 1, n // 2, n - 1]),
                    torch.randint(0, n, (2000,), generator=torch.Generator().manual_seed(91))])
    for r in range(2):
        c, tol, _ = ref.matmul(a[r].cpu(), sa[r].cpu(), b[at.cuda()].cpu(), sb[(at // 128).cuda()].cpu(),
                               torch.bfloat16, columns=at)
        ref.assert_within(out[r][:, at.cuda()], c, ref.rounded(c, tol, torch.bfloat16), f"rank {r}")
        assert not out[r].isnan().any()


# ---- kernels for more than 64 MiB ----------------------------------------------
def some_rows(rows, gen):
    return torch.cat([torch.tensor([0, 1, rows - 2, rows - 1]), torch.randint(0, rows, (40,), generator=gen)])


@pytest.mark.parametrize("quant", [False, True], ids=["same", "eight"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ranks,rows,cols", [
    # one, two, four and (float32) eight pieces a lane, in rows of whole pieces
    # and not; 3 and 7 ranks leave remainders in every batch of loads
    (3, 200_000, 65), (3, 120_000, 96), (3, 4000, 5001), (3, 4001, 5000), (7, 300, 12_345), (3, 700, 16_392),
    (3, 500, 32_763), (3, 499, 32_768)])
def test_norm_beyond_the_caches(comm, ranks, rows, cols, dtype, quant):
    g = torch.Generator("cpu").manual_seed(rows + cols)
    base = draw((997, cols), rows, DT[dtype])
    note(f"norm beyond the caches R={ranks} {rows}x{cols} {dtype} {quant}")
    send = Planes(ranks, rows, cols, DT[dtype])
    for r, t in enumerate(send.ranks):  # rank r's row i: row (i + 100 r) % 997 of `base`
        at = (torch.arange(rows) + 100 * r) % 997
        t.copy_(base.cuda()[at.cuda()])
    res = Planes(1, rows, cols, DT[dtype])
    res.ranks[0].copy_(base.cuda()[((torch.arange(rows) + 500) % 997).cuda()])
    w = (draw((cols,), 85) * 0.2 + 1).to(DT[dtype])
    kept, out = Planes(ranks, rows, cols, DT[dtype]), Planes(ranks, rows, cols, E4M3 if quant else DT[dtype])
    scales = Planes(ranks, ref.blocks(cols), rows, torch.float32) if quant else None
    assert ranks * rows * cols * (2 * send.es + out.es) > 64 << 20
    comm.all_reduce_norm(send.ranks, w.cuda(), 1e-5, res.ranks[0], kept.ranks, out.ranks,
                         scales.ranks if quant else None)
    torch.cuda.synchronize()
    for p in (send, res, kept, out, scales):
        assert p is None or p.untouched()
    i = some_rows(rows, g)
    x = torch.stack([base[(i + 100 * r) % 997] for r in range(ranks)])
    check_norm(x, base[(i + 500) % 997], w, 1e-5, [t[i.cuda()] for t in kept.ranks], [t[i.cuda()] for t in out.ranks],
               [t[:, i.cuda()] for t in scales.ranks] if quant else None, "beyond")
    for p in (kept, out, scales):  # every rank has the same, every row
        for t in p.ranks[1:] if p else ():
            assert torch.equal(t.view(torch.uint8), p.ranks[0].view(torch.uint8))
    # rows repeat after 997: all of them are like the first 997
    for p in (kept, out):
        t = p.ranks[0].view(torch.uint8)
        for at in range(997, rows, 997):
            assert torch.equal(t[at:at + 997], t[:min(997, rows - at)])
    if quant:
        t = scales.ranks[0]
        for at in range(997, rows, 997):
            assert torch.equal(t[:, at:at + 997], t[:, :min(997, rows - at)])


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ranks,rows,cols", [
    # blocks that are no multiple of four a group of lanes, last pieces of one
    # element and of all but one, rows that are no multiple of a workgroup's
    (2, 36_001, 520), (2, 18_001, 1001), (2, 14_003, 1289), (1, 40_007, 1152), (3, 90_001, 129), (2, 15, 1_200_007)])
def test_gate_beyond_the_caches(comm, ranks, rows, cols, dtype, act):
    g = torch.Generator("cuda").manual_seed(rows + cols)
    wide = 2 * cols if act == "silu" else cols
    note(f"gate beyond the caches R={ranks} {rows}x{cols} {dtype} {act}")
    src = Planes(ranks, rows, wide, DT[dtype])
    for t in src.ranks:
        for part in t.split(1 << 13):
            part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(3))
        if act == "silu":  # a few rows of gates far below zero, large values beside them
            far = torch.arange(rows // 7, rows, max(1, rows // 5), device="cuda")
            t[far, :cols] = -90.0
            t[far, cols:] *= 1e3
    out, scales = Planes(ranks, rows, cols, E4M3), Planes(ranks, ref.blocks(cols), rows, torch.float32)
    assert ranks * rows * (wide * src.es + cols) > 64 << 20
    comm.gate_quant(src.ranks, out.ranks, scales.ranks, act=act)
    torch.cuda.synchronize()
    assert src.untouched() and out.untouched() and scales.untouched()
    i = some_rows(rows, torch.Generator("cpu").manual_seed(1)) if rows > 100 else torch.arange(rows)
    i = torch.cat([i, torch.arange(rows // 7, rows, max(1, rows // 5))])
    for r in range(ranks):
        y, tol = ref.gate(src.ranks[r][i.cuda()].cpu(), act)
        check_eight(out.ranks[r][i.cuda()], scales.ranks[r][:, i.cuda()], y, tol + 2.0 ** -149, f"rank {r}")
        # all rows, coarsely: one step of e4m3
        for at in range(0, rows, 1 << 13):
            x = src.ranks[r][at:at + (1 << 13)].double()
            if act == "silu":
                x = x[:, :cols] * torch.sigmoid(x[:, :cols]) * x[:, cols:]
            s = scales.ranks[r][:, at:at + (1 << 13)].double().t().repeat_interleave(128, 1)[:, :cols]
            q = out.ranks[r][at:at + (1 << 13)].double()
            assert ((q * s - x).abs() <= x.abs() * 2.0 ** -3 + s * 2.0 ** -9).all(), f"rank {r} rows from {at}"
