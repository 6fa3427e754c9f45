"""The operators of ar_block.h on the GPU against their definitions in 64 bits
(tests/block_ref.py, with the bounds derived there): all-reduce with residual
and norm, gate with 8-bit output, block-scaled product; then the layer they
make together."""
import pytest
import torch

import all_reduce_amd as ar
import block_ref as ref
from gpu_util import bits, note

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
POISON = 0xA5


@pytest.fixture(scope="module")
def comm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = ar.Comm(device="cuda:0", max_ranks=32, max_ll_bytes_per_rank=1 << 16)
    yield c
    c.close()


class Planes:
    """Rank buffers [rows, cols] with poison around them, to see stray writes."""

    def __init__(self, ranks, rows, cols, dtype):
        es = torch.empty((), dtype=dtype).element_size()
        self.n, self.es = rows * cols, es
        stride = -(-(rows * cols * es + 512) // 256) * 256
        self.raw = torch.full((ranks, stride), POISON, dtype=torch.uint8, device="cuda:0")
        self.ranks = [r[256:256 + rows * cols * es].view(dtype).view(rows, cols) for r in self.raw]

    def fill(self, x):
        for t, v in zip(self.ranks, x):
            t.copy_(v)
        return self

    def untouched(self):
        a = self.raw[:, :256]
        b = self.raw[:, 256 + self.n * self.es:]
        return bool((a == POISON).all()) and bool((b == POISON).all())


def draw(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def eight(shape, seed):
    return draw(shape, seed, scale=110.0).clamp_(-448, 448).to(E4M3)


def same(a, b):
    """The same bytes, NaN included."""
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def check_eight(out, scales, y, tol, what):
    t, t_tol, s, s_tol = ref.quantised(y, tol)
    ref.assert_within(scales, s, s_tol, what + " scales")
    ref.assert_within(out.float(), t, t_tol, what + " values")


# ---- all-reduce, residual, norm ---------------------------------------------
NORMS = [
    # ranks, rows, cols, dtype: widths around a group of 8, a scale block, a wave,
    # a workgroup and the widest row; every remainder of the rank batches
    (1, 1, 1, "bf16"), (2, 3, 7, "fp16"), (3, 2, 8, "fp32"), (4, 5, 127, "bf16"),
    (5, 4, 128, "fp16"), (6, 3, 129, "fp32"), (7, 9, 512, "bf16"), (8, 1, 8192, "bf16"),
    (8, 64, 1000, "bf16"), (9, 2, 520, "fp32"), (12, 3, 5001, "fp16"), (13, 2, 8192, "fp16"),
    (15, 1, 4099, "fp32"), (16, 3, 8200, "fp32"), (31, 2, 1031, "bf16"), (32, 2, 16384, "bf16"),
    (32, 1, 16392, "fp32"), (2, 2, 24577, "bf16"), (1, 2, 32768, "fp32"), (8, 1, 32767, "fp16"),
    (3, 1500, 136, "bf16"), (1, 5000, 64, "fp16"), (8, 700, 2048, "bf16"),
]


def run_norm(comm, x, res, w, eps, quant, keep, inplace=None):
    ranks, rows, cols = x.shape
    note(f"norm R={ranks} {rows}x{cols} {x.dtype} quant={quant} keep={keep} inplace={inplace}")
    send = Planes(ranks, rows, cols, x.dtype).fill(x)
    r = Planes(1, rows, cols, x.dtype).fill([res]) if res is not None else None
    kept = Planes(ranks, rows, cols, x.dtype) if keep else None
    out = Planes(ranks, rows, cols, E4M3 if quant else x.dtype)
    scales = Planes(ranks, ref.blocks(cols), rows, torch.float32) if quant else None
    if inplace == "keep in send":
        kept = send
    elif inplace == "out in send":
        out = send
    keep_to = kept.ranks if kept else None
    if inplace == "keep in residual":
        keep_to = [r.ranks[0], *kept.ranks[1:]]
    comm.all_reduce_norm(send.ranks, w.cuda(), eps, residual=r.ranks[0] if r else None,
                         residual_out=keep_to, out=out.ranks, scales=scales.ranks if scales else None)
    torch.cuda.synchronize()
    for p in (send, r, kept, out, scales):
        assert p is None or p.untouched()
    if inplace != "keep in send" and inplace != "out in send":
        for t, v in zip(send.ranks, x):
            assert same([t.cpu()], [v.contiguous()]), "a send buffer changed"
    return keep_to, out.ranks, scales.ranks if scales else None


def check_norm(x, res, w, eps, kept, out, scales, what):
    h, h_tol, y, y_tol = ref.norm(x, res, w, eps)
    for r in range(len(out)):
        if kept is not None:
            ref.assert_within(kept[r], h, ref.rounded(h, h_tol, x.dtype), f"{what} h rank {r}")
        if scales is None:
            ref.assert_within(out[r], y, ref.rounded(y, y_tol, x.dtype), f"{what} out rank {r}")
        else:
            check_eight(out[r], scales[r], y, y_tol, f"{what} rank {r}")


@pytest.mark.parametrize("quant", [False, True], ids=["same", "eight"])
@pytest.mark.parametrize("ranks,rows,cols,dtype", NORMS)
def test_norm(comm, ranks, rows, cols, dtype, quant):
    seed = ranks * 1000 + rows + cols
    x = draw((ranks, rows, cols), seed, DT[dtype])
    x[:, :, ::97] *= 20
    with_res = (rows + cols) % 3 != 0
    res = draw((rows, cols), seed + 1, DT[dtype], 3.0) if with_res else None
    w = (draw((cols,), seed + 2) * 0.2 + 1).to(DT[dtype])
    got = run_norm(comm, x, res, w, 1e-5, quant, with_res or cols % 2 == 0)
    check_norm(x, res, w, 1e-5, *got, "norm")


@pytest.mark.parametrize("inplace", ["keep in send", "out in send", "keep in residual"])
@pytest.mark.parametrize("ranks,rows,cols,dtype", [(8, 5, 8192, "bf16"), (3, 7, 1001, "fp32"),
                                                   (2, 3, 20000, "fp16")])
def test_norm_in_place(comm, ranks, rows, cols, dtype, inplace):
    x = draw((ranks, rows, cols), 41, DT[dtype])
    res, w = draw((rows, cols), 42, DT[dtype]), draw((cols,), 43, DT[dtype])
    got = run_norm(comm, x, res, w, 1e-6, False, True, inplace)
    check_norm(x, res, w, 1e-6, *got, inplace)


@pytest.mark.parametrize("ranks,rows,cols,dtype", [(8, 5, 8192, "bf16"), (2, 600, 1001, "fp16"),
                                                   (3, 7, 30, "fp32")])
def test_norm_in_place_combined(comm, ranks, rows, cols, dtype):
    """Every exact overlap at once: the sums kept in the send buffers and an
    output in the residual; the residual that is rank 0's send buffer, with the
    sum kept there too.  Both against the same call with buffers of its own."""
    x = draw((ranks, rows, cols), 71, DT[dtype])
    w = draw((cols,), 72, DT[dtype]).cuda()
    for shared, res in ((False, draw((rows, cols), 73, DT[dtype])), (True, x[0])):
        note(f"norm in place, combined R={ranks} {rows}x{cols} {dtype}")
        own = [Planes(ranks, rows, cols, DT[dtype]) for _ in range(3)]
        own[0].fill(x)
        comm.all_reduce_norm(own[0].ranks, w, 1e-5, residual=res.cuda(), residual_out=own[1].ranks,
                             out=own[2].ranks)
        send = Planes(ranks, rows, cols, DT[dtype]).fill(x)
        out = Planes(ranks, rows, cols, DT[dtype])
        r = send.ranks[0] if shared else out.ranks[1].copy_(res)
        comm.all_reduce_norm(send.ranks, w, 1e-5, residual=r, residual_out=send.ranks,
                             out=out.ranks)
        torch.cuda.synchronize()
        assert send.untouched() and out.untouched()
        assert same(send.ranks, own[1].ranks) and same(out.ranks, own[2].ranks)


@pytest.mark.parametrize("ranks,rows,cols,dtype", [(8, 64, 8192, "bf16"), (5, 3, 777, "fp16"),
                                                   (32, 2, 4096, "fp32")])
def test_kept_sum_has_the_bits_of_the_all_reduce(comm, ranks, rows, cols, dtype):
    """Without a residual, what is kept is the all-reduce's own result."""
    x = draw((ranks, rows, cols), 51, DT[dtype])
    kept, _, _ = run_norm(comm, x, None, torch.ones(cols, dtype=DT[dtype]), 1e-6, True, True)
    bufs = Planes(ranks, rows, cols, DT[dtype]).fill(x)
    comm.all_reduce(bufs.ranks, protocol="hb")
    torch.cuda.synchronize()
    for a, b in zip(kept, bufs.ranks):
        assert (bits(a.cpu()) == bits(b.cpu())).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_norm_special_rows(comm, dtype):
    """Rows of zeros, with an infinity, with a NaN, of tiny and of large values:
    each changes itself alone."""
    x = draw((4, 7, 700), 61, DT[dtype])
    x[:, 1] = 0
    x[2, 2, 300] = float("inf")
    x[1, 3, 699] = float("nan")
    x[:, 4] *= 1e-4
    x[:, 5] *= 1e3
    x[:, 6, 128:256] = 0
    w = draw((700,), 62, DT[dtype])
    h, h_tol, y, y_tol = ref.norm(x, None, w, 1e-5)
    _, out, _ = run_norm(comm, x, None, w, 1e-5, False, False)
    # an infinite h: mean and root infinite, so 0 but at the infinity (inf * 0)
    y[2] = 0
    y[2, 300] = float("nan")
    y_tol[2:4] = 0
    for t in out:
        ref.assert_within(t, y, ref.rounded(y, y_tol, DT[dtype]).nan_to_num(), "special")
    _, out, scales = run_norm(comm, x, None, w, 1e-5, True, False)
    s, q = scales[3].cpu(), out[3].float().cpu()
    assert (s[:, 1] == 2.0 ** -126).all() and (q[1] == 0).all()
    assert s[2, 2].isnan() and q[2, 256:384].isnan().all()
    assert (s[[0, 1, 3, 4, 5], 2] == 2.0 ** -126).all() and (q[2, :256] == 0).all()
    assert s[:, 3].isnan().all() and q[3].isnan().all()
    assert s[1, 6] == 2.0 ** -126 and (q[6, 128:256] == 0).all()
    for row in (0, 4, 5, 6):
        check_eight(out[3][row:row + 1], scales[3][:, row:row + 1], y[row:row + 1],
                    y_tol[row:row + 1], f"row {row}")


def test_norm_zero_row_without_eps_is_nan(comm):
    x = torch.zeros((2, 2, 64))
    x[:, 1] = 1
    _, out, _ = run_norm(comm, x, None, torch.ones(64), 0.0, False, False)
    assert out[0][0].isnan().all() and torch.equal(out[0][1].cpu(), torch.ones(64))


# ---- gate and quantisation ----------------------------------------------------
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("ranks,rows,cols,dtype", [
    (1, 1, 1, "bf16"), (2, 3, 7, "fp16"), (3, 5, 128, "fp32"), (8, 64, 448, "bf16"),
    (4, 17, 129, "bf16"), (5, 33, 1001, "fp16"), (32, 2, 264, "bf16"), (1, 1000, 136, "fp32"),
    (2, 70, 3584, "bf16"), (1, 1, 16384, "fp16"), (7, 9, 1280, "fp32"), (3, 257, 200, "bf16"),
])
def test_gate_quant(comm, ranks, rows, cols, dtype, act):
    wide = 2 * cols if act == "silu" else cols
    x = draw((ranks, rows, wide), ranks + rows + cols, DT[dtype], 3.0)
    note(f"gate R={ranks} {rows}x{cols} {dtype} {act}")
    src = Planes(ranks, rows, wide, DT[dtype]).fill(x)
    out = Planes(ranks, rows, cols, E4M3)
    scales = Planes(ranks, ref.blocks(cols), rows, torch.float32)
    comm.gate_quant(src.ranks, out.ranks, scales.ranks, act=act)
    torch.cuda.synchronize()
    assert src.untouched() and out.untouched() and scales.untouched()
    for r in range(ranks):
        y, tol = ref.gate(x[r], act)
        check_eight(out.ranks[r], scales.ranks[r], y, tol, f"gate rank {r}")


def test_gate_special_values(comm):
    """Zeros, infinities, NaN and gates far from zero, each in a block of its own."""
    x = torch.ones((1, 3, 2 * 128))
    x[0, 0, :128] = 0
    x[0, 1, 5], x[0, 1, 6] = float("inf"), -1000.0
    x[0, 2, 7] = float("nan")
    src, out = x.cuda(), torch.empty((3, 128), dtype=E4M3, device="cuda:0")
    scales = torch.empty((1, 3), device="cuda:0")
    comm.gate_quant([src[0]], [out], [scales])
    torch.cuda.synchronize()
    s, q = scales.cpu(), out.float().cpu()
    assert s[0, 0] == 2.0 ** -126 and (q[0] == 0).all()
    assert s[0, 1] == float("inf") and q[1, 5].isnan() and (q[1, :5] == 0).all() and q[1, 6] == 0
    assert s[0, 2].isnan() and q[2].isnan().all()


# ---- block-scaled product -----------------------------------------------------
MATMULS = [
    # ranks, rows, n, k: one row to several tiles, ragged in every direction
    (1, 1, 1, 16), (1, 1, 16, 128), (2, 3, 17, 144), (1, 16, 64, 256), (3, 17, 100, 112),
    (8, 1, 512, 1024), (2, 64, 256, 512), (3, 77, 1000, 1040), (1, 65, 129, 2048),
    (2, 130, 384, 640), (1, 257, 300, 4096), (4, 256, 512, 384), (1, 300, 513, 1296),
    (8, 40, 136, 272), (32, 2, 48, 160), (1, 512, 768, 1024), (2, 1000, 264, 128),
    (1, 33, 8, 8192), (1, 5, 4100, 2064), (5, 128, 128, 128), (1, 8, 7, 96),
    (2, 2, 200, 1040), (3, 9, 1000, 640), (1, 30, 9000, 272), (8, 40, 2100, 400),
    # few tiles and a long k: workgroups share a summed tile's k
    (8, 91, 66, 6224), (6, 35, 130, 2064), (5, 1, 8, 4096), (32, 3, 100, 640),
    # enough tiles for 128 x 128 (each, sum) and 256 x 256 (each, sum)
    (8, 200, 2048, 1136), (2, 2100, 2000, 272), (8, 520, 2000, 1040), (2, 2100, 4000, 400),
]


def matmul_inputs(ranks, rows, n, k, seed):
    a, b = eight((ranks, rows, k), seed), eight((ranks, n, k), seed + 1)
    sa = draw((ranks, ref.blocks(k), rows), seed + 2, scale=0.5).exp() * 0.01
    sb = draw((ranks, ref.blocks(n), ref.blocks(k)), seed + 3, scale=0.5).exp() * 2e-4
    return a, sa, b, sb


def run_matmul(comm, a, sa, b, sb, dtype, reduce):
    ranks, rows, k = a.shape
    n = b.shape[1]
    note(f"matmul R={ranks} {rows}x{n}x{k} {dtype} reduce={reduce}")
    planes = [Planes(ranks, *t.shape[1:], t.dtype).fill(t) for t in (a, sa, b, sb)]
    out = Planes(ranks, rows, n, dtype)
    comm.matmul_scaled(*[p.ranks for p in planes], out.ranks, reduce=reduce)
    torch.cuda.synchronize()
    assert out.untouched()
    return out.ranks


@pytest.mark.parametrize("reduce", [False, True], ids=["each", "reduce"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ranks,rows,n,k", MATMULS)
def test_matmul(comm, ranks, rows, n, k, dtype, reduce):
    a, sa, b, sb = matmul_inputs(ranks, rows, n, k, rows + n + k)
    out = run_matmul(comm, a, sa, b, sb, DT[dtype], reduce)
    each = [ref.matmul(a[r], sa[r], b[r], sb[r], DT[dtype]) for r in range(ranks)]
    if reduce:
        # the ranks' blocks are added one after the other: one step a block
        total = sum(c for c, _, _ in each)
        tol = sum(t + ranks * ref.blocks(k) * step for _, t, step in each)
        each = [(total, tol)] * ranks
    else:
        each = [x[:2] for x in each]
    for r in range(ranks):
        c, tol = each[r]
        ref.assert_within(out[r], c, ref.rounded(c, tol, DT[dtype]), f"rank {r}")
        if reduce:
            assert (bits(out[r].cpu()) == bits(out[0].cpu())).all()


@pytest.mark.parametrize("reduce", [False, True], ids=["each", "reduce"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ranks,rows,n,k", [(8, 60, 2090, 4112), (8, 140, 1030, 8192),
                                            (8, 200, 2050, 4112), (8, 4, 4100, 2064)])
def test_matmul_from_memory(comm, ranks, rows, n, k, dtype, reduce):
    """More than 64 MB of inputs: other tiles, and other numbers of workgroups to
    share k, than smaller ones take."""
    test_matmul(comm, ranks, rows, n, k, dtype, reduce)


@pytest.mark.parametrize("rows,n,k", [(3, 40, 272), (100, 200, 400), (300, 520, 1040)])
def test_matmul_special_values(comm, rows, n, k):
    """A NaN in an activation takes its row alone, one in a weight its column,
    one in a scale what it scales; neighbours keep their values."""
    a, sa, b, sb = matmul_inputs(1, rows, n, k, 7)
    clean = run_matmul(comm, a, sa, b, sb, torch.float32, False)[0].cpu()
    a, b = a.float(), b.float()
    a[0, 1, k - 1] = float("nan")
    b[0, n - 1, 0] = float("nan")
    sa[0, 1, 2] = float("nan")
    got = run_matmul(comm, a.to(E4M3), sa, b.to(E4M3), sb, torch.float32, False)[0].cpu()
    hit = torch.zeros((rows, n), dtype=torch.bool)
    hit[1], hit[2], hit[:, n - 1] = True, True, True
    assert got[hit].isnan().all() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_matmul_special_values_where_k_is_shared(comm, dtype):
    """Few tiles and a long k, so that several workgroups share a tile's sums: a
    NaN or an infinity of one rank takes its row, in every rank's output."""
    a, sa, b, sb = matmul_inputs(8, 5, 40, 4096, 13)
    b = b.float().abs().clamp_min(1.0).to(E4M3)  # an infinity times these is one
    a = a.float().abs().clamp_min(1.0).to(E4M3)
    clean = run_matmul(comm, a, sa, b, sb, DT[dtype], True)[0].cpu()
    a = a.float()
    a[6, 1, 4095] = float("nan")
    sa[3, 17, 2] = float("inf")
    sa[0, 0, 4] = float("-inf")
    for out in run_matmul(comm, a.to(E4M3), sa, b, sb, DT[dtype], True):
        out = out.cpu()
        assert out[1].isnan().all() and (out[2] == float("inf")).all()
        assert (out[4] == float("-inf")).all()
        assert same([out[0], out[3]], [clean[0], clean[3]])


def test_matmul_with_shared_k_in_graphs_and_on_two_streams(comm):
    """The partial sums of workgroups that share a tile's k are the call's own:
    two captured graphs and eager calls on two streams do not disturb one another."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets, graphs, want = [], [], []
    for i, (rows, n, k, dtype) in enumerate([(3, 72, 4096, torch.bfloat16),
                                             (40, 66, 2064, torch.float32)]):
        planes = [Planes(8, *t.shape[1:], t.dtype).fill(t)
                  for t in matmul_inputs(8, rows, n, k, 30 + i)]
        out = Planes(8, rows, n, dtype)
        sets.append((planes, out))
        note(f"shared k {rows}x{n}x{k} {dtype}")
        call = comm.prepare_matmul_scaled(*[p.ranks for p in planes], out.ranks, reduce=True,
                                          stream=streams[i])
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out.ranks])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            comm.matmul_scaled(*[p.ranks for p in planes], out.ranks, reduce=True)
        graphs.append((graph, call))
    for turn in range(4):
        for (_, out), stream in zip(sets, streams):
            out.raw.fill_(POISON)
        torch.cuda.synchronize()
        for (graph, call), stream in zip(graphs, streams):
            if turn % 2 == 0:
                with torch.cuda.stream(stream):
                    graph.replay()
            else:
                call()
        torch.cuda.synchronize()
        for (_, out), w in zip(sets, want):
            assert same(out.ranks, w)


def test_matmul_is_repeatable(comm):
    """The same inputs give the same bits, call after call."""
    for rows, n, k in ((1, 1024, 4096), (64, 640, 2048), (512, 512, 512)):
        args = matmul_inputs(2, rows, n, k, 11)
        one = run_matmul(comm, *args, torch.float32, True)[0].cpu()
        for _ in range(3):
            assert torch.equal(one, run_matmul(comm, *args, torch.float32, True)[1].cpu())


def test_matmul_subnormal_values(comm):
    """The smallest 8-bit values, subnormal ones among them, keep their products:
    small whole multiples of 2^-18, exact in every type that can hold them."""
    g = torch.Generator("cpu").manual_seed(3)
    for rows, n, k in ((2, 40, 144), (40, 70, 272), (700, 900, 128)):
        a = torch.randint(-15, 16, (1, rows, k), generator=g).float() * 2.0 ** -9
        b = torch.randint(-15, 16, (1, n, k), generator=g).float() * 2.0 ** -9
        one = [torch.ones((1, ref.blocks(k), rows)), torch.ones((1, ref.blocks(n), ref.blocks(k)))]
        got = run_matmul(comm, a.to(E4M3), one[0], b.to(E4M3), one[1], torch.float32, False)[0].cpu()
        assert torch.equal(got.double(), a[0].double() @ b[0].double().t().contiguous())


# ---- past 32 bits ------------------------------------------------------------
def test_norm_past_32_bits(comm):
    """A message of 2.2e9 elements: rows at both ends and around 2^31 and 2^32
    bytes."""
    rows, cols = 135_000, 16_384
    note(f"norm {rows}x{cols} bf16")
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda:0").uniform_(-1, 1)
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda:0")
    q = torch.empty((rows, cols), dtype=E4M3, device="cuda:0")
    s = torch.empty((ref.blocks(cols), rows), device="cuda:0")
    h = torch.empty_like(x)
    comm.all_reduce_norm([x], w, 1e-5, residual_out=[h], out=[q], scales=[s])
    torch.cuda.synchronize()
    for row in (0, 65_535, 65_536, 131_071, 131_072, rows - 1):
        xr = x[row:row + 1].cpu()
        check_norm(xr[None], None, w.cpu(), 1e-5, [h[row:row + 1]], [q[row:row + 1]],
                   [s[:, row:row + 1]], f"row {row}")


def test_gate_past_32_bits(comm):
    rows, cols = 140_000, 8192
    note(f"gate {rows}x{cols} bf16")
    x = torch.empty((rows, 2 * cols), dtype=torch.bfloat16, device="cuda:0").uniform_(-4, 4)
    q = torch.empty((rows, cols), dtype=E4M3, device="cuda:0")
    s = torch.empty((ref.blocks(cols), rows), device="cuda:0")
    comm.gate_quant([x], [q], [s])
    torch.cuda.synchronize()
    for row in (0, 65_536, 131_072, rows - 1):
        y, tol = ref.gate(x[row:row + 1].cpu(), "silu")
        check_eight(q[row:row + 1], s[:, row:row + 1], y, tol, f"row {row}")


@pytest.mark.parametrize("rows,n,k,dtype", [(140_000, 16_400, 16, "bf16"), (300_000, 64, 8192, "fp16"),
                                            (300_000, 64, 8192, "bf16"), (40, 300_000, 8192, "bf16"), (1, 300_000, 8192, "fp32")])
def test_matmul_past_32_bits(comm, rows, n, k, dtype):
    """Outputs, activations and weights of more than 2^31 bytes."""
    note(f"matmul {rows}x{n}x{k} {dtype}")
    g = torch.Generator("cuda").manual_seed(5)

    def values(r):
        t = torch.empty((r, k), dtype=E4M3, device="cuda:0")
        for part in t.split(1 << 15):
            part.copy_(torch.randn(part.shape, generator=g, device="cuda:0").mul_(110).clamp_(-448, 448))
        return t

    a, b = values(rows), values(n)
    sa = torch.rand((ref.blocks(k), rows), generator=g, device="cuda:0").add_(0.5)
    sb = torch.rand((ref.blocks(n), ref.blocks(k)), generator=g, device="cuda:0").add_(0.5)
    out = torch.empty((rows, n), dtype=DT[dtype], device="cuda:0")
    comm.matmul_scaled([a], [sa], [b], [sb], [out])
    torch.cuda.synchronize()
    ri = torch.tensor(sorted({0, rows // 2, rows - 1}))
    ni = torch.tensor(sorted({0, n // 2, n - 1}))
    c, tol, _ = ref.matmul(a[ri.cuda()].cpu(), sa[:, ri.cuda()].cpu(), b[ni.cuda()].cpu(),
                           sb[(ni // 128).cuda()].cpu(), DT[dtype], columns=ni)
    ref.assert_within(out[ri.cuda()][:, ni.cuda()], c, ref.rounded(c, tol, DT[dtype]), "corners")


# ---- together -------------------------------------------------------------------
class Layer:
    """The MLP half of a layer over `ranks` ranks: norm, up product, gate, down
    product, all-reduce with the next norm."""

    def __init__(self, comm, ranks, rows, hidden, inner, dtype, seed, stream=None):
        self.comm, self.ranks, self.stream = comm, ranks, stream
        P = lambda r, c, d: Planes(ranks, r, c, d)  # noqa: E731
        self.x, self.h, self.h2 = P(rows, hidden, dtype), P(rows, hidden, dtype), P(rows, hidden, dtype)
        self.q, self.qs = P(rows, hidden, E4M3), P(ref.blocks(hidden), rows, torch.float32)
        self.up, self.gq = P(rows, 2 * inner, dtype), P(rows, inner, E4M3)
        self.gs = P(ref.blocks(inner), rows, torch.float32)
        self.part, self.y = P(rows, hidden, dtype), P(rows, hidden, dtype)
        self.fused = P(rows, hidden, dtype)
        self.w = (draw((2, hidden), seed) * 0.1 + 1).to(dtype).cuda()
        self.w1 = P(2 * inner, hidden, E4M3).fill(eight((ranks, 2 * inner, hidden), seed + 1))
        self.w2 = P(hidden, inner, E4M3).fill(eight((ranks, hidden, inner), seed + 2))
        self.s1 = P(ref.blocks(2 * inner), ref.blocks(hidden), torch.float32)
        self.s2 = P(ref.blocks(hidden), ref.blocks(inner), torch.float32)
        for p, k in ((self.s1, hidden), (self.s2, inner)):
            for t in p.ranks:
                t.fill_(1 / (110 * k ** 0.5))
        self.res = torch.empty((rows, hidden), dtype=dtype, device="cuda:0")

    def fill(self, seed):
        for r, t in enumerate(self.x.ranks):
            t.copy_(draw(t.shape, seed + r, t.dtype))
        self.res.copy_(draw(self.res.shape, seed + 99, self.res.dtype))

    def calls(self):
        """The calls of one pass, in order, as functions."""
        c, s = self.comm, self.stream
        return [
            lambda: c.all_reduce_norm(self.x.ranks, self.w[0], 1e-5, self.res, self.h.ranks,
                                      self.q.ranks, self.qs.ranks, stream=s),
            lambda: c.matmul_scaled(self.q.ranks, self.qs.ranks, self.w1.ranks, self.s1.ranks,
                                    self.up.ranks, stream=s),
            lambda: c.gate_quant(self.up.ranks, self.gq.ranks, self.gs.ranks, stream=s),
            lambda: c.matmul_scaled(self.gq.ranks, self.gs.ranks, self.w2.ranks, self.s2.ranks,
                                    self.part.ranks, stream=s),
            lambda: c.matmul_scaled(self.gq.ranks, self.gs.ranks, self.w2.ranks, self.s2.ranks,
                                    self.fused.ranks, reduce=True, stream=s),
            lambda: c.all_reduce_norm(self.part.ranks, self.w[1], 1e-5, self.h.ranks[0],
                                      self.h2.ranks, self.y.ranks, stream=s),
        ]

    def outputs(self):
        return [t.clone() for p in (self.h, self.q, self.qs, self.up, self.gq, self.gs, self.part,
                                    self.fused, self.h2, self.y) for t in p.ranks]


@pytest.mark.parametrize("ranks,rows,hidden,inner,dtype", [(8, 3, 1024, 448, "bf16"),
                                                           (2, 130, 640, 208, "fp16")])
def test_layer(comm, ranks, rows, hidden, inner, dtype):
    """Each step against the definition on the step's own inputs."""
    L = Layer(comm, ranks, rows, hidden, inner, DT[dtype], 5)
    L.fill(17)
    note(f"layer R={ranks} {rows}x{hidden}x{inner} {dtype}")
    for call in L.calls():
        call()
    torch.cuda.synchronize()
    cpu = lambda p: torch.stack([t.cpu() for t in p.ranks])  # noqa: E731
    check_norm(cpu(L.x), L.res.cpu(), L.w[0].cpu(), 1e-5, L.h.ranks, L.q.ranks, L.qs.ranks, "first")
    total, total_tol = 0, 0
    for r in range(ranks):
        c, tol, _ = ref.matmul(*[p.ranks[r].cpu() for p in (L.q, L.qs, L.w1, L.s1)], DT[dtype])
        ref.assert_within(L.up.ranks[r], c, ref.rounded(c, tol, DT[dtype]), f"up {r}")
        y, tol = ref.gate(L.up.ranks[r].cpu(), "silu")
        check_eight(L.gq.ranks[r], L.gs.ranks[r], y, tol, f"gate {r}")
        c, tol, step = ref.matmul(*[p.ranks[r].cpu() for p in (L.gq, L.gs, L.w2, L.s2)], DT[dtype])
        ref.assert_within(L.part.ranks[r], c, ref.rounded(c, tol, DT[dtype]), f"down {r}")
        total, total_tol = total + c, total_tol + tol + ranks * ref.blocks(inner) * step
    ref.assert_within(L.fused.ranks[-1], total, ref.rounded(total, total_tol, DT[dtype]), "reduced")
    check_norm(cpu(L.part), L.h.ranks[0].cpu(), L.w[1].cpu(), 1e-5, L.h2.ranks, L.y.ranks, None, "second")


def test_layer_in_a_graph(comm):
    """Captured once, replayed on new inputs with eager work between the
    replays: every replay equals the eager pass."""
    L = Layer(comm, 4, 5, 768, 272, torch.bfloat16, 6)
    L.fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for call in L.calls():
            call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in L.calls():
            call()
    for seed in (2, 3, 4):
        L.fill(seed)
        note(f"layer replay {seed}")
        g.replay()
        torch.cuda.synchronize()
        got = L.outputs()
        for p in (L.h, L.q, L.up, L.gq, L.part, L.fused, L.h2, L.y):
            p.raw.fill_(POISON)
        for call in L.calls():
            call()
        torch.cuda.synchronize()
        assert same(got, L.outputs())


def test_two_streams_at_once(comm):
    """Calls of one communicator on two streams that nothing orders."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    layers = [Layer(comm, 2, 40, 512, 256, torch.bfloat16, 7 + i, s) for i, s in enumerate(streams)]
    want = []
    for i, L in enumerate(layers):
        L.fill(20 + i)
        torch.cuda.synchronize()
        for call in L.calls():
            call()
        torch.cuda.synchronize()
        want.append(L.outputs())
    for _ in range(3):
        for calls in zip(*[L.calls() for L in layers]):
            for call in calls:
                call()
        torch.cuda.synchronize()
        assert all(same(w, L.outputs()) for w, L in zip(want, layers))


def test_refusals(comm):
    """What the binding refuses before the library is asked, and what the
    library refuses; nothing runs."""
    x = [torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda:0") for _ in range(2)]
    w = torch.zeros(64, dtype=torch.bfloat16, device="cuda:0")
    out = [torch.empty_like(t) for t in x]
    q = [torch.empty((2, 64), dtype=E4M3, device="cuda:0") for _ in range(2)]
    s = [torch.empty((1, 2), device="cuda:0") for _ in range(2)]
    with pytest.raises(ValueError, match="weight"):
        comm.all_reduce_norm(x, w[:32], 1e-5, out=out)
    with pytest.raises(ValueError, match="out"):
        comm.all_reduce_norm(x, w, 1e-5, out=out[:1])
    with pytest.raises(ValueError, match="out"):
        comm.all_reduce_norm(x, w, 1e-5, out=out, scales=s)
    with pytest.raises(ValueError, match="scales"):
        comm.all_reduce_norm(x, w, 1e-5, out=q, scales=[t.t() for t in s])
    with pytest.raises(ValueError, match="contiguous"):
        comm.all_reduce_norm([t.t().contiguous().t() for t in x], w, 1e-5, out=out)
    with pytest.raises(ValueError, match="residual"):
        comm.all_reduce_norm(x, w, 1e-5, residual=x[0].cpu(), out=out)
    with pytest.raises(ar.ArError) as e:
        comm.all_reduce_norm(x, w, -1.0, out=out)
    assert e.value.code == ar.arResult.arInvalidArgument
    with pytest.raises(ar.ArError) as e:
        comm.all_reduce_norm(x, w, 1e-5, out=[out[0], out[0]])
    assert e.value.code == ar.arResult.arInvalidArgument
    with pytest.raises(ValueError, match="even"):
        comm.gate_quant([t[:, :63].contiguous() for t in x], q, s)
    with pytest.raises(KeyError):
        comm.gate_quant(x, q, s, act="relu")
    a = [torch.zeros((2, 24), dtype=E4M3, device="cuda:0")]
    sc = [torch.zeros((1, 2), device="cuda:0")]
    with pytest.raises(ar.ArError) as e:
        comm.matmul_scaled(a, sc, a, [sc[0][:, :1].contiguous()], [x[0][:, :2].contiguous()])
    assert e.value.code == ar.arResult.arUnsupported
    empty = [torch.empty((0, 64), dtype=torch.bfloat16, device="cuda:0")]
    comm.all_reduce_norm(empty, w, 1e-5, out=empty)
    other = ar.Comm(device="cuda:0", max_ranks=1, max_ll_bytes_per_rank=0)
    call = other.prepare_all_reduce_norm(x, w, 1e-5, out=out)
    call()
    other.close()
    with pytest.raises(ValueError, match="closed"):
        call()
    torch.cuda.synchronize()
