"""The cases by which the tensor-parallel block operators are measured.

Three operators around the all-reduce of R rank buffers on one GPU:

* ``norm``   the all-reduce with the residual's addition, the root-mean-square
             norm and, where asked, an 8-bit output with a scale per row and
             128 columns (``Comm.prepare_all_reduce_norm``);
* ``gate``   SiLU gate (or nothing) and the same 8-bit output, per rank
             (``Comm.prepare_gate_quant``);
* ``matmul`` the product of 8-bit activations and weights with a scale per
             block of 128, per rank or summed over the ranks into every rank's
             output (``Comm.prepare_matmul_scaled``).

8-bit values are e4m3 (largest finite value 448).  Activation scales are laid
out [block of 128 columns, row], weight scales [block of 128 rows, block of
128 columns].
"""
import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": E4M3}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
EPS = 1e-5
TINY = 2.0 ** -126  # the smallest scale
GATE = {"silu": 2, "none": 1}  # input columns for each output column

# The largest listed cases: a drawn case costs no more.
MOST_NORM = 8 * 8192 * 8192
MOST_GATE = 8 * 8192 * 3584
MOST_FLOPS = 2 * 8 * 4096 * 7168 * 8192


def listed():
    return [
        # one new token of an 8-rank group: the smallest call of a decode loop
        dict(name="norm decode 1", op="norm", ranks=8, rows=1, cols=8192, dtype="bf16", out="e4m3", residual=True),
        # a decode batch of 64 tokens
        dict(name="norm decode 64", op="norm", ranks=8, rows=64, cols=8192, dtype="bf16", out="e4m3", residual=True),
        # a prefill of 8192 tokens whose next product is not in 8 bits
        dict(name="norm prefill 8192", op="norm", ranks=8, rows=8192, cols=8192, dtype="bf16", out="bf16", residual=True),
        # 16 ranks of float32 partial sums, 8-bit output
        dict(name="norm fp32 R16", op="norm", ranks=16, rows=1024, cols=7168, dtype="fp32", out="e4m3", residual=True),
        # a rank count, a row count and a width that no table is made for; the norm alone, no residual
        dict(name="norm odd", op="norm", ranks=3, rows=333, cols=5001, dtype="fp16", out="fp16", residual=False),
        # the MLP activation of a decode batch, each rank's share of a 28672-wide layer
        dict(name="gate decode 64", op="gate", ranks=8, rows=64, cols=3584, dtype="bf16", act="silu"),
        # and of a prefill
        dict(name="gate prefill 8192", op="gate", ranks=8, rows=8192, cols=3584, dtype="bf16", act="silu"),
        # the up product of one token: every rank's weights are read once
        dict(name="matmul decode 1", op="matmul", ranks=8, rows=1, n=7168, k=8192, out="bf16", reduce=False),
        # the row-parallel down product of a decode batch with its all-reduce
        dict(name="matmul decode 64", op="matmul", ranks=8, rows=64, n=8192, k=3584, out="bf16", reduce=True),
        # ragged everywhere: a batch of 77 rows, 3 ranks, float32 sums
        dict(name="matmul odd", op="matmul", ranks=3, rows=77, n=1000, k=1040, out="fp32", reduce=True),
        # the up product of a prefill
        dict(name="matmul prefill 4096", op="matmul", ranks=8, rows=4096, n=7168, k=8192, out="bf16", reduce=False),
        # the attention's output product of a prefill with its all-reduce
        dict(name="matmul prefill 8192", op="matmul", ranks=8, rows=8192, n=8192, k=1024, out="bf16", reduce=True),
    ]


def _log(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["norm", "norm", "gate", "matmul", "matmul"])
    if op == "matmul":
        ranks = rng.choice([1, 1, 2, 3, 4, 6, 8])
        rows, n, k = _log(rng, 1, 8192), _log(rng, 64, 8192), 16 * _log(rng, 8, 512)
        rows = max(1, min(rows, MOST_FLOPS // (2 * ranks * n * k)))
        return dict(op=op, ranks=ranks, rows=rows, n=n, k=k, out=rng.choice(["bf16", "fp16", "fp32"]), reduce=rng.random() < 0.5)
    ranks = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 24, 32])
    if op == "gate":
        cols = _log(rng, 64, 8192)
        rows = max(1, min(_log(rng, 1, 8192), MOST_GATE // (ranks * cols)))
        return dict(op=op, ranks=ranks, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), act=rng.choice(["silu", "silu", "none"]))
    cols = _log(rng, 64, 16384)
    cols = cols // 64 * 64 if rng.random() < 0.5 else cols
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    rows = max(1, min(_log(rng, 1, 8192), MOST_NORM * 2 // (ranks * cols * BYTES[dtype])))
    return dict(op=op, ranks=ranks, rows=rows, cols=cols, dtype=dtype, out=rng.choice([dtype, "e4m3"]), residual=rng.random() < 0.8)


def _plane(ranks, rows, cols, dtype):
    """One buffer a rank, each starting on a multiple of 256 bytes: [ranks, rows, cols]."""
    n = rows * cols
    at = 256 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((ranks, -(-n // at) * at), dtype=dtype, device="cuda")[:, :n].unflatten(1, (rows, cols))


def _blocks(cols):
    return -(-cols // 128)


def _eight(plane, gen):
    """Fills a plane with 8-bit values as a quantised normal variable has them: its blocks reach up to 448."""
    for rank in plane:
        rank.copy_(torch.randn(rank.shape, generator=gen, device="cuda").mul_(110).clamp_(-448, 448))


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    ranks, rows = case["ranks"], case["rows"]
    s = {"case": case}
    if case["op"] == "matmul":
        n, k = case["n"], case["k"]
        s["a"], s["b"] = _plane(ranks, rows, k, E4M3), _plane(ranks, n, k, E4M3)
        s["sa"], s["sb"] = _plane(ranks, _blocks(k), rows, torch.float32), _plane(ranks, _blocks(n), _blocks(k), torch.float32)
        _eight(s["a"], gen)
        _eight(s["b"], gen)
        s["sa"].copy_(torch.randn(s["sa"].shape, generator=gen, device="cuda").mul_(0.5).exp_().mul_(0.01))
        s["sb"].copy_(torch.randn(s["sb"].shape, generator=gen, device="cuda").mul_(0.3).exp_().mul_(2e-4))
        s["out"] = _plane(ranks, rows, n, TYPES[case["out"]])
    else:
        cols, dtype = case["cols"], TYPES[case["dtype"]]
        wide = cols * GATE[case["act"]] if case["op"] == "gate" else cols
        s["x"] = _plane(ranks, rows, wide, dtype)
        # hidden states: rows of differing size, and one column in a hundred that is far larger than the others
        size = torch.randn((rows, 1), generator=gen, device="cuda").mul_(0.5).exp_()
        far = torch.where(torch.rand((wide,), generator=gen, device="cuda") < 0.01, 20.0, 1.0)
        for rank in s["x"]:
            rank.copy_(torch.randn(rank.shape, generator=gen, device="cuda").mul_(size).mul_(far if case["op"] == "norm" else 1.0))
        to = TYPES[case["out"]] if case["op"] == "norm" else E4M3
        s["out"] = _plane(ranks, rows, cols, to)
        if to == E4M3:
            s["scales"] = _plane(ranks, _blocks(cols), rows, torch.float32)
        if case["op"] == "norm":
            s["weight"] = torch.randn((cols,), generator=gen, device="cuda").mul_(0.2).add_(1).to(dtype)
            if case["residual"]:
                s["res"] = torch.randn((rows, cols), generator=gen, device="cuda").mul_(size * 3).to(dtype)
                s["res_out"] = _plane(ranks, rows, cols, dtype)
    if own:  # the call, with its arguments marshalled once, as a decode loop over fixed buffers keeps it
        s["call"] = _call(s)
    return s


def _call(s):
    import all_reduce_amd as ar

    global _comm
    if _comm is None:
        _comm = ar.Comm(device="cuda", max_ranks=32, max_ll_bytes_per_rank=1 << 16)
    case = s["case"]
    at = {k: list(v.unbind(0)) for k, v in s.items() if k not in ("case", "weight", "res")}
    if case["op"] == "norm":
        return _comm.prepare_all_reduce_norm(at["x"], s["weight"], EPS, residual=s.get("res"), residual_out=at.get("res_out"), out=at["out"], scales=at.get("scales"))
    if case["op"] == "gate":
        return _comm.prepare_gate_quant(at["x"], at["out"], at["scales"], act=case["act"])
    return _comm.prepare_matmul_scaled(at["a"], at["sa"], at["b"], at["sb"], at["out"], reduce=case["reduce"])


_comm = None


def _results(s):
    return {k: s[k] for k in ("out", "scales", "res_out") if k in s}


def _in_blocks(y):
    """[..., rows, cols] as [..., rows, blocks, 128], filled up with zeros."""
    cols = y.shape[-1]
    return torch.nn.functional.pad(y, (0, _blocks(cols) * 128 - cols)).unflatten(-1, (-1, 128))


def _to_eight(y, out, scales):
    b = _in_blocks(y)
    scale = (b.abs().amax(-1) / 448).clamp_min(TINY)
    scales.copy_(scale.transpose(-1, -2))
    out.copy_((b / scale.unsqueeze(-1)).flatten(-2)[..., : y.shape[-1]].to(E4M3))


def run(s):
    if own:
        s["call"]()
        return _results(s)
    case = s["case"]
    if case["op"] == "norm":
        h = s["x"].float().sum(0)
        if case["residual"]:
            h = h + s["res"].float()
            s["res_out"].copy_(h.expand_as(s["res_out"]))
        y = h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * s["weight"].float()
        if case["out"] == "e4m3":
            _to_eight(y, s["out"], s["scales"])
        else:
            s["out"].copy_(y.expand_as(s["out"]))
    elif case["op"] == "gate":
        x = s["x"].float()
        if case["act"] == "silu":
            g, u = x.chunk(2, -1)
            x = g / (1 + (-g).exp()) * u
        _to_eight(x, s["out"], s["scales"])
    else:
        k, n = case["k"], case["n"]
        a = s["a"].float() * s["sa"].transpose(1, 2).repeat_interleave(128, 2)[:, :, :k]
        b = s["b"].float() * s["sb"].repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
        c = torch.bmm(a, b.transpose(1, 2))
        s["out"].copy_(c.sum(0).expand_as(c) if case["reduce"] else c)
    return _results(s)


def work(case):
    ranks, rows = case["ranks"], case["rows"]
    if case["op"] == "matmul":
        n, k = case["n"], case["k"]
        read = rows * k + n * k + 4 * _blocks(k) * (rows + _blocks(n))
        return {"bytes": ranks * (read + rows * n * BYTES[case["out"]]), "flops": 2 * ranks * rows * n * k}
    cols, es = case["cols"], BYTES[case["dtype"]]
    if case["op"] == "gate":
        wide = GATE[case["act"]] * es
        return {"bytes": ranks * rows * (cols * (wide + 1) + 4 * _blocks(cols)), "flops": ranks * rows * cols * 8}
    each = cols * BYTES[case["out"]] + (4 * _blocks(cols) if case["out"] == "e4m3" else 0)
    moved = ranks * rows * (cols * es + each) + cols * es
    if case["residual"]:
        moved += (ranks + 1) * rows * cols * es
    return {"bytes": moved, "flops": rows * cols * (ranks + 6)}


def exact(case, seed):
    """The definition in 64 bits; 8-bit values as they are before their rounding."""
    s = prepare(dict(case), seed)
    ranks, rows = case["ranks"], case["rows"]
    if case["op"] == "matmul":
        n, k = case["n"], case["k"]
        col, row = torch.arange(k, device="cuda") // 128, torch.arange(n, device="cuda") // 128
        c = []
        for r in range(ranks):  # one rank at a time: 64 bits of all of them are many bytes
            a = s["a"][r].double() * s["sa"][r].double().index_select(0, col).t()
            b = s["b"][r].double() * s["sb"][r].double().index_select(0, row).index_select(1, col)
            c.append(torch.mm(a, b.t().contiguous()))
        if case["reduce"]:
            total = c[0]
            for more in c[1:]:
                total = total + more
            c = [total] * ranks
        return {"out": torch.stack(c)}
    cols = case["cols"]
    start = torch.arange(0, cols, 128, device="cuda")
    outs, scales, res = [], [], []

    def eight(y):
        pad = y.new_zeros((rows, start.numel() * 128))
        pad[:, :cols] = y.abs()
        scale = torch.clamp(pad.view(rows, -1, 128).max(-1).values / 448.0, min=TINY)
        scales.append(scale.t().contiguous())
        return y / scale.index_select(1, torch.arange(cols, device="cuda") // 128)

    if case["op"] == "gate":
        for r in range(ranks):
            x = s["x"][r].double()
            outs.append(eight(x[:, :cols] * torch.sigmoid(x[:, :cols]) * x[:, cols:] if case["act"] == "silu" else x))
    else:
        h = s["res"].double() if case["residual"] else torch.zeros((rows, cols), dtype=torch.float64, device="cuda")
        for r in range(ranks):
            h = h + s["x"][r].double()
        y = h * torch.rsqrt((h * h).sum(-1, keepdim=True) / cols + EPS) * s["weight"].double()
        y = eight(y) if case["out"] == "e4m3" else y
        outs, scales, res = [y] * ranks, scales * ranks, [h] * ranks
    got = {"out": torch.stack(outs)}
    if scales:
        got["scales"] = torch.stack(scales)
    if case["op"] == "norm" and case["residual"]:
        got["res_out"] = torch.stack(res)
    return got
