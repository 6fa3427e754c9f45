"""The cases by which the operators of the paged key-value cache are measured.

Three operators over the R ranks of a tensor-parallel group on one GPU, each
rank with its share of the heads; slots, page table and lengths are the same on
every rank:

* ``write``   puts the keys and values of new tokens into the pages, as they are
              or in 8 bits with a scale per token and head
              (``Comm.prepare_cache_write``);
* ``read``    gets them back as dense rows (``Comm.prepare_cache_read``);
* ``attend``  attention of one new token a sequence over its cached tokens, with
              an output in the element type or in 8 bits with a scale per row and
              128 columns (``Comm.prepare_cache_attention``).

A cache is [pages, heads, tokens of a page, dim] (order "head") or [pages,
tokens of a page, heads, dim] (order "token"); scales are [pages, heads, tokens
of a page].  Token t of sequence s lies in page table[s, t // P], place t % P;
slot p * P + o is place o of page p.  8-bit values are e4m3.
"""
import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": E4M3}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
TINY = 2.0 ** -126  # the smallest scale

# The largest listed cases: a drawn case costs no more.
MOST_COPY = 8 * 16384 * 2 * 128  # ranks * tokens * heads * dim
MOST_READ = 8 * 64 * 8192 * 128 * 4  # bytes that an attention reads


def listed():
    return [
        # the new tokens of a decode batch of 64, cut out of the QKV product's rows (8 query heads, a key and a value head a rank)
        dict(name="write decode 64", op="write", ranks=8, tokens=64, heads=1, group=8, dim=128, dtype="bf16", cache="e4m3", page=64, order="head"),
        # a prefill's tokens, two key-value heads a rank
        dict(name="write prefill 16384", op="write", ranks=8, tokens=16384, heads=2, group=4, dim=128, dtype="bf16", cache="e4m3", page=64, order="head"),
        # sizes that no table is made for, a cache in the element type; every eleventh row of the batch is padding
        dict(name="write odd", op="write", ranks=3, tokens=333, heads=5, group=1, dim=80, dtype="fp16", cache="fp16", page=20, order="token"),
        # a cached prefix as dense rows, for a prefill that continues it
        dict(name="read prefix 16384", op="read", ranks=8, tokens=16384, heads=2, group=4, dim=128, dtype="bf16", cache="e4m3", page=64, order="head"),
        # a float32 cache, a page a token
        dict(name="read odd", op="read", ranks=3, tokens=777, heads=2, group=1, dim=192, dtype="fp32", cache="fp32", page=1, order="token"),
        # one sequence of ordinary length: the smallest call of a decode loop
        dict(name="attend 1 x 1000", op="attend", ranks=8, seqs=1, longest=1000, ragged=False, heads=1, group=8, dim=128, dtype="bf16", cache="bf16", page=64, order="head", window=0, out="bf16", lse=False),
        # a large decode batch of long sequences
        dict(name="attend 64 x 8192", op="attend", ranks=8, seqs=64, longest=8192, ragged=False, heads=1, group=8, dim=128, dtype="bf16", cache="bf16", page=64, order="head", window=0, out="bf16", lse=False),
        # a batch in every state from its first tokens to 32768, cache and output in 8 bits
        dict(name="attend ragged e4m3", op="attend", ranks=8, seqs=64, longest=32768, ragged=True, heads=1, group=8, dim=128, dtype="bf16", cache="e4m3", page=64, order="head", window=0, out="e4m3", lse=False),
        # one long document: every compute unit on one sequence
        dict(name="attend 1 x 131072", op="attend", ranks=8, seqs=1, longest=131072, ragged=False, heads=1, group=8, dim=128, dtype="bf16", cache="e4m3", page=256, order="head", window=0, out="bf16", lse=False),
        # odd everywhere, empty sequences, heads of 80, pages of 20, with the logarithm of the sums
        dict(name="attend odd", op="attend", ranks=3, seqs=29, longest=999, ragged=True, heads=5, group=3, dim=80, dtype="fp16", cache="fp16", page=20, order="token", window=0, out="fp16", lse=True),
        # every head with keys of its own, in float32
        dict(name="attend fp32", op="attend", ranks=2, seqs=16, longest=4096, ragged=True, heads=16, group=1, dim=64, dtype="fp32", cache="fp32", page=16, order="token", window=0, out="fp32", lse=True),
        # many query heads on one key-value head of 256, the last 4096 tokens alone
        dict(name="attend window wide", op="attend", ranks=4, seqs=32, longest=16384, ragged=True, heads=1, group=32, dim=256, dtype="bf16", cache="bf16", page=128, order="head", window=4096, out="e4m3", lse=False),
    ]


def _log(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    case = dict(op=op, ranks=rng.choice([1, 1, 2, 3, 4, 8, 8, 16]), heads=rng.choice([1, 1, 2, 3, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16, 24]),
                dim=rng.choice([64, 128, 128, 128, 256, 16 * rng.randint(2, 16)]), dtype=dtype, cache=rng.choice([dtype, "e4m3"]),
                page=rng.choice([1, 16, 32, 64, 128, 256, rng.randint(1, 100)]), order=rng.choice(["head", "token"]))
    each = case["ranks"] * case["heads"] * case["dim"]
    if op != "attend":
        case["tokens"] = max(1, min(_log(rng, 1, 16384), MOST_COPY * 2 // (each * BYTES[dtype])))
        return case
    seqs, longest = _log(rng, 1, 256), _log(rng, 1, 65536)
    fits = MOST_READ // (2 * BYTES[case["cache"]] * each)  # tokens of all sequences
    fits = min(fits, MOST_READ // (8 * case["ranks"] * case["heads"] * case["group"] * 4))  # and the plain form's scores stay small
    longest = max(1, min(longest, fits))
    case.update(seqs=max(1, min(seqs, fits // longest)), longest=longest, ragged=rng.random() < 0.7, window=rng.choice([0, 0, 0, _log(rng, 16, 8192)]),
                out=rng.choice([dtype, "e4m3"]) if case["dim"] % 128 == 0 else dtype, lse=rng.random() < 0.3)
    return case


def _plane(ranks, shape, dtype):
    """One buffer a rank, each starting on a multiple of 256 bytes: [ranks, *shape]."""
    n = torch.Size(shape).numel()
    at = 256 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((ranks, -(-n // at) * at), dtype=dtype, device="cuda")[:, :n].unflatten(1, shape)


def _blocks(cols):
    return -(-cols // 128)


def _lengths(case, seed):
    """Cached tokens of each sequence, the new one among them."""
    if not case["ragged"]:
        return torch.full((case["seqs"],), case["longest"])
    gen = torch.Generator().manual_seed(seed)
    share = torch.rand((case["seqs"],), generator=gen)
    n = (case["longest"] * share * share).long()  # many short ones, few long ones; one in a batch of some is empty
    n[0] = case["longest"]
    if case["seqs"] > 8:
        n[3], n[5] = 0, 1
    return n


def _tokens_of(case, lengths):
    return lengths.clamp_max(case["window"]) if case["window"] else lengths


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    ranks, heads, dim, page, dtype = case["ranks"], case["heads"], case["dim"], case["page"], TYPES[case["dtype"]]
    host = torch.Generator().manual_seed(seed)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] == "attend":
        lengths = _lengths(case, seed)
        per = -(-int(lengths.max()) // page) + 2  # a table with room for the next pages
        used = -(-lengths // page)
        pages = int(used.sum()) + 3
    else:
        pages = -(-case["tokens"] * 5 // (4 * page)) + 1
    # the pool, as long serving leaves it: pages of a sequence lie anywhere
    places = (pages, heads, page, dim) if case["order"] == "head" else (pages, page, heads, dim)
    channel = normal(ranks, 1, 1, 1, dim).mul(0.5).exp()  # some channels of the keys are larger
    for name in ("key", "value"):
        s[name + "_pages"] = pool = _plane(ranks, places, TYPES[case["cache"]])
        if case["cache"] == "e4m3":
            s[name + "_scales"] = _plane(ranks, (pages, heads, page), torch.float32)
            s[name + "_scales"].copy_(normal(ranks, pages, heads, page).mul_(0.3).exp_().mul_(0.01))
        for r in range(ranks):
            x = normal(*places)
            if case["cache"] == "e4m3":
                x = x.mul_(110).clamp_(-448, 448)
            elif name == "key":
                x = x.mul_(channel[r])
            pool[r].copy_(x)
    if case["op"] == "attend":
        table = torch.full((case["seqs"], per), -1, dtype=torch.int32)
        order = torch.randperm(pages, generator=host).int()
        where = torch.arange(per).expand_as(table) < used[:, None]
        table[where] = order[: int(used.sum())]
        s["page_table"], s["lengths"] = table.cuda(), lengths.int().cuda()
        s["queries"] = _plane(ranks, (case["seqs"], heads * case["group"], dim), dtype)
        s["queries"].copy_(normal(*s["queries"].shape).mul_(2))
        s["out"] = _plane(ranks, (case["seqs"], heads * case["group"], dim), TYPES[case["out"]])
        if case["out"] == "e4m3":
            s["out_scales"] = _plane(ranks, (_blocks(heads * case["group"] * dim), case["seqs"]), torch.float32)
        if case["lse"]:
            s["lse"] = _plane(ranks, (case["seqs"], heads * case["group"]), torch.float32)
    else:
        tokens = case["tokens"]
        slots = torch.randperm(pages * page, generator=host)[:tokens]
        slots[10::11] = -1  # padding of the batch
        s["slots"], s["there"] = slots.cuda(), (slots >= 0).nonzero()[:, 0].cuda()
        if case["op"] == "write":  # rows of the QKV product: queries, keys, values
            wide = (case["group"] + 2) * heads * dim
            qkv = _plane(ranks, (tokens, wide), dtype)
            qkv.copy_(normal(ranks, tokens, wide).mul_(normal(tokens, 1).mul_(0.3).exp_()))
            s["keys"] = qkv[:, :, -2 * heads * dim: -heads * dim].unflatten(2, (heads, dim))
            s["values"] = qkv[:, :, -heads * dim:].unflatten(2, (heads, dim))
        else:
            s["keys"], s["values"] = (_plane(ranks, (tokens, heads, dim), dtype).zero_() for _ in range(2))
    if own:  # the call, with its arguments marshalled once, as a decode loop over fixed buffers keeps it
        s["call"] = _call(s)
    return s


def _call(s):
    import all_reduce_amd as ar

    global _comm
    if _comm is None:
        _comm = ar.Comm(device="cuda", max_ranks=32, max_ll_bytes_per_rank=1 << 16)
    case = s["case"]
    shared = ("case", "slots", "there", "page_table", "lengths")
    at = {k: list(v.unbind(0)) for k, v in s.items() if k not in shared}
    if case["order"] == "token":  # [pages, heads, tokens, dim] whatever the order in memory
        for name in ("key_pages", "value_pages"):
            at[name] = [t.transpose(1, 2) for t in at[name]]
    scales = dict(key_scales=at.get("key_scales"), value_scales=at.get("value_scales"))
    if case["op"] == "write":
        return _comm.prepare_cache_write(at["keys"], at["values"], s["slots"], at["key_pages"], at["value_pages"], **scales)
    if case["op"] == "read":
        return _comm.prepare_cache_read(s["slots"], at["key_pages"], at["value_pages"], at["keys"], at["values"], **scales)
    return _comm.prepare_cache_attention(at["queries"], at["key_pages"], at["value_pages"], s["page_table"], s["lengths"], at["out"], window=case["window"],
                                         out_scales=at.get("out_scales"), lse=at.get("lse"), **scales)


_comm = None


def _results(s):
    names = {"write": ("key_pages", "value_pages", "key_scales", "value_scales"), "read": ("keys", "values"), "attend": ("out", "out_scales", "lse")}
    return {k: s[k] for k in names[s["case"]["op"]] if k in s}


def _places(case, page, place, scales=False):
    """Of every head: the row of a rank's pool (or the place among its scales) that holds these tokens: [..., heads]."""
    head = torch.arange(case["heads"], device="cuda")
    page, place = page.unsqueeze(-1), place.unsqueeze(-1)
    if scales or case["order"] == "head":
        return (page * case["heads"] + head) * case["page"] + place
    return (page * case["page"] + place) * case["heads"] + head


def _bytes(x):
    """8-bit values as whole numbers, which every indexing operation takes."""
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def _put(s, name, x, page, place):
    """x [ranks, tokens, heads, dim] into the pool, rounded to its type."""
    case, pool = s["case"], s[name + "_pages"]
    x = x.float()
    if case["cache"] == "e4m3":
        scale = (x.abs().amax(-1, keepdim=True) / 448).clamp_min(TINY)
        at = _places(case, page, place, True).flatten()
        s[name + "_scales"].flatten(1).index_copy_(1, at, scale.flatten(1))
        x = x / scale
    at = _places(case, page, place).flatten()
    _bytes(pool).flatten(1, 3).index_copy_(1, at, _bytes(x.to(pool.dtype)).flatten(1, 2))


def _get(s, name, page, place):
    """The rows at these places in 32 bits: [ranks, *page.shape, heads, dim]."""
    case, pool = s["case"], s[name + "_pages"]
    at = _places(case, page, place)
    x = _bytes(pool).flatten(1, 3).index_select(1, at.flatten()).view(pool.dtype).float()
    if case["cache"] == "e4m3":
        x = x * s[name + "_scales"].flatten(1).index_select(1, _places(case, page, place, True).flatten()).unsqueeze(-1)
    return x.unflatten(1, at.shape)


def _attend(s):
    case = s["case"]
    group, dim, page = case["group"], case["dim"], case["page"]
    t = torch.arange(case["longest"], device="cuda")
    n = s["lengths"].long().unsqueeze(1)
    there = t < n
    if case["window"]:
        there = there & (t >= n - case["window"])
    pages = s["page_table"].long()[:, t // page].clamp_min(0)
    # [ranks, sequences, heads, tokens, ...]
    k = _get(s, "key", pages, (t % page).expand_as(pages)).transpose(2, 3).contiguous()
    q = s["queries"].float().unflatten(2, (case["heads"], group))
    x = torch.matmul(k, q.transpose(3, 4).contiguous()) * dim ** -0.5
    del k
    x = x.masked_fill(~there[None, :, None, :, None], -torch.inf)
    m = x.amax(3, keepdim=True)
    p = (x - m.masked_fill(m == -torch.inf, 0)).exp()
    total = p.sum(3)
    v = _get(s, "value", pages, (t % page).expand_as(pages)).transpose(2, 3).contiguous()
    y = torch.matmul(p.transpose(3, 4).contiguous(), v)
    y = (y / total.unsqueeze(-1)).masked_fill((total == 0).unsqueeze(-1), 0).flatten(2, 3)
    if case["lse"]:
        s["lse"].copy_((total.log() + m.squeeze(3)).flatten(2))
    if case["out"] == "e4m3":
        b = y.flatten(2).unflatten(2, (-1, 128))
        scale = (b.abs().amax(-1) / 448).clamp_min(TINY)
        s["out_scales"].copy_(scale.transpose(1, 2))
        y = (b / scale.unsqueeze(-1)).view_as(y)
    s["out"].copy_(y)


def run(s):
    if own:
        s["call"]()
        return _results(s)
    case = s["case"]
    if case["op"] == "attend":
        _attend(s)
        return _results(s)
    slots = s["slots"][s["there"]]
    page, place = slots // case["page"], slots % case["page"]
    if case["op"] == "write":
        _put(s, "key", s["keys"][:, s["there"]], page, place)
        _put(s, "value", s["values"][:, s["there"]], page, place)
    else:
        s["keys"].index_copy_(1, s["there"], _get(s, "key", page, place).to(s["keys"].dtype))
        s["values"].index_copy_(1, s["there"], _get(s, "value", page, place).to(s["values"].dtype))
    return _results(s)


def work(case):
    ranks, heads, dim = case["ranks"], case["heads"], case["dim"]
    scale = 8 if case["cache"] == "e4m3" else 0
    if case["op"] != "attend":
        there = case["tokens"] - case["tokens"] // 11
        return {"bytes": there * ranks * heads * (2 * dim * (BYTES[case["dtype"]] + BYTES[case["cache"]]) + scale) + 8 * case["tokens"], "flops": there * ranks * heads * dim * 4}
    share = 1 / 3 if case["ragged"] else 1  # (the lengths go by the seed: the mean of a square)
    tokens = case["longest"] * (1 + (case["seqs"] - 1) * share)
    if case["window"]:  # the mean of min(longest x^2, window)
        w = min(1.0, case["window"] / case["longest"])
        share = w ** 1.5 / 3 + w * (1 - w ** 0.5) if case["ragged"] else w
        tokens = case["longest"] * (w + (case["seqs"] - 1) * share)
    rows = ranks * case["seqs"] * heads * case["group"]
    moved = ranks * heads * tokens * (2 * dim * BYTES[case["cache"]] + scale) + rows * dim * (BYTES[case["dtype"]] + BYTES[case["out"]])
    moved += 4 * case["seqs"] + 4 * tokens / case["page"] + (4 * rows if case["lse"] else 0) + (rows * dim // 32 if case["out"] == "e4m3" else 0)
    return {"bytes": moved, "flops": 4 * ranks * heads * case["group"] * dim * tokens}


def exact(case, seed):
    """The definition in 64 bits; 8-bit values as they are before their rounding."""
    s = prepare(dict(case), seed)
    ranks, heads, dim, page = case["ranks"], case["heads"], case["dim"], case["page"]
    eight = case["cache"] == "e4m3"

    def ordered(pool):  # [pages, tokens of a page, heads, dim], a view
        return pool.transpose(1, 2) if case["order"] == "head" else pool

    if case["op"] != "attend":
        slots = s["slots"].cpu()
        token = [t for t, slot in enumerate(slots.tolist()) if slot >= 0]
        p, o = slots[token].div(page, rounding_mode="floor").cuda(), slots[token].remainder(page).cuda()
        token = torch.tensor(token, device="cuda", dtype=torch.long)
        got = {k: v.double().clone() for k, v in _results(s).items()}
        for name in ("key", "value"):
            for r in range(ranks):
                if case["op"] == "write":
                    x = s[name + "s"][r].double()[token]
                    if eight:
                        scale = torch.clamp(x.abs().max(-1).values / 448.0, min=TINY)
                        got[name + "_scales"][r].transpose(1, 2)[p, o] = scale
                        x = x / scale[..., None]
                    ordered(got[name + "_pages"][r])[p, o] = x
                else:
                    x = ordered(s[name + "_pages"][r].double())[p, o]
                    if eight:
                        x = x * s[name + "_scales"][r].double().transpose(1, 2)[p, o][..., None]
                    got[name + "s"][r][token] = x
        return got
    lengths, table = s["lengths"].tolist(), s["page_table"].long()
    y = torch.zeros((ranks, case["seqs"], heads, case["group"], dim), dtype=torch.float64, device="cuda")
    lse = torch.full(y.shape[:-1], -torch.inf, dtype=torch.float64, device="cuda")
    for r in range(ranks):
        for i, n in enumerate(lengths):
            if n == 0:
                continue
            t = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
            p, o = table[i].index_select(0, t // page), t % page
            kv = []
            for name in ("key", "value"):
                x = _bytes(ordered(s[name + "_pages"][r]))[p, o].view(TYPES[case["cache"]]).double()
                kv.append(x * s[name + "_scales"][r].transpose(1, 2)[p, o].double()[..., None] if eight else x)
            q = s["queries"][r, i].double().view(heads, case["group"], dim) / dim ** 0.5
            x = torch.bmm(q, kv[0].permute(1, 2, 0).contiguous())
            y[r, i] = torch.bmm(torch.softmax(x, -1), kv[1].transpose(0, 1).contiguous())
            lse[r, i] = torch.logsumexp(x, -1)
    got = {}
    cols = y.flatten(2)
    if case["out"] == "e4m3":
        block = torch.arange(cols.shape[2], device="cuda") // 128
        scale = torch.clamp(cols.abs().view(ranks, case["seqs"], -1, 128).max(-1).values / 448.0, min=TINY)
        got["out_scales"] = scale.transpose(1, 2).contiguous()
        cols = cols / scale.index_select(2, block)
    got["out"] = cols.view(ranks, case["seqs"], -1, dim)
    if case["lse"]:
        got["lse"] = lse.flatten(2)
    return got
