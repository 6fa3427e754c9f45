"""The product's sizes on the host: what no launch holds is refused before
anything else is looked at, and the sizes that the GPU tests list take the
kernels that they are listed for.  No GPU is needed."""
import ctypes
import json
import random
import re
import subprocess
import sys

import pytest

import all_reduce_amd as ar
from block_shapes import CUS, KERNELS
from test_block_host import CHILD, MM, ROOT

# (label, changes to a valid call, code, log): 16 bytes of k, so that weights
# and outputs have room between the made-up addresses
CASES = [
    ("1 row of 2^30", dict(rows=1, n=1 << 30), "arInvalidArgument", "NULL comm"),
    ("256 rows of 2^30", dict(rows=256, n=1 << 30), "arInvalidArgument", "NULL comm"),
    ("2^30 rows of 1", dict(rows=1 << 30, n=1), "arInvalidArgument", "NULL comm"),
    ("2^19 rows of 2^19", dict(rows=1 << 19, n=1 << 19), "arInvalidArgument", "NULL comm"),
    ("257 rows of 2^29.99, summed", dict(rows=257, n=(1 << 38) // 257, reduce=1), "arUnsupported", "launch"),
    ("2^19 rows of 2^19 floats", dict(rows=1 << 19, n=1 << 19, out_dtype=2), "arUnsupported", "launch"),
    ("128 rows of 2^30 floats", dict(rows=128, n=1 << 30, out_dtype=2), "arInvalidArgument", "NULL comm"),
    ("15000000 tiles of floats", dict(rows=128 * 3000, n=128 * 5000, out_dtype=2), "arInvalidArgument", "NULL comm"),
]


@pytest.fixture(scope="module")
def results():
    tb = 1 << 42
    at = lambda i: (1 << 44) + i * tb  # noqa: E731
    base = dict(MM, abufs=[at(0), at(1)], ascales=[at(2), at(3)], bbufs=[at(4), at(5)], bscales=[at(6), at(7)],
                outbufs=[at(8), at(9)], k=16)
    calls = [(label, "arMatmulScaled", dict(base, **kw)) for label, kw, _, _ in CASES]
    res = subprocess.run([sys.executable, "-c", CHILD, str(ROOT), json.dumps(calls)], capture_output=True,
                         text=True, env={"AR_DEBUG": "1", "PATH": "/usr/bin:/bin"}, timeout=120)
    assert res.returncode == 0, res.stderr
    codes = dict(json.loads(line) for line in res.stdout.splitlines())
    logs = dict(part.split("\n", 1) for part in res.stderr.split("@@")[1:])
    return codes, logs


@pytest.mark.parametrize("label,kw,code,why", CASES, ids=[c[0] for c in CASES])
def test_tiles_of_a_launch(results, label, kw, code, why):
    codes, logs = results
    assert codes[label] == ar.arResult[code] and why in logs[label], (codes[label], logs[label])


def choice(ranks, rows, n, k, dtype, reduce, cus):
    out = (ctypes.c_int * 4)()
    assert ar.library().ar_block_matmul_choice(
        ctypes.c_size_t(rows), ctypes.c_size_t(n), ctypes.c_size_t(k), int(dtype), reduce, ranks, cus, out) == 1
    return tuple(out)


def form(shared, reduce):
    return "shared" if shared > 1 else "sum" if reduce else "each"


@pytest.mark.parametrize("kernel,form_,bits,shapes", KERNELS, ids=str)
def test_listed_sizes_take_their_kernels(kernel, form_, bits, shapes):
    for dtype in ((0, 1) if bits == 16 else (2,)):
        for ranks, rows, n, k in shapes:
            *got, shared = choice(ranks, rows, n, k, dtype, int(form_ != "each"), CUS)
            assert (tuple(got), form(shared, form_ != "each")) == (kernel, form_), (ranks, rows, n, k)


def test_every_kernel_is_listed():
    """Whatever a call may take, over sizes of all kinds, is in the list, with
    whole and with ragged k."""
    listed = {(kernel, form_, bits): shapes for kernel, form_, bits, shapes in KERNELS}
    for shapes in listed.values():
        assert any(k % 128 for *_, k in shapes)
    rng, taken = random.Random(1), set()
    for _ in range(60000):
        ranks = rng.choice([1, 2, 3, 4, 6, 8, 16, 32])
        rows, n, k = (int(2 ** rng.uniform(0, 13)) for _ in range(3))
        dtype, reduce = rng.choice([0, 2]), rng.randrange(2)
        *got, shared = choice(ranks, rows, n, 16 * -(-k // 16), dtype, reduce, CUS)
        taken.add((tuple(got), form(shared, reduce), 32 if dtype == 2 else 16))
    assert taken == set(listed), taken ^ set(listed)


def test_no_choice_where_no_launch_holds_the_tiles():
    out = (ctypes.c_int * 4)()
    args = [ctypes.c_size_t(v) for v in (1, 1 << 30, 16)]
    assert ar.library().ar_block_matmul_choice(*args, 0, 0, 2, CUS, out) == 0
    assert ar.library().ar_block_matmul_choice(*args, 0, 0, 1, CUS, out) == 1


def test_inline_assembly_names_the_registers_it_writes():
    """An asm statement that sets m0 says so: the compiler may keep a value there."""
    statements = [s for f in sorted((ROOT / "all_reduce_amd" / "csrc").glob("*.h*"))
                  for s in re.findall(r"\basm\b[^;]*;", f.read_text())]
    setting = [s for s in statements if re.search(r"s_mov_b32 m0,", s)]
    assert setting
    for s in setting:
        assert '"m0"' in s.rsplit(":", 1)[1], s
