"""The entry points of ar_block.h on the host: symbols, constants and argument
validation.  No GPU is needed: every argument check runs before any HIP call.
"""
import json
import re
import subprocess
import sys

import pytest

import all_reduce_amd as ar

HEADER = ar.BLOCK_HEADER.read_text()
ROOT = ar.HEADER.parent.parent
A = 0x7F0000000000  # 16-byte aligned fake device addresses; never dereferenced
GAP = 1 << 24


def test_library_exports_every_declared_function():
    body = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    names = sorted(set(re.findall(r"^arResult_t (ar[A-Z]\w*)\(", body, re.M)))
    assert names == ["arAllReduceNorm", "arGateQuant", "arMatmulScaled"]
    exported = subprocess.run(["nm", "-D", "--defined-only", str(ar.LIBRARY)],
                              capture_output=True, text=True, check=True).stdout
    for n in names:
        assert re.search(rf"\bT {n}$", exported, re.M), n


def test_constants_match_header():
    for member in ar.arActivation:
        assert int(re.search(rf"\b{member.name} = (\d+)", HEADER).group(1)) == member.value
    for name in ("AR_SCALE_BLOCK", "AR_NORM_MAX_COLS"):
        assert int(re.search(rf"#define {name} (\d+)", HEADER).group(1)) == getattr(ar, name)


def test_header_is_c99(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "ar_block.h"\narResult_t (*const call)(const void *const *, void *const *, float *const *, size_t, size_t,\n'
                   '    arDataType_t, arActivation_t, int, arComm_t, arStream_t) = arGateQuant;\n')
    res = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-c", str(src),
                          f"-I{ROOT / 'include'}", "-o", str(tmp_path / "t.o")],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def at(i):
    return A + i * GAP


NORM = dict(sendbufs=[at(0), at(1)], residual=at(2), weight=at(3), eps=1e-5,
            residual_out=[at(4), at(5)], outbufs=[at(6), at(7)], scalebufs=[at(8), at(9)],
            rows=4, cols=256, dtype=0, nranks=2)
NORM16 = dict(NORM, scalebufs=None)
GATE = dict(inbufs=[at(0), at(1)], outbufs=[at(2), at(3)], scalebufs=[at(4), at(5)], rows=4,
            cols=256, dtype=0, act=1, nranks=2)
MM = dict(abufs=[at(0), at(1)], ascales=[at(2), at(3)], bbufs=[at(4), at(5)],
          bscales=[at(6), at(7)], outbufs=[at(8), at(9)], rows=4, n=256, k=256, out_dtype=0,
          reduce=0, nranks=2)
BYTES = 4 * 256 * 2

# (label, entry point, arguments, expected code, expected log text)
CASES = [
    ("norm valid", "arAllReduceNorm", NORM, "arInvalidArgument", "NULL comm"),
    ("norm valid 16 bit", "arAllReduceNorm", NORM16, "arInvalidArgument", "NULL comm"),
    ("norm no residual", "arAllReduceNorm", dict(NORM, residual=None, residual_out=None),
     "arInvalidArgument", "NULL comm"),
    ("norm h in place of send", "arAllReduceNorm", dict(NORM, residual_out=[at(0), at(1)]),
     "arInvalidArgument", "NULL comm"),
    ("norm h in place of residual", "arAllReduceNorm", dict(NORM, residual_out=[at(2), at(5)]),
     "arInvalidArgument", "NULL comm"),
    ("norm out in place of send", "arAllReduceNorm", dict(NORM16, outbufs=[at(0), at(1)]),
     "arInvalidArgument", "NULL comm"),
    ("norm sends may be shared", "arAllReduceNorm", dict(NORM, sendbufs=[at(0), at(0)]),
     "arInvalidArgument", "NULL comm"),
    ("norm rows 0", "arAllReduceNorm", dict(NORM, rows=0, sendbufs=None), "arSuccess", None),
    ("norm bad dtype", "arAllReduceNorm", dict(NORM, dtype=3), "arUnsupported", "dtype"),
    ("norm 0 ranks", "arAllReduceNorm", dict(NORM, nranks=0), "arUnsupported", "nranks"),
    ("norm 33 ranks", "arAllReduceNorm", dict(NORM, nranks=33), "arUnsupported", "nranks"),
    ("norm cols 0", "arAllReduceNorm", dict(NORM, cols=0), "arUnsupported", "cols"),
    ("norm cols 32769", "arAllReduceNorm", dict(NORM, cols=32769), "arUnsupported", "cols"),
    ("norm eps negative", "arAllReduceNorm", dict(NORM, eps=-1.0), "arInvalidArgument", "eps"),
    ("norm eps nan", "arAllReduceNorm", dict(NORM, eps=float("nan")), "arInvalidArgument", "eps"),
    ("norm rows huge", "arAllReduceNorm", dict(NORM, rows=1 << 60), "arInvalidArgument", "rows"),
    ("norm NULL sends", "arAllReduceNorm", dict(NORM, sendbufs=None), "arInvalidArgument", "NULL"),
    ("norm NULL outs", "arAllReduceNorm", dict(NORM, outbufs=None), "arInvalidArgument", "NULL"),
    ("norm NULL weight", "arAllReduceNorm", dict(NORM, weight=None), "arInvalidArgument", "NULL"),
    ("norm NULL send", "arAllReduceNorm", dict(NORM, sendbufs=[at(0), 0]), "arInvalidArgument", "NULL"),
    ("norm NULL scale", "arAllReduceNorm", dict(NORM, scalebufs=[at(8), 0]), "arInvalidArgument", "NULL"),
    ("norm misaligned", "arAllReduceNorm", dict(NORM, residual=at(2) + 8), "arInvalidArgument", "aligned"),
    ("norm out overlaps 8 bit", "arAllReduceNorm", dict(NORM, outbufs=[at(0), at(7)]),
     "arInvalidArgument", "overlaps"),
    ("norm h partly over send", "arAllReduceNorm", dict(NORM, residual_out=[at(0) + 16, at(5)]),
     "arInvalidArgument", "overlaps"),
    ("norm h over another rank's send", "arAllReduceNorm", dict(NORM, residual_out=[at(1), at(5)]),
     "arInvalidArgument", "overlaps"),
    ("norm h over a shared send", "arAllReduceNorm",
     dict(NORM, sendbufs=[at(0), at(0)], residual_out=[at(0), at(5)]), "arInvalidArgument", "overlaps"),
    ("norm h twice the residual", "arAllReduceNorm", dict(NORM, residual_out=[at(2), at(2)]),
     "arInvalidArgument", "overlaps"),
    ("norm out over h", "arAllReduceNorm", dict(NORM16, outbufs=[at(4), at(7)]),
     "arInvalidArgument", "overlaps"),
    ("norm scales over the weight", "arAllReduceNorm", dict(NORM, scalebufs=[at(3), at(9)]),
     "arInvalidArgument", "overlaps"),
    ("norm outs overlap by a byte", "arAllReduceNorm",
     dict(NORM16, outbufs=[at(6), at(6) + BYTES - 16]), "arInvalidArgument", "overlaps"),
    ("norm outs next to each other", "arAllReduceNorm",
     dict(NORM16, outbufs=[at(6), at(6) + BYTES]), "arInvalidArgument", "NULL comm"),
    ("gate valid", "arGateQuant", GATE, "arInvalidArgument", "NULL comm"),
    ("gate rows 0", "arGateQuant", dict(GATE, rows=0), "arSuccess", None),
    ("gate cols 0", "arGateQuant", dict(GATE, cols=0), "arSuccess", None),
    ("gate bad dtype", "arGateQuant", dict(GATE, dtype=-1), "arUnsupported", "dtype"),
    ("gate bad act", "arGateQuant", dict(GATE, act=2), "arUnsupported", "activation"),
    ("gate 33 ranks", "arGateQuant", dict(GATE, nranks=33), "arUnsupported", "nranks"),
    ("gate huge", "arGateQuant", dict(GATE, rows=1 << 40, cols=1 << 40), "arInvalidArgument", "large"),
    ("gate NULL scales", "arGateQuant", dict(GATE, scalebufs=None), "arInvalidArgument", "NULL"),
    ("gate out over in", "arGateQuant", dict(GATE, outbufs=[at(0), at(3)]), "arInvalidArgument", "overlaps"),
    ("gate in is as wide as gate and up", "arGateQuant",
     dict(GATE, outbufs=[at(0) + 2 * BYTES - 16, at(3)]), "arInvalidArgument", "overlaps"),
    ("matmul valid", "arMatmulScaled", MM, "arInvalidArgument", "NULL comm"),
    ("matmul weights shared", "arMatmulScaled", dict(MM, bbufs=[at(4), at(4)]), "arInvalidArgument",
     "NULL comm"),
    ("matmul rows 0", "arMatmulScaled", dict(MM, rows=0), "arSuccess", None),
    ("matmul n 0", "arMatmulScaled", dict(MM, n=0), "arSuccess", None),
    ("matmul k 0", "arMatmulScaled", dict(MM, k=0), "arUnsupported", "multiple of 16"),
    ("matmul k 24", "arMatmulScaled", dict(MM, k=24), "arUnsupported", "multiple of 16"),
    ("matmul bad dtype", "arMatmulScaled", dict(MM, out_dtype=7), "arUnsupported", "outDtype"),
    ("matmul bad reduce", "arMatmulScaled", dict(MM, reduce=2), "arInvalidArgument", "reduce"),
    ("matmul 0 ranks", "arMatmulScaled", dict(MM, nranks=0), "arUnsupported", "nranks"),
    ("matmul rows huge", "arMatmulScaled", dict(MM, rows=(1 << 30) + 1), "arInvalidArgument", "2^30"),
    ("matmul k huge", "arMatmulScaled", dict(MM, k=(1 << 23) + 16), "arUnsupported", "2^23"),
    ("matmul output huge", "arMatmulScaled", dict(MM, rows=1 << 20, n=1 << 19), "arInvalidArgument",
     "2^38"),
    ("matmul NULL a", "arMatmulScaled", dict(MM, abufs=None), "arInvalidArgument", "NULL"),
    ("matmul NULL scale", "arMatmulScaled", dict(MM, bscales=[0, at(7)]), "arInvalidArgument", "NULL"),
    ("matmul misaligned", "arMatmulScaled", dict(MM, outbufs=[at(8) + 4, at(9)]), "arInvalidArgument",
     "aligned"),
    ("matmul out over a", "arMatmulScaled", dict(MM, outbufs=[at(0), at(9)]), "arInvalidArgument",
     "overlaps"),
    ("matmul outs the same", "arMatmulScaled", dict(MM, outbufs=[at(8), at(8)], reduce=1),
     "arInvalidArgument", "overlaps"),
    ("matmul short list", "arMatmulScaled", dict(MM, nranks=3), "arInvalidArgument", "NULL"),
]

CHILD = r"""
import json, sys
sys.path.insert(0, sys.argv[1])
import all_reduce_amd as ar
for label, name, kw in json.loads(sys.argv[2]):
    sys.stderr.write(f"@@{label}\n"); sys.stderr.flush()
    r = getattr(ar, name)(**kw, comm=None, stream=None)
    sys.stderr.flush()
    print(json.dumps([label, r]), flush=True)
"""


@pytest.fixture(scope="module")
def results():
    res = subprocess.run([sys.executable, "-c", CHILD, str(ROOT), json.dumps([c[:3] for c in CASES])],
                         capture_output=True, text=True,
                         env={"AR_DEBUG": "1", "PATH": "/usr/bin:/bin"}, timeout=120)
    assert res.returncode == 0, res.stderr
    codes = dict(json.loads(line) for line in res.stdout.splitlines())
    logs = {}
    for part in res.stderr.split("@@")[1:]:
        label, _, text = part.partition("\n")
        logs[label] = text
    return codes, logs


@pytest.mark.parametrize("label,name,kw,code,why", CASES, ids=[c[0] for c in CASES])
def test_validation(results, label, name, kw, code, why):
    codes, logs = results
    assert codes[label] == ar.arResult[code], (label, codes[label], logs[label])
    assert (why in logs[label]) if why else logs[label].strip() == "", logs[label]


def test_helpers():
    assert [ar.scale_blocks(c) for c in (1, 128, 129, 8192)] == [1, 1, 2, 64]
    assert ar.activation_code("SiLU") == ar.arActivation.arActSiLU
    assert ar.activation_code(0) == ar.arActivation.arActNone
