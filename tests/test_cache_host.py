"""The entry points of ar_cache.h on the host: symbols, constants and argument
validation.  No GPU is needed: every argument check runs before any HIP call.
"""
import json
import re
import subprocess
import sys

import pytest

import all_reduce_amd as ar

HEADER = ar.CACHE_HEADER.read_text()
ROOT = ar.HEADER.parent.parent
A = 0x7F0000000000  # 16-byte aligned fake device addresses; never dereferenced
GAP = 1 << 24


def test_library_exports_every_declared_function():
    body = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    names = sorted(set(re.findall(r"^arResult_t (ar[A-Z]\w*)\(", body, re.M)))
    assert names == ["arCacheAttention", "arCacheAttentionWorkspace", "arCacheRead", "arCacheWrite"]
    exported = subprocess.run(["nm", "-D", "--defined-only", str(ar.LIBRARY)],
                              capture_output=True, text=True, check=True).stdout
    for n in names:
        assert re.search(rf"\bT {n}$", exported, re.M), n


def test_constants_and_layout_match_the_header():
    assert int(re.search(r"#define AR_CACHE_MAX_DIM (\d+)", HEADER).group(1)) == ar.AR_CACHE_MAX_DIM
    body = re.search(r"typedef struct \{(.*?)\} arCacheLayout_t;", HEADER, re.S).group(1)
    assert re.findall(r"size_t (\w+);", body) == [n for n, _ in ar.arCacheLayout._fields_]


def test_header_is_c99(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "ar_cache.h"\narCacheLayout_t layout = {4, 16, 2, 128, 4096, 2048, 128};\n'
                   'arResult_t (*const call)(size_t, size_t, arComm_t, size_t *) = arCacheAttentionWorkspace;\n')
    res = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-c", str(src),
                          f"-I{ROOT / 'include'}", "-o", str(tmp_path / "t.o")],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def at(i):
    return A + i * GAP


LAYOUT = dict(pages=8, pageTokens=16, heads=2, dim=128, pageStride=4096, headStride=2048, tokenStride=128)
POOL = 8 * 4096 * 2
WRITE = dict(keys=[at(0), at(1)], values=[at(2), at(3)], row_stride=256, slots=at(4), tokens=5, cache=LAYOUT,
             key_pages=[at(5), at(6)], value_pages=[at(7), at(8)], key_scales=None, value_scales=None, dtype=0,
             nranks=2)
SCALES = dict(key_scales=[at(9), at(10)], value_scales=[at(11), at(12)])
READ = dict(WRITE)
ATTEND = dict(queries=[at(0), at(1)], query_stride=1024, cache=LAYOUT, key_pages=[at(5), at(6)],
              value_pages=[at(7), at(8)], key_scales=None, value_scales=None, page_table=at(2), table_pages=4,
              lengths=at(3), seqs=3, heads=8, scale=0.1, window=0, outbufs=[at(13), at(14)], out_scales=None,
              lse=None, workspace=at(20), workspace_bytes=1 << 20, dtype=0, nranks=2)


def layout(**kw):
    return dict(LAYOUT, **kw)


OK = ("arInvalidArgument", "NULL comm")  # every other check has passed
W, R, T = "arCacheWrite", "arCacheRead", "arCacheAttention"

# (label, entry point, arguments, expected code, expected log text)
CASES = [
    ("write valid", W, WRITE, *OK),
    ("write 8 bit", W, dict(WRITE, **SCALES), *OK),
    ("write sources shared", W, dict(WRITE, values=[at(0), at(1)]), *OK),
    ("write parts of a row", W, dict(WRITE, row_stride=1024, values=[at(0) + 512, at(1) + 512]), *OK),
    ("write other order", W, dict(WRITE, cache=layout(headStride=128, tokenStride=256)), *OK),
    ("write heads outermost", W, dict(WRITE, cache=layout(headStride=8 * 2048, pageStride=2048)), *OK),
    ("write gaps", W, dict(WRITE, cache=layout(pageStride=5000, headStride=2400, tokenStride=144)), *OK),
    ("write pairs in a page", W, dict(WRITE, cache=layout(pageStride=8192), key_pages=[at(5), at(6)],
                                      value_pages=[at(5) + 8192, at(6) + 8192]), *OK),
    ("write pairs, values first", W, dict(WRITE, cache=layout(pageStride=8192), key_pages=[at(5) + 8192, at(6) + 8192],
                                          value_pages=[at(5), at(6)]), *OK),
    ("write pairs that overlap", W, dict(WRITE, cache=layout(pageStride=8192), value_pages=[at(5) + 8176, at(8)]),
     "arInvalidArgument", "overlaps"),
    ("write pairs past the page", W, dict(WRITE, cache=layout(pageStride=8176), value_pages=[at(5) + 8192, at(8)]),
     "arInvalidArgument", "overlaps"),
    ("write pairs of tokens", W, dict(WRITE, cache=layout(pageStride=8192, tokenStride=512, headStride=128),
                                      value_pages=[at(5) + 512, at(6) + 512]), *OK),
    ("write pairs of heads", W, dict(WRITE, cache=layout(pageStride=8192, headStride=4096), value_pages=[at(5) + 4096, at(6) + 4096]),
     *OK),
    ("write pairs of places", W, dict(WRITE, cache=layout(pageStride=8192, headStride=4096, tokenStride=256),
                                      value_pages=[at(5) + 256, at(6) + 256]), *OK),
    ("write pairs of one page's tokens", W, dict(WRITE, cache=layout(pages=1, tokenStride=512, headStride=128),
                                                 value_pages=[at(5) + 512, at(6) + 512]), *OK),
    ("write pairs of tokens that overlap", W, dict(WRITE, cache=layout(pageStride=8192, tokenStride=512, headStride=128),
                                                   value_pages=[at(5) + 496, at(6) + 496]), "arInvalidArgument", "overlaps"),
    ("write pairs of tokens past the token", W, dict(WRITE, cache=layout(pageStride=8192, tokenStride=512, headStride=128),
                                                     value_pages=[at(5) + 528, at(6) + 528]), "arInvalidArgument", "overlaps"),
    ("write pairs of tokens past the page", W, dict(WRITE, cache=layout(pageStride=8184, tokenStride=512, headStride=128),
                                                    value_pages=[at(5) + 512, at(6) + 512]), "arInvalidArgument", "overlaps"),
    ("write pairs of heads past the page", W, dict(WRITE, cache=layout(pageStride=6144, headStride=4096),
                                                   value_pages=[at(5) + 4096, at(6) + 4096]), "arInvalidArgument", "overlaps"),
    ("write pairs a token apart", W, dict(WRITE, cache=layout(pageStride=8192, tokenStride=512, headStride=128),
                                          value_pages=[at(5) + 1024, at(6) + 1024]), "arInvalidArgument", "overlaps"),
    ("write pair over another rank's", W, dict(WRITE, cache=layout(pageStride=8192), key_pages=[at(5), at(5) + 8192],
                                               value_pages=[at(7), at(8)]), "arInvalidArgument", "overlaps"),
    ("write no tokens", W, dict(WRITE, tokens=0, keys=None, slots=None), "arSuccess", None),
    ("write bad dtype", W, dict(WRITE, dtype=3), "arUnsupported", "dtype"),
    ("write 0 ranks", W, dict(WRITE, nranks=0), "arUnsupported", "nranks"),
    ("write 33 ranks", W, dict(WRITE, nranks=33), "arUnsupported", "nranks"),
    ("write one scale table", W, dict(WRITE, key_scales=[at(9), at(10)]), "arInvalidArgument", "scales"),
    ("write no layout", W, dict(WRITE, cache=None), "arInvalidArgument", "layout"),
    ("write dim 8", W, dict(WRITE, cache=layout(dim=8)), "arUnsupported", "dim"),
    ("write dim 100", W, dict(WRITE, cache=layout(dim=100)), "arUnsupported", "dim"),
    ("write dim 272", W, dict(WRITE, cache=layout(dim=272)), "arUnsupported", "dim"),
    ("write 0 heads", W, dict(WRITE, cache=layout(heads=0)), "arUnsupported", "heads"),
    ("write 4097 heads", W, dict(WRITE, cache=layout(heads=4097)), "arUnsupported", "heads"),
    ("write 0 pages", W, dict(WRITE, cache=layout(pages=0)), "arInvalidArgument", "pages"),
    ("write pages of 0", W, dict(WRITE, cache=layout(pageTokens=0)), "arInvalidArgument", "pages"),
    ("write 2^31 slots", W, dict(WRITE, cache=layout(pages=1 << 27)), "arInvalidArgument", "pages"),
    ("write slots that wrap", W, dict(WRITE, cache=layout(pages=1 << 60, pageTokens=16)), "arInvalidArgument", "pages"),
    ("write odd stride", W, dict(WRITE, cache=layout(tokenStride=132)), "arInvalidArgument", "multiples"),
    ("write odd stride 8 bit", W, dict(WRITE, **SCALES, cache=layout(tokenStride=136, headStride=4096, pageStride=16384)),
     "arInvalidArgument", "multiples"),
    ("write rows overlap", W, dict(WRITE, cache=layout(tokenStride=112)), "arInvalidArgument", "rows of the cache"),
    ("write heads overlap", W, dict(WRITE, cache=layout(headStride=2040)), "arInvalidArgument", "rows of the cache"),
    ("write pages overlap", W, dict(WRITE, cache=layout(pageStride=4088)), "arInvalidArgument", "rows of the cache"),
    ("write cache huge", W, dict(WRITE, cache=layout(pageStride=1 << 61)), "arInvalidArgument", "too large"),
    ("write one page, any stride", W, dict(WRITE, cache=layout(pages=1, pageStride=3)), *OK),
    ("write one place, any stride", W, dict(WRITE, cache=layout(pageTokens=1, tokenStride=3)), *OK),
    ("write rows closer than a row", W, dict(WRITE, row_stride=248), "arInvalidArgument", "row stride"),
    ("write odd row stride", W, dict(WRITE, row_stride=260), "arInvalidArgument", "row stride"),
    ("write rows huge", W, dict(WRITE, row_stride=1 << 62), "arInvalidArgument", "rows"),
    ("write tokens huge", W, dict(WRITE, tokens=1 << 31), "arInvalidArgument", "tokens"),
    ("write NULL keys", W, dict(WRITE, keys=None), "arInvalidArgument", "NULL"),
    ("write NULL pages", W, dict(WRITE, value_pages=None), "arInvalidArgument", "NULL"),
    ("write NULL key", W, dict(WRITE, keys=[at(0), 0]), "arInvalidArgument", "NULL"),
    ("write NULL page", W, dict(WRITE, key_pages=[0, at(6)]), "arInvalidArgument", "NULL"),
    ("write NULL slots", W, dict(WRITE, slots=None), "arInvalidArgument", "NULL"),
    ("write NULL scale", W, dict(WRITE, **dict(SCALES, key_scales=[at(9), 0])), "arInvalidArgument", "NULL"),
    ("write slots off", W, dict(WRITE, slots=at(4) + 4), "arInvalidArgument", "aligned"),
    ("write slots at 8", W, dict(WRITE, slots=at(4) + 8), *OK),
    ("write keys off", W, dict(WRITE, keys=[at(0) + 8, at(1)]), "arInvalidArgument", "aligned"),
    ("write pages over keys", W, dict(WRITE, key_pages=[at(0), at(6)]), "arInvalidArgument", "overlaps"),
    ("write pages over slots", W, dict(WRITE, key_pages=[at(4), at(6)]), "arInvalidArgument", "overlaps"),
    ("write values over keys", W, dict(WRITE, value_pages=[at(5), at(8)]), "arInvalidArgument", "overlaps"),
    ("write scales over pages", W, dict(WRITE, **dict(SCALES, key_scales=[at(5), at(10)])), "arInvalidArgument",
     "overlaps"),
    ("write pools next to each other", W, dict(WRITE, value_pages=[at(5) + POOL, at(8)]), *OK),
    ("write pools that overlap by a piece", W, dict(WRITE, value_pages=[at(5) + POOL - 16, at(8)]),
     "arInvalidArgument", "overlaps"),
    ("read valid", R, READ, *OK),
    ("read 8 bit", R, dict(READ, **SCALES), *OK),
    ("read caches shared", R, dict(READ, value_pages=[at(5), at(6)], key_pages=[at(5), at(5)]), *OK),
    ("read into parts of a row", R, dict(READ, row_stride=512, values=[at(0) + 512, at(1) + 512]), *OK),
    ("read into parts that overlap", R, dict(READ, row_stride=512, values=[at(0) + 496, at(3)]), "arInvalidArgument",
     "overlaps"),
    ("read into parts past the row", R, dict(READ, row_stride=504, values=[at(0) + 512, at(3)]), "arInvalidArgument",
     "overlaps"),
    ("read no tokens", R, dict(READ, tokens=0, values=None), "arSuccess", None),
    ("read rows over cache", R, dict(READ, keys=[at(5), at(1)]), "arInvalidArgument", "overlaps"),
    ("read keys over values", R, dict(READ, keys=[at(2), at(1)]), "arInvalidArgument", "overlaps"),
    ("read rows over slots", R, dict(READ, values=[at(4), at(3)]), "arInvalidArgument", "overlaps"),
    ("read bad dtype", R, dict(READ, dtype=-1), "arUnsupported", "dtype"),
    ("read one scale table", R, dict(READ, value_scales=[at(9), at(10)]), "arInvalidArgument", "scales"),
    ("read dim 0", R, dict(READ, cache=layout(dim=0)), "arUnsupported", "dim"),
    ("attend valid", T, ATTEND, *OK),
    ("attend everything", T, dict(ATTEND, **SCALES, out_scales=[at(15), at(16)], lse=[at(17), at(18)], window=7), *OK),
    ("attend caches shared", T, dict(ATTEND, value_pages=[at(5), at(5)]), *OK),
    ("attend queries shared", T, dict(ATTEND, queries=[at(0), at(0)]), *OK),
    ("attend no sequences", T, dict(ATTEND, seqs=0, queries=None, workspace=None), "arSuccess", None),
    ("attend bad dtype", T, dict(ATTEND, dtype=9), "arUnsupported", "dtype"),
    ("attend 33 ranks", T, dict(ATTEND, nranks=33), "arUnsupported", "nranks"),
    ("attend one scale table", T, dict(ATTEND, value_scales=[at(9), at(10)]), "arInvalidArgument", "scales"),
    ("attend 7 heads on 2", T, dict(ATTEND, heads=7), "arUnsupported", "multiple"),
    ("attend 0 heads", T, dict(ATTEND, heads=0), "arUnsupported", "multiple"),
    ("attend 4098 heads", T, dict(ATTEND, heads=4098), "arUnsupported", "4096"),
    ("attend 8-bit output of 64", T, dict(ATTEND, cache=layout(dim=64), query_stride=512, out_scales=[at(15), at(16)]),
     "arUnsupported", "128 or 256"),
    ("attend dim 24", T, dict(ATTEND, cache=layout(dim=24)), "arUnsupported", "dim"),
    ("attend scale nan", T, dict(ATTEND, scale=float("nan")), "arInvalidArgument", "scale"),
    ("attend scale inf", T, dict(ATTEND, scale=float("inf")), "arInvalidArgument", "scale"),
    ("attend scale that overflows", T, dict(ATTEND, scale=-1.7e38), "arInvalidArgument", "scale"),
    ("attend 65537 sequences", T, dict(ATTEND, seqs=65537), "arUnsupported", "65536"),
    ("attend too many units", T, dict(ATTEND, seqs=65536, heads=130), "arUnsupported", "2^24"),
    ("attend no table", T, dict(ATTEND, table_pages=0), "arInvalidArgument", "tablePages"),
    ("attend table huge", T, dict(ATTEND, table_pages=1 << 31), "arInvalidArgument", "tablePages"),
    ("attend query rows closer than a row", T, dict(ATTEND, query_stride=1016), "arInvalidArgument", "row stride"),
    ("attend NULL queries", T, dict(ATTEND, queries=None), "arInvalidArgument", "NULL"),
    ("attend NULL out", T, dict(ATTEND, outbufs=[at(13), 0]), "arInvalidArgument", "NULL"),
    ("attend NULL table", T, dict(ATTEND, page_table=None), "arInvalidArgument", "NULL"),
    ("attend NULL lengths", T, dict(ATTEND, lengths=None), "arInvalidArgument", "NULL"),
    ("attend NULL workspace", T, dict(ATTEND, workspace=None), "arInvalidArgument", "NULL"),
    ("attend NULL lse", T, dict(ATTEND, lse=[0, at(18)]), "arInvalidArgument", "NULL"),
    ("attend lengths off", T, dict(ATTEND, lengths=at(3) + 2), "arInvalidArgument", "aligned"),
    ("attend lengths at 4", T, dict(ATTEND, lengths=at(3) + 4), *OK),
    ("attend workspace off", T, dict(ATTEND, workspace=at(20) + 8), "arInvalidArgument", "aligned"),
    ("attend out over queries", T, dict(ATTEND, outbufs=[at(0), at(14)]), "arInvalidArgument", "overlaps"),
    ("attend out over cache", T, dict(ATTEND, outbufs=[at(13), at(8)]), "arInvalidArgument", "overlaps"),
    ("attend out over table", T, dict(ATTEND, outbufs=[at(2), at(14)]), "arInvalidArgument", "overlaps"),
    ("attend outs the same", T, dict(ATTEND, outbufs=[at(13), at(13)]), "arInvalidArgument", "overlaps"),
    ("attend out in the workspace", T, dict(ATTEND, outbufs=[at(20) + 4096, at(14)]), "arInvalidArgument", "overlaps"),
    ("attend lse over scales", T, dict(ATTEND, out_scales=[at(15), at(16)], lse=[at(15), at(18)]),
     "arInvalidArgument", "overlaps"),
    ("attend 8-bit outs next to each other", T,
     dict(ATTEND, out_scales=[at(15), at(16)], outbufs=[at(13), at(13) + 3 * 8 * 128]), *OK),
    ("attend short list", T, dict(ATTEND, nranks=3), "arInvalidArgument", "NULL"),
]

CHILD = r"""
import json, sys
sys.path.insert(0, sys.argv[1])
import all_reduce_amd as ar
for label, name, kw in json.loads(sys.argv[2]):
    sys.stderr.write(f"@@{label}\n"); sys.stderr.flush()
    if kw["cache"] is not None:
        kw["cache"] = ar.arCacheLayout(**kw["cache"])
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


def test_workspace_query_refusals():
    assert ar.arCacheAttentionWorkspace(100, 8, None)[0] == ar.arResult.arUnsupported
    assert ar.arCacheAttentionWorkspace(128, 0, None)[0] == ar.arResult.arUnsupported
    assert ar.arCacheAttentionWorkspace(128, 8, None)[0] == ar.arResult.arInvalidArgument


def test_zeros_of_a_workspace_match_the_header():
    assert int(re.search(r"#define AR_CACHE_WORKSPACE_ZEROS (\d+)", HEADER).group(1)) == ar.AR_CACHE_WORKSPACE_ZEROS
