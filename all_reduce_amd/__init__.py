"""Python binding of the MI355X sum all-reduce over R simulated ranks, and of
the operators around it in a tensor-parallel layer, its key-value cache among them.

The functions named ``ar*`` are the C ABI of ``include/ar_allreduce.h``,
``include/ar_block.h`` and ``include/ar_cache.h``, one for one, over ctypes:
arguments are marshalled and the result code is returned, nothing else happens
here.  :class:`Comm` and :func:`rank_buffers` are conveniences on top for torch
tensors; torch supplies device memory and streams only.  Every step of the
all-reduce runs in the HIP kernels of ``libar_allreduce.so``; there is no other
implementation to fall back to, so a missing library raises instead of running
anything.
"""
from __future__ import annotations

import contextlib
import ctypes
from enum import IntEnum
from pathlib import Path
from typing import Sequence

LIBRARY = Path(__file__).resolve().parent / "_lib" / "libar_allreduce.so"
HEADER = Path(__file__).resolve().parent.parent / "include" / "ar_allreduce.h"
BLOCK_HEADER = HEADER.with_name("ar_block.h")
CACHE_HEADER = HEADER.with_name("ar_cache.h")


class arResult(IntEnum):
    arSuccess = 0
    arInvalidArgument = 1
    arUnsupported = 2
    arInvalidUsage = 3
    arHipError = 4
    arTimeout = 5
    arInternalError = 6


class arDataType(IntEnum):
    arBfloat16 = 0
    arFloat16 = 1
    arFloat32 = 2


class arRedOp(IntEnum):
    arSum = 0


class arProtocol(IntEnum):
    arProtoLL = 0
    arProtoHB = 1
    arProtoAuto = 2


class arOption(IntEnum):
    arOptPollTimeoutUs = 0
    arOptLLBlocksPerRank = 1
    arOptHBBlocks = 2
    arOptHBNonTemporal = 3
    arOptDebugFlagSkew = 4
    arOptHBUnroll = 5
    arOptLLThreads = 6
    arOptHBThreads = 7
    arOptHBChunkLayout = 8
    arOptNodeRanks = 9
    arOptLLPacketBytes = 10
    arOptHBStaged = 11
    arOptLLFlagScheme = 12
    arOptDebugSeqStart = 13
    arOptTuneFreshInputs = 14
    arOptLLDense = 15


class arActivation(IntEnum):
    arActNone = 0
    arActSiLU = 1


AR_SCALE_BLOCK = 128
AR_NORM_MAX_COLS = 32768
AR_CACHE_MAX_DIM = 256
AR_CACHE_WORKSPACE_ZEROS = 65536

AR_MAX_RANKS = 32
AR_NOALLOC_SCRATCH_BYTES = 64 << 20


class arTunedShape(ctypes.Structure):
    """Mirror of arTunedShape_t."""
    _fields_ = [("tuned", ctypes.c_int), ("threads", ctypes.c_int), ("blocks", ctypes.c_int),
                ("packetBytes", ctypes.c_int), ("nonTemporal", ctypes.c_int),
                ("us", ctypes.c_float)]


class arLaunchInfo(ctypes.Structure):
    """Mirror of arLaunchInfo_t."""
    _fields_ = [("protocol", ctypes.c_int), ("kernels", ctypes.c_int), ("grid", ctypes.c_uint),
                ("threads", ctypes.c_uint), ("packetBytes", ctypes.c_int),
                ("nonTemporal", ctypes.c_int), ("nodeRanks", ctypes.c_int),
                ("staged", ctypes.c_int), ("packetPayloadBytes", ctypes.c_int)]


class arCacheLayout(ctypes.Structure):
    """Mirror of arCacheLayout_t."""
    _fields_ = [("pages", ctypes.c_size_t), ("pageTokens", ctypes.c_size_t),
                ("heads", ctypes.c_size_t), ("dim", ctypes.c_size_t),
                ("pageStride", ctypes.c_size_t), ("headStride", ctypes.c_size_t),
                ("tokenStride", ctypes.c_size_t)]


class ArError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = arResult(code)
        super().__init__(f"{where}: {arGetErrorString(code)}")


_lib = None


def library() -> ctypes.CDLL:
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIBRARY.exists():
        raise RuntimeError(f"{LIBRARY} is missing: build it with `python -m all_reduce_amd.build`")
    lib = ctypes.CDLL(str(LIBRARY))
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    pvp, layout = ctypes.POINTER(vp), ctypes.POINTER(arCacheLayout)
    sig = {
        "arCommCreate": ([ctypes.POINTER(vp), i32, i32, sz], i32),
        "arCommDestroy": ([vp], i32),
        "arCommReset": ([vp, vp], i32),
        "arCommGetAsyncError": ([vp, ctypes.POINTER(i32)], i32),
        "arCommSetOption": ([vp, i32, i64], i32),
        "arCommGetOption": ([vp, i32, ctypes.POINTER(i64)], i32),
        "arAllReduce": ([ctypes.POINTER(vp), ctypes.POINTER(vp), sz, i32, i32, i32, i32, vp, vp], i32),
        "arCommTune": ([vp, i32, i32, sz, vp], i32),
        "arCommGetTunedShape": ([vp, i32, i32, i32, sz, i32, ctypes.POINTER(arTunedShape)], i32),
        "arCommGetLastLaunch": ([vp, ctypes.POINTER(arLaunchInfo)], i32),
        "arCommSetWorkspace": ([vp, vp, sz], i32),
        "arAllReduceNoAlloc": ([ctypes.POINTER(vp), ctypes.POINTER(vp), sz, i32, i32, i32, i32,
                                vp], i32),
        "arAllReduceNorm": ([pvp, vp, vp, ctypes.c_float, pvp, pvp, pvp, sz, sz, i32, i32, vp, vp],
                            i32),
        "arGateQuant": ([pvp, pvp, pvp, sz, sz, i32, i32, i32, vp, vp], i32),
        "arMatmulScaled": ([pvp, pvp, pvp, pvp, pvp, sz, sz, sz, i32, i32, i32, vp, vp], i32),
        "arCacheWrite": ([pvp, pvp, sz, vp, sz, layout, pvp, pvp, pvp, pvp, i32, i32, vp, vp], i32),
        "arCacheRead": ([vp, sz, layout, pvp, pvp, pvp, pvp, pvp, pvp, sz, i32, i32, vp, vp], i32),
        "arCacheAttention": ([pvp, sz, layout, pvp, pvp, pvp, pvp, vp, sz, vp, sz, sz,
                              ctypes.c_float, sz, pvp, pvp, pvp, vp, sz, i32, i32, vp, vp], i32),
        "arCacheAttentionWorkspace": ([sz, sz, vp, ctypes.POINTER(sz)], i32),
        "arGetErrorString": ([i32], ctypes.c_char_p),
        "arGetVersion": ([], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


# ---- the C ABI, one Python function per entry point -----------------------
def arGetErrorString(result: int) -> str:
    return library().arGetErrorString(int(result)).decode()


def arGetVersion() -> int:
    return library().arGetVersion()


def arCommCreate(device: int, max_ranks: int, max_ll_bytes_per_rank: int):
    """Returns (result code, communicator handle or None)."""
    h = ctypes.c_void_p()
    r = library().arCommCreate(ctypes.byref(h), device, max_ranks, max_ll_bytes_per_rank)
    return r, (h.value if r == 0 else None)


def arCommDestroy(comm) -> int:
    return library().arCommDestroy(comm)


def arCommReset(comm, stream) -> int:
    return library().arCommReset(comm, stream)


def arCommGetAsyncError(comm):
    """Returns (result code, recorded asynchronous error)."""
    e = ctypes.c_int(0)
    r = library().arCommGetAsyncError(comm, ctypes.byref(e))
    return r, e.value


def arCommSetOption(comm, option: int, value: int) -> int:
    return library().arCommSetOption(comm, int(option), int(value))


def arCommGetOption(comm, option: int):
    v = ctypes.c_int64(0)
    r = library().arCommGetOption(comm, int(option), ctypes.byref(v))
    return r, v.value


def arCommTune(comm, dtype: int, nranks: int, max_bytes_per_rank: int, stream) -> int:
    return library().arCommTune(comm, int(dtype), nranks, max_bytes_per_rank, stream)


def arCommGetTunedShape(comm, dtype: int, nranks: int, protocol: int, bytes_per_rank: int,
                        in_place: int = 0):
    """Returns (result code, arTunedShape)."""
    shape = arTunedShape()
    r = library().arCommGetTunedShape(comm, int(dtype), nranks, int(protocol), bytes_per_rank,
                                      int(in_place), ctypes.byref(shape))
    return r, shape


def arCommSetWorkspace(comm, workspace, nbytes: int) -> int:
    """``workspace`` a device pointer as an integer, or None with 0."""
    return library().arCommSetWorkspace(comm, workspace, nbytes)


def arCommGetLastLaunch(comm):
    """Returns (result code, arLaunchInfo)."""
    info = arLaunchInfo()
    r = library().arCommGetLastLaunch(comm, ctypes.byref(info))
    return r, info


def _pointer_array(ptrs: Sequence[int] | None, nranks: int):
    """ctypes array of device pointers, NULL-padded to ``nranks`` entries so the
    library never reads past it (it rejects nranks > AR_MAX_RANKS before reading
    any pointer, and reports a NULL entry as arInvalidArgument)."""
    if ptrs is None:
        return None
    n = max(1, len(ptrs), min(max(int(nranks), 0), AR_MAX_RANKS))
    return (ctypes.c_void_p * n)(*ptrs)


def arAllReduce(sendbufs: Sequence[int] | None, recvbufs: Sequence[int] | None, count: int,
                dtype: int, op: int, nranks: int, protocol: int, comm, stream) -> int:
    """Device pointers as integers; ``None`` passes a NULL array."""
    s = _pointer_array(sendbufs, nranks)
    d = _pointer_array(recvbufs, nranks)
    return library().arAllReduce(s, d, count, int(dtype), int(op), nranks, int(protocol),
                                 comm, stream)


def arAllReduceNoAlloc(sendbufs: Sequence[int] | None, recvbufs: Sequence[int] | None,
                       count: int, dtype: int, op: int, nranks: int, node_ranks: int,
                       stream) -> int:
    """Device pointers as integers; ``None`` passes a NULL array."""
    s = _pointer_array(sendbufs, nranks)
    d = _pointer_array(recvbufs, nranks)
    return library().arAllReduceNoAlloc(s, d, count, int(dtype), int(op), nranks,
                                        int(node_ranks), stream)


def arAllReduceNorm(sendbufs, residual, weight, eps: float, residual_out, outbufs, scalebufs,
                    rows: int, cols: int, dtype: int, nranks: int, comm, stream) -> int:
    """Device pointers as integers, sequences of them for the rank tables;
    ``None`` passes NULL."""
    return library().arAllReduceNorm(
        _pointer_array(sendbufs, nranks), residual, weight, eps,
        _pointer_array(residual_out, nranks), _pointer_array(outbufs, nranks),
        _pointer_array(scalebufs, nranks), rows, cols, int(dtype), nranks, comm, stream)


def arGateQuant(inbufs, outbufs, scalebufs, rows: int, cols: int, dtype: int, act: int,
                nranks: int, comm, stream) -> int:
    """Device pointers as integers, sequences of them for the rank tables;
    ``None`` passes NULL."""
    return library().arGateQuant(
        _pointer_array(inbufs, nranks), _pointer_array(outbufs, nranks),
        _pointer_array(scalebufs, nranks), rows, cols, int(dtype), int(act), nranks, comm, stream)


def arMatmulScaled(abufs, ascales, bbufs, bscales, outbufs, rows: int, n: int, k: int,
                   out_dtype: int, reduce: int, nranks: int, comm, stream) -> int:
    """Device pointers as integers, sequences of them for the rank tables;
    ``None`` passes NULL."""
    return library().arMatmulScaled(
        _pointer_array(abufs, nranks), _pointer_array(ascales, nranks),
        _pointer_array(bbufs, nranks), _pointer_array(bscales, nranks),
        _pointer_array(outbufs, nranks), rows, n, k, int(out_dtype), int(reduce), nranks, comm,
        stream)


def arCacheWrite(keys, values, row_stride: int, slots, tokens: int, cache, key_pages, value_pages,
                 key_scales, value_scales, dtype: int, nranks: int, comm, stream) -> int:
    """Device pointers as integers, sequences of them for the rank tables;
    ``cache`` an arCacheLayout; ``None`` passes NULL."""
    return library().arCacheWrite(
        _pointer_array(keys, nranks), _pointer_array(values, nranks), row_stride, slots, tokens,
        cache, _pointer_array(key_pages, nranks), _pointer_array(value_pages, nranks),
        _pointer_array(key_scales, nranks), _pointer_array(value_scales, nranks), int(dtype),
        nranks, comm, stream)


def arCacheRead(slots, tokens: int, cache, key_pages, value_pages, key_scales, value_scales, keys,
                values, row_stride: int, dtype: int, nranks: int, comm, stream) -> int:
    """As arCacheWrite."""
    return library().arCacheRead(
        slots, tokens, cache, _pointer_array(key_pages, nranks),
        _pointer_array(value_pages, nranks), _pointer_array(key_scales, nranks),
        _pointer_array(value_scales, nranks), _pointer_array(keys, nranks),
        _pointer_array(values, nranks), row_stride, int(dtype), nranks, comm, stream)


def arCacheAttention(queries, query_stride: int, cache, key_pages, value_pages, key_scales,
                     value_scales, page_table, table_pages: int, lengths, seqs: int, heads: int,
                     scale: float, window: int, outbufs, out_scales, lse, workspace,
                     workspace_bytes: int, dtype: int, nranks: int, comm, stream) -> int:
    """As arCacheWrite."""
    return library().arCacheAttention(
        _pointer_array(queries, nranks), query_stride, cache, _pointer_array(key_pages, nranks),
        _pointer_array(value_pages, nranks), _pointer_array(key_scales, nranks),
        _pointer_array(value_scales, nranks), page_table, table_pages, lengths, seqs, heads, scale,
        window, _pointer_array(outbufs, nranks), _pointer_array(out_scales, nranks),
        _pointer_array(lse, nranks), workspace, workspace_bytes, int(dtype), nranks, comm, stream)


def arCacheAttentionWorkspace(dim: int, group: int, comm):
    """Returns (result code, bytes)."""
    n = ctypes.c_size_t(0)
    r = library().arCacheAttentionWorkspace(dim, group, comm, ctypes.byref(n))
    return r, n.value


# ---- torch conveniences ---------------------------------------------------
def _torch():
    import torch
    return torch


def dtype_code(dtype) -> arDataType:
    torch = _torch()
    table = {torch.bfloat16: arDataType.arBfloat16, torch.float16: arDataType.arFloat16,
             torch.float32: arDataType.arFloat32}
    if dtype not in table:
        raise ArError(arResult.arUnsupported, f"dtype {dtype}")
    return table[dtype]


def protocol_code(protocol) -> arProtocol:
    if isinstance(protocol, str):
        return {"ll": arProtocol.arProtoLL, "hb": arProtocol.arProtoHB,
                "auto": arProtocol.arProtoAuto}[protocol.lower()]
    return arProtocol(protocol)


def activation_code(act) -> arActivation:
    if isinstance(act, str):
        return {"none": arActivation.arActNone, "silu": arActivation.arActSiLU}[act.lower()]
    return arActivation(act)


def scale_blocks(cols: int) -> int:
    """Scales that `cols` columns (or a weight's rows) have: one for each 128, the
    last block shorter."""
    return -(-cols // AR_SCALE_BLOCK)


def rank_buffers(nranks: int, count: int, dtype, device, align: int = 256):
    """One allocation holding ``nranks`` buffers of ``count`` elements.

    Rank r's buffer starts at ``base + r * stride`` with the stride rounded up
    to ``align`` bytes.  Returns (plane, views): ``plane`` is the
    (nranks, stride_elems) tensor, ``views[r]`` rank r's ``count`` elements."""
    torch = _torch()
    es = torch.empty((), dtype=dtype).element_size()
    stride = -(-max(count, 1) * es // align) * align // es
    plane = torch.empty((nranks, stride), dtype=dtype, device=device)
    return plane, [plane[r, :count] for r in range(nranks)]


class Comm:
    """Owns an ``arComm_t`` on one device; ``all_reduce`` over torch tensors."""

    def __init__(self, device=None, max_ranks: int = AR_MAX_RANKS,
                 max_ll_bytes_per_rank: int = 1 << 20):
        torch = _torch()
        dev = torch.device("cuda") if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"a communicator needs a GPU device, not {dev}")
        # "cuda" without an index means the current device; resolve it now, so
        # that tensors on "cuda:<i>" compare equal to the communicator's device.
        dev = torch.device("cuda", dev.index if dev.index is not None
                           else torch.cuda.current_device())
        self.device = dev
        r, h = arCommCreate(dev.index, max_ranks, max_ll_bytes_per_rank)
        if r != 0:
            raise ArError(r, "arCommCreate")
        self.handle = h
        self.max_ranks = max_ranks
        self.max_ll_bytes_per_rank = max_ll_bytes_per_rank
        self._workspace = None

    def close(self):
        """Free the communicator after the device has finished the work using it."""
        if self.handle is not None:
            _torch().cuda.synchronize(self.device)
            r = arCommDestroy(self.handle)
            self.handle = None
            if r != 0:
                raise ArError(r, "arCommDestroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _stream(self, stream):
        torch = _torch()
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        return s.cuda_stream

    def set_option(self, option, value: int):
        r = arCommSetOption(self.handle, option, value)
        if r != 0:
            raise ArError(r, "arCommSetOption")

    def get_option(self, option) -> int:
        r, v = arCommGetOption(self.handle, option)
        if r != 0:
            raise ArError(r, "arCommGetOption")
        return v

    def tune(self, dtype, nranks: int, max_bytes_per_rank: int, stream=None):
        """Measure launch shapes per power-of-two size (see arCommTune)."""
        r = arCommTune(self.handle, dtype_code(dtype), nranks, max_bytes_per_rank,
                       self._stream(stream))
        if r != 0:
            raise ArError(r, "arCommTune")

    def tuned_shape(self, dtype, nranks: int, protocol, bytes_per_rank: int,
                    in_place: bool = False):
        """(threads, blocks, us, packet_bytes, non_temporal) stored for that size
        and mode -- threads and blocks 0 when the built-in default won;
        packet_bytes 8 or 16 for LL, 0 for HB; non_temporal 1 or 0 for HB, 0 for
        LL -- or None if never tuned."""
        r, s = arCommGetTunedShape(self.handle, dtype_code(dtype), nranks,
                                   protocol_code(protocol), bytes_per_rank, 1 if in_place else 0)
        if r != 0:
            raise ArError(r, "arCommGetTunedShape")
        return None if s.tuned == 0 else (s.threads, s.blocks, s.us, s.packetBytes, s.nonTemporal)

    def set_workspace(self, workspace):
        """Attach a device tensor (256-byte aligned, on the communicator's
        device) as the staged two-level form's workspace, or None to detach.
        The tensor is kept alive while attached."""
        if workspace is None:
            r = arCommSetWorkspace(self.handle, None, 0)
        else:
            if not workspace.is_contiguous() or workspace.device != self.device:
                raise ValueError("the workspace must be a contiguous tensor on the "
                                 "communicator's device")
            r = arCommSetWorkspace(self.handle, workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size())
        if r != 0:
            raise ArError(r, "arCommSetWorkspace")
        self._workspace = workspace

    def last_launch(self) -> dict | None:
        """The shape of the communicator's most recent launch (see
        arCommGetLastLaunch) as a dict, or None before the first one."""
        r, info = arCommGetLastLaunch(self.handle)
        if r != 0:
            raise ArError(r, "arCommGetLastLaunch")
        if info.protocol < 0:
            return None
        return {name: getattr(info, name) for name, _ in info._fields_}

    def reset(self, stream=None):
        r = arCommReset(self.handle, self._stream(stream))
        if r != 0:
            raise ArError(r, "arCommReset")

    def async_error(self) -> arResult:
        r, e = arCommGetAsyncError(self.handle)
        if r != 0:
            raise ArError(r, "arCommGetAsyncError")
        return arResult(e)

    def all_reduce(self, send, recv=None, protocol="auto", stream=None):
        """Sum all-reduce of the tensors in ``send`` into ``recv`` (default: in place).

        ``protocol`` is "ll", "hb" or "auto" (the tuned faster one; HB where
        nothing was tuned)."""
        send, recv = self._check_ranks(send, recv)
        t0 = send[0]
        r = arAllReduce([t.data_ptr() for t in send], [t.data_ptr() for t in recv],
                        t0.numel(), dtype_code(t0.dtype), arRedOp.arSum, len(send),
                        protocol_code(protocol), self.handle, self._stream(stream))
        if r != 0:
            raise ArError(r, "arAllReduce")
        return recv

    def prepare(self, send, recv=None, protocol="auto", stream=None) -> "PreparedAllReduce":
        """``all_reduce(send, recv, protocol, stream)`` with its arguments
        marshalled once, for a loop that reduces the same buffers again and
        again without a graph.  The stream is fixed here (default: the current
        stream now); the tensors are kept alive by the returned call."""
        send, recv = self._check_ranks(send, recv)
        return PreparedAllReduce(self, send, recv, protocol_code(protocol), self._stream(stream))

    def all_reduce_norm(self, send, weight, eps: float, residual=None, residual_out=None,
                        out=None, scales=None, stream=None):
        """All-reduce, residual addition and root-mean-square norm in one pass
        (see arAllReduceNorm).  ``send``, ``residual_out`` (or None: not kept) and
        ``out`` are lists of one [rows, cols] tensor a rank, ``residual`` (or
        None) one such tensor, ``weight`` [cols].  ``out`` has the element type,
        or torch.float8_e4m3fn with ``scales`` a list of float32
        [scale_blocks(cols), rows].  Returns ``out``."""
        self.prepare_all_reduce_norm(send, weight, eps, residual, residual_out, out, scales,
                                     stream)()
        return out

    def prepare_all_reduce_norm(self, send, weight, eps: float, residual=None,
                                residual_out=None, out=None, scales=None,
                                stream=None) -> "PreparedCall":
        """``all_reduce_norm`` with its arguments marshalled once (see ``prepare``)."""
        torch = _torch()
        rows, cols, dtype = self._matrix(send)
        if out is None:
            raise ValueError("need one output tensor per rank")
        n = len(send)
        eight = scales is not None
        self._check("send", send, n, (rows, cols), dtype)
        self._check("weight", [weight], 1, (cols,), dtype)
        if residual is not None:
            self._check("residual", [residual], 1, (rows, cols), dtype)
        if residual_out is not None:
            self._check("residual_out", residual_out, n, (rows, cols), dtype)
        self._check("out", out, n, (rows, cols), torch.float8_e4m3fn if eight else dtype)
        if eight:
            self._check("scales", scales, n, (scale_blocks(cols), rows), torch.float32)
        return PreparedCall(self, "arAllReduceNorm", (
            _rank_table(send), None if residual is None else residual.data_ptr(),
            weight.data_ptr(), float(eps), _rank_table(residual_out), _rank_table(out),
            _rank_table(scales), rows, cols, int(dtype_code(dtype)), n), self._stream(stream),
            (send, weight, residual, residual_out, out, scales))

    def gate_quant(self, x, out, scales, act="silu", stream=None):
        """Activation and quantisation to 8 bits for every rank (see arGateQuant).
        ``x`` is a list of one [rows, cols] tensor a rank, or [rows, 2 * cols]
        with ``act`` "silu" (gate, then up); ``out`` of [rows, cols]
        torch.float8_e4m3fn, ``scales`` of float32 [scale_blocks(cols), rows].
        Returns ``out``."""
        self.prepare_gate_quant(x, out, scales, act, stream)()
        return out

    def prepare_gate_quant(self, x, out, scales, act="silu", stream=None) -> "PreparedCall":
        """``gate_quant`` with its arguments marshalled once (see ``prepare``)."""
        torch = _torch()
        rows, wide, dtype = self._matrix(x)
        code = activation_code(act)
        n, cols = len(x), wide // 2 if code == arActivation.arActSiLU else wide
        if code == arActivation.arActSiLU and wide % 2 != 0:
            raise ValueError("gated inputs need an even number of columns")
        self._check("x", x, n, (rows, wide), dtype)
        self._check("out", out, n, (rows, cols), torch.float8_e4m3fn)
        self._check("scales", scales, n, (scale_blocks(cols), rows), torch.float32)
        return PreparedCall(self, "arGateQuant", (
            _rank_table(x), _rank_table(out), _rank_table(scales), rows, cols,
            int(dtype_code(dtype)), int(code), n), self._stream(stream), (x, out, scales))

    def matmul_scaled(self, a, a_scales, b, b_scales, out, reduce: bool = False, stream=None):
        """The product of 8-bit activations and weights with a scale per block of
        128 (see arMatmulScaled).  Lists of one tensor a rank: ``a`` [rows, k] and
        ``b`` [n, k] torch.float8_e4m3fn, ``a_scales`` float32
        [scale_blocks(k), rows], ``b_scales`` float32
        [scale_blocks(n), scale_blocks(k)], ``out`` [rows, n] bfloat16, float16 or
        float32: each rank's own product, or with ``reduce`` the sum of all of
        them in every rank's output.  Returns ``out``."""
        self.prepare_matmul_scaled(a, a_scales, b, b_scales, out, reduce, stream)()
        return out

    def prepare_matmul_scaled(self, a, a_scales, b, b_scales, out, reduce: bool = False,
                              stream=None) -> "PreparedCall":
        """``matmul_scaled`` with its arguments marshalled once (see ``prepare``)."""
        torch = _torch()
        eight = torch.float8_e4m3fn
        rows, k, _ = self._matrix(a)
        cols, _, _ = self._matrix(b)
        _, _, dtype = self._matrix(out)
        n = len(a)
        self._check("a", a, n, (rows, k), eight)
        self._check("a_scales", a_scales, n, (scale_blocks(k), rows), torch.float32)
        self._check("b", b, n, (cols, k), eight)
        self._check("b_scales", b_scales, n, (scale_blocks(cols), scale_blocks(k)), torch.float32)
        self._check("out", out, n, (rows, cols), dtype)
        return PreparedCall(self, "arMatmulScaled", (
            _rank_table(a), _rank_table(a_scales), _rank_table(b), _rank_table(b_scales),
            _rank_table(out), rows, cols, k, int(dtype_code(dtype)), int(bool(reduce)), n),
            self._stream(stream), (a, a_scales, b, b_scales, out))

    def cache_write(self, keys, values, slots, key_pages, value_pages, key_scales=None,
                    value_scales=None, stream=None):
        """New tokens' keys and values into the paged cache (see arCacheWrite).
        Lists of one tensor a rank: ``keys`` and ``values`` [tokens, heads, dim],
        which may be parts of the wider rows of a product; ``key_pages`` and
        ``value_pages`` [pages, heads, tokens of a page, dim] in any order of memory
        whose last dimension is dense, of the element type, or torch.float8_e4m3fn
        with ``key_scales`` and ``value_scales`` float32 [pages, heads, tokens of a
        page].  ``slots``, int64 [tokens], is the ranks' common one; tokens whose
        slot is negative are skipped."""
        self.prepare_cache_write(keys, values, slots, key_pages, value_pages, key_scales,
                                 value_scales, stream)()

    def prepare_cache_write(self, keys, values, slots, key_pages, value_pages, key_scales=None,
                            value_scales=None, stream=None) -> "PreparedCall":
        """``cache_write`` with its arguments marshalled once (see ``prepare``)."""
        dtype, n = self._rows(keys, "keys").dtype, len(keys)
        layout = self._pages(key_pages, value_pages, key_scales, value_scales, n, dtype)
        stride = self._check_rows(keys, values, slots, layout, dtype)
        return PreparedCall(self, "arCacheWrite", (
            _rank_table(keys), _rank_table(values), stride, slots.data_ptr(), slots.numel(), layout,
            _rank_table(key_pages), _rank_table(value_pages), _rank_table(key_scales),
            _rank_table(value_scales), int(dtype_code(dtype)), n), self._stream(stream),
            (keys, values, slots, key_pages, value_pages, key_scales, value_scales))

    def cache_read(self, slots, key_pages, value_pages, keys, values, key_scales=None,
                   value_scales=None, stream=None):
        """The cached rows of ``slots`` into ``keys`` and ``values`` (see arCacheRead;
        shapes as for ``cache_write``).  Rows whose slot is negative are left as
        they were.  Returns ``(keys, values)``."""
        self.prepare_cache_read(slots, key_pages, value_pages, keys, values, key_scales,
                                value_scales, stream)()
        return keys, values

    def prepare_cache_read(self, slots, key_pages, value_pages, keys, values, key_scales=None,
                           value_scales=None, stream=None) -> "PreparedCall":
        """``cache_read`` with its arguments marshalled once (see ``prepare``)."""
        dtype, n = self._rows(keys, "keys").dtype, len(keys)
        layout = self._pages(key_pages, value_pages, key_scales, value_scales, n, dtype)
        stride = self._check_rows(keys, values, slots, layout, dtype)
        return PreparedCall(self, "arCacheRead", (
            slots.data_ptr(), slots.numel(), layout, _rank_table(key_pages),
            _rank_table(value_pages), _rank_table(key_scales), _rank_table(value_scales),
            _rank_table(keys), _rank_table(values), stride, int(dtype_code(dtype)), n),
            self._stream(stream),
            (keys, values, slots, key_pages, value_pages, key_scales, value_scales))

    def cache_attention(self, queries, key_pages, value_pages, page_table, lengths, out,
                        key_scales=None, value_scales=None, scale: float | None = None,
                        window: int = 0, out_scales=None, lse=None, workspace=None, stream=None):
        """Attention of one new token a sequence over the paged cache (see
        arCacheAttention).  Lists of one tensor a rank: ``queries`` [seqs, heads,
        dim], which may be parts of the wider rows of a product; the cache as for
        ``cache_write``; ``out`` [seqs, heads, dim] of the element type, or
        torch.float8_e4m3fn with ``out_scales`` float32 [heads * dim / 128, seqs];
        ``lse`` (or None: not wanted) float32 [seqs, heads].  ``page_table`` int32
        [seqs, pages of a sequence] and ``lengths`` int32 [seqs] are the ranks'
        common ones.  ``scale``: 1 / sqrt(dim) if None; ``window``: attend to the
        last tokens alone, 0: to all.  ``workspace``: one of ``cache_workspace``
        that no other call uses at the same time; None: one of the call's own.
        Returns ``out``."""
        self.prepare_cache_attention(queries, key_pages, value_pages, page_table, lengths, out,
                                     key_scales, value_scales, scale, window, out_scales, lse,
                                     workspace, stream)()
        return out

    def prepare_cache_attention(self, queries, key_pages, value_pages, page_table, lengths, out,
                                key_scales=None, value_scales=None, scale: float | None = None,
                                window: int = 0, out_scales=None, lse=None, workspace=None,
                                stream=None) -> "PreparedCall":
        """``cache_attention`` with its arguments marshalled once (see ``prepare``).
        The workspace is part of the prepared call, so calls that may run at once
        need to be prepared apart."""
        torch = _torch()
        first, n = self._rows(queries, "queries"), len(queries)
        dtype = first.dtype
        seqs, heads, dim = first.shape
        layout = self._pages(key_pages, value_pages, key_scales, value_scales, n, dtype)
        if layout.dim != dim:
            raise ValueError(f"queries of {dim}, cache of {layout.dim}")
        if window < 0:
            raise ValueError(f"window must not be negative, got {window}")
        stride = self._strided("queries", queries, n, (seqs, heads, dim), dtype)
        self._check("out", out, n, (seqs, heads, dim), dtype if out_scales is None else torch.float8_e4m3fn)
        if out_scales is not None:
            self._check("out_scales", out_scales, n, (scale_blocks(heads * dim), seqs), torch.float32)
        if lse is not None:
            self._check("lse", lse, n, (seqs, heads), torch.float32)
        if page_table.dim() != 2:
            raise ValueError("page_table: need [seqs, pages of a sequence]")
        self._check("page_table", [page_table], 1, (seqs, page_table.shape[1]), torch.int32)
        self._check("lengths", [lengths], 1, (seqs,), torch.int32)
        if workspace is None:
            workspace = self.cache_workspace(dim, max(1, heads // max(1, layout.heads)), stream)
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError("the workspace must be a contiguous tensor on the communicator's device")
        return PreparedCall(self, "arCacheAttention", (
            _rank_table(queries), stride, layout, _rank_table(key_pages), _rank_table(value_pages),
            _rank_table(key_scales), _rank_table(value_scales), page_table.data_ptr(),
            page_table.shape[1], lengths.data_ptr(), seqs, heads,
            float(dim ** -0.5 if scale is None else scale), int(window), _rank_table(out),
            _rank_table(out_scales), _rank_table(lse), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), int(dtype_code(dtype)), n),
            self._stream(stream), (queries, key_pages, value_pages, key_scales, value_scales,
                                   page_table, lengths, out, out_scales, lse, workspace))

    def cache_workspace(self, dim: int, group: int, stream=None):
        """A workspace for ``cache_attention`` with heads of ``dim`` and ``group``
        query heads to a key-value head (or fewer of either), ready on ``stream``
        (default: the current one).  Calls one after the other may share it; calls
        that may run at once need one each."""
        torch = _torch()
        r, n = arCacheAttentionWorkspace(dim, group, self.handle)
        if r != 0:
            raise ArError(r, "arCacheAttentionWorkspace")
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            work = torch.empty(n, dtype=torch.uint8, device=self.device)
            work[:AR_CACHE_WORKSPACE_ZEROS].zero_()
        return work

    @staticmethod
    def _rows(tensors, name):
        """The first of a list of [rows, heads, dim] tensors."""
        if not tensors or tensors[0].dim() != 3:
            raise ValueError(f"{name}: need one three-dimensional tensor per rank")
        return tensors[0]

    def _strided(self, name, tensors, count, shape, dtype, stride=None):
        """Checks [rows, heads, dim] tensors with dense rows; returns the elements
        from one row to the next, the same for all (``stride`` if given)."""
        if len(tensors) != count:
            raise ValueError(f"{name}: need {count} tensors, got {len(tensors)}")
        rows, heads, dim = shape
        if stride is None:
            stride = tensors[0].stride(0) if rows > 1 else heads * dim
        want = (stride, dim, 1)
        for t in tensors:
            if t.device != self.device:
                raise ValueError(f"{name}: tensor on {t.device}, communicator on {self.device}")
            if tuple(t.shape) != shape or t.dtype != dtype:
                raise ValueError(f"{name}: need {shape} of {dtype}, got {tuple(t.shape)} of "
                                 f"{t.dtype}")
            if any(n > 1 and a != b for n, a, b in zip(shape, t.stride(), want)):
                raise ValueError(f"{name}: need dense rows, equally far apart in all tensors")
        return stride

    def _check_rows(self, keys, values, slots, layout, dtype):
        """Checks the rows of a write or read; returns their stride."""
        torch = _torch()
        if slots.dim() != 1:
            raise ValueError("slots: need [tokens]")
        self._check("slots", [slots], 1, (slots.shape[0],), torch.int64)
        shape = (slots.shape[0], layout.heads, layout.dim)
        stride = self._strided("keys", keys, len(keys), shape, dtype)
        return self._strided("values", values, len(keys), shape, dtype, stride)

    def _pages(self, key_pages, value_pages, key_scales, value_scales, count, dtype):
        """Checks a cache's tensors; returns its layout."""
        torch = _torch()
        if (key_scales is None) != (value_scales is None):
            raise ValueError("need scales of keys and of values, or of neither")
        if not key_pages or key_pages[0].dim() != 4:
            raise ValueError("key_pages: need one four-dimensional tensor per rank")
        shape, strides = tuple(key_pages[0].shape), key_pages[0].stride()
        want = dtype if key_scales is None else torch.float8_e4m3fn
        for name, tensors in (("key_pages", key_pages), ("value_pages", value_pages)):
            if len(tensors) != count:
                raise ValueError(f"{name}: need {count} tensors, got {len(tensors)}")
            for t in tensors:
                if t.device != self.device:
                    raise ValueError(f"{name}: tensor on {t.device}, communicator on {self.device}")
                if tuple(t.shape) != shape or t.dtype != want:
                    raise ValueError(f"{name}: need {shape} of {want}, got {tuple(t.shape)} of "
                                     f"{t.dtype}")
                if t.stride(3) != 1 or any(n > 1 and a != b
                                           for n, a, b in zip(shape, t.stride(), strides)):
                    raise ValueError(f"{name}: need dense rows and the same strides in all tensors")
        if key_scales is not None:
            self._check("key_scales", key_scales, count, shape[:3], torch.float32)
            self._check("value_scales", value_scales, count, shape[:3], torch.float32)
        pages, heads, tokens, dim = shape
        return arCacheLayout(pages, tokens, heads, dim, strides[0], strides[1], strides[2])

    @staticmethod
    def _matrix(tensors):
        """(rows, columns, dtype) of the first of a list of matrices."""
        if not tensors or tensors[0].dim() != 2:
            raise ValueError("need one two-dimensional tensor per rank")
        return (*tensors[0].shape, tensors[0].dtype)

    def _check(self, name, tensors, count, shape, dtype):
        if len(tensors) != count:
            raise ValueError(f"{name}: need {count} tensors, got {len(tensors)}")
        for t in tensors:
            if t.device != self.device:
                raise ValueError(f"{name}: tensor on {t.device}, communicator on {self.device}")
            if tuple(t.shape) != shape or t.dtype != dtype:
                raise ValueError(f"{name}: need {shape} of {dtype}, got {tuple(t.shape)} of "
                                 f"{t.dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{name}: tensors must be contiguous")

    def _check_ranks(self, send, recv):
        if recv is None:
            recv = send
        if len(send) != len(recv) or not send:
            raise ValueError("need one receive tensor per send tensor")
        t0 = send[0]
        for t in (*send, *recv):
            if t.device != self.device:
                raise ValueError(f"tensor on {t.device}, communicator on {self.device}")
            if t.dtype != t0.dtype or t.numel() != t0.numel():
                raise ValueError("all rank tensors need the same dtype and size")
            if not t.is_contiguous():
                raise ValueError("rank tensors must be contiguous")
        return list(send), list(recv)


class PreparedAllReduce:
    """One ``arAllReduce`` call whose arguments (pointer arrays, count, dtype,
    protocol, stream) were marshalled once: calling it is a single foreign
    call.  Made by ``Comm.prepare``.  The communicator's handle is read at each
    call, so a call after ``Comm.close()`` raises instead of passing a freed
    communicator to the library."""

    __slots__ = ("_fn", "_head", "_tail", "_comm", "_keep")

    def __init__(self, comm, send, recv, protocol, stream):
        n = len(send)
        t0 = send[0]
        self._fn = library().arAllReduce
        self._head = (_pointer_array([t.data_ptr() for t in send], n),
                      _pointer_array([t.data_ptr() for t in recv], n),
                      t0.numel(), int(dtype_code(t0.dtype)), int(arRedOp.arSum), n,
                      int(protocol))
        self._tail = stream
        self._comm = comm
        self._keep = (send, recv)

    def __call__(self):
        h = self._comm.handle
        if h is None:
            raise ValueError("the communicator of this prepared call was closed")
        r = self._fn(*self._head, h, self._tail)
        if r != 0:
            raise ArError(r, "arAllReduce")


def _rank_table(tensors):
    """The pointer array of one tensor a rank; None passes NULL."""
    return None if tensors is None else \
        (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


class PreparedCall:
    """One call of an operator of ``ar_block.h`` or ``ar_cache.h`` whose arguments
    were marshalled once: calling it is a single foreign call.  Made by the
    ``Comm.prepare_*`` methods; the tensors are kept alive.  A call after
    ``Comm.close()`` raises instead of passing a freed communicator to the library.

    The arguments are kept as ctypes objects and passed to a function object
    without argument types, which converts nothing (0.4 us less a call)."""

    __slots__ = ("_fn", "_name", "_args", "_comm", "_keep")

    def __init__(self, comm, name, head, stream, keep):
        types = getattr(library(), name).argtypes
        values = (*head, comm.handle, stream)
        self._fn = library()[name]
        self._fn.restype = ctypes.c_int
        self._name = name
        self._args = tuple(v if isinstance(v, ctypes.Array) else
                           ctypes.c_void_p(None) if v is None else t(v)
                           for t, v in zip(types, values))
        self._comm = comm
        self._keep = keep

    def __call__(self):
        if self._comm.handle is None:
            raise ValueError("the communicator of this prepared call was closed")
        r = self._fn(*self._args)
        if r != 0:
            raise ArError(r, self._name)
