// block_api.hip -- the entry points declared in include/ar_block.h.
//
// Host side of each call: check the arguments without touching the device,
// pack the rank tables into the kernel arguments and enqueue one launch on
// the caller's stream.  Nothing here allocates, synchronises or records a
// memset, so calls can be captured into a HIP graph.
#include <math.h>

#include "api_checks.hpp"
#include "block_internal.hpp"

using namespace ar;

extern "C" {

arResult_t arAllReduceNorm(const void *const *sendbufs, const void *residual, const void *weight,
                           float eps, void *const *residualOut, void *const *outbufs,
                           float *const *scalebufs, size_t rows, size_t cols,
                           arDataType_t dtype_arg, int nranks, arComm_t comm, arStream_t stream)
{
    const int dtype = raw(dtype_arg);
    if (!is_dtype(dtype))
        return reject(arUnsupported, "dtype must be bf16, fp16 or fp32");
    if (nranks < 1 || nranks > AR_MAX_RANKS)
        return reject(arUnsupported, "nranks must be in 1..32");
    if (cols < 1 || cols > AR_NORM_MAX_COLS)
        return reject(arUnsupported, "cols must be in 1..32768");
    if (!(eps >= 0.0f) || !isfinite(eps))
        return reject(arInvalidArgument, "eps must be finite and not negative");
    if (rows == 0)
        return arSuccess;
    if (too_large(rows, cols))
        return reject(arInvalidArgument, "rows too large");
    if (sendbufs == nullptr || outbufs == nullptr)
        return reject(arInvalidArgument, "NULL buffer array");
    const size_t bytes = rows * cols * elem_bytes(dtype);
    const bool eight = scalebufs != nullptr;
    Ranges mem;
    bool residual_written = false, in_place = false, ok = true;
    for (int r = 0; r < nranks && ok; ++r) {
        // A written buffer that is exactly this rank's send buffer, or the
        // residual, stands for both: a row is read before it is written.
        bool send_written = false;
        if (residualOut != nullptr) {
            send_written |= residualOut[r] == sendbufs[r];
            residual_written |= residualOut[r] == residual;
            ok = mem.add(residualOut[r], bytes, true);
        }
        if (!eight) {
            send_written |= outbufs[r] == sendbufs[r];
            residual_written |= outbufs[r] == residual;
        }
        ok = ok && mem.add(outbufs[r], eight ? rows * cols : bytes, true);
        if (eight)
            ok = ok && mem.add(scalebufs[r], scale_blocks(cols) * rows * sizeof(float), true);
        ok = ok && (send_written || mem.add(sendbufs[r], bytes, false));
        in_place |= send_written;
    }
    if (residual != nullptr && !residual_written)
        ok = ok && mem.add(residual, bytes, false);
    ok = ok && mem.add(weight, cols * elem_bytes(dtype), false);
    if (!ok || !mem.disjoint())
        return reject(arInvalidArgument, mem.why());
    const arResult_t usage = check_comm(comm);
    if (usage != arSuccess)
        return usage;

    ar::NormArgs args = {};
    for (int r = 0; r < nranks; ++r) {
        args.send[r] = (const char *)sendbufs[r];
        args.res_out[r] = residualOut != nullptr ? (char *)residualOut[r] : nullptr;
        args.out[r] = (char *)outbufs[r];
        args.scales[r] = eight ? scalebufs[r] : nullptr;
    }
    args.residual = (const char *)residual;
    args.weight = (const char *)weight;
    args.rows = rows;
    args.cols = (uint32_t)cols;
    args.nranks = (uint32_t)nranks;
    args.has_res_out = residualOut != nullptr;
    args.in_place = in_place || (residual != nullptr && residual_written);
    args.eps = eps;
    return launched(ar::launch_norm(args, dtype, eight, comm->cu_count, (hipStream_t)stream));
}

arResult_t arGateQuant(const void *const *inbufs, void *const *outbufs, float *const *scalebufs,
                       size_t rows, size_t cols, arDataType_t dtype_arg, arActivation_t act_arg,
                       int nranks, arComm_t comm, arStream_t stream)
{
    const int dtype = raw(dtype_arg), act = raw(act_arg);
    if (!is_dtype(dtype))
        return reject(arUnsupported, "dtype must be bf16, fp16 or fp32");
    if (act != arActNone && act != arActSiLU)
        return reject(arUnsupported, "unknown activation");
    if (nranks < 1 || nranks > AR_MAX_RANKS)
        return reject(arUnsupported, "nranks must be in 1..32");
    if (rows == 0 || cols == 0)
        return arSuccess;
    if (too_large(rows, cols))
        return reject(arInvalidArgument, "rows or cols too large");
    const size_t in = rows * cols * elem_bytes(dtype) * (act == arActSiLU ? 2 : 1);
    Ranges mem;
    if (!mem.add_ranks(inbufs, nranks, in, false) ||
        !mem.add_ranks(outbufs, nranks, rows * cols, true) ||
        !mem.add_ranks((const void *const *)scalebufs, nranks,
                       scale_blocks(cols) * rows * sizeof(float), true) ||
        !mem.disjoint())
        return reject(arInvalidArgument, mem.why());
    const arResult_t usage = check_comm(comm);
    if (usage != arSuccess)
        return usage;

    ar::GateArgs args = {};
    for (int r = 0; r < nranks; ++r) {
        args.in[r] = (const char *)inbufs[r];
        args.out[r] = (char *)outbufs[r];
        args.scales[r] = scalebufs[r];
    }
    args.rows = rows;
    args.cols = cols;
    return launched(ar::launch_gate(args, dtype, act, nranks, comm->cu_count, (hipStream_t)stream));
}

arResult_t arMatmulScaled(const void *const *abufs, const float *const *ascales,
                          const void *const *bbufs, const float *const *bscales,
                          void *const *outbufs, size_t rows, size_t n, size_t k,
                          arDataType_t outDtype_arg, int reduce, int nranks, arComm_t comm,
                          arStream_t stream)
{
    const int dtype = raw(outDtype_arg);
    if (!is_dtype(dtype))
        return reject(arUnsupported, "outDtype must be bf16, fp16 or fp32");
    if (nranks < 1 || nranks > AR_MAX_RANKS)
        return reject(arUnsupported, "nranks must be in 1..32");
    if (k < 16 || k % 16 != 0)
        return reject(arUnsupported, "k must be a positive multiple of 16");
    if (k > ar::kMatmulMaxK)
        return reject(arUnsupported, "k must be at most 2^23");
    if (reduce != 0 && reduce != 1)
        return reject(arInvalidArgument, "reduce must be 0 or 1");
    if (rows == 0 || n == 0)
        return arSuccess;
    const size_t most = (size_t)1 << 30;
    if (rows > most || n > most)
        return reject(arInvalidArgument, "rows and n must be at most 2^30");
    if (rows * n > ((size_t)1 << 38))
        return reject(arInvalidArgument, "rows * n must be at most 2^38");
    if (!ar::matmul_fits(rows, n, dtype))
        return reject(arUnsupported, "more tiles than a launch holds");
    Ranges mem;
    if (!mem.add_ranks(abufs, nranks, rows * k, false) ||
        !mem.add_ranks((const void *const *)ascales, nranks,
                       scale_blocks(k) * rows * sizeof(float), false) ||
        !mem.add_ranks(bbufs, nranks, n * k, false) ||
        !mem.add_ranks((const void *const *)bscales, nranks,
                       scale_blocks(n) * scale_blocks(k) * sizeof(float), false) ||
        !mem.add_ranks(outbufs, nranks, rows * n * elem_bytes(dtype), true) || !mem.disjoint())
        return reject(arInvalidArgument, mem.why());
    const arResult_t usage = check_comm(comm);
    if (usage != arSuccess)
        return usage;

    ar::MatmulArgs args = {};
    for (int r = 0; r < nranks; ++r) {
        args.a[r] = (const char *)abufs[r];
        args.sa[r] = ascales[r];
        args.b[r] = (const char *)bbufs[r];
        args.sb[r] = bscales[r];
        args.out[r] = (char *)outbufs[r];
    }
    args.rows = (uint32_t)rows;
    args.n = (uint32_t)n;
    args.k = (uint32_t)k;
    args.kblocks = (uint32_t)scale_blocks(k);
    args.nranks = (uint32_t)nranks;
    return launched(ar::launch_matmul(args, dtype, reduce != 0, comm->cu_count,
                                      (hipStream_t)stream));
}

// For tests, on the host: which kernel arMatmulScaled launches for a call of
// these sizes on a card of `cu_count` compute units: tile rows and columns (16
// x 16: the kernel for one or two rows), waves that share a tile's k, workgroups
// that do.  0 where the call would be split or refused.
int ar_block_matmul_choice(size_t rows, size_t n, size_t k, int outDtype, int reduce, int nranks,
                           int cu_count, int choice[4])
{
    ar::MatmulArgs args = {};
    args.rows = (uint32_t)rows;
    args.n = (uint32_t)n;
    args.k = (uint32_t)k;
    args.kblocks = (uint32_t)scale_blocks(k);
    args.nranks = (uint32_t)nranks;
    ar::MatmulChoice c;
    if (!ar::choose_matmul(args, outDtype, reduce != 0, cu_count, &c))
        return 0;
    choice[0] = (int)c.rows;
    choice[1] = (int)c.cols;
    choice[2] = (int)c.waves;
    choice[3] = (int)c.split;
    return 1;
}

}  // extern "C"
