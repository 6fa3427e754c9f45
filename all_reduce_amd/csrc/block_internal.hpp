// block_internal.hpp -- what the entry points of ar_block.h and their kernel
// files share.
#pragma once

#include "ar_allreduce.h"
#include "ar_block.h"
#include "ar_internal.hpp"

namespace ar {

// Rank tables of the block operators, passed by value in the kernel arguments
// and indexed at run time: the index is the same in every lane, so a pointer
// is one scalar load, and one kernel serves every rank count.
struct NormArgs {
    const char *send[AR_MAX_RANKS];
    char *res_out[AR_MAX_RANKS];  // unused where has_res_out is 0
    char *out[AR_MAX_RANKS];
    float *scales[AR_MAX_RANKS];  // unused for an output in the element type
    const char *residual;         // nullptr: none
    const char *weight;
    uint64_t rows;
    uint32_t cols;
    uint32_t nranks;
    uint32_t has_res_out;
    uint32_t in_place;  // a written buffer is also a read one
    uint32_t split;     // workgroups a row (the launcher sets it)
    float eps;
};

struct GateArgs {
    const char *in[AR_MAX_RANKS];
    char *out[AR_MAX_RANKS];
    float *scales[AR_MAX_RANKS];
    uint64_t rows;
    uint64_t cols;
    uint32_t tall;  // rows a workgroup takes at once (the launcher sets it)
};

struct MatmulArgs {
    const char *a[AR_MAX_RANKS];
    const float *sa[AR_MAX_RANKS];
    const char *b[AR_MAX_RANKS];
    const float *sb[AR_MAX_RANKS];
    char *out[AR_MAX_RANKS];
    uint32_t rows;
    uint32_t n;
    uint32_t k;
    uint32_t kblocks;  // ceil(k / 128)
    uint32_t nranks;
    uint32_t split;    // workgroups that share a tile's k (the launcher sets it)
};

// Launchers: validate nothing (the entry points did), pick the kernel and
// enqueue it on `stream`.
hipError_t launch_norm(const NormArgs &args, int dtype, bool eight, int cu_count,
                       hipStream_t stream);
hipError_t launch_gate(const GateArgs &args, int dtype, int act, int nranks, int cu_count,
                       hipStream_t stream);
hipError_t launch_matmul(const MatmulArgs &args, int out_dtype, bool reduce, int cu_count,
                         hipStream_t stream);
// What it launches: tiles of rows x cols (16 x 16: the kernel for one or two
// rows; from 128 x 128 on the ones for many), the waves that share a tile's k
// and the workgroups that do.  False where no kernel's launch holds the tiles;
// it then takes the ranks in two launches.  One rank's tiles (or all, summed)
// fit where matmul_fits says so.
struct MatmulChoice {
    uint32_t rows, cols, waves, split;
};
bool choose_matmul(const MatmulArgs &args, int out_dtype, bool reduce, int cu_count,
                   MatmulChoice *choice);
bool matmul_fits(uint64_t rows, uint64_t n, int out_dtype);
// Its kernels for a batch of rows (block_matmul_mid.hip; mt, nt: tiles of 32
// rows and columns, 1 and 1, 2 and 1 or 2 and 2) and for many
// (block_matmul_tile.hip; tiles of 256 x 256 or 128 x 128).  Their 32-bit
// offsets inside a tile limit k.  `split` > 1: that many workgroups share the k
// of a tile, in the summed form only, and at most matmul_most_split of them.
constexpr uint32_t kMatmulMaxK = 1u << 23;
inline uint32_t matmul_most_split(int out_dtype, uint32_t nranks)
{
    return out_dtype == kFp32 ? nranks : nranks / 2u > 0u ? nranks / 2u : 1u;
}
hipError_t launch_matmul_mid(const MatmulArgs &args, int out_dtype, bool reduce, int mt, int nt,
                             uint32_t waves, uint32_t split, hipStream_t stream);
hipError_t launch_matmul_tile(const MatmulArgs &args, int out_dtype, bool reduce, bool large,
                              hipStream_t stream);

}  // namespace ar
