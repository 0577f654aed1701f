// vrc_ops_host.hpp -- host-side pieces of libvrc_ops.so: the operators'
// internal entry points (one per source file), buffer checks and the 32-bit
// division by a launch constant.  Internal; the C ABI is include/vrc_ops.h.
#pragma once

#include "vrc_host.hpp"
#include "vrc_ops.h"

namespace vrc {

// n / d for n < 2^31 and a divisor known at launch: with L = ceil(log2 d) and
// m = ceil(2^(31+L) / d), m fits 32 bits and floor(n * m / 2^(31+L)) is exact
// (n * m < 2^63).  A 64-bit division takes over 100 instructions per lane.
struct FastDiv {
    uint32_t m, s;
    __host__ static FastDiv of(uint64_t d)
    {
        FastDiv f = {0, 0};
        if (d == 0 || d > 0x7fffffffull) return f;
        uint32_t lg = 0;
        while ((1ull << lg) < d) lg++;
        f.m = (uint32_t)((((unsigned __int128)1 << (31 + lg)) + d - 1) / d);
        f.s = 31 + lg;
        return f;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> s); }
};

namespace host {

// One buffer of an operator's call.
struct Buf {
    uintptr_t p;
    uint64_t bytes;
};

// Outputs against every other buffer: out[i] may be in[j] itself only where
// same(i, j) says so (same address and the same layout); outputs never overlap
// each other.
template <class Same>
vrc_status_t check_outputs(const Buf* out, int n_out, const Buf* in, int n_in, Same same)
{
    for (int i = 0; i < n_out; i++) {
        for (int j = 0; j < n_in; j++) {
            if (!overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) continue;
            if (out[i].p == in[j].p && out[i].bytes == in[j].bytes && same(i, j)) continue;
            return VRC_ERR_ALIAS;
        }
        for (int j = 0; j < i; j++)
            if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return VRC_ERR_ALIAS;
    }
    return VRC_OK;
}

// Read the device's CU count and clear the thread's pending HIP error, as
// every launching call of the library does first.
inline vrc_status_t begin_launch(int* cus)
{
    const hipError_t e = cu_count(cus);
    if (e != hipSuccess) return hip_fail(e);
    (void)hipGetLastError();
    return VRC_OK;
}

inline bool float_dtype(int d) { return d == VRC_FP32 || d == VRC_FP16 || d == VRC_BF16; }

// The mask of one call, as its kernels take it.
struct MaskArgs {
    uint64_t seed, offset;
    const uint64_t* offset_dev;  // added to offset when the kernel runs
    float scale;
    uint32_t thr;   // a word below it drops its element
    uint32_t kind;  // 0: nothing is dropped, 1: by the generator, 2: everything is dropped
};

// Launchers, on checked arguments.  residual: null for none.
vrc_status_t run_allreduce_dropout(const char* const* x, const char* const* res, char* const* y, int n, uint64_t count,
                                   vrc_dtype_t dt, const MaskArgs& m, int cus, hipStream_t st);
vrc_status_t run_reduce_scatter_dropout(const char* const* x, const char* const* res, char* const* y, int n,
                                        uint64_t count, uint64_t outer, vrc_dtype_t dt, const MaskArgs& m, int cus,
                                        hipStream_t st);
vrc_status_t run_all_gather_dropout(const char* const* x, char* const* y, int n, uint64_t total, uint64_t outer,
                                    vrc_dtype_t dt, const MaskArgs& m, int cus, hipStream_t st);
vrc_status_t run_mx4_quantize(const char* const* x, char* const* codes, char* const* scales, int n, uint64_t rows,
                              uint64_t cols, vrc_dtype_t dt, bool along_rows, int cus, hipStream_t st);
// Rank q's block (row, j) decodes to row `row` and column 32 j of slab q: at
// q * slab + row * stride elements of each of the n_out outputs, or of y[q]
// alone where n_out == 0.
vrc_status_t run_mx4_decode(const char* const* codes, const char* const* scales, char* const* y, int n, int n_out,
                            uint64_t rows, uint64_t cols, uint64_t slab, uint64_t stride, vrc_dtype_t dt, int cus,
                            hipStream_t st);
vrc_status_t run_mx4_matmul(const char* const* ac, const char* const* as, const char* const* bc, const char* const* bs,
                            char* const* y, int n, uint64_t m, uint64_t cols, uint64_t kblocks, vrc_dtype_t dt,
                            bool sum, int cus, hipStream_t st);

}  // namespace host
}  // namespace vrc
