// vrc_ops_host.hpp -- host-side pieces of libvrc_ops.so: the operators'
// internal entry points (one per source file), buffer checks and the 32-bit
// division by a launch constant.  Internal; the C ABI is include/vrc_ops.h.
#pragma once

#include <atomic>
#include <cstring>

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

// Grids of many workgroups.  A grid has less than 2^32 work items along each
// axis, so workgroups beyond kWideX (of up to 1024 lanes) go along z.  blockIdx.y is
// the caller's; the last workgroups may have no tile.
constexpr uint64_t kWideX = 1ull << 21;

__host__ inline dim3 wide_grid(uint64_t tiles, int y)
{
    return dim3((unsigned)(tiles < kWideX ? tiles : kWideX), (unsigned)y, (unsigned)((tiles + kWideX - 1) / kWideX));
}

__device__ __forceinline__ uint32_t wide_tile() { return blockIdx.z * (uint32_t)kWideX + blockIdx.x; }

namespace host {

constexpr int kMaxDevices = 64;
inline std::atomic<int> g_cu_count[kMaxDevices];

inline hipError_t cu_count(int* out)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) {
        int c = g_cu_count[dev].load(std::memory_order_relaxed);
        if (c > 0) {
            *out = c;
            return hipSuccess;
        }
    }
    int c = 0;
    e = hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    if (c < 1) c = 1;
    if (dev >= 0 && dev < kMaxDevices) g_cu_count[dev].store(c, std::memory_order_relaxed);
    *out = c;
    return hipSuccess;
}

inline bool overlap(uintptr_t a, uint64_t na, uintptr_t b, uint64_t nb)
{
    if (na == 0 || nb == 0) return false;
    return a < b + nb && b < a + na;
}

// Counts above 2^56 elements are rejected: every byte size computed from
// them (at most count * 16 ranks * 4 bytes) then fits in 64 bits.
constexpr uint64_t kMaxCount = 1ull << 56;

// The enum arguments of the C ABI hold whatever int a C caller passes.  In
// C++ an enum object whose value lies outside its enumerators' range may not
// be read as that enum, so every entry point reads them as plain ints (from
// the object's bytes) and the implementations check the ints before turning
// them back into enums.
template <class E>
inline int raw(const E& e)
{
    static_assert(sizeof(E) == sizeof(int), "the C enums of vrc.h are int-sized");
    int v;
    std::memcpy(&v, &e, sizeof v);
    return v;
}

inline bool dtype_valid(int d) { return d >= VRC_INT32 && d <= VRC_BF16; }

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
