// vrc_mx4_matmul.hip -- the product of microscaled 4-bit matrices, summed over
// the ranks' parts of the contraction or one per rank.
//
// C = sum_q A_q B_q^T on the matrix cores: v_mfma_scale_f32_32x32x64 takes, per
// lane, one block of 32 codes of a row of each operand with its scale byte, and
// adds 64 exact products per output to an fp32 accumulator.
#include <hip/hip_runtime.h>

#include "vrc_ops_host.hpp"

namespace vrc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct MatmulArgs {
    const char* ac[kMaxRanks];
    const char* as[kMaxRanks];
    const char* bc[kMaxRanks];
    const char* bs[kMaxRanks];
    char* dst[kMaxRanks];
    uint32_t m, n, kb;
    int ranks;
    uint32_t tiles_n;
};

// One wave a 32 x 32 tile, fed straight from memory.  Lane l has row l % 32 of
// both operands and block l / 32 of each pair; its results are column l % 32,
// rows 8 (i / 4) + 4 (l / 32) + i % 4.
template <class T, bool SUM>
__global__ __launch_bounds__(64) void k_mx4_matmul(MatmulArgs a)
{
    const uint32_t lane = threadIdx.x;
    const uint32_t m0 = blockIdx.x / a.tiles_n * 32, n0 = blockIdx.x % a.tiles_n * 32;
    const uint32_t ra = min(m0 + (lane & 31), a.m - 1), rb = min(n0 + (lane & 31), a.n - 1);
    f32x16 acc = {};
    const int q0 = SUM ? 0 : (int)blockIdx.y, q1 = SUM ? a.ranks : q0 + 1;
    for (int q = q0; q < q1; q++) {
        const uint64_t ia = (uint64_t)ra * a.kb, ib = (uint64_t)rb * a.kb;
        for (uint32_t k = lane >> 5; k < ((a.kb + 1) & ~1u); k += 2) {
            u32x4 x = {}, y = {};
            int sx = 127, sy = 127;
            if (k < a.kb) {
                x = *(global_ptr<const u32x4>)(a.ac[q] + (ia + k) * 16);
                y = *(global_ptr<const u32x4>)(a.bc[q] + (ib + k) * 16);
                sx = *(global_ptr<const uint8_t>)(a.as[q] + ia + k);
                sy = *(global_ptr<const uint8_t>)(a.bs[q] + ib + k);
            }
            const i32x8 p = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
            const i32x8 r = {(int)y.x, (int)y.y, (int)y.z, (int)y.w, 0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(p, r, acc, 4, 4, 0, sx, 0, sy);
        }
    }
    const uint32_t col = n0 + (lane & 31);
    if (col >= a.n) return;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const uint32_t row = m0 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
        if (row >= a.m) continue;
        const typename T::S s = T::narrow(acc[i]);
        const uint64_t at = ((uint64_t)row * a.n + col) * T::ESZ;
        for (int q = SUM ? 0 : q0; q < q1; q++) store_s<T>(a.dst[q] + at, s);
    }
}

using namespace host;

template <class T>
vrc_status_t matmul_typed(const MatmulArgs& a, bool sum, int cus, hipStream_t st)
{
    (void)cus;
    const uint64_t tiles = (uint64_t)((a.m + 31) / 32) * a.tiles_n;
    if (tiles > 0x7fffffffull) return VRC_ERR_INVALID_ARG;
    if (sum) k_mx4_matmul<T, true><<<dim3((unsigned)tiles), 64, 0, st>>>(a);
    else k_mx4_matmul<T, false><<<dim3((unsigned)tiles, (unsigned)a.ranks), 64, 0, st>>>(a);
    return check_launch();
}

}  // namespace

namespace host {

vrc_status_t run_mx4_matmul(const char* const* ac, const char* const* as, const char* const* bc, const char* const* bs,
                            char* const* y, int n, uint64_t m, uint64_t cols, uint64_t kblocks, vrc_dtype_t dt,
                            bool sum, int cus, hipStream_t st)
{
    MatmulArgs a = {};
    for (int r = 0; r < n; r++) {
        a.ac[r] = ac[r];
        a.as[r] = as[r];
        a.bc[r] = bc[r];
        a.bs[r] = bs[r];
        a.dst[r] = y[r];
    }
    a.m = (uint32_t)m;
    a.n = (uint32_t)cols;
    a.kb = (uint32_t)kblocks;
    a.ranks = n;
    a.tiles_n = (a.n + 31) / 32;
    switch (dt) {
    case VRC_FP32: return matmul_typed<F32>(a, sum, cus, st);
    case VRC_FP16: return matmul_typed<F16>(a, sum, cus, st);
    case VRC_BF16: return matmul_typed<BF16>(a, sum, cus, st);
    default: return VRC_ERR_UNSUPPORTED;
    }
}

}  // namespace host
}  // namespace vrc
