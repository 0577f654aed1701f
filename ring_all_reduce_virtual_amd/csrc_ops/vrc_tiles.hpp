// vrc_tiles.hpp -- a tile of a matrix product on the matrix cores, whose operands
// come into a ring of stages in LDS by direct loads.  Internal.
//
// acc += A B over a walk of the contraction in tiles of KT elements (128 bytes of
// a row).  An operand lies in memory either along the contraction (ALONG: [rows,
// k], k contiguous) or across it (ACROSS: [k, columns], columns contiguous); the
// result is the same, so no operand is ever transposed in memory:
//   * ALONG: LDS holds a row's eight 16-byte granules with granule j at place j ^
//     (row / 2 mod 8), so that the rows a matrix operand reads at one granule spread
//     over all banks;
//   * ACROSS: LDS holds the tile's KT rows of B columns.  16-bit operands are read
//     by ds_read_b64_tr_b16: of each 16 lanes, lane j addresses row j / 4 and four
//     columns from 4 (j mod 4), and receives column j of the four rows.  Runs of 32
//     columns are permuted within a row by the row's number, so that the rows that
//     one read takes lie on other banks.  32-bit operands are read element by element.
// Both loads permute their global addresses to that end, as a direct load writes
// consecutive lanes to consecutive places.
//
// B is the instruction's first operand, so that a lane's results are four
// consecutive columns (of B) of a row (of A).
#pragma once

#include "vrc_elem.hpp"

namespace vrc {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kAlong = 0, kAcross = 1;
constexpr uint32_t kTileRow = 128;  // bytes of the contraction in a tile
template <class T>
constexpr uint32_t kTileK = kTileRow / T::ESZ;

// What is read in place of elements past the end of the contraction.
__device__ const u32x4 kZeroGranule = {0, 0, 0, 0};

// `x`, whose origin the compiler is not to see: an address is then a uniform base
// and a 32-bit lane offset, instead of a 64-bit address per lane and load kept in
// registers over the whole loop.
__device__ __forceinline__ uint32_t hidden_offset(uint32_t x)
{
    __asm__ volatile("" : "+v"(x));
    return x;
}

// A barrier behind this wave's LDS reads and writes, with its direct loads left
// under way (__syncthreads() may wait for them).
__device__ __forceinline__ void tile_barrier()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// 16 bytes a lane, lane l's to place l after `to`.
__device__ __forceinline__ void granules_to_lds(global_ptr<const char> from, char* to)
{
    __builtin_amdgcn_global_load_lds((global_ptr<const void>)from, (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Workgroup b's tile.  Workgroups are handed to the 8 XCDs in turn; each XCD takes
// a run of consecutive tiles, in groups of G rows of tiles walked column by
// column, so that the tiles it works on at once share their operands in its L2.
template <uint32_t G>
__device__ __forceinline__ void xcd_tile(uint32_t b, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn)
{
    const uint32_t total = tiles_m * tiles_n, each = total / 8, more = total % 8, x = b % 8;
    const uint32_t t = x * each + (x < more ? x : more) + b / 8;
    const uint32_t group = t / (G * tiles_n), left = tiles_m - group * G, rows = left < G ? left : G;
    const uint32_t i = t - group * G * tiles_n;
    tm = group * G + i % rows;
    tn = i / rows;
}

// F matrix operands of 16-bit elements read across: for each, two transposing reads of four
// rows at a lane's address `at` and at OFF and STEP bytes behind it.  As assembly with its own
// wait: the compiler takes the builtin for an access that direct loads to LDS may write, and
// waits for all of those, the next tile's, before every one (4096 x 16384 x 4096: the
// weights' gradients 528 us with the builtin, 460 with this).  The tile's barrier orders both.
template <int F, int OFF, int STEP>
__device__ __forceinline__ void read_across(const uint32_t (&at)[F], u32x4 (&out)[F])
{
    u32x2 a[F], b[F];
#define VRC_TR(d, s, o) "ds_read_b64_tr_b16 %" #d ", %" #s " offset:%" #o "\n\t"
    static_assert(F == 1 || F == 2 || F == 4 || F == 6, "operands of a wave");
    if constexpr (F == 1) {
        __asm__ volatile(VRC_TR(0, 2, 3) VRC_TR(1, 2, 4) "s_waitcnt lgkmcnt(0)"
                         : "=&v"(a[0]), "=&v"(b[0]) : "v"(at[0]), "n"(OFF), "n"(OFF + STEP) : "memory");
    } else if constexpr (F == 2) {
        __asm__ volatile(VRC_TR(0, 4, 6) VRC_TR(1, 4, 7) VRC_TR(2, 5, 6) VRC_TR(3, 5, 7) "s_waitcnt lgkmcnt(0)"
                         : "=&v"(a[0]), "=&v"(b[0]), "=&v"(a[1]), "=&v"(b[1])
                         : "v"(at[0]), "v"(at[1]), "n"(OFF), "n"(OFF + STEP) : "memory");
    } else if constexpr (F == 4) {
        __asm__ volatile(VRC_TR(0, 8, 12) VRC_TR(1, 8, 13) VRC_TR(2, 9, 12) VRC_TR(3, 9, 13) VRC_TR(4, 10, 12) VRC_TR(5, 10, 13)
                         VRC_TR(6, 11, 12) VRC_TR(7, 11, 13) "s_waitcnt lgkmcnt(0)"
                         : "=&v"(a[0]), "=&v"(b[0]), "=&v"(a[1]), "=&v"(b[1]), "=&v"(a[2]), "=&v"(b[2]), "=&v"(a[3]), "=&v"(b[3])
                         : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF), "n"(OFF + STEP) : "memory");
    } else {
        __asm__ volatile(VRC_TR(0, 12, 18) VRC_TR(1, 12, 19) VRC_TR(2, 13, 18) VRC_TR(3, 13, 19) VRC_TR(4, 14, 18) VRC_TR(5, 14, 19)
                         VRC_TR(6, 15, 18) VRC_TR(7, 15, 19) VRC_TR(8, 16, 18) VRC_TR(9, 16, 19) VRC_TR(10, 17, 18) VRC_TR(11, 17, 19)
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(a[0]), "=&v"(b[0]), "=&v"(a[1]), "=&v"(b[1]), "=&v"(a[2]), "=&v"(b[2]), "=&v"(a[3]), "=&v"(b[3]),
                           "=&v"(a[4]), "=&v"(b[4]), "=&v"(a[5]), "=&v"(b[5])
                         : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]), "n"(OFF), "n"(OFF + STEP)
                         : "memory");
    }
#undef VRC_TR
#pragma unroll
    for (int f = 0; f < F; f++) out[f] = u32x4{a[f].x, a[f].y, b[f].x, b[f].y};
}

// One operand of a tile: B rows (ALONG) or columns (ACROSS).
template <class T, int KIND, int B>
struct TileOperand {
    static constexpr uint32_t KT = kTileK<T>;
    static constexpr uint32_t BYTES = B * kTileRow;             // of a stage
    static constexpr uint32_t LOADS = BYTES / 1024;             // by a wave, 64 granules each
    static constexpr uint32_t ROW = B * T::ESZ, ROW_GRANULES = ROW / 16;  // ACROSS
    static constexpr uint32_t RUN = 32 * T::ESZ, RUNS = B / 32;          // bytes of 32 columns; such runs in a row

    // Where run `run` of row k lies.
    static __device__ __forceinline__ uint32_t run_place(uint32_t run, uint32_t k)
    {
        if constexpr (T::ESZ == 4) return RUNS >= 2 ? run ^ (k >> 2 & 1) : run;
        else return RUNS >= 4 ? run ^ (k & 3) : RUNS == 2 ? run ^ (k >> 1 & 1) : run;
    }

    // Granule `g` (of the stage, in LDS order): its offset in memory from the tile's
    // first element, and its element of the contraction (ALONG: the first).  pitch: bytes
    // of a row in memory.  `last`: the last row (ALONG) or granule of a row (ACROSS)
    // that there is; those past it read it again.
    static __device__ __forceinline__ void source(uint32_t g, uint32_t pitch, uint32_t last, uint32_t& offset, uint32_t& k)
    {
        if constexpr (KIND == kAlong) {
            const uint32_t row = g / 8, j = (g & 7) ^ (row >> 1 & 7);
            offset = (row < last ? row : last) * pitch + j * 16;
            k = j * (16 / T::ESZ);
        } else {
            constexpr uint32_t RG = RUN / 16;
            k = g / ROW_GRANULES;
            const uint32_t p = g % ROW_GRANULES, j = run_place(p / RG, k) * RG + p % RG;
            offset = k * pitch + (j < last ? j : last) * 16;
        }
    }

    // ACROSS of 16 bits: what read_across() takes of columns c0 .. c0 + 31 at step 0; a
    // step is 16 rows on.
    static constexpr bool TRANSPOSED = KIND == kAcross && T::ESZ == 2;
    static __device__ __forceinline__ uint32_t across_at(uint32_t c0, uint32_t lane)
    {
        const uint32_t j = lane & 15, k = 8 * (lane >> 5) + j / 4;
        return k * ROW + run_place(c0 / 32, k) * RUN + (lane >> 4 & 1) * 32 + (j & 3) * 8;
    }

    // Else a lane's operand of step s (of four): rows or columns c0 .. c0 + 31, one a lane;
    // elements 2 s + half granules on.
    static __device__ __forceinline__ u32x4 read(const char* stage, uint32_t c0, int s, uint32_t lane)
    {
        const uint32_t half = lane >> 5;
        if constexpr (KIND == kAlong) {
            const uint32_t row = c0 + (lane & 31);
            return *(const u32x4*)(stage + row * kTileRow + (((2 * s + half) ^ (row >> 1 & 7)) * 16));
        } else {
            const uint32_t k = 8 * s + 4 * half;
            const char* at = stage + k * ROW + run_place(c0 / 32, k) * RUN + (lane & 31) * 4;
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = *(const uint32_t*)(at + e * ROW);
            return v;
        }
    }
};

// acc += the products of one step.
template <class T>
__device__ __forceinline__ f32x16 tile_mfma(u32x4 b, u32x4 a, f32x16 acc)
{
    if constexpr (T::ESZ == 4) {
#pragma unroll
        for (int e = 0; e < 4; e++)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(b[e]), __uint_as_float(a[e]), acc, 0, 0, 0);
        return acc;
    } else if constexpr (__is_same(T, BF16)) {
        typedef __bf16 v8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, b), __builtin_bit_cast(v8, a), acc, 0, 0, 0);
    } else {
        typedef _Float16 v8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, b), __builtin_bit_cast(v8, a), acc, 0, 0, 0);
    }
}

// The column, among a tile of 32, of a lane's result e.
__device__ __forceinline__ uint32_t result_col(int e, uint32_t half) { return 8 * (e / 4) + 4 * half + e % 4; }

}  // namespace vrc
