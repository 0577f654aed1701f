// vrc_mx4.hip -- microscaled 4-bit blocks: quantisation along either axis, and
// decoding (each rank's own matrix, or the gather of all of them).
//
// A block of 32 values shares 2^X, X = floor(log2 max|v|) - 2: the exponent
// field of the largest magnitude less two, so no logarithm is taken.  v / 2^X is
// exact (a power of two) and rounded to E2M1 by the target's conversions, which
// equal the definition (nearest, ties to even, saturating at 6) on every finite
// fp16 and bf16 value under every scale.  Both directions are streams: 2 or 4
// bytes a value on one side, 17/32 on the other.
#include <hip/hip_runtime.h>

#include "vrc_ops_host.hpp"

namespace vrc {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Two values to two codes in byte SEL of `old`, two codes to two values.  `s` is
// the scale's byte in a float's exponent field (byte 0, a zero there, stands for
// 2^-127 to these conversions; byte 255 decodes to NaN).
template <class T>
struct Mx4;

template <>
struct Mx4<F32> {
    template <int SEL>
    __device__ static uint32_t encode(uint32_t old, uint32_t a, uint32_t b, float s)
    {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __uint_as_float(a), __uint_as_float(b), s, SEL);
    }
};

template <>
struct Mx4<BF16> {
    template <int SEL>
    __device__ static uint32_t encode(uint32_t old, uint32_t pair, float s)
    {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), s, SEL);
    }
    template <int SEL>
    __device__ static uint32_t decode(uint32_t codes, float s)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, SEL));
    }
};

template <>
struct Mx4<F16> {
    template <int SEL>
    __device__ static uint32_t encode(uint32_t old, uint32_t pair, float s)
    {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, pair), s, SEL);
    }
    template <int SEL>
    __device__ static uint32_t decode(uint32_t codes, float s)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, SEL));
    }
};

constexpr uint32_t kNanScale = 255;

// The scale byte of a block whose largest magnitude has the bits m (sign
// cleared): the exponent as a float's, less two, at least 0; 255 where m is an
// infinity's or a NaN's.
template <class T>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m)
{
    uint32_t e;
    if constexpr (T::ESZ == 4) e = m >> 23;
    else if constexpr (std::is_same<T, BF16>::value) e = m >> 7;
    else e = m >= 0x7c00u ? 255u : __float_as_uint(F16::widen((uint16_t)m)) >> 23;
    return e == 255u ? kNanScale : (e > 2u ? e - 2u : 0u);
}

__device__ __forceinline__ float scale_float(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(
        uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// The larger of x over a lane's quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t x)
{
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xf, 0xf, true);  // lanes 1 0 3 2
    x = x > y ? x : y;
    const uint32_t z = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xf, 0xf, true);  // lanes 2 3 0 1
    return x > z ? x : z;
}

// Eight consecutive values as they are stored: ESZ * 8 bytes.
template <class T>
struct Eight {
    static constexpr int D = T::ESZ * 2;  // dwords
    uint32_t w[D];

    __device__ __forceinline__ void load(const char* p)
    {
#pragma unroll
        for (int i = 0; i < D / 4; i++) {
            const u32x4 v = ld16<true>(p + 16 * i);
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    }
    // The first `left` of them, zero after.
    __device__ __forceinline__ void load_part(const char* p, int left)
    {
#pragma unroll
        for (int i = 0; i < D; i++) w[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (i >= left) continue;
            const uint32_t s = load_s<T>(p + i * T::ESZ);
            if constexpr (T::ESZ == 4) w[i] = s;
            else w[i / 2] |= s << (16 * (i & 1));
        }
    }
    // Bits of the largest magnitude.
    __device__ __forceinline__ uint32_t top() const
    {
        constexpr uint32_t ABS = T::ESZ == 4 ? 0x7fffffffu : 0x7fff7fffu;
        uint32_t m = w[0] & ABS;
#pragma unroll
        for (int i = 1; i < D; i++) {
            const uint32_t x = w[i] & ABS;
            if constexpr (T::ESZ == 4) m = m > x ? m : x;
            else m = max_u16x2(m, x);
        }
        if constexpr (T::ESZ == 2) m = (m >> 16) > (m & 0xffffu) ? m >> 16 : m & 0xffffu;
        return m;
    }
    __device__ __forceinline__ uint32_t encode(float s) const
    {
        uint32_t c = 0;
        if constexpr (T::ESZ == 4) {
            c = Mx4<T>::template encode<0>(c, w[0], w[1], s);
            c = Mx4<T>::template encode<1>(c, w[2], w[3], s);
            c = Mx4<T>::template encode<2>(c, w[4], w[5], s);
            c = Mx4<T>::template encode<3>(c, w[6], w[7], s);
        } else {
            c = Mx4<T>::template encode<0>(c, w[0], s);
            c = Mx4<T>::template encode<1>(c, w[1], s);
            c = Mx4<T>::template encode<2>(c, w[2], s);
            c = Mx4<T>::template encode<3>(c, w[3], s);
        }
        return c;
    }
};

// ---------------------------------------------------------------------------
// Quantisation along the rows.  A quad of lanes has a block, eight values a
// lane: 16-byte loads (two for fp32) and 4-byte stores, consecutive over the
// wave, and the block's maximum in two lane exchanges.  A lane keeps U groups'
// loads in flight.  blockIdx.y is the rank.
// FLAT: cols is a multiple of 32, so block b starts at value 32 b.
// ---------------------------------------------------------------------------
struct QuantArgs {
    const char* src[kMaxRanks];
    char* codes[kMaxRanks];
    char* scales[kMaxRanks];
    uint64_t cols, kb;
    uint64_t groups;  // rows * kb * 4
    FastDiv by_kb;
};

template <class T, bool FLAT>
__global__ __launch_bounds__(256) void k_mx4_quantize(QuantArgs a)
{
    constexpr int U = 4;
    constexpr uint64_t E = T::ESZ;
    const char* src = a.src[blockIdx.y];
    const auto codes = (global_ptr<uint32_t>)a.codes[blockIdx.y];
    const auto scales = (global_ptr<uint8_t>)a.scales[blockIdx.y];
    const uint64_t step = (uint64_t)gridDim.x * 256 * U;
    for (uint64_t g0 = (uint64_t)blockIdx.x * 256 * U + threadIdx.x; g0 < a.groups; g0 += step) {
        Eight<T> x[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint64_t g = g0 + u * 256;
            if (g >= a.groups) continue;
            if constexpr (FLAT) {
                x[u].load(src + g * 8 * E);
            } else {
                const uint64_t b = g >> 2;
                const uint64_t row = (a.groups >> 33) ? b / a.kb : a.by_kb.div((uint32_t)b);
                const uint64_t col = (b - row * a.kb) * 32 + (g & 3) * 8;
                const int64_t left = (int64_t)a.cols - (int64_t)col;
                const char* p = src + (row * a.cols + col) * E;
                if (left >= 8) x[u].load(p);
                else x[u].load_part(p, left > 0 ? (int)left : 0);
            }
        }
        issue_loads_first();
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint64_t g = g0 + u * 256;
            if (g >= a.groups) continue;
            const uint32_t byte = scale_byte<T>(quad_max(x[u].top()));
            codes[g] = byte == kNanScale ? 0u : x[u].encode(scale_float(byte));
            if ((g & 3) == 0) scales[g >> 2] = (uint8_t)byte;
        }
    }
}

// ---------------------------------------------------------------------------
// Quantisation down the columns, stored transposed.  A workgroup has 256 rows
// (eight blocks) of 64 C columns, a wave two of the blocks.  A lane has one dword
// of every row (C = 2 columns of a 16-bit type, 1 of fp32) and reads a block's 32
// rows, each a consecutive run over the wave; the maximum needs no exchange.
// Codes and scales go out through LDS, so that a column's eight blocks, 128 bytes
// of its row of codes and eight of its scales, leave at once: stored by the lanes
// that made them, 16 bytes and one byte at a time on different rows, 2 x 8200 x
// 4100 bf16 took 73 us instead of 39 us.
// The values are read past the caches, and codes that fill memory lines are written
// past them, which leaves the scales' eight-byte pieces in L2 until their neighbours
// join them: 8192 x 8192 fp32 71 -> 62 us, bf16 45 -> 36, 8 x (8192 x 4096) bf16 142 ->
// 122 (137 with cached codes); 2 x 8200 x 4100, codes off the lines, 47 -> 40 (52 if
// those went past the caches too).
// blockIdx.y is the rank.  LINES: a tile's codes of a column are a whole memory line.
// ---------------------------------------------------------------------------
struct QuantTArgs {
    const char* src[kMaxRanks];
    char* codes[kMaxRanks];
    char* scales[kMaxRanks];
    uint64_t rows, cols, kb;
    uint32_t col_tiles, tiles;
};

// Workgroups are handed to the 8 XCDs in turn; each XCD takes a run of consecutive
// tiles, whose neighbours share the memory lines at their edges.
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t total)
{
    const uint32_t each = total / 8, more = total % 8, x = b % 8;
    return x * each + (x < more ? x : more) + b / 8;
}

template <class T, bool LINES>
__global__ __launch_bounds__(256) void k_mx4_quantize_t(QuantTArgs a)
{
    constexpr uint64_t E = T::ESZ;
    constexpr int C = 4 / T::ESZ;  // columns per lane
    constexpr uint32_t COLS = 64 * C;
    __shared__ u32x4 out_codes[COLS][8];  // block b of column c at b ^ (c / C mod 8), against bank conflicts
    __shared__ __attribute__((aligned(8))) uint8_t out_scales[COLS][8];
    if (wide_tile() >= a.tiles) return;
    const uint32_t tile = xcd_run(wide_tile(), a.tiles);
    const uint64_t rt = tile / a.col_tiles, col0 = (uint64_t)(tile % a.col_tiles) * COLS;
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t col = col0 + lane * C;
    const uint64_t row_bytes = a.cols * E;
    if (col < a.cols) {
        // The last lane of an odd count of 16-bit columns reads its column and the
        // one before, and shifts; a single column is read by itself.
        const bool whole = col + C <= a.cols;
        const bool single = C == 2 && a.cols == 1;
        const uint32_t shift = whole || single ? 0 : 16;
        const char* src = a.src[blockIdx.y] + (shift ? col - 1 : col) * E;
        for (uint32_t k = 0; k < 2; k++) {
            const uint32_t lb = (threadIdx.x >> 6) + 4 * k;
            const uint64_t b = rt * 8 + lb;
            if (b >= a.kb) break;
            // Rows past the end read the last row again and count as zeros.
            const uint64_t left = a.rows - b * 32;
            const uint32_t last = left < 32 ? (uint32_t)left - 1 : 31;
            const char* p = src + b * 32 * row_bytes;
            uint32_t x[32];
#pragma unroll
            for (uint32_t i = 0; i < 32; i++) {
                typedef uint32_t u32_any __attribute__((aligned(2)));
                const char* at = p + (i < last ? i : last) * row_bytes;
                if (single) x[i] = load_s<T>(at);
                else x[i] = __builtin_nontemporal_load((global_ptr<const u32_any>)at);
            }
            issue_loads_first();
#pragma unroll
            for (uint32_t i = 0; i < 32; i++) x[i] = i <= last ? x[i] >> shift : 0;
            constexpr uint32_t ABS = C == 1 ? 0x7fffffffu : 0x7fff7fffu;
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 32; i++) {
                const uint32_t m = x[i] & ABS;
                if constexpr (C == 1) top = top > m ? top : m;
                else top = max_u16x2(top, m);
            }
#pragma unroll
            for (int c = 0; c < C; c++) {
                const uint32_t byte = scale_byte<T>(C == 1 ? top : (c ? top >> 16 : top & 0xffffu));
                const float s = scale_float(byte);
                uint32_t w[4];
#pragma unroll
                for (int d = 0; d < 4; d++) {
                    uint32_t code = 0;
                    if constexpr (C == 1) {
                        code = Mx4<T>::template encode<0>(code, x[8 * d], x[8 * d + 1], s);
                        code = Mx4<T>::template encode<1>(code, x[8 * d + 2], x[8 * d + 3], s);
                        code = Mx4<T>::template encode<2>(code, x[8 * d + 4], x[8 * d + 5], s);
                        code = Mx4<T>::template encode<3>(code, x[8 * d + 6], x[8 * d + 7], s);
                    } else {
                        // column c of two rows side by side
                        const auto pair = [&](int i) {
                            return c ? (x[i] >> 16) | (x[i + 1] & 0xffff0000u) : (x[i] & 0xffffu) | (x[i + 1] << 16);
                        };
                        code = Mx4<T>::template encode<0>(code, pair(8 * d), s);
                        code = Mx4<T>::template encode<1>(code, pair(8 * d + 2), s);
                        code = Mx4<T>::template encode<2>(code, pair(8 * d + 4), s);
                        code = Mx4<T>::template encode<3>(code, pair(8 * d + 6), s);
                    }
                    w[d] = byte == kNanScale ? 0u : code;
                }
                out_codes[lane * C + c][lb ^ (lane & 7)] = u32x4{w[0], w[1], w[2], w[3]};
                out_scales[lane * C + c][lb] = (uint8_t)byte;
            }
        }
    }
    __syncthreads();
    const uint64_t b0 = rt * 8;
    const uint32_t blocks = a.kb - b0 < 8 ? (uint32_t)(a.kb - b0) : 8;
    const uint32_t cols = a.cols - col0 < COLS ? (uint32_t)(a.cols - col0) : COLS;
    char* codes = a.codes[blockIdx.y] + (col0 * a.kb + b0) * 16;
    char* scales = a.scales[blockIdx.y] + col0 * a.kb + b0;
    for (uint32_t v = threadIdx.x; v < cols * 8; v += 256) {
        const uint32_t c = v / 8, b = v % 8;
        if (b >= blocks) continue;
        const u32x4 x = out_codes[c][b ^ (c / C & 7)];
        const auto to = (global_ptr<u32x4>)(codes + (c * a.kb + b) * 16);
        if constexpr (LINES) __builtin_nontemporal_store(x, to);
        else *to = x;
    }
    if (threadIdx.x < cols) {
        char* to = scales + threadIdx.x * a.kb;
        typedef uint64_t u64_any __attribute__((aligned(1)));
        if (blocks == 8) {
            *(global_ptr<u64_any>)to = *(const uint64_t*)out_scales[threadIdx.x];
        } else {
            for (uint32_t b = 0; b < blocks; b++) *(global_ptr<uint8_t>)(to + b) = out_scales[threadIdx.x][b];
        }
    }
}

// ---------------------------------------------------------------------------
// Decoding.  A lane has one vector of the output's type (eight codes, or four for
// fp32), written to every output: a wave's stores fill whole lines.  (With eight codes
// a lane in fp32 too, 32 bytes in two stores, each wrote half of every line: gather of
// 8 x [20480, 128] 300 us, and 540 us where the halves were kept apart by THROTTLE.)
// blockIdx.y is the rank whose codes are read.
// FLAT: cols is a multiple of 32 and rows are packed in the outputs.  THROTTLE: a
// wave waits for each store before the next, which keeps the outputs' streams from
// crowding one another out.
// ---------------------------------------------------------------------------
struct DecodeArgs {
    const char* codes[kMaxRanks];
    const char* scales[kMaxRanks];
    char* dst[kMaxRanks];
    int n_out;  // outputs that every rank's values go to; 0: rank q's go to dst[q] alone
    uint64_t cols, kb, groups, slab, stride;
    FastDiv by_kb;
};

// One vector of a type from its codes.
template <class T>
__device__ __forceinline__ u32x4 decode_vec(uint32_t c, float s)
{
    if constexpr (T::ESZ == 4) {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
        return u32x4{__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)};
    } else {
        return u32x4{Mx4<T>::template decode<0>(c, s), Mx4<T>::template decode<1>(c, s), Mx4<T>::template decode<2>(c, s),
                     Mx4<T>::template decode<3>(c, s)};
    }
}

template <class T, bool FLAT, bool THROTTLE>
__global__ __launch_bounds__(256) void k_mx4_decode(DecodeArgs a)
{
    constexpr uint64_t E = T::ESZ;
    constexpr int V = T::VEC, LG = V == 8 ? 2 : 3;  // 2^LG vectors of a block
    typedef typename std::conditional<V == 8, uint32_t, uint16_t>::type Codes;
    const int q = blockIdx.y;
    const auto codes = (global_ptr<const Codes>)a.codes[q];
    const auto scales = (global_ptr<const uint8_t>)a.scales[q];
    const int r0 = a.n_out ? 0 : q, r1 = a.n_out ? a.n_out : q + 1;
    const uint64_t step = (uint64_t)gridDim.x * 256;
    for (uint64_t g = (uint64_t)blockIdx.x * 256 + threadIdx.x; g < a.groups; g += step) {
        const u32x4 x = decode_vec<T>(codes[g], scale_float(scales[g >> LG]));
        uint64_t at = (uint64_t)q * a.slab;
        int64_t left = V;
        if constexpr (FLAT) {
            at += g * V;
        } else {
            const uint64_t b = g >> LG;
            const uint64_t row = (a.groups >> (31 + LG)) ? b / a.kb : a.by_kb.div((uint32_t)b);
            const uint64_t col = (b - row * a.kb) * 32 + (g & ((1 << LG) - 1)) * V;
            left = (int64_t)a.cols - (int64_t)col;
            at += row * a.stride + col;
        }
        if (left >= V) {
            for (int r = r0; r < r1; r++) {
                st16<true>(a.dst[r] + at * E, x);
                if constexpr (THROTTLE) wait_vmem_below<0>();
            }
        } else {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < V; i++) {
                if (i >= left) continue;
                const uint32_t s = E == 4 ? w[i % 4] : w[i / 2 % 4] >> (16 * (i & 1));
                for (int r = r0; r < r1; r++) store_s<T>(a.dst[r] + (at + i) * E, (typename T::S)s);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
using namespace host;

unsigned block_grid(uint64_t items, uint64_t per_block, int n, int cus, int per_cu)
{
    uint64_t want = (items + per_block - 1) / per_block;
    uint64_t cap = (uint64_t)cus * (uint64_t)per_cu / (uint64_t)n;
    if (cap < 1) cap = 1;
    if (want > cap) want = cap;
    return (unsigned)(want < 1 ? 1 : want);
}

template <class T>
vrc_status_t quantize_typed(const char* const* x, char* const* codes, char* const* scales, int n, uint64_t rows,
                            uint64_t cols, bool along_rows, int cus, hipStream_t st)
{
    if (along_rows) {
        QuantTArgs a = {};
        for (int r = 0; r < n; r++) {
            a.src[r] = x[r];
            a.codes[r] = codes[r];
            a.scales[r] = scales[r];
        }
        a.rows = rows;
        a.cols = cols;
        a.kb = (rows + 31) / 32;
        constexpr uint64_t wide = 64 * (4 / T::ESZ);
        const uint64_t ct = (cols + wide - 1) / wide, rt = (a.kb + 7) / 8;
        if (ct > 0x7fffffffull || ct * rt > 0x7fffffffull) return VRC_ERR_INVALID_ARG;
        a.col_tiles = (uint32_t)ct;
        a.tiles = (uint32_t)(ct * rt);
        bool lines = a.kb % 8 == 0;
        for (int r = 0; r < n; r++) lines = lines && (uintptr_t)codes[r] % 128 == 0;
        if (lines) k_mx4_quantize_t<T, true><<<wide_grid(a.tiles, n), 256, 0, st>>>(a);
        else k_mx4_quantize_t<T, false><<<wide_grid(a.tiles, n), 256, 0, st>>>(a);
        return check_launch();
    }
    QuantArgs a = {};
    for (int r = 0; r < n; r++) {
        a.src[r] = x[r];
        a.codes[r] = codes[r];
        a.scales[r] = scales[r];
    }
    a.cols = cols;
    a.kb = (cols + 31) / 32;
    a.groups = rows * a.kb * 4;
    a.by_kb = FastDiv::of(a.kb);
    // 32 workgroups per CU with four groups a lane: 8 x [8192, 4096] bf16 108 us
    // (6.3 TB/s), 8 per CU 113 us, one group a lane 109-125 us.
    const dim3 grid(block_grid(a.groups, 1024, n, cus, 32), (unsigned)n);
    if (cols % 32 == 0) k_mx4_quantize<T, true><<<grid, 256, 0, st>>>(a);
    else k_mx4_quantize<T, false><<<grid, 256, 0, st>>>(a);
    return check_launch();
}

template <class T>
vrc_status_t decode_typed(const char* const* codes, const char* const* scales, char* const* y, int n, int n_out,
                          uint64_t rows, uint64_t cols, uint64_t slab, uint64_t stride, int cus, hipStream_t st)
{
    DecodeArgs a = {};
    for (int r = 0; r < n; r++) {
        a.codes[r] = codes[r];
        a.scales[r] = scales[r];
        a.dst[r] = y[r];
    }
    a.n_out = n_out;
    a.cols = cols;
    a.kb = (cols + 31) / 32;
    a.groups = rows * a.kb * (32 / T::VEC);
    a.slab = slab;
    a.stride = stride;
    a.by_kb = FastDiv::of(a.kb);
    // A gather keeps one store in flight per wave, 16 workgroups per CU: us with / without
    // that wait, along the rows 8 x [8192, 4096] bf16 773 / 893, [20480, 128] fp16 61 / 66,
    // fp32 119 / 127, 2 x [65536, 512] fp32 92 / 97, 4 x [4096, 4096] fp16 103 / 98, 16 x
    // [4096, 1024] bf16 389 / 383; along the columns within 3 % either way (8 x [8192, 4096]
    // 799 / 794); 8 x [1, 4096] 4.8 / 4.2.  64 workgroups per CU come to the same, but for
    // rows of odd lengths (8 x [5003, 1001] fp16 170, by 64 154).
    const dim3 grid(block_grid(a.groups, 256, n, cus, n_out > 1 ? 16 : 32), (unsigned)n);
    const bool flat = cols % 32 == 0 && stride == cols;
    if (n_out > 1) {
        if (flat) k_mx4_decode<T, true, true><<<grid, 256, 0, st>>>(a);
        else k_mx4_decode<T, false, true><<<grid, 256, 0, st>>>(a);
    } else {
        if (flat) k_mx4_decode<T, true, false><<<grid, 256, 0, st>>>(a);
        else k_mx4_decode<T, false, false><<<grid, 256, 0, st>>>(a);
    }
    return check_launch();
}

}  // namespace

namespace host {

vrc_status_t run_mx4_quantize(const char* const* x, char* const* codes, char* const* scales, int n, uint64_t rows,
                              uint64_t cols, vrc_dtype_t dt, bool along_rows, int cus, hipStream_t st)
{
    switch (dt) {
    case VRC_FP32: return quantize_typed<F32>(x, codes, scales, n, rows, cols, along_rows, cus, st);
    case VRC_FP16: return quantize_typed<F16>(x, codes, scales, n, rows, cols, along_rows, cus, st);
    case VRC_BF16: return quantize_typed<BF16>(x, codes, scales, n, rows, cols, along_rows, cus, st);
    default: return VRC_ERR_UNSUPPORTED;
    }
}

vrc_status_t run_mx4_decode(const char* const* codes, const char* const* scales, char* const* y, int n, int n_out,
                            uint64_t rows, uint64_t cols, uint64_t slab, uint64_t stride, vrc_dtype_t dt, int cus,
                            hipStream_t st)
{
    switch (dt) {
    case VRC_FP32: return decode_typed<F32>(codes, scales, y, n, n_out, rows, cols, slab, stride, cus, st);
    case VRC_FP16: return decode_typed<F16>(codes, scales, y, n, n_out, rows, cols, slab, stride, cus, st);
    case VRC_BF16: return decode_typed<BF16>(codes, scales, y, n, n_out, rows, cols, slab, stride, cus, st);
    default: return VRC_ERR_UNSUPPORTED;
    }
}

}  // namespace host
}  // namespace vrc
