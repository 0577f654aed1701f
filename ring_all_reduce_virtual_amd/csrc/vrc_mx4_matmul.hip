// vrc_mx4_matmul.hip -- the product of microscaled 4-bit matrices, summed over
// the ranks' parts of the contraction or one per rank.
//
// C = sum_q A_q B_q^T on the matrix cores: v_mfma_scale_f32_32x32x64 takes, per
// lane, one block of 32 codes of a row of each operand with its scale byte, and
// adds 64 exact products per output to an fp32 accumulator.  B is the first
// operand, so that a lane's results are four consecutive columns of a row of C.
//
// The contraction is walked in tiles of eight blocks (256 codes, 128 bytes a
// row) of one rank; a row's last tile may hold fewer, whose missing blocks count
// as zero codes with scale 1.
#include <hip/hip_runtime.h>

#include "vrc_ops_host.hpp"

namespace vrc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

constexpr uint32_t kTileBlocks = 8;                // blocks per row of a tile
constexpr uint32_t kTileBytes = kTileBlocks * 16;  // codes of a row of a tile

struct MatmulArgs {
    const char* ac[kMaxRanks];
    const char* as[kMaxRanks];
    const char* bc[kMaxRanks];
    const char* bs[kMaxRanks];
    char* dst[kMaxRanks];
    uint32_t m, n, kb;
    int ranks;
    uint32_t tiles_m, tiles_n;
};

// acc += the 64 products per output of step S (blocks 2S and 2S + 1) of a tile;
// byte S of sb and sa is this lane's block's scale.
template <int S>
__device__ __forceinline__ f32x16 mfma(u32x4 b, u32x4 a, f32x16 acc, uint32_t sb, uint32_t sa)
{
    const i32x8 x = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    const i32x8 y = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 4, 4, S, (int)sb, S, (int)sa);
}

// The four scale bytes that a lane needs of a row's eight: those of blocks
// half, 2 + half, 4 + half and 6 + half, in step order.
__device__ __forceinline__ uint32_t step_scales(u32x2 bytes, uint32_t half)
{
    return __builtin_amdgcn_perm(bytes.y, bytes.x, half ? 0x07050301u : 0x06040200u);
}

// A row's eight scale bytes of the tile at `p`, or the `left` that it has and 127
// (scale 1) for the rest.
__device__ __forceinline__ u32x2 load_scales(const char* p, uint32_t left)
{
    if (left >= kTileBlocks) return *(global_ptr<const u32x2_any>)p;
    uint64_t v = 0x7f7f7f7f7f7f7f7full;
    for (uint32_t i = 0; i < left; i++)
        v = (v & ~(0xffull << (8 * i))) | (uint64_t)*(global_ptr<const uint8_t>)(p + i) << (8 * i);
    return u32x2{(uint32_t)v, (uint32_t)(v >> 32)};
}

// Four consecutive columns, rounded.
template <class T>
struct Four {
    uint32_t w[T::ESZ];  // 4 * ESZ bytes
    __device__ __forceinline__ explicit Four(const float* v)
    {
        if constexpr (T::ESZ == 4) {
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 2; i++)
                w[i] = (uint32_t)T::narrow(v[2 * i]) | (uint32_t)T::narrow(v[2 * i + 1]) << 16;
        }
    }
};

// ---------------------------------------------------------------------------
// Tiled product.  A workgroup of WM x WN waves has a BM x BN tile of C, a wave MI
// x NI matrix-instruction tiles of it.  Each tile of the contraction is brought
// into LDS by direct loads (16 bytes a lane, no registers) while the one before is
// multiplied.
//
// LDS holds a row's eight 16-byte blocks with block j at place j ^ (row / 2 mod
// 8), so that the 32 rows that a matrix operand reads at one block spread
// over all banks; the loads permute their global addresses within the row's
// 128 bytes to that end, as a direct load writes consecutive lanes to consecutive
// places.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t place(uint32_t row, uint32_t block) { return block ^ (row >> 1 & 7); }

// Every wave's direct loads have landed (a barrier alone does not wait for
// them), and every wave is done with the stage it read.
__device__ __forceinline__ void stage_barrier()
{
    wait_vmem_below<0>();
    __syncthreads();
}

template <int BM, int BN>
struct Stage {
    char codes[(BM + BN) * kTileBytes];  // A's rows, then B's
    u32x2 scales[BM + BN];
};

template <class T, bool SUM, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void k_mx4_matmul_tiled(MatmulArgs a)
{
    constexpr int MI = BM / WM / 32, NI = BN / WN / 32, WAVES = WM * WN, THREADS = WAVES * 64;
    constexpr int CHUNKS = (BM + BN) / 8;  // of eight rows: 1 KiB, one load of a wave
    static_assert(CHUNKS % WAVES == 0 && THREADS == BM + BN && BM % 64 == 0, "loads are shared out evenly");
    __shared__ __attribute__((aligned(16))) Stage<BM, BN> stage[2];

    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t m0 = blockIdx.x % a.tiles_m * BM, n0 = blockIdx.x / a.tiles_m * BN;
    const uint32_t ktiles = (a.kb + kTileBlocks - 1) / kTileBlocks;
    const int q0 = SUM ? 0 : (int)blockIdx.y;
    const uint32_t total = ktiles * (SUM ? (uint32_t)a.ranks : 1u);
    const uint64_t row_bytes = (uint64_t)a.kb * 16;

    // This lane's part of each of its wave's loads: a row's offset from the tile's
    // first row (rows past the end read the last one again) and its block.
    uint32_t off[CHUNKS / WAVES];
#pragma unroll
    for (int i = 0; i < CHUNKS / WAVES; i++) {
        const uint32_t chunk = wave * (CHUNKS / WAVES) + i;
        const bool isb = chunk >= BM / 8;
        const uint32_t row = (isb ? chunk - BM / 8 : chunk) * 8 + lane / 8;
        const uint32_t last = isb ? a.n - 1 - n0 : a.m - 1 - m0;
        off[i] = (row < last ? row : last) * (uint32_t)row_bytes + place(row, lane & 7) * 16;
    }
    const uint32_t srow = tid < BM ? (tid < a.m - m0 ? m0 + tid : a.m - 1)
                                   : (tid - BM < a.n - n0 ? n0 + tid - BM : a.n - 1);

    // Tile t of the contraction into a stage.
    const auto fetch_codes = [&](Stage<BM, BN>& s, int q, uint32_t kt) {
        const auto pa = (global_ptr<const char>)a.ac[q] + m0 * row_bytes + (uint64_t)kt * kTileBytes;
        const auto pb = (global_ptr<const char>)a.bc[q] + n0 * row_bytes + (uint64_t)kt * kTileBytes;
        const uint32_t left = a.kb - kt * kTileBlocks;
        if (left >= kTileBlocks) {
#pragma unroll
            for (int i = 0; i < CHUNKS / WAVES; i++) {
                const uint32_t chunk = wave * (CHUNKS / WAVES) + i;
                __builtin_amdgcn_global_load_lds(
                    (global_ptr<const void>)((chunk >= BM / 8 ? pb : pa) + off[i]),
                    (__attribute__((address_space(3))) void*)(s.codes + chunk * 1024), 16, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < CHUNKS / WAVES; i++) {
                const uint32_t chunk = wave * (CHUNKS / WAVES) + i;
                u32x4 v = {};
                if (place(chunk * 8 + lane / 8, lane & 7) < left) v = *(global_ptr<const u32x4>)((chunk >= BM / 8 ? pb : pa) + off[i]);
                *(u32x4*)(s.codes + chunk * 1024 + lane * 16) = v;
            }
        }
    };
    const auto fetch_scales = [&](int q, uint32_t kt) {
        const char* p = wave < BM / 64 ? a.as[q] : a.bs[q];  // one array per wave
        return load_scales(p + (uint64_t)srow * a.kb + kt * kTileBlocks, a.kb - kt * kTileBlocks);
    };

    f32x16 acc[MI][NI] = {};
    const uint32_t wm = wave % WM * (BM / WM), wn = wave / WM * (BN / WN);
    const uint32_t r = lane & 31, half = lane >> 5;
    const auto multiply = [&](const Stage<BM, BN>& s) {
        uint32_t sa[MI], sb[NI];
#pragma unroll
        for (int i = 0; i < MI; i++) sa[i] = step_scales(s.scales[wm + i * 32 + r], half);
#pragma unroll
        for (int j = 0; j < NI; j++) sb[j] = step_scales(s.scales[BM + wn + j * 32 + r], half);
        // The next step's operands are read while one is multiplied; the scheduling
        // barriers keep the compiler from reading all four at once, which takes
        // more registers than there are.
        u32x4 x[2][MI], y[2][NI];
        const auto read = [&](int k) {
            const uint32_t at = place(r, 2 * k + half) * 16;
#pragma unroll
            for (int j = 0; j < NI; j++) y[k & 1][j] = *(const u32x4*)(s.codes + (BM + wn + j * 32 + r) * kTileBytes + at);
#pragma unroll
            for (int i = 0; i < MI; i++) x[k & 1][i] = *(const u32x4*)(s.codes + (wm + i * 32 + r) * kTileBytes + at);
        };
        const auto step = [&](auto S) {
            constexpr int k = decltype(S)::value;
            if constexpr (k < 3) read(k + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int j = 0; j < NI; j++) acc[i][j] = mfma<k>(y[k & 1][j], x[k & 1][i], acc[i][j], sb[j], sa[i]);
            __builtin_amdgcn_sched_barrier(0);
        };
        read(0);
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
    };

    int q = q0;
    uint32_t kt = 0;
    if (total) {
        fetch_codes(stage[0], q, kt);
        const u32x2 sc = fetch_scales(q, kt);
        stage[0].scales[tid] = sc;
    }
    for (uint32_t t = 0; t < total; t++) {
        stage_barrier();
        const uint32_t cur = t & 1, next = cur ^ 1;
        if (++kt == ktiles) {
            kt = 0;
            q++;
        }
        u32x2 sc = {};
        if (t + 1 < total) {
            fetch_codes(stage[next], q, kt);
            sc = fetch_scales(q, kt);
        }
        multiply(stage[cur]);
        stage[next].scales[tid] = sc;
    }
    stage_barrier();

    // The wave's results, 32 rows at a time through its own part of LDS, so that
    // they leave in 16-byte stores along the rows of C.
    // Row r's 16-byte piece c is at c ^ (r mod 8), which spreads a column over the banks.
    constexpr uint32_t PITCH = NI * 32 * T::ESZ;
    static_assert(WAVES * 32 * PITCH <= sizeof(stage[0].codes), "the epilogue fits a stage");
    char* own = stage[0].codes + wave * 32 * PITCH;
    const uint32_t vecs = NI * 32 / T::VEC;  // per row
    const int dst0 = SUM ? 0 : q0, dst1 = SUM ? a.ranks : q0 + 1;
#pragma unroll
    for (int i = 0; i < MI; i++) {
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const float v[4] = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                const Four<T> f(v);
                if constexpr (T::ESZ == 4) {
                    *(u32x4*)(own + r * PITCH + ((j * 8 + 2 * g + half) ^ (r & 7)) * 16) =
                        u32x4{f.w[0], f.w[1], f.w[2], f.w[3]};
                } else {
                    *(u32x2*)(own + r * PITCH + ((j * 4 + g) ^ (r & 7)) * 16 + half * 8) = u32x2{f.w[0], f.w[1]};
                }
            }
        __builtin_amdgcn_wave_barrier();
        for (uint32_t v = lane; v < 32 * vecs; v += 64) {
            const uint32_t row = m0 + wm + i * 32 + v / vecs, c = v % vecs * T::VEC, col = n0 + wn + c;
            const u32x4 x = *(const u32x4*)(own + v / vecs * PITCH + (v % vecs ^ (v / vecs & 7)) * 16);
            if (row >= a.m || col >= a.n) continue;
            const uint64_t at = ((uint64_t)row * a.n + col) * T::ESZ;
            if (col + T::VEC <= a.n) {
                for (int d = dst0; d < dst1; d++) st16<true>(a.dst[d] + at, x);
            } else {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < T::VEC; e++) {
                    if (col + e >= a.n) continue;
                    const auto s = (typename T::S)(T::ESZ == 4 ? w[e % 4] : w[e / 2 % 4] >> (16 * (e & 1)));
                    for (int d = dst0; d < dst1; d++) store_s<T>(a.dst[d] + at + e * T::ESZ, s);
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ---------------------------------------------------------------------------
// Few rows of A: a stream of B.  A workgroup has 32 columns of C (rows of B) and
// all of C's rows (MI x 32); its waves take the contraction's tiles in turn,
// straight from memory into registers, the next tile's loads in flight while one is
// multiplied, and the waves' sums meet in LDS, added in wave order.
// ---------------------------------------------------------------------------
template <int MI>
struct Frag {
    u32x4 b[4], a[MI][4];
    u32x2 sb, sa[MI];
};

template <class T, bool SUM, int MI, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_mx4_matmul_few(MatmulArgs a)
{
    __shared__ float part[WAVES][MI * 32 * 33];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t r = lane & 31, half = lane >> 5;
    const uint32_t n0 = blockIdx.x * 32;
    const uint32_t ktiles = (a.kb + kTileBlocks - 1) / kTileBlocks;
    const int q0 = SUM ? 0 : (int)blockIdx.y;
    const uint32_t total = ktiles * (SUM ? (uint32_t)a.ranks : 1u);
    const uint64_t rb = n0 + r < a.n ? n0 + r : a.n - 1;
    uint64_t ra[MI];
#pragma unroll
    for (int i = 0; i < MI; i++) ra[i] = i * 32 + r < a.m ? i * 32 + r : a.m - 1;

    const auto fetch = [&](Frag<MI>& f, uint32_t t) {
        const uint32_t qi = t / ktiles, kt = t - qi * ktiles;
        const int q = q0 + (int)qi;
        const uint64_t k0 = (uint64_t)kt * kTileBlocks;
        const uint32_t left = a.kb - kt * kTileBlocks;
        const char* pb = a.bc[q] + (rb * a.kb + k0 + half) * 16;
        f.sb = load_scales(a.bs[q] + rb * a.kb + k0, left);
#pragma unroll
        for (int i = 0; i < MI; i++) f.sa[i] = load_scales(a.as[q] + ra[i] * a.kb + k0, left);
        if (left >= kTileBlocks) {
#pragma unroll
            for (int s = 0; s < 4; s++) f.b[s] = *(global_ptr<const u32x4>)(pb + 32 * s);
#pragma unroll
            for (int i = 0; i < MI; i++) {
                const char* pa = a.ac[q] + (ra[i] * a.kb + k0 + half) * 16;
#pragma unroll
                for (int s = 0; s < 4; s++) f.a[i][s] = *(global_ptr<const u32x4>)(pa + 32 * s);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; s++) f.b[s] = 2 * s + half < left ? *(global_ptr<const u32x4>)(pb + 32 * s) : u32x4{};
#pragma unroll
            for (int i = 0; i < MI; i++) {
                const char* pa = a.ac[q] + (ra[i] * a.kb + k0 + half) * 16;
#pragma unroll
                for (int s = 0; s < 4; s++)
                    f.a[i][s] = 2 * s + half < left ? *(global_ptr<const u32x4>)(pa + 32 * s) : u32x4{};
            }
        }
    };
    f32x16 acc[MI] = {};
    const auto multiply = [&](const Frag<MI>& f) {
        const uint32_t sb = step_scales(f.sb, half);
#pragma unroll
        for (int i = 0; i < MI; i++) {
            const uint32_t sa = step_scales(f.sa[i], half);
            acc[i] = mfma<0>(f.b[0], f.a[i][0], acc[i], sb, sa);
            acc[i] = mfma<1>(f.b[1], f.a[i][1], acc[i], sb, sa);
            acc[i] = mfma<2>(f.b[2], f.a[i][2], acc[i], sb, sa);
            acc[i] = mfma<3>(f.b[3], f.a[i][3], acc[i], sb, sa);
        }
    };
    Frag<MI> f0, f1;
    uint32_t t = wave;
    if (t < total) fetch(f0, t);
    for (; t < total; t += 2 * WAVES) {
        if (t + WAVES < total) fetch(f1, t + WAVES);
        multiply(f0);
        if (t + WAVES >= total) break;
        if (t + 2 * WAVES < total) fetch(f0, t + 2 * WAVES);
        multiply(f1);
    }
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) part[wave][(i * 32 + r) * 33 + 8 * (e / 4) + 4 * half + e % 4] = acc[i][e];
    __syncthreads();
    const int dst0 = SUM ? 0 : q0, dst1 = SUM ? a.ranks : q0 + 1;
    for (uint32_t o = tid; o < MI * 32 * 32; o += WAVES * 64) {
        const uint32_t row = o / 32, col = o % 32;
        if (row >= a.m || n0 + col >= a.n) continue;
        float s = part[0][row * 33 + col];
#pragma unroll
        for (int w = 1; w < WAVES; w++) s += part[w][row * 33 + col];
        const typename T::S v = T::narrow(s);
        const uint64_t at = ((uint64_t)row * a.n + n0 + col) * T::ESZ;
        for (int d = dst0; d < dst1; d++) store_s<T>(a.dst[d] + at, v);
    }
}

using namespace host;

template <class T, bool SUM, int BM, int BN, int WM, int WN>
vrc_status_t launch_tiled(MatmulArgs& a, hipStream_t st)
{
    a.tiles_m = (a.m + BM - 1) / BM;
    a.tiles_n = (a.n + BN - 1) / BN;
    const uint64_t tiles = (uint64_t)a.tiles_m * a.tiles_n;
    if (tiles > 0x7fffffffull) return VRC_ERR_INVALID_ARG;
    const dim3 grid((unsigned)tiles, SUM ? 1u : (unsigned)a.ranks);
    k_mx4_matmul_tiled<T, SUM, BM, BN, WM, WN><<<grid, WM * WN * 64, 0, st>>>(a);
    return check_launch();
}

template <class T, bool SUM, int MI>
vrc_status_t launch_few(const MatmulArgs& a, hipStream_t st)
{
    constexpr int WAVES = 8;
    const dim3 grid((a.n + 31) / 32, SUM ? 1u : (unsigned)a.ranks);
    k_mx4_matmul_few<T, SUM, MI, WAVES><<<grid, WAVES * 64, 0, st>>>(a);
    return check_launch();
}

template <class T, bool SUM>
vrc_status_t matmul_typed(MatmulArgs& a, int cus, hipStream_t st)
{
    if (a.m <= 32) return launch_few<T, SUM, 1>(a, st);
    if (a.m <= 64) return launch_few<T, SUM, 2>(a, st);
    const uint64_t big = (uint64_t)((a.m + 255) / 256) * ((a.n + 255) / 256) * (SUM ? 1 : a.ranks);
    if (big >= (uint64_t)cus) return launch_tiled<T, SUM, 256, 256, 2, 4>(a, st);
    return launch_tiled<T, SUM, 128, 128, 2, 2>(a, st);
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
    switch (dt) {
    case VRC_FP32: return sum ? matmul_typed<F32, true>(a, cus, st) : matmul_typed<F32, false>(a, cus, st);
    case VRC_FP16: return sum ? matmul_typed<F16, true>(a, cus, st) : matmul_typed<F16, false>(a, cus, st);
    case VRC_BF16: return sum ? matmul_typed<BF16, true>(a, cus, st) : matmul_typed<BF16, false>(a, cus, st);
    default: return VRC_ERR_UNSUPPORTED;
    }
}

}  // namespace host
}  // namespace vrc
