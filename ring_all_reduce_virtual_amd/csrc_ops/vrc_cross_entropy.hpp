// vrc_cross_entropy.hpp -- kernels of the cross entropy over a split vocabulary
// and of its gradient.  Internal; one unit per element type compiles them.
//
// Three products on the matrix cores (vrc_tiles.hpp), none of whose results leaves
// the chip as logits:
//   LOGITS   z = hidden W^T.  Its end is, for the loss, a maximum and a sum of
//            exponentials of every row of a tile (and the target's logit from the one
//            tile that has it), which a second launch joins; for the gradient, the
//            tile of G = a exp(z - lse) - b [target], rounded to the type, of a piece
//            of the vocabulary at a time;
//   DWEIGHT  G^T hidden, whole for each row of the weights;
//   DHIDDEN  G W, summed over the pieces (and over splits of the contraction, where
//            there are few tiles) in fp32.
// G is the only thing kept, [tokens, a piece's columns]; DHIDDEN reads it along its
// rows, DWEIGHT across them.
//
// G of 16-bit types is rounded to the type, for the matrix cores.  However many tokens there are,
// a row of either gradient is mostly one element of G, the target's, so that the error of one value
// of each adds to that of the output's rounding: where tokens weigh differently, errors are 0.0022
// of the norm in bf16 (the output's rounding alone 0.0017) and 0.00028 (0.00021) in fp16, for 129
// tokens and for 4096; of a mean over tokens of small probability, whose elements of G are close
// to the unit, 0.0017 and 0.00021.
// Few tokens (kFewTokens at most) are bound by the weights' bytes and their gradients'.  There G is held
// as its transpose, a row of the vocabulary a row, and, of 16-bit types, as two values each, G rounded and
// what that left, which keeps errors at the output's rounding (7 tokens 0.0017, with one value 0.0028).
// It is a choice by what it costs, 65536 x 4096 bf16 with two values and (by the other kernels) with one:
// 33 tokens 402 us and 367, 64 404 and 375, 96 508 and 405, 128 534 and 432; 128 tokens of 8000 x 1024
// 59 and 37.  Where the matrix instructions bound, it would be two of three products made twice (4096
// tokens: some 9,000 us for 5,400).
//
// Measured on MI355X, 4096 tokens and 8 x (8192 x 4096) bf16, calls one after the other on other
// inputs: the loss 1,732 us (1.27 PFLOP/s, matrix pipes busy for 71 % of all cycles), the gradients
// 5,369 to 5,548 us (1.19 to 1.23 PFLOP/s: for each of four pieces LOGITS 437, DHIDDEN 466, DWEIGHT 435
// us).  One token 107 us for 537 MB; the gradients of 7 tokens, 8 x (4096 x 4096), 171 us (LOGITS 58,
// DHIDDEN 53, DWEIGHT 51).  fp32, 2048 x 16384 x 2048: 138 TFLOP/s.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "vrc_model_host.hpp"
#include "vrc_tiles.hpp"

namespace vrc {
namespace {

using host::EntropyCall;

constexpr uint64_t kFewTokens = 128, kStreamTokens = 32;

// kDsums: DHIDDEN's sums, in fp32.  kGradT, kDweightT and kDsumsT: of few tokens, by G's transpose.
enum EntropyOp { kStats, kGrad, kGradT, kDweight, kDweightT, kDhidden, kDsums, kDsumsT };

// A run of one rank's weight rows.
struct Piece {
    const char* w;       // its first row (packed or the caller's)
    char* out;           // DWEIGHT: the first row's gradient
    uint32_t len;        // rows
    uint32_t first;      // of the whole vocabulary
    uint32_t col;        // G: its first column, a multiple of 256
    uint32_t tile;       // its first tile along the vocabulary, or (DHIDDEN) of the contraction
};

// A token's part of the gradient: a and b, scaled; lse; its target in the whole
// vocabulary, or none.  Tokens without gradient have a = b = 0.
struct Coef {
    float a, b, lse;
    uint32_t target;
};
constexpr uint32_t kNoTarget = 0xffffffffu;

struct EntropyArgs {
    Piece piece[kMaxRanks];
    const char* a;        // LOGITS: hidden; else G
    const char* b;        // DWEIGHT: hidden
    uint64_t pitch_a, pitch_b, pitch_out;  // bytes of a row; pitch_b: of the weights', but for DWEIGHT
    char* out;            // G, dhidden, or DHIDDEN's fp32 sums [split][token][pitch_out]
    const Coef* coef;     // kGrad
    const float* unscale; // what the products of G are multiplied by (null: nothing)
    const long long* target;  // kStats
    float2* stats;            // kStats: [tile along the vocabulary][token]
    float* picked;            // kStats: [token]
    uint32_t tiles_m, tiles_n;
    uint32_t tokens, rows_a, width, granules;  // rows_a: rows that LOGITS and DHIDDEN read of A; granules: of a row of B (across)
    uint32_t ktiles;          // of the contraction
    uint32_t kwidth;          // LOGITS: elements of the contraction; DWEIGHT: whole tiles of it
    int pieces;
    int first_piece;          // DHIDDEN to fp32 sums: this launch is the first
};

// Four consecutive columns, rounded.
template <class T>
struct Quad {
    uint32_t w[T::ESZ];
    __device__ __forceinline__ explicit Quad(const float* v)
    {
        if constexpr (T::ESZ == 4) {
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 2; i++) w[i] = (uint32_t)T::narrow(v[2 * i]) | (uint32_t)T::narrow(v[2 * i + 1]) << 16;
        }
    }
};

// A wave's results to sink(row, column, 16 bytes), 32 rows at a time through `own`,
// the wave's part of LDS, so that they leave along the rows.  value(i, j, e): result e of
// the instruction tile (i, j).  Row r's 16-byte piece c is at c ^ (r mod 8) (mod 4 where
// a row has four), which spreads a column over the banks.
template <class T, int MI, int NI, class Value, class Sink>
__device__ __forceinline__ void drain(char* own, uint32_t lane, Value value, Sink sink)
{
    constexpr uint32_t PITCH = NI * 32 * T::ESZ, VECS = NI * 32 / T::VEC, MIX = VECS < 8 ? VECS - 1 : 7;
    const uint32_t r = lane & 31, half = lane >> 5;
#pragma unroll
    for (int i = 0; i < MI; i++) {
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = value(i, j, 4 * g + e);
                const Quad<T> f(v);
                if constexpr (T::ESZ == 4)
                    *(u32x4*)(own + r * PITCH + ((j * 8 + 2 * g + half) ^ (r & MIX)) * 16) = u32x4{f.w[0], f.w[1], f.w[2], f.w[3]};
                else
                    *(u32x2*)(own + r * PITCH + ((j * 4 + g) ^ (r & MIX)) * 16 + half * 8) = u32x2{f.w[0], f.w[1]};
            }
        __builtin_amdgcn_wave_barrier();
        for (uint32_t v = lane; v < 32 * VECS; v += 64)
            sink(i * 32 + v / VECS, v % VECS * T::VEC, *(const u32x4*)(own + v / VECS * PITCH + ((v % VECS) ^ (v / VECS & MIX)) * 16));
        __builtin_amdgcn_wave_barrier();
    }
}

// `left` (1 to VEC and more) elements of x to `to`, at any element's address.
template <class T>
__device__ __forceinline__ void store_some(char* to, u32x4 x, uint32_t left)
{
    if (left >= T::VEC) {
        st16<true>(to, x);
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < T::VEC; e++)
        if (e < (int)left) store_s<T>(to + e * T::ESZ, (typename T::S)(T::ESZ == 4 ? w[e % 4] : w[e / 2 % 4] >> (16 * (e & 1))));
}

// exp(x) for x <= 0 (or NaN): the hardware's 2^x, whose error and that of the product
// before it are below half a step of a 16-bit result by far; fp32's own for fp32.
template <class T>
__device__ __forceinline__ float exp_of(float x)
{
    if constexpr (T::ESZ == 4) return expf(x);
    else return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

// A workgroup of WM x WN waves has a BM x BN tile of the result, a wave MI x NI
// matrix-instruction tiles of it.  A ring of S stages, up to S - 1 tiles of the
// contraction ahead; one barrier a tile, between its last read and its last step, behind
// which the next tile has landed for every wave and this tile's stage is free.  Past the last tile the
// loop goes on fetching that tile again, so that every wave always has the same number of
// loads under way, which is what its waits count.
// CUT (LOGITS): B's elements past the end of a row are read from a constant zero (A's
// are zero in memory).
// KS: 1, or 4 groups of waves that each take one step of every tile of the contraction, and
// join their sums in LDS (ALONG operands): where the matrix instructions bound and tiles are
// few, smaller ones then fill the CUs.
template <class T, int OP, int BM, int BN, int WM, int WN, int S, bool CUT, int KS>
__global__ __launch_bounds__(WM * WN * KS * 64) void k_entropy(EntropyArgs a)
{
    constexpr int MI = BM / WM / 32, NI = BN / WN / 32, WAVES = WM * WN * KS;
    constexpr bool DHIDDEN = OP == kDhidden || OP == kDsums || OP == kDsumsT, LOGITS = OP == kStats || OP == kGrad || OP == kGradT;
    constexpr bool DWEIGHT = OP == kDweight || OP == kDweightT;
    typedef TileOperand<T, OP == kDweight || OP == kDsumsT ? kAcross : kAlong, BM> A;
    typedef TileOperand<T, LOGITS ? kAlong : kAcross, BN> B;
    constexpr uint32_t LOADS = (A::LOADS + B::LOADS) / WAVES, STAGE = A::BYTES + B::BYTES, KT = kTileK<T>;
    static_assert((A::LOADS + B::LOADS) % WAVES == 0 && S >= 2 && LOADS * (S - 1) < 64, "loads are shared out evenly");
    __shared__ __attribute__((aligned(16))) char ring[S][STAGE];

    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t tm, tn;
    xcd_tile<4>(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);

    // The piece of the vocabulary, and the tile's first row and column in it.
    uint32_t m0 = tm * BM, n0 = tn * BN;
    int p = 0;
    if constexpr (!DHIDDEN) {
        const uint32_t t = DWEIGHT ? tm : tn;
        while (p + 1 < a.pieces && t >= a.piece[p + 1].tile) p++;
        if constexpr (DWEIGHT) m0 = (tm - a.piece[p].tile) * BM;
        else n0 = (tn - a.piece[p].tile) * BN;
    }
    uint32_t t0 = 0, total = a.ktiles;
    if constexpr (DHIDDEN) {  // this split's tiles
        const uint64_t splits = gridDim.y;
        t0 = (uint32_t)(a.ktiles * (uint64_t)blockIdx.y / splits);
        total = (uint32_t)(a.ktiles * (uint64_t)(blockIdx.y + 1) / splits) - t0;
        while (p + 1 < a.pieces && t0 >= a.piece[p + 1].tile) p++;
    }

    // This lane's part of each of its wave's loads.
    uint32_t off[LOADS], kk[LOADS];
#pragma unroll
    for (uint32_t i = 0; i < LOADS; i++) {
        const uint32_t at = wave * LOADS + i;
        if (at < A::LOADS) {
            // across: a piece's columns of G are there up to a multiple of 256
            const uint32_t last = OP == kDweight || OP == kDsumsT ? 0xffffffffu : (OP == kDweightT ? a.piece[p].len : a.rows_a) - 1 - m0;
            A::source(at * 64 + lane, (uint32_t)a.pitch_a, last, off[i], kk[i]);
            kk[i] = 0;
        } else {
            const uint32_t last = LOGITS ? a.piece[p].len - 1 - n0 : a.granules - 1 - n0 * T::ESZ / 16;
            B::source((at - A::LOADS) * 64 + lane, (uint32_t)a.pitch_b, last, off[i], kk[i]);
        }
    }
    // The tile that is fetched next, and where it lies: found while the one before it is
    // multiplied, so that behind the barrier its loads go out at once.
    uint32_t kt = t0, fetched = 0, fstage = 0, left = ~0u;
    const char *pa = nullptr, *pb = nullptr;
    const auto aim = [&] {
        if constexpr (DHIDDEN) {
            const Piece& q = a.piece[p];
            const uint32_t k = (kt - q.tile) * KT;
            if constexpr (OP == kDsumsT) pa = a.a + (uint64_t)(q.col + k) * a.pitch_a + (uint64_t)m0 * T::ESZ;
            else pa = a.a + m0 * a.pitch_a + (uint64_t)(q.col + k) * T::ESZ;
            pb = q.w + (uint64_t)k * a.pitch_b + (uint64_t)n0 * T::ESZ;
            left = q.len - k;
        } else if constexpr (OP == kDweight) {
            pa = a.a + (uint64_t)(a.piece[p].col + m0) * T::ESZ + (uint64_t)kt * KT * a.pitch_a;
            pb = a.b + (uint64_t)n0 * T::ESZ + (uint64_t)kt * KT * a.pitch_b;
        } else if constexpr (OP == kDweightT) {  // the tokens once for each of their two values
            pa = a.a + (uint64_t)(a.piece[p].col + m0) * a.pitch_a + (uint64_t)kt * kTileRow;
            pb = a.b + (uint64_t)n0 * T::ESZ + (uint64_t)(kt * KT < a.rows_a ? kt * KT : kt * KT - a.rows_a) * a.pitch_b;
        } else {
            pa = a.a + m0 * a.pitch_a + (uint64_t)kt * kTileRow;
            pb = a.piece[p].w + n0 * a.pitch_b + (uint64_t)kt * kTileRow;
            left = a.kwidth - kt * KT;
        }
    };
    const auto load = [&](uint32_t i) {
        const uint32_t at = wave * LOADS + i;
        uint32_t o = off[i];
        if constexpr (DHIDDEN)  // rows of the weights past a piece's end, times G's zeros: its last row again
            o -= kk[i] < left ? 0 : (kk[i] - left + 1) * (uint32_t)a.pitch_b;
        auto from = (global_ptr<const char>)(at < A::LOADS ? pa : pb) + hidden_offset(o);
        if constexpr (CUT && !DHIDDEN)
            if (kk[i] >= left) from = (global_ptr<const char>)&kZeroGranule;
        granules_to_lds(from, ring[fstage] + at * 1024);
    };
    const auto advance = [&] {
        fstage = fstage + 1 == S ? 0 : fstage + 1;
        fetched++;
        if (fetched < total) {
            kt++;
            if constexpr (DHIDDEN) p += p + 1 < a.pieces && kt >= a.piece[p + 1].tile;
        }
    };
    const auto fetch = [&] {
        aim();
#pragma unroll
        for (uint32_t i = 0; i < LOADS; i++) load(i);
        advance();
    };

    f32x16 acc[MI][NI] = {};
    const uint32_t member = wave % (WM * WN), group = wave / (WM * WN);
    const uint32_t wm = member % WM * (BM / WM), wn = member / WM * (BN / WN), r = lane & 31, half = lane >> 5;
    // A step's operands, one ahead of the matrix instructions.  The scheduling barriers
    // keep the reads in front of the step before theirs: left alone, the compiler reads each
    // operand right before its use.  Transposing reads (LATE) hold their wait, and stand
    // behind that step.
    constexpr bool TA = A::TRANSPOSED, TB = B::TRANSPOSED, LATE = TA || TB;
    constexpr int FRAGS = (TA ? MI : 0) + (TB ? NI : 0);
    u32x4 x[2][MI], y[2][NI];
    uint32_t places[FRAGS ? FRAGS : 1], base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)&ring[0][0];
    if constexpr (TB)
#pragma unroll
        for (int j = 0; j < NI; j++) places[j] = base + A::BYTES + B::across_at(wn + j * 32, lane);
    if constexpr (TA)
#pragma unroll
        for (int i = 0; i < MI; i++) places[(TB ? NI : 0) + i] = base + A::across_at(wm + i * 32, lane);
    const auto settle = [] { __builtin_amdgcn_sched_barrier(0); };
    // Transposing reads of a step: `count` operands from number `first` on, B's before A's.
    const auto across = [&](auto count, auto step, auto row, int first, uint32_t at) {
        constexpr int F = decltype(count)::value, s = decltype(step)::value, ROW = decltype(row)::value;
        uint32_t from[F];
        u32x4 out[F];
#pragma unroll
        for (int f = 0; f < F; f++) from[f] = places[first + f] + at * STAGE;
        read_across<F, s * 16 * ROW, 4 * ROW>(from, out);
#pragma unroll
        for (int f = 0; f < F; f++) {
            const int g = first + f;
            if (TB && g < NI) y[s & 1][g] = out[f];
            else x[s & 1][TB ? g - NI : g] = out[f];
        }
    };
    const auto read = [&](uint32_t at, auto step) {
        constexpr int s = decltype(step)::value;
        const char* stage = ring[at];
        if constexpr (!TB)
#pragma unroll
            for (int j = 0; j < NI; j++) y[s & 1][j] = B::read(stage + A::BYTES, wn + j * 32, s, lane);
        if constexpr (!TA)
#pragma unroll
            for (int i = 0; i < MI; i++) x[s & 1][i] = A::read(stage, wm + i * 32, s, lane);
        if constexpr (TA && TB && (int)A::ROW == (int)B::ROW) {
            across(std::integral_constant<int, NI + MI>{}, step, std::integral_constant<int, B::ROW>{}, 0, at);
        } else {
            if constexpr (TB) across(std::integral_constant<int, NI>{}, step, std::integral_constant<int, B::ROW>{}, 0, at);
            if constexpr (TA) across(std::integral_constant<int, MI>{}, step, std::integral_constant<int, A::ROW>{}, TB ? NI : 0, at);
        }
        settle();
    };
    const auto multiply = [&](int s, int i) {
#pragma unroll
        for (int j = 0; j < NI; j++)  // G's transpose: rows of it to lanes
            acc[i][j] = OP == kGradT ? tile_mfma<T>(x[s & 1][i], y[s & 1][j], acc[i][j]) : tile_mfma<T>(y[s & 1][j], x[s & 1][i], acc[i][j]);
    };
    const auto step = [&](int s) {
#pragma unroll
        for (int i = 0; i < MI; i++) multiply(s, i);
        settle();
    };
    if constexpr (KS == 4) {
        static_assert(!LATE, "a step by number");
        const auto mine = [&](uint32_t at) {
#pragma unroll
            for (int j = 0; j < NI; j++) y[0][j] = B::read(ring[at] + A::BYTES, wn + j * 32, group, lane);
#pragma unroll
            for (int i = 0; i < MI; i++) x[0][i] = A::read(ring[at], wm + i * 32, group, lane);
            settle();
        };
        if (total) {
#pragma unroll
            for (int t = 0; t < S; t++) fetch();
            wait_vmem_below<LOADS*(S - 1)>();
            tile_barrier();
            uint32_t cur = 0;
            mine(0);
            for (uint32_t t = 1; t < total; t++) {
                aim();
                wait_vmem_below<LOADS*(S - 2)>();
                tile_barrier();
                cur = cur + 1 == S ? 0 : cur + 1;
#pragma unroll
                for (uint32_t i = 0; i < LOADS; i++) load(i);
                advance();
                step(0);
                mine(cur);
            }
            step(0);
            wait_vmem_below<0>();
        }
        __syncthreads();
        static_assert((KS - 1) * WM * WN * MI * NI * 4096 <= S * STAGE, "the groups' sums fit the ring");
        char* const sums = &ring[0][0] + member * (MI * NI * 4096) + lane * 16;
        if (group) {
#pragma unroll
            for (int i = 0; i < MI * NI; i++)
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    const f32x16& v = acc[i / NI][i % NI];
                    *(u32x4*)(sums + ((group - 1) * WM * WN * MI * NI + i) * 4096 + g * 1024) =
                        u32x4{__float_as_uint(v[4 * g]), __float_as_uint(v[4 * g + 1]), __float_as_uint(v[4 * g + 2]), __float_as_uint(v[4 * g + 3])};
                }
        }
        __syncthreads();
        if (group == 0)
            for (int k = 0; k < KS - 1; k++)
#pragma unroll
                for (int i = 0; i < MI * NI; i++)
#pragma unroll
                    for (int g = 0; g < 4; g++) {
                        float v[4];
                        F32::unpack(*(const u32x4*)(sums + (k * WM * WN * MI * NI + i) * 4096 + g * 1024), v);
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[i / NI][i % NI][4 * g + e] += v[e];
                    }
    } else if (total) {
#pragma unroll
        for (int t = 0; t < S; t++) fetch();
        wait_vmem_below<LOADS*(S - 1)>();
        tile_barrier();
        uint32_t cur = 0;
        typedef std::integral_constant<int, 0> First;
        read(0, First{});
        const auto one = [&](auto next) {  // the step before `next`, and its operands
            constexpr int s = decltype(next)::value;
            if constexpr (LATE) step(s - 1);
            read(cur, next);
            if constexpr (!LATE) step(s - 1);
        };
        const auto first_steps = [&] {
            one(std::integral_constant<int, 1>{});
            one(std::integral_constant<int, 2>{});
            one(std::integral_constant<int, 3>{});
        };
        for (uint32_t t = 1; t < total; t++) {
            aim();
            first_steps();
            // the next tile has landed, for every wave behind the barrier, and this one's stage is free
            wait_vmem_below<LOADS*(S - 2)>();
            tile_barrier();
            cur = cur + 1 == S ? 0 : cur + 1;
            if constexpr (!LATE) read(cur, First{});
            // the loads between the matrix instructions of the last step
#pragma unroll
            for (int i = 0; i < MI; i++) {
                multiply(3, i);
                settle();
#pragma unroll
                for (uint32_t l = i * LOADS / MI; l < (i + 1) * LOADS / MI; l++) load(l);
                settle();
            }
            advance();
            if constexpr (LATE) read(cur, First{});
        }
        first_steps();
        step(3);
        wait_vmem_below<0>();
    }
    __syncthreads();

    if constexpr (OP == kStats) {
        const uint32_t cols = a.piece[p].len - n0;  // that the tile has
        float2* const part = (float2*)&ring[0][0];  // [WN][BM]
#pragma unroll
        for (int i = 0; i < (KS > 1 && group ? 0 : MI); i++) {
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NI; j++)
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    if (wn + j * 32 + result_col(e, half) >= cols) acc[i][j][e] = -INFINITY;
                    top = fmaxf(top, acc[i][j][e]);
                }
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            // rows of infinities: differences from 0 instead, whose exponentials are 0 and infinity
            const float from = __builtin_isinf(top) ? 0.0f : top;
#pragma unroll
            for (int j = 0; j < NI; j++)
#pragma unroll
                for (int e = 0; e < 16; e++) sum += exp_of<T>(acc[i][j][e] - from);
            sum += __shfl_xor(sum, 32, 64);
            if (half == 0) part[member / WM * BM + wm + i * 32 + r] = make_float2(top, sum);
            const uint32_t token = m0 + wm + i * 32 + r;
            if (a.target && token < a.tokens) {
                const unsigned long long at = (unsigned long long)a.target[token] - a.piece[p].first - n0 - wn;
                if (at < BN / WN && wn + at < cols) {
                    float z = 0.0f;
#pragma unroll
                    for (int j = 0; j < NI; j++)
#pragma unroll
                        for (int e = 0; e < 16; e++) z = j * 32 + result_col(e, half) == at ? acc[i][j][e] : z;
                    if ((at >> 2 & 1) == half) a.picked[token] = z;
                }
            }
        }
        __syncthreads();
        for (uint32_t m = tid; m < BM; m += WAVES * 64) {
            if (m0 + m >= a.tokens) continue;
            float top = part[m].x;
#pragma unroll
            for (int w = 1; w < WN; w++) top = fmaxf(top, part[w * BM + m].x);
            const float from = __builtin_isinf(top) ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < WN; w++) {
                const float2 v = part[w * BM + m];
                sum += v.y * exp_of<T>(v.x - from);
            }
            a.stats[(uint64_t)tn * a.tokens + m0 + m] = make_float2(top, sum);
        }
    } else {
        [[maybe_unused]] constexpr uint32_t PART = 32 * NI * 32;  // results of a wave on their way out
        if constexpr (OP == kGrad) {
            if (KS > 1 && group) return;
            static_assert(WAVES * PART * T::ESZ <= S * STAGE, "the results' way out fits the ring");
            const uint32_t cols = a.piece[p].len - n0;
            Coef c[MI];
            bool live[MI];
#pragma unroll
            for (int i = 0; i < MI; i++) {
                const uint32_t token = m0 + wm + i * 32 + r;
                c[i] = a.coef[token < a.rows_a ? token : a.rows_a - 1];
                live[i] = (c[i].a != 0.0f) | (c[i].b != 0.0f);  // NaN too
                c[i].target -= a.piece[p].first + n0 + wn;
            }
            drain<T, MI, NI>(&ring[0][0] + wave * PART * T::ESZ, lane,
                [&](int i, int j, int e) {
                    const uint32_t col = j * 32 + result_col(e, half);
                    float g = c[i].a * exp_of<T>(acc[i][j][e] - c[i].lse);
                    g = col == c[i].target ? g - c[i].b : g;
                    return (live[i] & (wn + col < cols)) ? g : 0.0f;
                },
                [&](uint32_t row, uint32_t col, u32x4 x) {
                    const uint32_t token = m0 + wm + row;
                    if (token < a.rows_a) st16<false>(a.out + token * a.pitch_out + (uint64_t)(a.piece[p].col + n0 + wn + col) * T::ESZ, x);
                });
        } else if constexpr (OP == kGradT) {
            // a lane has a row of the transpose, four consecutive tokens at a time
            const uint32_t cols = a.piece[p].len - n0;
            if (KS > 1 && group) return;
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    const uint32_t token = m0 + wm + i * 32 + result_col(4 * g, half);
                    Coef c[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) c[e] = a.coef[token + e];
#pragma unroll
                    for (int j = 0; j < NI; j++) {
                        const uint32_t col = wn + j * 32 + r, v = a.piece[p].first + n0 + col;
                        float hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            float x = c[e].a * exp_of<T>(acc[i][j][4 * g + e] - c[e].lse);
                            x = v == c[e].target ? x - c[e].b : x;
                            hi[e] = (((c[e].a != 0.0f) | (c[e].b != 0.0f)) & (col < cols)) ? x : 0.0f;
                            const float kept = T::widen(T::narrow(hi[e]));
                            lo[e] = __builtin_isfinite(kept) ? hi[e] - kept : 0.0f;
                        }
                        char* const to = a.out + (uint64_t)(a.piece[p].col + n0 + col) * a.pitch_out + token * T::ESZ;
                        const Quad<T> h(hi), l(lo);
                        if constexpr (T::ESZ == 4) {
                            *(u32x4*)to = u32x4{h.w[0], h.w[1], h.w[2], h.w[3]};
                        } else {
                            *(u32x2*)to = u32x2{h.w[0], h.w[1]};
                            *(u32x2*)(to + a.rows_a * T::ESZ) = u32x2{l.w[0], l.w[1]};
                        }
                    }
                }
        } else if constexpr (OP == kDsums || OP == kDsumsT) {
            static_assert(WAVES * PART * 4 <= S * STAGE, "the results' way out fits the ring");
            char* const out = a.out + blockIdx.y * (uint64_t)a.tokens * a.pitch_out;
            drain<F32, MI, NI>(&ring[0][0] + wave * PART * 4, lane, [&](int i, int j, int e) { return acc[i][j][e]; },
                [&](uint32_t row, uint32_t col, u32x4 x) {
                    const uint64_t m = m0 + wm + row;
                    const uint32_t n = n0 + wn + col;
                    if (m >= a.tokens || n >= a.width) return;  // rows of sums are padded to whole vectors
                    char* const to = out + m * a.pitch_out + (uint64_t)n * 4;
                    if (!a.first_piece) {
                        const u32x4 old = ld16<false>(to);
#pragma unroll
                        for (int e = 0; e < 4; e++) x[e] = __float_as_uint(__uint_as_float(old[e]) + __uint_as_float(x[e]));
                    }
                    st16<false>(to, x);
                });
        } else {
            const float u = a.unscale ? *a.unscale : 1.0f;
            const uint32_t rows = DWEIGHT ? a.piece[p].len : a.tokens;
            char* const out = DWEIGHT ? a.piece[p].out : a.out;
            static_assert(WAVES * PART * T::ESZ <= S * STAGE, "the results' way out fits the ring");
            drain<T, MI, NI>(&ring[0][0] + wave * PART * T::ESZ, lane, [&](int i, int j, int e) { return acc[i][j][e] * u; },
                [&](uint32_t row, uint32_t col, u32x4 x) {
                    const uint64_t m = m0 + wm + row;
                    const uint32_t n = n0 + wn + col;
                    if (m < rows && n < a.width) store_some<T>(out + m * a.pitch_out + (uint64_t)n * T::ESZ, x, a.width - n);
                });
        }
    }
}

// DWEIGHT of up to kStreamTokens: a stream of stores (32 tokens, 65536 x 4096 bf16: 114 us of
// 107 for the bytes; from 64 on tiles take no longer: 166 us of tiles, 172 of this).  A wave keeps the hidden states of its NI x
// 32 columns in registers and walks a run of the vocabulary, 32 rows at a time, whose
// rows of G's transpose (`steps` granules a lane, the next 32 rows' under way while these
// are multiplied) are its other operand.  Neighbouring waves have neighbouring columns
// of the same rows, so that lines of a row are written at about the same time.
// a.b: the hidden states' transpose, [columns, STEPS * 2 granules].
template <class T, int STEPS, int NI>
__global__ __launch_bounds__(512) void k_entropy_dweight_few(EntropyArgs a, uint32_t waves)
{
    constexpr int PARTS = T::ESZ == 2 ? 2 : 1;
    constexpr uint32_t PART = 32 * NI * 32;
    __shared__ __attribute__((aligned(16))) char out[8][PART * T::ESZ];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = lane & 31, half = lane >> 5, id = blockIdx.x * 8 + wave;
    if (id >= waves) return;  // no barrier follows
    const uint32_t groups = a.tiles_n, runs = waves / groups, run = id / groups, n0 = id % groups * (NI * 32);
    const uint32_t t0 = (uint32_t)(a.ktiles * (uint64_t)run / runs), t1 = (uint32_t)(a.ktiles * (uint64_t)(run + 1) / runs);
    if (t0 >= t1) return;
    u32x4 y[STEPS][NI];
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const uint32_t col = n0 + j * 32 + r;
        const char* from = a.b + (col < a.width ? col : a.width - 1) * a.pitch_b + half * 16;
#pragma unroll
        for (int s = 0; s < STEPS; s++) y[s][j] = ld16<false>(from + s * 32);
    }
    int p = 0;
    while (p + 1 < a.pieces && t0 >= a.piece[p + 1].tile) p++;
    const float u = *a.unscale;
    u32x4 x[PARTS * STEPS];
    const auto fetch = [&](uint32_t t, int q) {  // rows past a piece's end are zero or those of a multiple of 256, and not stored
        const char* from = a.a + (uint64_t)(a.piece[q].col + (t - a.piece[q].tile) * 32 + r) * a.pitch_a + half * 16;
#pragma unroll
        for (int s = 0; s < PARTS * STEPS; s++) x[s] = ld16<false>(from + s * 32);
    };
    fetch(t0, p);
    for (uint32_t t = t0; t < t1; t++) {
        f32x16 acc[1][NI] = {};
#pragma unroll
        for (int s = 0; s < PARTS * STEPS; s++)
#pragma unroll
            for (int j = 0; j < NI; j++) acc[0][j] = tile_mfma<T>(y[s % STEPS][j], x[s], acc[0][j]);
        const uint32_t v0 = (t - a.piece[p].tile) * 32, rows = a.piece[p].len;
        char* const to = a.piece[p].out;
        if (t + 1 < t1) {
            p += p + 1 < a.pieces && t + 1 >= a.piece[p + 1].tile;
            fetch(t + 1, p);
        }
        drain<T, 1, NI>(out[wave], lane, [&](int i, int j, int e) { return acc[i][j][e] * u; },
            [&](uint32_t row, uint32_t col, u32x4 v) {
                const uint32_t n = n0 + col;
                if (v0 + row < rows && n < a.width) store_some<T>(to + (v0 + row) * a.pitch_out + (uint64_t)n * T::ESZ, v, a.width - n);
            });
    }
}

// ---------------------------------------------------------------------------
// What stands around the products.
// ---------------------------------------------------------------------------

__device__ __forceinline__ float group_max(float v, float* lds)
{
#pragma unroll
    for (int m = 32; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
    for (uint32_t w = 1; w < blockDim.x / 64; w++) v = fmaxf(v, lds[w]);
    return v;
}

// (maximum, sum of exponentials of the differences from it) of two sets together.  A
// maximum that is infinite takes differences from 0 instead, whose exponentials are 0 and
// infinity; NaN stays in the sum.
__device__ __forceinline__ float2 join_sums(float2 p, float2 q)
{
    const float top = fmaxf(p.x, q.x), from = __builtin_isinf(top) ? 0.0f : top;
    return make_float2(top, p.y * expf(p.x - from) + q.y * expf(q.x - from));
}

// The tiles' maxima and sums of each token, joined: RUNS lanes have a token, whose tiles
// they take in turn.  16 lanes, so that neighbouring ones read neighbouring tokens;
// where tokens are few 256, as a lane's tiles follow one another at memory's latency (one
// token's 512 tiles: 17 us with 16 lanes, 4 us with 256; a loss over 65536 of width 64 of 64 tokens 20.0
// and 9.7, 1,024 39.8 and 37.7, 2,048 68.2 and 71.6).
template <int RUNS>
__global__ __launch_bounds__(256) void k_entropy_loss(const float2* stats, const float* picked, uint32_t tiles, uint32_t tokens,
                                                      const long long* target, long long ignore, uint32_t vocab, float* loss,
                                                      float* lse)
{
    constexpr uint32_t TOKENS = 256 / RUNS;
    __shared__ float2 part[RUNS][TOKENS + 1];
    const uint32_t c = threadIdx.x % TOKENS, run = threadIdx.x / TOKENS, token = blockIdx.x * TOKENS + c;
    float2 s = make_float2(-INFINITY, 0.0f);
    if (token < tokens)
        for (uint32_t i = run; i < tiles; i += RUNS) s = join_sums(s, stats[(uint64_t)i * tokens + token]);
    part[run][c] = s;
    __syncthreads();
    for (uint32_t half = RUNS / 2; half; half /= 2) {
        if (run < half) part[run][c] = join_sums(part[run][c], part[run + half][c]);
        __syncthreads();
    }
    if (run || token >= tokens) return;
    s = part[0][c];
    const float l = (__builtin_isinf(s.x) ? 0.0f : s.x) + logf(s.y);
    lse[token] = l;
    if (!loss) return;
    const long long t = target[token];
    loss[token] = t == ignore ? 0.0f : (unsigned long long)t < vocab ? l - picked[token] : __builtin_nanf("");
}

// What the gradient's launches share of the call.
struct TokenArgs {
    const long long* target;
    const float* lse;
    const float* dloss;
    const float* dlse;  // or null
    long long ignore;
    uint32_t vocab, tokens, padded;
};

__device__ __forceinline__ Coef coef_of(const TokenArgs& a, uint32_t t)
{
    const long long at = a.target[t];
    const bool none = at == a.ignore, bad = !none && (unsigned long long)at >= a.vocab;
    const float dloss = a.dloss[t], dlse = a.dlse ? a.dlse[t] : 0.0f;
    Coef c;
    c.b = none ? 0.0f : dloss;
    c.a = c.b + dlse;
    if (bad && (c.a != 0.0f || c.b != 0.0f)) c.a = __builtin_nanf("");  // without weight it has no gradient to spoil
    c.lse = a.lse[t];
    c.target = none || bad ? kNoTarget : (uint32_t)at;
    return c;
}

// Whether a token has any gradient; what the others' hidden states hold reaches nothing.
__device__ __forceinline__ bool live(const TokenArgs& a, uint32_t t)
{
    if (t >= a.tokens) return false;
    const Coef c = coef_of(a, t);
    return c.a != 0.0f || c.b != 0.0f;
}

// The tokens' coefficients, by one workgroup.  16-bit G is held in units of the largest
// |a| or |b| (fp16: 2^-14 of it): the targets' elements of a loss whose tokens weigh
// the same are then rounded from 1 - p instead of from an arbitrary weight, and the loss's
// scale does not matter.  fp16 then keeps all bits of elements from 2^-28 of the largest on; smaller
// ones are multiples of 2^-38 of it.  A unit for each token would save those of tokens that weigh little
// from one product, by the hidden states' rows, and lose as much in the other, whose sum is over
// tokens.  scale[0]: one such unit.
template <class T>
__device__ __forceinline__ void write_coefs(const TokenArgs& a, Coef* coef, float* scale, float* lds)
{
    const uint32_t lanes = blockDim.x;
    float unit = 1.0f, up = 1.0f;
    if constexpr (T::ESZ == 2) {
        float most = 0.0f;
        for (uint32_t t = threadIdx.x; t < a.tokens; t += lanes) {
            const Coef c = coef_of(a, t);
            const float x = fmaxf(fabsf(c.a), fabsf(c.b));
            most = fmaxf(most, __builtin_isfinite(x) ? x : 0.0f);
        }
        most = group_max(most, lds);
        // between 2^-100 and 2^100, where neither the unit nor its inverse leaves fp32's range
        most = most == 0.0f ? 1.0f : fminf(fmaxf(most, 0x1p-100f), 0x1p100f);
        unit = __is_same(T, F16) ? most * 0x1p-14f : most;
        up = 1.0f / unit;
    }
    for (uint32_t t = threadIdx.x; t < a.padded; t += lanes) {
        Coef c = {0.0f, 0.0f, 0.0f, kNoTarget};
        if (t < a.tokens) {
            c = coef_of(a, t);
            c.a *= up;
            c.b *= up;
        }
        coef[t] = c;
    }
    if (threadIdx.x == 0) scale[0] = unit;
}

// Matrices of one width, and how many rows of each there are and are written.
struct PackArgs {
    const char* src[kMaxRanks];
    char* dst[kMaxRanks];
    uint32_t rows[kMaxRanks], padded[kMaxRanks];
};

// Granule g of a row of `width` elements, zero behind its end.
template <class T>
__device__ __forceinline__ u32x4 row_granule(const char* row, uint32_t g, uint32_t width)
{
    const uint32_t col = g * T::VEC;
    if (col + T::VEC <= width) return ld16<false>(row + (uint64_t)g * 16);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t e = 0; e < T::VEC; e++) {
        if (col + e >= width) continue;
        const uint32_t s = load_s<T>(row + (uint64_t)(col + e) * T::ESZ);
        if constexpr (T::ESZ == 4) w[e] = s;
        else w[e / 2] |= s << (16 * (e & 1));
    }
    return u32x4{w[0], w[1], w[2], w[3]};
}

// Rows at a pitch of whole tiles, zero behind each row's end and behind the last row.
// `lanes` (a power of two up to 256) have a row.
template <class T>
__global__ __launch_bounds__(256) void k_entropy_pack(PackArgs a, uint32_t width, uint32_t granules, uint32_t lanes)
{
    const uint32_t m = blockIdx.y, per = 256 / lanes, lane = threadIdx.x & (lanes - 1);
    for (uint32_t row = blockIdx.x * per + threadIdx.x / lanes; row < a.padded[m]; row += gridDim.x * per) {
        const char* from = a.src[m] + (uint64_t)row * width * T::ESZ;
        for (uint32_t g = lane; g < granules; g += lanes) {
            u32x4 x = {0, 0, 0, 0};
            if (row < a.rows[m]) x = row_granule<T>(from, g, width);
            st16<false>(a.dst[m] + ((uint64_t)row * granules + g) * 16, x);
        }
    }
}

// What the gradient's products start from, in one launch of 1024 lanes a workgroup (the
// coefficients' one takes the longest: 4096 tokens 22 us with 256).  blockIdx.y 0: the tokens'
// coefficients (one workgroup); 1: the hidden states packed, rows of tokens without
// gradient zero, so that what those hold reaches no product; 2 (for k_entropy_dweight_few): their
// transpose, [width][padded].
template <class T>
__global__ __launch_bounds__(1024) void k_entropy_prepare(TokenArgs a, const char* hidden, uint32_t width, uint32_t granules,
                                                         uint32_t lanes, char* packed, char* transpose, Coef* coef, float* scale)
{
    __shared__ float lds[16];
    if (blockIdx.y == 0) {
        if (blockIdx.x == 0) write_coefs<T>(a, coef, scale, lds);
    } else if (blockIdx.y == 1) {
        const uint32_t per = 1024 / lanes, lane = threadIdx.x & (lanes - 1);
        for (uint32_t row = blockIdx.x * per + threadIdx.x / lanes; row < a.padded; row += gridDim.x * per) {
            // loaded whether the token is live or not: the two do not wait for each other
            const char* from = hidden + (uint64_t)row * width * T::ESZ;
            bool has = false;
            for (uint32_t g = lane; g < granules; g += 4 * lanes) {
                u32x4 x[4] = {};
#pragma unroll
                for (uint32_t i = 0; i < 4; i++)
                    if (row < a.tokens && g + i * lanes < granules) x[i] = row_granule<T>(from, g + i * lanes, width);
                if (g == lane) has = live(a, row);
#pragma unroll
                for (uint32_t i = 0; i < 4; i++) {
#pragma unroll
                    for (int e = 0; e < 4; e++) x[i][e] = has ? x[i][e] : 0;
                    if (g + i * lanes < granules) st16<false>(packed + ((uint64_t)row * granules + g + i * lanes) * 16, x[i]);
                }
            }
        }
    } else {
        static_assert(kStreamTokens <= 64, "a bit of the wave's mask for each token");
        const uint64_t mask = __ballot(live(a, threadIdx.x & 63));
        const uint32_t each = a.padded / T::VEC;  // granules of a column
        const uint64_t count = (uint64_t)width * each;
        for (uint64_t i = blockIdx.x * 1024ull + threadIdx.x; i < count; i += gridDim.x * 1024ull) {
            const uint32_t g = (uint32_t)(i / width), col = (uint32_t)(i - (uint64_t)g * width);
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (uint32_t e = 0; e < T::VEC; e++) {
                const uint32_t t = g * T::VEC + e;
                uint32_t v = 0;
                if (a.tokens) v = load_s<T>(hidden + ((uint64_t)(t < a.tokens ? t : a.tokens - 1) * width + col) * T::ESZ);
                const uint32_t s = mask >> t & 1 ? v : 0;
                if constexpr (T::ESZ == 4) w[e] = s;
                else w[e / 2] |= s << (16 * (e & 1));
            }
            st16<false>(transpose + ((uint64_t)col * a.padded * T::ESZ + g * 16), u32x4{w[0], w[1], w[2], w[3]});
        }
    }
}

// out = unscale x the sums of every split and, in it, of every part (few tokens: of G
// rounded and of what that left), rounded: in their order within each of RUNS interleaved
// runs and then of the runs.  16 runs where there are many sums (eight and more), which one
// lane would fetch one after the other (3 tokens of 17 values, 109 splits: 27 us; the gradient by hidden
// states of 33 tokens, 4000 x 512, 24.5 us with one run and 22.6 with 16, of 300, 65536 x 1024, 155.8 and 157.4).
template <class T, int RUNS>
__global__ __launch_bounds__(256) void k_entropy_join(const float* sums, uint32_t count, uint32_t rows, uint32_t tokens,
                                                      uint32_t width, uint32_t pitch, const float* unscale, char* out)
{
    constexpr uint32_t QUADS = 256 / RUNS;
    __shared__ float part[RUNS > 1 ? RUNS : 1][QUADS][RUNS > 1 ? 4 : 1];
    const float u = *unscale;
    const uint32_t c = threadIdx.x % QUADS, run = threadIdx.x / QUADS, q = blockIdx.x * QUADS + c, quads = (width + 3) / 4;
    for (uint32_t row = blockIdx.y; row < tokens; row += gridDim.y) {
        float s[4] = {};
        if (q < quads) {
#pragma unroll 4
            for (uint32_t i = run; i < count; i += RUNS) {
                float v[4];
                F32::unpack(ld16<false>((const char*)(sums + ((uint64_t)i * rows + row) * pitch + q * 4)), v);
#pragma unroll
                for (int e = 0; e < 4; e++) s[e] += v[e];
            }
        }
        if constexpr (RUNS > 1) {
#pragma unroll
            for (int e = 0; e < 4; e++) part[run][c][e] = s[e];
            __syncthreads();
            if (run == 0)
                for (int i = 1; i < RUNS; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) s[e] += part[i][c][e];
            __syncthreads();
        }
        if (run || q >= quads) continue;
        char* const to = out + ((uint64_t)row * width + q * 4) * T::ESZ;
        const uint32_t left = width - q * 4;
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (e < (int)left) store_s<T>(to + e * T::ESZ, T::narrow(s[e] * u));
    }
}

template <class T>
__global__ __launch_bounds__(256) void k_entropy_zero(char* out, uint64_t count)
{
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < count; i += gridDim.x * 256ull) store_s<T>(out + i * T::ESZ, 0);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
using namespace host;

constexpr uint64_t kCus = 256;               // of the card this library is built for; plans do not ask the device
constexpr uint64_t kPieceBytes = 128u << 20; // G of one piece of the vocabulary: half the last-level cache
constexpr uint64_t kPackBytes = 1u << 30;    // packed weights of one piece: enough tiles for all CUs

inline uint64_t up_to(uint64_t x, uint64_t m) { return (x + m - 1) / m * m; }

// What fp32 tiles take: rounds of one a CU, times what a tile of that kind takes.  A tile of 64
// is a quarter of one of 128 and takes a twentieth more for its work, and a seventh where its
// contraction is split.
constexpr uint64_t kTile128 = 80, kTile64 = 21, kTile64Split = 23;
inline uint64_t rounds(uint64_t tiles, uint64_t each) { return (tiles + kCus - 1) / kCus * each; }

// What one call does, from its sizes and alignments alone, so that the workspace's
// size can be asked for beforehand.
template <class T>
struct EntropyPlan {
    static constexpr uint64_t KT = kTileK<T>;
    bool few = false, stream = false; // tokens: up to kFewTokens, kStreamTokens
    bool fine = false;                // LOGITS by the smallest tiles
    uint64_t parts = 1, rows = 0;     // of G's elements (few tokens); rows of DHIDDEN's sums, parts of `padded` each
    uint64_t vocab = 0, columns = 0;  // the whole; the same with each rank's rounded up to 256
    uint64_t padded, wide;            // tokens rounded up to 64; elements of a packed row
    bool pack_hidden, pack_weight, cut;
    uint64_t piece;                   // columns of a piece at most, a multiple of 256
    uint64_t tokens;                  // of one pass (the loss)
    int side = 0, splits = 1;         // of DHIDDEN: of a tile; of its contraction
    bool sums = false;                // whether DHIDDEN goes by fp32 sums
    uint64_t at_hidden = 0, at_transpose = 0, at_weight = 0, at_stats = 0, at_picked = 0, at_coef = 0, at_scale = 0, at_g = 0, at_sums = 0, bytes = 0;

    uint64_t take(uint64_t size)
    {
        const uint64_t at = bytes;
        bytes += up_to(size, 256);
        return at;
    }
    static bool direct(uint64_t width, uintptr_t p) { return width * T::ESZ % 16 == 0 && p % 16 == 0; }
    uint64_t pieces_of(uint64_t piece_columns) const { return (columns + piece_columns - 1) / piece_columns; }

    EntropyPlan(const EntropyCall& c, bool gradient)
    {
        pack_weight = false;
        uint64_t along = 0;
        for (int r = 0; r < c.n; r++) {
            vocab += c.vocab[r];
            along += (c.vocab[r] + 63) / 64;
            columns += up_to(c.vocab[r], 256);
            if (c.vocab[r]) pack_weight |= !direct(c.width, (uintptr_t)c.weight[r]);
        }
        wide = up_to(c.width, KT);
        few = gradient && c.tokens <= kFewTokens;
        stream = gradient && c.tokens <= kStreamTokens;
        padded = few ? (c.tokens <= 32 ? 32 : c.tokens <= 64 ? 64 : 128) : up_to(c.tokens ? c.tokens : 1, 64);
        parts = few && T::ESZ == 2 ? 2 : 1;
        rows = few ? parts * padded : c.tokens;
        fine = T::ESZ == 4 && !few && (c.tokens + 63) / 64 * along <= 2 * kCus;
        cut = c.width % KT != 0 && !pack_weight;
        // the gradient's hidden states are always packed: rows of tokens without gradient are zero
        pack_hidden = gradient ? true : c.width % KT != 0 || !direct(c.width, (uintptr_t)c.hidden);
        piece = up_to(columns, 256);
        if (pack_weight) piece = limit(piece, kPackBytes / (wide * T::ESZ), 256);
        tokens = c.tokens;
        if (!gradient) {
            tokens = c.tokens < 16384 ? c.tokens : 16384;
            if (pack_hidden) at_hidden = take(c.tokens * wide * T::ESZ);
            if (pack_weight) at_weight = take(piece * wide * T::ESZ);
            at_stats = take(columns / (T::ESZ == 4 && (tokens <= 64 || fine) ? 32 : 64) * tokens * sizeof(float2));
            at_picked = take(tokens * sizeof(float));
            return;
        }
        if (columns == 0) return;
        // pieces of a few thousand columns at least, so that the sums over them cost little
        piece = limit(piece, kPieceBytes / (padded * parts * T::ESZ), 4096);
        piece = up_to((columns + pieces_of(piece) - 1) / pieces_of(piece), 256);  // of about one size
        at_coef = take(padded * sizeof(Coef));
        at_scale = take(16);
        at_hidden = take(padded * wide * T::ESZ);
        if (pack_weight) at_weight = take(piece * wide * T::ESZ);
        if (stream && c.want_dweight) at_transpose = take(c.width * padded * T::ESZ);
        at_g = take(few ? piece * pitch_gt() : padded * pitch_g());
        if (c.want_dhidden) {
            // Few tiles: the contraction is split until each CU has one (256 x 256) or two,
            // of four tiles at least.
            const auto tiles = [&](uint64_t bm, uint64_t bn) { return ((rows + bm - 1) / bm) * ((c.width + bn - 1) / bn); };
            const auto parts_of = [&](uint64_t bm, uint64_t bn) {
                uint64_t s = (bm == 256 ? kCus : 2 * kCus) / tiles(bm, bn);
                const uint64_t most = piece / KT / 4;
                s = s < most ? s : most;
                return s < 1 ? 1 : s > 128 ? 128 : s;
            };
            // Sides of 16-bit types, us with 64, 128 and 256 (the hidden states' gradient alone): 200 x 16384 x 512,
            // 8 tiles of 128, 39, 40, 40; 200 x 65536 x 1024, 16 of 128, 136, 119, 108.  128 and 256 are within a
            // tenth of each other from 8 to 32 tiles of 256, as the contraction is split over all CUs in any case:
            // 8 tiles, 500 x 16384 x 1024, 67, 67, 73, but 500 x 65536 x 1024 238, 193, 173; 16 tiles, 1024 x 65536
            // x 1024, 440, 338, 298; 32 tiles, 300 x 65536 x 4096, 782, 462, 484.
            if (!few) side = T::ESZ == 2 && tiles(256, 256) > 8 ? 256 : tiles(128, 128) > 8 ? 128 : 64;
            if (T::ESZ == 4 && side == 128) {
                const uint64_t t64 = tiles(64, 64), t128 = tiles(128, 128), s64 = parts_of(64, 64), s128 = parts_of(128, 128);
                // 315 x 1915 x 5678: 108 us with its join and 89; 515 x 35809 x 864: 351 and 367
                if (rounds(t64 * s64, kTile64Split) * s128 < rounds(t128 * s128, kTile128) * s64) side = 64;
            }
            const uint64_t bm = few ? rows : side, bn = few ? (rows == 256 ? 256 : 128) : side;
            splits = (int)parts_of(bm, bn);
            sums = few || splits > 1 || pieces_of(piece) > 1;
            if (sums) at_sums = take((uint64_t)splits * rows * wide * sizeof(float));
        }
    }
    // At most `most` columns (rounded down to 256), but no fewer than `least`.
    static uint64_t limit(uint64_t piece, uint64_t most, uint64_t least)
    {
        most = most / 256 * 256;
        most = most > least ? most : least;
        return piece < most ? piece : most;
    }
    // A row of G: 128 bytes more than its columns, so that rows start on other memory channels.
    uint64_t pitch_g() const { return piece * T::ESZ + 128; }
    // Rows from one part of the sums to the next.
    uint64_t padded_rows() const { return few ? padded : rows; }
    uint64_t pitch_gt() const { return padded * parts * T::ESZ; }
};

// The pieces of the vocabulary, a few at a time: `columns` of them at most.
struct PieceWalk {
    const EntropyCall& c;
    uint64_t columns;
    int r = 0;
    uint64_t at = 0;     // of rank r's rows
    uint64_t first = 0;  // of the whole vocabulary

    // The next launch's pieces; tile sizes are set by the caller.
    int next(Piece* piece, int esz)
    {
        int n = 0;
        uint64_t col = 0;
        while (r < c.n && col < columns && n < kMaxRanks) {
            const uint64_t left = c.vocab[r] - at, room = columns - col;
            if (left == 0) {
                r++;
                at = 0;
                continue;
            }
            const uint64_t len = left < room ? left : room, row = c.width * (uint64_t)esz;
            Piece& q = piece[n++];
            q = {};
            q.w = c.weight[r] + at * row;
            q.out = c.dweight[r] ? c.dweight[r] + at * row : nullptr;
            q.len = (uint32_t)len;
            q.first = (uint32_t)first;
            q.col = (uint32_t)col;
            col += up_to(len, 256);
            first += len;
            at += len;
        }
        return n;
    }
};

template <class T, int OP, int BM, int BN, int WM, int WN, int S, int KS = 1>
vrc_status_t launch_entropy(EntropyArgs& a, uint64_t rows, uint64_t cols, bool cut, int splits, hipStream_t st)
{
    a.tiles_m = (uint32_t)((rows + BM - 1) / BM);
    a.tiles_n = (uint32_t)((cols + BN - 1) / BN);
    constexpr bool DHIDDEN = OP == kDhidden || OP == kDsums || OP == kDsumsT;
    if constexpr (DHIDDEN) {
        uint32_t t = 0;
        for (int i = 0; i < a.pieces; i++) {
            a.piece[i].tile = t;
            t += (uint32_t)((a.piece[i].len + kTileK<T> - 1) / kTileK<T>);
        }
        a.ktiles = t;
    } else {
        constexpr bool DWEIGHT = OP == kDweight || OP == kDweightT;
        constexpr uint32_t B = DWEIGHT ? BM : BN;
        uint32_t t = 0;
        for (int i = 0; i < a.pieces; i++) {
            a.piece[i].tile = t;
            t += (a.piece[i].len + B - 1) / B;
        }
        (DWEIGHT ? a.tiles_m : a.tiles_n) = t;
    }
    const uint64_t tiles = (uint64_t)a.tiles_m * a.tiles_n;
    constexpr int LANES = WM * WN * KS * 64;
    if (tiles * LANES > 0xffffffffull) return VRC_ERR_INVALID_ARG;  // not with sizes that the entry points let pass
    const dim3 grid((unsigned)tiles, (unsigned)splits);
    if constexpr (OP == kDweight || OP == kDweightT) {
        k_entropy<T, OP, BM, BN, WM, WN, S, false, KS><<<grid, LANES, 0, st>>>(a);
    } else if constexpr (DHIDDEN) {
        k_entropy<T, OP, BM, BN, WM, WN, S, false, KS><<<grid, LANES, 0, st>>>(a);
    } else {
        if (cut) k_entropy<T, OP, BM, BN, WM, WN, S, true, KS><<<grid, LANES, 0, st>>>(a);
        else k_entropy<T, OP, BM, BN, WM, WN, S, false, KS><<<grid, LANES, 0, st>>>(a);
    }
    return check_launch();
}

// Tiles of b x b in a product of rows x cols, whose vocabulary side (if any) is in pieces.
template <int OP>
uint64_t tiles_of(const EntropyArgs& a, uint64_t rows, uint64_t cols, uint64_t b)
{
    uint64_t along = 0;
    for (int i = 0; i < a.pieces; i++) along += (a.piece[i].len + b - 1) / b;
    if constexpr (OP == kStats || OP == kGrad) return (rows + b - 1) / b * along;
    else return (cols + b - 1) / b * along;
}

// The tile's side of a product of `tiles(b)` tiles of b x b: the smallest of which two a CU
// are enough (bf16, LOGITS with its join, us with sides of 64, 128 and 256: 80 x 8192 x 1024, 256 tiles of
// 64, 13.6, 19.9, 30.6; 500 x 4096 x 2048, 512 of 64, 20.4, 28.2, 47.6; 80 x 65536 x 4096, 512 of 128, 155,
// 111, 127; 1024 x 8192 x 1024, 512 of 128, 37, 26, 31; 200 x 65536 x 4096, 1,024 of 128, 239, 154, 126;
// 300 x 65536 x 4096, 1,536 of 128, 353, 214, 212; the gradients, whose LOGITS and DWEIGHT go by it, of
// 1024 x 8192 x 1024 115, 93, 106, of 1024 x 16384 x 1024 206, 145, 130).  fp32's matrix instructions take so long that the rounds in which CUs compute
// tiles decide (LOGITS of 900 x 9000 x 1000 in 7: 616 tiles of 128 273 us, 2,205 of 64 187;
// 2048 x 8192 x 512: 1,024 of 128 150 us, 4,096 of 64 157).
template <class T, class Tiles>
int tile_side(Tiles tiles)
{
    if constexpr (T::ESZ == 4) return rounds(tiles(64), kTile64) < rounds(tiles(128), kTile128) ? 64 : 128;
    if (tiles(64) <= 2 * kCus) return 64;
    return tiles(128) <= 2 * kCus ? 128 : 256;
}

// The product, by tiles of one side.
template <class T, int OP>
vrc_status_t launch_side(EntropyArgs& a, int side, uint64_t rows, uint64_t cols, bool cut, int splits, hipStream_t st)
{
    if (side == 64) return launch_entropy<T, OP, 64, 64, 2, 2, T::ESZ == 4 ? 2 : 4>(a, rows, cols, cut, splits, st);
    if constexpr (T::ESZ == 2)
        if (side == 256) return launch_entropy<T, OP, 256, 256, 2, 4, 2>(a, rows, cols, cut, splits, st);
    return launch_entropy<T, OP, 128, 128, 2, 2, 2>(a, rows, cols, cut, splits, st);
}

template <class T, int OP>
vrc_status_t launch_tiles(EntropyArgs& a, uint64_t rows, uint64_t cols, bool cut, hipStream_t st)
{
    const int side = tile_side<T>([&](uint64_t b) { return tiles_of<OP>(a, rows, cols, b); });
    return launch_side<T, OP>(a, side, rows, cols, cut, 1, st);
}

// LOGITS.  fp32's are bound by the matrix instructions: up to two tiles of 64 a CU, of which some
// CUs have twice as many as others, tiles of 32 by four waves that share the contraction are
// faster (LOGITS of 315 x 1915 x 5678 in 7, 175 tiles, 127 -> 83 us; 2285 x 462 x 3231 in 5, 360,
// 119 -> 90; 640 x 4096 x 1024, 640 tiles, 60 and 58, but 1024 tiles 78 and 89).
template <class T, int OP>
vrc_status_t launch_logits(EntropyArgs& a, uint64_t rows, bool fine, bool cut, hipStream_t st)
{
    if constexpr (T::ESZ == 4)
        if (fine) return launch_entropy<T, OP, 32, 32, 1, 1, 4, 4>(a, rows, 0, cut, 1, st);
    return launch_tiles<T, OP>(a, rows, 0, cut, st);
}

// Few rows (tokens): one tile has all of them, and its other side is as small as keeps two
// workgroups' rings in a CU's LDS.
template <class T, int OP>
vrc_status_t launch_few(EntropyArgs& a, uint64_t rows, uint64_t cols, bool cut, int splits, hipStream_t st)
{
    // fp32's are bound by the matrix instructions: where tiles of 128 columns leave CUs idle, of
    // 32 by four waves that share the contraction (28 x 191 x 768 20 -> 10.5 us, 48 x 20011 x 1000
    // 46 -> 43; but 64 x 65536 x 4096 305 -> 325)
    if (T::ESZ == 4 && OP != kDsumsT && tiles_of<kStats>(a, rows, cols, 128) <= kCus) {
        if constexpr (T::ESZ == 4 && OP != kDsumsT) {
            if (rows <= 32) return launch_entropy<T, OP, 32, 32, 1, 1, 4, 4>(a, rows, cols, cut, splits, st);
            if (rows <= 64) return launch_entropy<T, OP, 64, 32, 1, 1, 4, 4>(a, rows, cols, cut, splits, st);
        }
    }
    if (rows <= 32) return launch_entropy<T, OP, 32, 128, 1, 4, 4>(a, rows, cols, cut, splits, st);
    if (rows <= 64) return launch_entropy<T, OP, 64, 128, 1, 4, 3>(a, rows, cols, cut, splits, st);
    if constexpr (OP == kDsumsT && T::ESZ == 2)
        if (rows > 128) return launch_entropy<T, OP, 256, 256, 2, 4, 2>(a, rows, cols, cut, splits, st);
    return launch_entropy<T, OP, 128, 128, 2, 2, 2>(a, rows, cols, cut, splits, st);
}

template <class T>
vrc_status_t dweight_few(EntropyArgs& a, hipStream_t st)
{
    constexpr int STEPS = T::ESZ, NI = T::ESZ == 2 ? 4 : 2;  // steps of 32 bytes
    uint32_t t = 0;
    for (int i = 0; i < a.pieces; i++) {
        a.piece[i].tile = t;
        t += (a.piece[i].len + 31) / 32;
    }
    a.ktiles = t;
    a.tiles_n = (a.width + NI * 32 - 1) / (NI * 32);
    // two workgroups of eight waves a CU
    uint64_t runs = (2 * 8 * kCus + a.tiles_n - 1) / a.tiles_n;
    runs = runs < t ? runs : t;
    const uint64_t waves = runs * a.tiles_n;
    k_entropy_dweight_few<T, STEPS, NI><<<(unsigned)((waves + 7) / 8), 512, 0, st>>>(a, (uint32_t)waves);
    return check_launch();
}

// Lanes for a row of granules.
inline uint32_t row_lanes(uint32_t granules)
{
    uint32_t lanes = 8;
    while (lanes < 256 && lanes < granules) lanes *= 2;
    return lanes;
}

template <class T>
vrc_status_t pack(const PackArgs& p, int count, uint64_t width, uint64_t wide, hipStream_t st)
{
    const uint32_t granules = (uint32_t)(wide * T::ESZ / 16), lanes = row_lanes(granules);
    uint32_t most = 0;
    for (int i = 0; i < count; i++) most = p.padded[i] > most ? p.padded[i] : most;
    const uint32_t groups = most / (256 / lanes) + 1;
    k_entropy_pack<T><<<dim3(groups < 65536 ? groups : 65536, (unsigned)count), 256, 0, st>>>(p, (uint32_t)width, granules, lanes);
    return check_launch();
}

// The launch's pieces in the packed form.
template <class T>
vrc_status_t pack_pieces(const EntropyCall& c, const EntropyPlan<T>& plan, EntropyArgs& a, hipStream_t st)
{
    char* to = c.workspace + plan.at_weight;
    PackArgs p = {};
    for (int i = 0; i < a.pieces; i++) {
        p.src[i] = a.piece[i].w;
        p.dst[i] = to;
        p.rows[i] = p.padded[i] = a.piece[i].len;
        a.piece[i].w = to;  // one behind the other
        to += (uint64_t)a.piece[i].len * plan.wide * T::ESZ;
    }
    return pack<T>(p, a.pieces, c.width, plan.wide, st);
}

template <class T>
vrc_status_t cross_entropy_typed(const EntropyCall& c, hipStream_t st)
{
    const EntropyPlan<T> plan(c, false);
    const char* hidden = c.hidden;
    if (plan.pack_hidden) {
        char* const to = c.workspace + plan.at_hidden;
        PackArgs p = {};
        p.src[0] = c.hidden;
        p.dst[0] = to;
        p.rows[0] = p.padded[0] = (uint32_t)c.tokens;
        const vrc_status_t rc = pack<T>(p, 1, c.width, plan.wide, st);
        if (rc) return rc;
        hidden = to;
    }
    float2* const stats = (float2*)(c.workspace + plan.at_stats);
    float* const picked = (float*)(c.workspace + plan.at_picked);
    for (uint64_t t0 = 0; t0 < c.tokens; t0 += plan.tokens) {
        const uint64_t tokens = c.tokens - t0 < plan.tokens ? c.tokens - t0 : plan.tokens;
        uint64_t tiles = 0;
        PieceWalk walk = {c, plan.piece};
        EntropyArgs a = {};
        while ((a.pieces = walk.next(a.piece, T::ESZ)) != 0) {
            if (plan.pack_weight) {
                const vrc_status_t rc = pack_pieces(c, plan, a, st);
                if (rc) return rc;
                // packed they are one matrix, whose tiles cross the ranks' ends
                for (int i = 1; i < a.pieces; i++) a.piece[0].len += a.piece[i].len;
                a.pieces = 1;
            }
            a.pitch_a = (plan.pack_hidden ? plan.wide : c.width) * T::ESZ;
            a.pitch_b = (plan.pack_weight ? plan.wide : c.width) * T::ESZ;
            a.a = hidden + t0 * a.pitch_a;
            a.target = c.loss ? c.target + t0 : nullptr;
            a.stats = stats + tiles * tokens;
            a.picked = picked;
            a.tokens = a.rows_a = (uint32_t)tokens;
            a.kwidth = (uint32_t)c.width;
            a.ktiles = (uint32_t)(plan.wide / plan.KT);
            const vrc_status_t rc = tokens <= 64 ? launch_few<T, kStats>(a, tokens, 0, plan.cut, 1, st)
                                                 : launch_logits<T, kStats>(a, tokens, plan.fine, plan.cut, st);
            if (rc) return rc;
            tiles += a.tiles_n;
        }
        const long long* const target = c.loss ? c.target + t0 : nullptr;
        float* const loss = c.loss ? c.loss + t0 : nullptr;
        if (tokens <= 1024)
            k_entropy_loss<256><<<(unsigned)tokens, 256, 0, st>>>(stats, picked, (uint32_t)tiles, (uint32_t)tokens, target,
                                                                  c.ignore_index, (uint32_t)plan.vocab, loss, c.lse + t0);
        else
            k_entropy_loss<16><<<(unsigned)((tokens + 15) / 16), 256, 0, st>>>(stats, picked, (uint32_t)tiles, (uint32_t)tokens,
                                                                               target, c.ignore_index, (uint32_t)plan.vocab, loss,
                                                                               c.lse + t0);
        const vrc_status_t rc = check_launch();
        if (rc) return rc;
    }
    return VRC_OK;
}

template <class T>
vrc_status_t cross_entropy_grad_typed(const EntropyCall& c, hipStream_t st)
{
    const EntropyPlan<T> plan(c, true);
    if (plan.columns == 0) {  // nothing to add up
        if (c.want_dhidden) {
            const uint64_t count = c.tokens * c.width, groups = (count + 255) / 256;
            k_entropy_zero<T><<<(unsigned)(groups < 65536 ? groups : 65536), 256, 0, st>>>(c.dhidden, count);
            return check_launch();
        }
        return VRC_OK;
    }
    Coef* const coef = (Coef*)(c.workspace + plan.at_coef);
    float* const scale = (float*)(c.workspace + plan.at_scale);
    char* const hidden = c.workspace + plan.at_hidden;
    char* const g = c.workspace + plan.at_g;
    char* const sums = c.workspace + plan.at_sums;
    const TokenArgs tokens = {c.target, c.lse, c.dloss, c.dlse, c.ignore_index, (uint32_t)plan.vocab, (uint32_t)c.tokens, (uint32_t)plan.padded};
    const uint32_t granules = (uint32_t)(plan.wide * T::ESZ / 16), lanes = row_lanes(granules), groups = (uint32_t)plan.padded / (1024 / lanes) + 1;
    k_entropy_prepare<T><<<dim3(groups < 65536 ? groups : 65536, plan.stream && c.want_dweight ? 3 : 2), 1024, 0, st>>>(
        tokens, c.hidden, (uint32_t)c.width, granules, lanes, hidden, c.workspace + plan.at_transpose, coef, scale);
    vrc_status_t rc = check_launch();
    if (rc) return rc;

    EntropyArgs a = {};
    PieceWalk walk = {c, plan.piece};
    bool first = true;
    while ((a.pieces = walk.next(a.piece, T::ESZ)) != 0) {
        if (plan.pack_weight) {
            rc = pack_pieces(c, plan, a, st);
            if (rc) return rc;
        }
        const uint64_t pitch_w = (plan.pack_weight ? plan.wide : c.width) * T::ESZ;
        a.tokens = (uint32_t)c.tokens;
        a.width = (uint32_t)c.width;
        a.rows_a = (uint32_t)plan.padded;
        // G
        a.a = hidden;
        a.pitch_a = plan.wide * T::ESZ;
        a.pitch_b = pitch_w;
        a.kwidth = a.width;
        a.ktiles = (uint32_t)(plan.wide / plan.KT);
        a.coef = coef;
        a.out = g;
        a.pitch_out = plan.few ? plan.pitch_gt() : plan.pitch_g();
        rc = plan.few ? launch_few<T, kGradT>(a, plan.padded, 0, plan.cut, 1, st)
                      : launch_logits<T, kGrad>(a, plan.padded, plan.fine, plan.cut, st);
        if (rc) return rc;
        a.unscale = scale;
        a.a = g;
        a.pitch_a = a.pitch_out;
        if (c.want_dhidden) {
            a.pitch_b = pitch_w;
            a.granules = (uint32_t)(pitch_w / 16);
            a.first_piece = first;
            if (plan.sums) {
                a.out = sums;
                a.pitch_out = plan.wide * sizeof(float);
                a.tokens = (uint32_t)plan.rows;
                rc = plan.few ? launch_few<T, kDsumsT>(a, plan.rows, c.width, true, plan.splits, st)
                              : launch_side<T, kDsums>(a, plan.side, plan.rows, c.width, true, plan.splits, st);
            } else {
                a.out = c.dhidden;
                a.pitch_out = c.width * T::ESZ;
                rc = launch_side<T, kDhidden>(a, plan.side, c.tokens, c.width, true, 1, st);
            }
            if (rc) return rc;
        }
        if (c.want_dweight) {
            a.pitch_out = c.width * T::ESZ;
            a.b = hidden;
            a.pitch_b = plan.wide * T::ESZ;
            a.granules = (uint32_t)(plan.wide * T::ESZ / 16);
            if (plan.stream) {
                a.b = c.workspace + plan.at_transpose;
                a.pitch_b = plan.padded * T::ESZ;
                rc = dweight_few<T>(a, st);
            } else if (plan.few) {
                a.ktiles = (uint32_t)(plan.pitch_gt() / kTileRow);
                rc = launch_tiles<T, kDweightT>(a, 0, c.width, false, st);
            } else {
                a.ktiles = (uint32_t)(plan.padded / plan.KT);
                rc = launch_tiles<T, kDweight>(a, 0, c.width, false, st);
            }
            if (rc) return rc;
        }
        first = false;
    }
    if (!plan.sums) return VRC_OK;
    const uint32_t count = (uint32_t)(plan.splits * plan.parts), gy = (uint32_t)(c.tokens < 32768 ? c.tokens : 32768);
    const auto join = [&](auto runs) {
        constexpr int RUNS = decltype(runs)::value;
        constexpr uint64_t COLUMNS = 256 / RUNS * 4;
        k_entropy_join<T, RUNS><<<dim3((unsigned)((c.width + COLUMNS - 1) / COLUMNS), gy), 256, 0, st>>>(
            (const float*)sums, count, (uint32_t)plan.padded_rows(), (uint32_t)c.tokens, (uint32_t)c.width, (uint32_t)plan.wide,
            scale, c.dhidden);
    };
    if (count >= 8) join(std::integral_constant<int, 16>{});
    else join(std::integral_constant<int, 1>{});
    return check_launch();
}

}  // namespace
}  // namespace vrc
