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
//
// Measured on MI355X, random codes: 8 x (4096 x 8192 x 4096) summed, eight bf16
// outputs, 552 us with other operands at each call (3.98 PFLOP/s; 531 us with the same
// ones; 107 us of it are the 537 MB of stores at the end of each tile; the matrix pipes
// are busy for 53 % of all cycles); 8192 x 8192 x 8192 255 us (4.31).  The matrix
// instructions alone, operands from LDS but nothing loaded, take 213 us: random operands
// hold the clock down (205 us whole on zeros), and 41 us of either are tile starts and
// ends.  8 x (1 x 8192 x 4096) summed, a stream of 143 MB: 27.0 us, 5.3 TB/s (28.6 us
// under the profiler).
#include <hip/hip_runtime.h>

#include <utility>

#include "vrc_ops_host.hpp"

namespace vrc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
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
    uint64_t sm, sn;  // strides of C's rows and columns, and division by a row's
    FastDiv by_ktiles;  // tiles (the few-rows kernel)
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

// What a block past the end of a row is read from.
__device__ const u32x4 kZeroCodes = {0, 0, 0, 0};

// `x`, whose origin the compiler is not to see: an address is then a uniform base
// and a 32-bit lane offset, which a load takes as they are, instead of a 64-bit
// address per lane and load kept in registers over the whole loop.
__device__ __forceinline__ uint32_t opaque(uint32_t x)
{
    __asm__ volatile("" : "+v"(x));
    return x;
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

// A wave's results to its outputs: MI x NI matrix-instruction tiles at (row0, col0)
// of C, 32 rows at a time through `own`, the wave's part of LDS, so that they leave
// in 16-byte stores along the rows.  Row r's 16-byte piece c is at c ^ (r mod 8)
// (mod 4 where a row has four), which spreads a column over the banks.
template <class T, int MI, int NI>
__device__ __forceinline__ void store_results(const MatmulArgs& a, const f32x16 (&acc)[MI][NI], char* own, uint32_t lane,
                                              uint32_t row0, uint32_t col0, int dst0, int dst1)
{
    constexpr uint32_t PITCH = NI * 32 * T::ESZ, VECS = NI * 32 / T::VEC, MIX = VECS < 8 ? VECS - 1 : 7;
    const uint32_t r = lane & 31, half = lane >> 5;
#pragma unroll
    for (int i = 0; i < MI; i++) {
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const float v[4] = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                const Four<T> f(v);
                if constexpr (T::ESZ == 4) {
                    *(u32x4*)(own + r * PITCH + ((j * 8 + 2 * g + half) ^ (r & MIX)) * 16) =
                        u32x4{f.w[0], f.w[1], f.w[2], f.w[3]};
                } else {
                    *(u32x2*)(own + r * PITCH + ((j * 4 + g) ^ (r & MIX)) * 16 + half * 8) = u32x2{f.w[0], f.w[1]};
                }
            }
        __builtin_amdgcn_wave_barrier();
        for (uint32_t v = lane; v < 32 * VECS; v += 64) {
            const uint32_t row = row0 + i * 32 + v / VECS, col = col0 + v % VECS * T::VEC;
            const u32x4 x = *(const u32x4*)(own + v / VECS * PITCH + (v % VECS ^ (v / VECS & MIX)) * 16);
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
// Tiled product.  A workgroup of WM x WN waves has a BM x BN tile of C, a wave MI
// x NI matrix-instruction tiles of it.  The contraction's tiles come into a ring of
// S stages in LDS by direct loads (no registers), up to S - 1 ahead.
//
// LDS holds a row's eight 16-byte blocks with block j at place j ^ (row / 2 mod
// 8), so that the rows that a matrix operand reads at one block spread over all
// banks; the loads permute their global addresses within the row's 128 bytes to
// that end, as a direct load writes consecutive lanes to consecutive places.
//
// A row's scale bytes are in a memory line of their own, and a line costs the CU's
// cache as much as one of 128 bytes of codes, so where rows allow (EVEN: kb a
// multiple of 16, 16-byte aligned arrays) they come 16 at a time in the same way,
// with the first of each two tiles.  Else a lane reads a row's eight bytes a tile
// ahead and writes them to LDS, and blocks past a row's end come from a constant,
// zero codes, and have scale 1.
//
// The loop over the tiles has no branch in it.  Past the last tile it goes on
// fetching one word of it that nobody reads, so every wave always has the same
// number of loads under way, which is what its waits count; and with a branch the
// compiler moves the matrix instructions behind it, all four steps' operands live.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t place(uint32_t row, uint32_t block) { return block ^ (row >> 1 & 7); }

// A barrier behind this wave's LDS reads and writes, with its direct loads left
// under way (__syncthreads() may wait for them).
__device__ __forceinline__ void lds_barrier()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// A ring of S tiles, A's rows and then B's in each.
template <int ROWS, int S, bool EVEN>
struct Ring {
    char codes[S][ROWS * kTileBytes];
    u32x2 scales[EVEN ? S / 2 + 1 : S][ROWS][EVEN ? 2 : 1];  // a row's of two tiles or one
};

// One X a lane, lane l's to place l after `to` (a byte fills a dword there).
template <class X>
__device__ __forceinline__ void load_to_lds(global_ptr<const char> from, X* to)
{
    const auto g = (global_ptr<const void>)from;
    const auto l = (__attribute__((address_space(3))) void*)to;
    if constexpr (sizeof(X) == 16) __builtin_amdgcn_global_load_lds(g, l, 16, 0, 0);
    else if constexpr (sizeof(X) == 4) __builtin_amdgcn_global_load_lds(g, l, 4, 0, 0);
    else __builtin_amdgcn_global_load_lds(g, l, 1, 0, 0);
}

// Workgroup b's tile.  Workgroups are handed to the 8 XCDs in turn; each XCD takes
// a run of consecutive tiles, in groups of G rows of tiles walked column by
// column, so that the 32 or 64 tiles it works on at once share their operands'
// rows in its L2.
template <uint32_t G>
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn)
{
    const uint32_t total = tiles_m * tiles_n, each = total / 8, more = total % 8, x = b % 8;
    const uint32_t t = x * each + (x < more ? x : more) + b / 8;
    const uint32_t group = t / (G * tiles_n), left = tiles_m - group * G, rows = left < G ? left : G;
    const uint32_t i = t - group * G * tiles_n;
    tm = group * G + i % rows;
    tn = i / rows;
}

template <class T, bool SUM, bool EVEN, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(WM * WN * 64) void k_mx4_matmul_tiled(MatmulArgs a)
{
    constexpr int MI = BM / WM / 32, NI = BN / WN / 32, WAVES = WM * WN;
    constexpr int CODE_LOADS = (BM + BN) / 8 / WAVES;                      // of eight rows: 1 KiB
    constexpr int SCALE_LOADS = (BM + BN) / 64 / WAVES;  // a tile's (EVEN: two tiles'), of 64 rows
    constexpr int PAIR = EVEN ? 2 : 1;                   // tiles that scales come for at once
    constexpr int NB = EVEN ? S / 2 + 1 : S;             // scale buffers
    // Loads of the W tiles after one, where that one is (EVEN) the second of its two or the first.
    constexpr auto loads = [](int w, bool second) {
        return w * CODE_LOADS + (EVEN ? (second ? (w + 1) / 2 : w / 2) : w) * SCALE_LOADS;
    };
    static_assert((BM + BN) % (64 * WAVES) == 0 && BM % 64 == 0 && S >= 2, "loads are shared out evenly");
    static_assert(EVEN || (S == 2 && SCALE_LOADS == 1), "rows' scales pass through a lane's registers");
    static_assert(loads(S - 1, true) < 64, "the waits count at most 63 loads");
    __shared__ __attribute__((aligned(16))) Ring<BM + BN, S, EVEN> ring;

    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t tm, tn;
    tile_of<8>(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * BN;
    const uint32_t ktiles = (a.kb + kTileBlocks - 1) / kTileBlocks;
    const int q0 = SUM ? 0 : (int)blockIdx.y;
    const uint32_t total = ktiles * (SUM ? (uint32_t)a.ranks : 1u);
    const uint64_t row_bytes = (uint64_t)a.kb * 16;

    // This lane's part of each of its wave's loads, from the tile's first row (rows
    // past the end read the last one again).
    uint32_t off[CODE_LOADS], soff[SCALE_LOADS];
#pragma unroll
    for (int i = 0; i < CODE_LOADS; i++) {
        const uint32_t at = (wave * CODE_LOADS + i) * 8;
        const uint32_t row = (at >= BM ? at - BM : at) + lane / 8, last = at >= BM ? a.n - 1 - n0 : a.m - 1 - m0;
        off[i] = (row < last ? row : last) * (uint32_t)row_bytes + place(row, lane & 7) * 16;
    }
#pragma unroll
    for (int i = 0; i < SCALE_LOADS; i++) {
        const uint32_t at = (wave * SCALE_LOADS + i) * 64;
        const uint32_t row = (at >= BM ? at - BM : at) + lane, last = at >= BM ? a.n - 1 - n0 : a.m - 1 - m0;
        soff[i] = (row < last ? row : last) * a.kb;
    }
    int fq = q0;  // the next tile to fetch
    uint32_t fkt = 0, fetched = 0, fstage = 0, fbuf = 0;
    // A wave's loads are all of A's rows or all of B's, so it has one pair of arrays.
    constexpr uint32_t A_WAVES = BM / 8 / CODE_LOADS;
    static_assert(BM % (8 * CODE_LOADS) == 0, "a wave loads rows of one operand");
    const bool isb = wave >= A_WAVES;
    const uint64_t row0 = isb ? n0 : m0;
    global_ptr<const char> pcodes = nullptr, pscales = nullptr;
    uint32_t live = 0, left = 0;
    const auto aim = [&] {  // at the next tile
        live = fetched < total ? ~0u : 0u;
        left = a.kb - fkt * kTileBlocks;
        pcodes = (global_ptr<const char>)(isb ? a.bc[fq] : a.ac[fq]) + row0 * row_bytes + (uint64_t)fkt * kTileBytes;
        pscales = (global_ptr<const char>)(isb ? a.bs[fq] : a.as[fq]) + row0 * a.kb +
                  (EVEN ? fkt & ~1u : fkt) * kTileBlocks;  // past the end fkt may be odd
    };
    const auto load_codes = [&](int i) {
        const uint32_t at = (wave * CODE_LOADS + i) * 8;
        auto from = pcodes + opaque(off[i] & live);
        if constexpr (!EVEN)
            if ((place(at + lane / 8, lane & 7) & live) >= left) from = (global_ptr<const char>)&kZeroCodes;
        load_to_lds(from, (u32x4*)(ring.codes[fstage] + at * kTileBytes));
    };
    const auto load_scales = [&](int i) {
        const uint32_t at = (wave * SCALE_LOADS + i) * 64;
        load_to_lds(pscales + opaque(soff[i] & live), (u32x4*)ring.scales[fbuf][at]);
    };
    // !EVEN: this lane's row's eight bytes, to be written with keep_scales().  They
    // are read at most seven bytes early, where eight would end past the array (which
    // holds eight or more).
    uint64_t held = 0;
    uint32_t held_skip = 0, held_left = 0;
    const uint64_t array_end = (isb ? a.n : a.m) * (uint64_t)a.kb - 8;
    const auto hold_scales = [&] {
        const uint64_t want = row0 * a.kb + (soff[0] & live) + fkt * kTileBlocks, from = want < array_end ? want : array_end;
        typedef uint64_t u64_any __attribute__((aligned(1)));
        held = *(global_ptr<const u64_any>)((global_ptr<const char>)(isb ? a.bs[fq] : a.as[fq]) + from);
        held_skip = (uint32_t)(want - from);
        held_left = left < kTileBlocks ? left : kTileBlocks;
    };
    const auto keep_scales = [&](uint32_t to) {
        const uint64_t ones = held_left == kTileBlocks ? 0 : 0x7f7f7f7f7f7f7f7full << (8 * held_left);
        const uint64_t keep = held_left == kTileBlocks ? ~0ull : ~(~0ull << (8 * held_left));
        const uint64_t v = (held >> (8 * held_skip) & keep) | ones;
        ring.scales[to][tid][0] = u32x2{(uint32_t)v, (uint32_t)(v >> 32)};
    };
    const auto advance = [&](auto first) {
        if constexpr (decltype(first)::value) fbuf = fbuf + 1 == NB ? 0 : fbuf + 1;
        fstage = fstage + 1 == S ? 0 : fstage + 1;
        fetched++;
        const bool more = fetched < total, wrap = fkt + 1 == ktiles;
        fq += more && wrap;
        fkt = !more ? fkt : wrap ? 0 : fkt + 1;
    };
    const auto fetch = [&](auto first) {
        aim();
#pragma unroll
        for (int i = 0; i < CODE_LOADS; i++) load_codes(i);
        if constexpr (!EVEN) {
            hold_scales();
        } else if constexpr (decltype(first)::value) {
#pragma unroll
            for (int i = 0; i < SCALE_LOADS; i++) load_scales(i);
        }
        advance(first);
    };

    f32x16 acc[MI][NI] = {};
    const uint32_t wm = wave % WM * (BM / WM), wn = wave / WM * (BN / WN);
    const uint32_t r = lane & 31, half = lane >> 5;
    // A step's operands and a tile's scales, one ahead of the matrix instructions.
    u32x4 x[2][MI], y[2][NI];
    uint32_t sa[MI], sb[NI];
    const auto read = [&](uint32_t cur, int k) {
        const char* codes = ring.codes[cur];
        const uint32_t at = place(r, 2 * k + half) * 16;
#pragma unroll
        for (int j = 0; j < NI; j++) y[k & 1][j] = *(const u32x4*)(codes + (BM + wn + j * 32 + r) * kTileBytes + at);
#pragma unroll
        for (int i = 0; i < MI; i++) x[k & 1][i] = *(const u32x4*)(codes + (wm + i * 32 + r) * kTileBytes + at);
    };
    const auto row_scales = [&](uint32_t buf, uint32_t second, uint32_t row) {
        return step_scales(ring.scales[buf][row][second], half);
    };
    const auto read_scales = [&](uint32_t buf, uint32_t second, uint32_t* ua, uint32_t* ub) {
#pragma unroll
        for (int i = 0; i < MI; i++) ua[i] = row_scales(buf, second, wm + i * 32 + r);
#pragma unroll
        for (int j = 0; j < NI; j++) ub[j] = row_scales(buf, second, BM + wn + j * 32 + r);
    };
    const auto step = [&](auto K) {
        constexpr int k = decltype(K)::value;
#pragma unroll
        for (int i = 0; i < MI; i++)
#pragma unroll
            for (int j = 0; j < NI; j++) acc[i][j] = mfma<k>(y[k & 1][j], x[k & 1][i], acc[i][j], sb[j], sa[i]);
    };
    // The scheduling barriers keep a step's reads before the step that they are to
    // run behind: left alone, the compiler reads all four steps at once, which takes
    // more registers than there are.
    const auto settle = [] { __builtin_amdgcn_sched_barrier(0); };

    // One tile: its first three steps, then, between its last read and its last
    // step, the next tile's: it has landed for every wave, this tile's stage is
    // free, and the next tile's first operands are on their way while the last step
    // runs.  `second`: the tile is (EVEN) the second of its two.
    uint32_t cur = 0, buf = 0;
    const auto first_steps = [&] {
        read(cur, 1);
        settle();
        step(std::integral_constant<int, 0>{});
        settle();
        read(cur, 2);
        settle();
        step(std::integral_constant<int, 1>{});
        settle();
        read(cur, 3);
        settle();
        step(std::integral_constant<int, 2>{});
        settle();
    };
    const auto tile = [&](auto second) {
        constexpr bool SECOND = decltype(second)::value;
        first_steps();
        wait_vmem_below<loads(S - 2, !SECOND)>();
        if constexpr (!EVEN) keep_scales(cur ^ 1);  // the next tile's
        __syncthreads();
        // the tile S after this one, of the same place in its pair where S is even
        fetch(std::integral_constant<bool, !EVEN || SECOND == (S % 2 != 0)>{});
        cur = cur + 1 == S ? 0 : cur + 1;
        if (!EVEN || SECOND) buf = buf + 1 == NB ? 0 : buf + 1;
        uint32_t ua[MI], ub[NI];
        read_scales(buf, EVEN && !SECOND, ua, ub);
        read(cur, 0);
        settle();
        step(std::integral_constant<int, 3>{});
        settle();
#pragma unroll
        for (int i = 0; i < MI; i++) sa[i] = ua[i];
#pragma unroll
        for (int j = 0; j < NI; j++) sb[j] = ub[j];
    };
    if (total) {
#pragma unroll
        for (int t = 0; t < S; t++) {
            if (t % PAIR == 0) fetch(std::true_type{});
            else fetch(std::false_type{});
            if (!EVEN && t == 0) keep_scales(0);
        }
        wait_vmem_below<loads(S - 1, false)>();
        __syncthreads();
        read_scales(0, 0, sa, sb);
        read(0, 0);
        if constexpr (EVEN) {
            for (uint32_t t = 2; t < total; t += 2) {
                tile(std::false_type{});
                tile(std::true_type{});
            }
            tile(std::false_type{});
        } else {
            for (uint32_t t = 1; t < total; t++) tile(std::false_type{});
        }
        first_steps();
        step(std::integral_constant<int, 3>{});
        wait_vmem_below<0>();
    }
    __syncthreads();

    static_assert(WAVES * 32 * NI * 32 * T::ESZ <= sizeof(ring.codes), "the results' way out fits the ring");
    store_results<T, MI, NI>(a, acc, ring.codes[0] + wave * 32 * NI * 32 * T::ESZ, lane, m0 + wm, n0 + wn, SUM ? 0 : q0,
                             SUM ? a.ranks : q0 + 1);
}

// ---------------------------------------------------------------------------
// Tiled product, large: 256 x 256 tiles, eight waves of 128 x 64.
//
// The waves of each half of the workgroup, one per SIMD, take turns: while one
// half multiplies a step (256 cycles of matrix instructions), the other reads its
// next step's operands from LDS, and a barrier swaps them.  Two stages: the next
// tile's loads go out between the matrix instructions of a tile's first two steps,
// into the stage that both halves have left, and have the last two steps to
// land.  Scales come a group of G tiles ahead, 8 G bytes of a row at once, and are
// read from LDS two tiles at a time behind the steps of the second.
//
// RAGGED: rows whose blocks are not whole groups of G tiles, or scales that are not
// 16-byte aligned.  A rank's tiles are then rounded up to whole pairs (G = 2); blocks
// past a row's end come from a constant, zero codes with scale 1, and a lane reads a
// row's 16 scale bytes from any address and writes them to LDS itself.
// Rows that do not start on a memory line have each tile's 128 bytes on two, twice
// the CU's cache look-ups: 18 tiles each of 4 x (2048 x 1024), fp32 outputs, take 29.5
// us whole, 34 us ragged and 43 us ragged with rows of 2064 bytes (4 x (2056 x 1000 x
// 4100): 2.1 L2 requests for each row's 128 bytes, scales included, against 1.25 where
// rows are whole).  Reading the lines of the tile after next ahead of time changes none
// of the three.
// ---------------------------------------------------------------------------
template <int G>
struct TurnsLds {
    char codes[2][512 * kTileBytes];
    u32x4 scales[2][512][G / 2];  // of two tiles each
};

template <class T, bool SUM, int G, bool RAGGED>
__global__ __launch_bounds__(512) void k_mx4_matmul_turns(MatmulArgs a)
{
    constexpr int BM = 256, BN = 256, MI = 4, NI = 2, WAVES = 8;
    static_assert(G == 2 || (G == 4 && !RAGGED), "scales of one or two pairs of tiles");
    __shared__ __attribute__((aligned(16))) TurnsLds<G> lds;

    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t tm, tn;
    tile_of<4>(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * BN;
    const uint32_t ktiles = RAGGED ? (a.kb + 2 * kTileBlocks - 1) / (2 * kTileBlocks) * 2 : a.kb / kTileBlocks;
    const int q0 = SUM ? 0 : (int)blockIdx.y;
    const uint32_t total = ktiles * (SUM ? (uint32_t)a.ranks : 1u);
    const uint64_t row_bytes = (uint64_t)a.kb * 16;

    // Waves 0-3 load A's rows and 4-7 B's, 64 rows each: eight loads of eight rows'
    // codes a tile, G / 2 loads of scales a group.  Offsets are from the operand's
    // first row of the tile; rows past the end read the last one again.
    const bool isb = wave >= 4;
    const uint64_t row0 = isb ? n0 : m0;
    const uint32_t last = isb ? a.n - 1 - n0 : a.m - 1 - m0, wrow = (wave & 3) * 64;
    uint32_t off[8], soff[G / 2];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t row = wrow + i * 8 + lane / 8;
        off[i] = (row < last ? row : last) * (uint32_t)row_bytes + place(row, lane & 7) * 16;
    }
#pragma unroll
    for (int i = 0; i < G / 2; i++) {
        constexpr uint32_t L = G / 2;  // lanes of a row
        const uint32_t row = wrow + (i * 64 + lane) / L;
        soff[i] = (row < last ? row : last) * a.kb + lane % L * 16;
    }
    // RAGGED: this lane's row's scales on their way to LDS.  They are read at most 15
    // bytes early, where 16 would end past the array (which holds 16 or more).
    const uint32_t blk = place(lane / 8, lane & 7);  // this lane's block of rows 0-7; of rows 8-15, ^ 4; and so on
    u32x4 held = {};
    uint32_t held_skip = 0, held_left = 0, left = 0;
    const uint64_t array_end = (isb ? a.n : a.m) * (uint64_t)a.kb - 16;

    // The tile that is fetched next, and the group of scales after it.
    int fq = q0;
    uint32_t fkt = 0, fetched = 0, live = 0, slive = 0;
    global_ptr<const char> pcodes = nullptr, pscales = nullptr;
    const auto aim = [&] {
        live = fetched < total ? ~0u : 0u;
        left = fkt * kTileBlocks < a.kb ? a.kb - fkt * kTileBlocks : 0;
        pcodes = (global_ptr<const char>)(isb ? a.bc[fq] : a.ac[fq]) + row0 * row_bytes + (uint64_t)fkt * kTileBytes;
    };
    const auto aim_scales = [&](int q, uint32_t kt, bool more) {
        slive = more ? ~0u : 0u;
        pscales = (global_ptr<const char>)(isb ? a.bs[q] : a.as[q]) + row0 * a.kb + kt * kTileBlocks;
    };
    const auto load_codes = [&](uint32_t stage, int i) {
        auto from = pcodes + opaque(off[i] & live);
        if constexpr (RAGGED)
            if ((opaque(blk) ^ (i & 1) * 4) >= left) from = (global_ptr<const char>)&kZeroCodes;
        load_to_lds(from, (u32x4*)(lds.codes[stage] + ((isb ? BM : 0) + wrow + i * 8) * kTileBytes));
    };
    const auto hold_scales = [&](int q, uint32_t kt) {
        const uint64_t want = row0 * a.kb + soff[0] + kt * kTileBlocks, from = want < array_end ? want : array_end;
        typedef u32x4 u32x4_at __attribute__((aligned(1)));
        held = *(global_ptr<const u32x4_at>)((global_ptr<const char>)(isb ? a.bs[q] : a.as[q]) + from);
        held_skip = (uint32_t)(want - from);
        held_left = a.kb - kt * kTileBlocks;
    };
    const auto keep_scales = [&](uint32_t buf) {
        uint64_t lo = (uint64_t)held.y << 32 | held.x, hi = (uint64_t)held.w << 32 | held.z;
        const bool far = held_skip >= 8;
        const uint32_t bits = 8 * (held_skip & 7);
        lo = far ? hi : lo;
        hi = far ? 0 : hi;
        lo = lo >> bits | hi << 1 << (63 - bits);
        hi >>= bits;
        // bytes from held_left on are scale 1; no branches
        const uint32_t n0 = held_left < 8 ? held_left : 8, n1 = (held_left < 16 ? held_left : 16) - n0;
        const uint64_t gone0 = ~0ull << 4 * n0 << 4 * n0, gone1 = ~0ull << 4 * n1 << 4 * n1;
        lo = (lo & ~gone0) | (0x7f7f7f7f7f7f7f7full & gone0);
        hi = (hi & ~gone1) | (0x7f7f7f7f7f7f7f7full & gone1);
        lds.scales[buf][(isb ? BM : 0) + wrow + lane][0] =
            u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    };
    const auto load_scales = [&](uint32_t buf, int i) {
        load_to_lds(pscales + opaque(soff[i] & slive), &lds.scales[buf][(isb ? BM : 0) + wrow][0] + i * 64);
    };
    const auto advance = [&] {
        fetched++;
        const bool more = fetched < total, wrap = fkt + 1 == ktiles;
        fq += more && wrap;
        fkt = !more ? fkt : wrap ? 0 : fkt + 1;
    };

    f32x16 acc[MI][NI] = {};
    const uint32_t wm = wave % 2 * 128, wn = wave / 2 * 64;
    const uint32_t r = lane & 31, half = lane >> 5;
    u32x4 x[MI], y[NI];
    uint32_t sa[2][MI], sb[2][NI];  // of the pair of tiles at work
    uint32_t ta[2][MI], tb[2][NI];  // of the next
    const auto read_scales = [&](uint32_t buf, int pair, int i) {  // rows' tile i of six: A's four, B's two
        const u32x4 v = lds.scales[buf][i < MI ? wm + i * 32 + r : BM + wn + (i - MI) * 32 + r][pair];
        const uint32_t u0 = step_scales(u32x2{v.x, v.y}, half), u1 = step_scales(u32x2{v.z, v.w}, half);
        if (i < MI) { ta[0][i] = u0; ta[1][i] = u1; }
        else { tb[0][i - MI] = u0; tb[1][i - MI] = u1; }
    };
    const auto take_scales = [&] {
#pragma unroll
        for (int t = 0; t < 2; t++) {
#pragma unroll
            for (int i = 0; i < MI; i++) sa[t][i] = ta[t][i];
#pragma unroll
            for (int j = 0; j < NI; j++) sb[t][j] = tb[t][j];
        }
    };
    const auto settle = [] { __builtin_amdgcn_sched_barrier(0); };
    const auto meet = [&] {
        settle();
        lds_barrier();
        settle();
    };

    uint32_t buf = 0;
    // Step K of tile g of a group (stage g mod 2).
    const auto turn = [&](auto K, auto tile) {
        constexpr int k = decltype(K)::value, g = decltype(tile)::value, stage = g & 1;
        const char* codes = lds.codes[stage];
        const uint32_t at = place(r, 2 * k + half) * 16;
#pragma unroll
        for (int j = 0; j < NI; j++) y[j] = *(const u32x4*)(codes + (BM + wn + j * 32 + r) * kTileBytes + at);
#pragma unroll
        for (int i = 0; i < MI; i++) x[i] = *(const u32x4*)(codes + (wm + i * 32 + r) * kTileBytes + at);
        if constexpr (g % 2 == 1 && k > 0) {
            read_scales(g == G - 1 ? buf ^ 1 : buf, g == G - 1 ? 0 : g / 2 + 1, 2 * k - 2);
            read_scales(g == G - 1 ? buf ^ 1 : buf, g == G - 1 ? 0 : g / 2 + 1, 2 * k - 1);
        }
        if constexpr (k == 0) {
            aim();
            if constexpr (g == 0) {
                // the group after this one: G - 1 tiles after the tile that is fetched next
                const uint32_t kt = fkt + (G - 1);
                const bool more = fetched + (G - 1) < total, wrap = kt == ktiles;
                if constexpr (RAGGED) hold_scales(fq + (more && wrap), !more || wrap ? 0 : kt);
                else aim_scales(fq + (more && wrap), !more || wrap ? 0 : kt, more);
            }
        }
        if constexpr (k == 3) {
            advance();
            wait_vmem_below<0>();
            if constexpr (RAGGED && g == 0) keep_scales(buf ^ 1);
        }
        meet();
        __builtin_amdgcn_s_setprio(1);
        if constexpr (k == 0 && g == 0 && !RAGGED)
#pragma unroll
            for (int i = 0; i < G / 2; i++) load_scales(buf ^ 1, i);
#pragma unroll
        for (int i = 0; i < MI; i++) {
#pragma unroll
            for (int j = 0; j < NI; j++) acc[i][j] = mfma<k>(y[j], x[i], acc[i][j], sb[g & 1][j], sa[g & 1][i]);
            settle();
            if constexpr (k < 2) load_codes(stage ^ 1, k * 4 + i);
            settle();
        }
        __builtin_amdgcn_s_setprio(0);
        meet();
    };
    const auto whole = [&](auto tile) {
        turn(std::integral_constant<int, 0>{}, tile);
        turn(std::integral_constant<int, 1>{}, tile);
        turn(std::integral_constant<int, 2>{}, tile);
        turn(std::integral_constant<int, 3>{}, tile);
        if constexpr (decltype(tile)::value % 2 == 1) take_scales();
    };

    aim();
#pragma unroll
    for (int i = 0; i < 8; i++) load_codes(0, i);
    if constexpr (RAGGED) {
        hold_scales(fq, 0);
        keep_scales(0);
    } else {
        aim_scales(fq, 0, true);
#pragma unroll
        for (int i = 0; i < G / 2; i++) load_scales(0, i);
    }
    advance();
    wait_vmem_below<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 6; i++) read_scales(0, 0, i);
    take_scales();
    if (wave >= 4) meet();
    for (uint32_t t = 0; t < total; t += G) {
        whole(std::integral_constant<int, 0>{});
        whole(std::integral_constant<int, 1>{});
        if constexpr (G == 4) {
            whole(std::integral_constant<int, 2>{});
            whole(std::integral_constant<int, 3>{});
        }
        buf ^= 1;
    }
    if (wave < 4) meet();
    wait_vmem_below<0>();
    __syncthreads();
    static_assert(WAVES * 32 * NI * 32 * T::ESZ <= sizeof(lds.codes), "the results' way out fits the stages");
    store_results<T, MI, NI>(a, acc, lds.codes[0] + wave * 32 * NI * 32 * T::ESZ, lane, m0 + wm, n0 + wn, SUM ? 0 : q0,
                             SUM ? a.ranks : q0 + 1);
}

// ---------------------------------------------------------------------------
// Few rows of one operand, A here: a stream of the other.  A workgroup has W (32
// or 16) columns of C (rows of B) and MI x W of its rows; its waves take the
// contraction's tiles in turn, straight from memory into registers, the next
// two tiles' loads in flight while one is multiplied, and the waves' sums meet in
// LDS, added in wave order.
// ---------------------------------------------------------------------------
template <int W>
struct Wide;
template <>
struct Wide<32> {
    typedef f32x16 Acc;
    static constexpr int STEPS = 4;
    // A lane's scales of a tile's steps, from its row's eight bytes, or from its own.
    __device__ static void scales(u32x2 bytes, uint32_t part, uint32_t* s)
    {
        s[0] = s[1] = s[2] = s[3] = step_scales(bytes, part);
    }
    __device__ static void own_scales(const uint32_t* bytes, uint32_t* s)
    {
        s[0] = s[1] = s[2] = s[3] = bytes[0] | bytes[1] << 8 | bytes[2] << 16 | bytes[3] << 24;
    }
    template <int S>
    __device__ static Acc mul(u32x4 b, u32x4 a, Acc acc, uint32_t sb, uint32_t sa) { return mfma<S>(b, a, acc, sb, sa); }
    // The column of result e.
    __device__ static uint32_t col(int e, uint32_t part) { return 8 * (e / 4) + 4 * part + e % 4; }
};
template <>
struct Wide<16> {
    typedef f32x4 Acc;
    static constexpr int STEPS = 2;
    __device__ static void scales(u32x2 bytes, uint32_t part, uint32_t* s)
    {
        s[0] = bytes.x >> (8 * part);
        s[1] = bytes.y >> (8 * part);
    }
    __device__ static void own_scales(const uint32_t* bytes, uint32_t* s)
    {
        s[0] = bytes[0];
        s[1] = bytes[1];
    }
    template <int S>
    __device__ static Acc mul(u32x4 b, u32x4 a, Acc acc, uint32_t sb, uint32_t sa)
    {
        const i32x8 x = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
        const i32x8 y = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, 0, (int)sb, 0, (int)sa);
    }
    __device__ static uint32_t col(int e, uint32_t part) { return 4 * part + e; }
};

// A lane's part of a row of a tile: the blocks that it multiplies, and their scales.
// WHOLE: rows are whole tiles, and a row's eight scales are read at once.  Else a lane
// reads the bytes of its own blocks; a block past the row's end comes from a
// constant, zero codes, and has scale 1.
template <int W, bool WHOLE>
struct RowPart {
    static constexpr int STEPS = Wide<W>::STEPS, PARTS = 64 / W;
    u32x4 codes[STEPS];
    u32x2 scales;             // WHOLE
    uint32_t bytes[STEPS];    // else

    // codes and scales: of the tile's first row, at this tile; off: the row's offset in
    // scale bytes (in codes 16 times that); left: blocks that the tile has.
    __device__ __forceinline__ void load(global_ptr<const char> c, global_ptr<const char> sc, uint32_t off,
                                         uint32_t part, uint32_t left)
    {
        const auto at = c + opaque((off + part) * 16);
#pragma unroll
        for (int s = 0; s < STEPS; s++) {
            auto from = at + (PARTS * 16 * s);
            if constexpr (!WHOLE) from = PARTS * s + part < left ? from : (global_ptr<const char>)&kZeroCodes;
            codes[s] = *(global_ptr<const u32x4>)from;
        }
        if constexpr (WHOLE) {
            scales = *(global_ptr<const u32x2_any>)(sc + opaque(off));
        } else {
#pragma unroll
            for (int s = 0; s < STEPS; s++) {
                const uint32_t b = PARTS * s + part;
                bytes[s] = *(global_ptr<const uint8_t>)(sc + opaque(off + (b < left ? b : left - 1)));
            }
        }
    }
    __device__ __forceinline__ void steps(uint32_t part, uint32_t left, uint32_t* s) const
    {
        if constexpr (WHOLE) {
            Wide<W>::scales(scales, part, s);
        } else {
            uint32_t b[STEPS];
#pragma unroll
            for (int i = 0; i < STEPS; i++) b[i] = PARTS * i + part < left ? bytes[i] : 127u;
            Wide<W>::own_scales(b, s);
        }
    }
};

template <int W, int MI, bool WHOLE>
struct Frag {
    RowPart<W, WHOLE> b, a[MI];
    uint32_t left;  // blocks that the tile has
};

template <class T, bool SUM, bool WHOLE, int W, int MI, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_mx4_matmul_few(MatmulArgs a)
{
    typedef Wide<W> Op;
    constexpr int STEPS = Op::STEPS, RESULTS = W * W / 64;
    __shared__ float part_sum[WAVES][MI * W * (W + 1)];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t r = lane % W, part = lane / W;
    const uint32_t tile = wide_tile();
    if (tile >= a.tiles_m * a.tiles_n) return;
    const uint32_t n0 = tile % a.tiles_n * W, m0 = tile / a.tiles_n * (MI * W);
    const uint32_t ktiles = (a.kb + kTileBlocks - 1) / kTileBlocks;
    const int q0 = SUM ? 0 : (int)blockIdx.y;
    const uint32_t total = ktiles * (SUM ? (uint32_t)a.ranks : 1u);
    // Rows past the end read the last one again.
    const uint32_t last_b = a.n - 1 - n0, last_a = a.m - 1 - m0;
    const uint32_t off_b = (r < last_b ? r : last_b) * a.kb;
    uint32_t off_a[MI];
#pragma unroll
    for (int i = 0; i < MI; i++) off_a[i] = (i * W + r < last_a ? i * W + r : last_a) * a.kb;

    const auto fetch = [&](Frag<W, MI, WHOLE>& f, uint32_t t) {
        const uint32_t qi = a.by_ktiles.div(t), kt = t - qi * ktiles;
        const int q = q0 + (int)qi;
        const uint64_t k0 = (uint64_t)kt * kTileBlocks, at_b = (uint64_t)n0 * a.kb + k0, at_a = (uint64_t)m0 * a.kb + k0;
        f.left = a.kb - kt * kTileBlocks;
        f.b.load((global_ptr<const char>)a.bc[q] + at_b * 16, (global_ptr<const char>)a.bs[q] + at_b, off_b, part, f.left);
#pragma unroll
        for (int i = 0; i < MI; i++)
            f.a[i].load((global_ptr<const char>)a.ac[q] + at_a * 16, (global_ptr<const char>)a.as[q] + at_a, off_a[i], part,
                        f.left);
    };
    typename Op::Acc acc[MI] = {};
    const auto multiply = [&](const Frag<W, MI, WHOLE>& f) {
        uint32_t sb[STEPS];
        f.b.steps(part, f.left, sb);
#pragma unroll
        for (int i = 0; i < MI; i++) {
            uint32_t sa[STEPS];
            f.a[i].steps(part, f.left, sa);
            acc[i] = Op::template mul<0>(f.b.codes[0], f.a[i].codes[0], acc[i], sb[0], sa[0]);
            acc[i] = Op::template mul<1>(f.b.codes[1], f.a[i].codes[1], acc[i], sb[1], sa[1]);
            if constexpr (STEPS == 4) {
                acc[i] = Op::template mul<2>(f.b.codes[2], f.a[i].codes[2], acc[i], sb[2], sa[2]);
                acc[i] = Op::template mul<3>(f.b.codes[3], f.a[i].codes[3], acc[i], sb[3], sa[3]);
            }
        }
    };
    // Two tiles ahead, without a branch around the loads: where some may not be under
    // way, the compiler waits for all of them before each product (on one card 8 x (1 x
    // 8192 x 4096) 32.5 us instead of 30.5, 4 x (1 x 5120 x 640) 5.3 instead of 4.3).  Three
    // tiles ahead or 16 waves gain nothing; loads that pass by the caches take 46 us,
    // as a row's line is read in four pieces.
    Frag<W, MI, WHOLE> f[2];
    uint32_t t = wave, left = t < total ? (total - t + WAVES - 1) / WAVES : 0;
    const auto turn = [&](int d) {
        multiply(f[d]);
        __builtin_amdgcn_sched_barrier(0);
        fetch(f[d], t + (2 + d) * WAVES);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (left >= 2) {
        fetch(f[0], t);
        fetch(f[1], t + WAVES);
        for (; left >= 4; left -= 2, t += 2 * WAVES) {
            turn(0);
            turn(1);
        }
        if (left == 3) turn(0);
        else multiply(f[0]);
        multiply(f[1]);
        if (left == 3) multiply(f[0]);
    } else if (left) {
        fetch(f[0], t);
        multiply(f[0]);
    }
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int e = 0; e < RESULTS; e++) part_sum[wave][(i * W + r) * (W + 1) + Op::col(e, part)] = acc[i][e];
    __syncthreads();
    const int dst0 = SUM ? 0 : q0, dst1 = SUM ? a.ranks : q0 + 1;
    for (uint32_t o = tid; o < MI * W * W; o += WAVES * 64) {
        const uint32_t row = o / W, col = o % W;
        if (m0 + row >= a.m || n0 + col >= a.n) continue;
        float s = part_sum[0][row * (W + 1) + col];
#pragma unroll
        for (int w = 1; w < WAVES; w++) s += part_sum[w][row * (W + 1) + col];
        const typename T::S v = T::narrow(s);
        const uint64_t at = ((m0 + row) * a.sm + (n0 + col) * a.sn) * T::ESZ;
        for (int d = dst0; d < dst1; d++) store_s<T>(a.dst[d] + at, v);
    }
}

using namespace host;

template <class T, bool SUM, bool EVEN, int BM, int BN, int WM, int WN, int S>
vrc_status_t launch_tiled(MatmulArgs& a, hipStream_t st)
{
    a.tiles_m = (a.m + BM - 1) / BM;
    a.tiles_n = (a.n + BN - 1) / BN;
    const uint64_t tiles = (uint64_t)a.tiles_m * a.tiles_n;
    if (tiles * (WM * WN * 64) > 0xffffffffull) return VRC_ERR_INVALID_ARG;  // C of 2^38 elements
    const dim3 grid((unsigned)tiles, SUM ? 1u : (unsigned)a.ranks);
    k_mx4_matmul_tiled<T, SUM, EVEN, BM, BN, WM, WN, S><<<grid, WM * WN * 64, 0, st>>>(a);
    return check_launch();
}

template <class T, bool SUM, int G, bool RAGGED>
vrc_status_t launch_turns(MatmulArgs& a, hipStream_t st)
{
    a.tiles_m = (a.m + 255) / 256;
    a.tiles_n = (a.n + 255) / 256;
    const uint64_t tiles = (uint64_t)a.tiles_m * a.tiles_n;
    if (tiles * 512 > 0xffffffffull) return VRC_ERR_INVALID_ARG;  // C of 2^39 elements
    k_mx4_matmul_turns<T, SUM, G, RAGGED><<<dim3((unsigned)tiles, SUM ? 1u : (unsigned)a.ranks), 512, 0, st>>>(a);
    return check_launch();
}

// `swap`: B is the operand of few rows.
template <class T, bool SUM, int W, int MI, int WAVES>
vrc_status_t launch_few(MatmulArgs a, bool swap, hipStream_t st)
{
    a.sm = a.n;
    a.sn = 1;
    if (swap) {
        for (int r = 0; r < a.ranks; r++) {
            std::swap(a.ac[r], a.bc[r]);
            std::swap(a.as[r], a.bs[r]);
        }
        std::swap(a.m, a.n);
        std::swap(a.sm, a.sn);
    }
    a.tiles_m = (a.m + MI * W - 1) / (MI * W);
    a.tiles_n = (a.n + W - 1) / W;
    static_assert(WAVES * 64 <= 1024, "wide_grid's workgroups");
    a.by_ktiles = FastDiv::of((a.kb + kTileBlocks - 1) / kTileBlocks);
    const dim3 grid = wide_grid((uint64_t)a.tiles_m * a.tiles_n, SUM ? 1 : a.ranks);
    if (a.kb % kTileBlocks == 0) k_mx4_matmul_few<T, SUM, true, W, MI, WAVES><<<grid, WAVES * 64, 0, st>>>(a);
    else k_mx4_matmul_few<T, SUM, false, W, MI, WAVES><<<grid, WAVES * 64, 0, st>>>(a);
    return check_launch();
}

// The kernel by sizes.  One operand of up to 64 rows: a stream of the other, by 16
// columns where that makes at most a workgroup per CU and by 32 otherwise (us; 16 /
// 32 columns: 1 x 4096 x 16384 9.9 / 13.9, 32 x 4096 x 16384 19.1 / 20.6, 8 x (7 x
// 4096 x 2048) 10.4 / 14.5; but 8 x (1 x 8192 x 4096) 33.8 / 31.0, 32 x 8192 x 4096
// 11.2 / 7.9, and from 33 rows 4 x (48 x 5003 x 1000) 14.5 / 9.5).  Else the smallest tiles of which at most two a CU
// are needed: a tile of the contraction takes 0.5 us with 64 x 64 tiles, 0.7 us with
// 128 x 128 and 1.2 us with 256 x 256, whatever the grid, until the CUs are full
// (us; 64 / 128 / 256: 256 x 8192 x 4096 12.5 / 15.0 / 24.0, 512 x 8192 x 4096
// 23.4 / 16.7 / 25.3, 1024 x 8192 x 4096 45.7 / 25.6 / 28.1, 2048 x 8192 x 4096
// 84.5 / 48.9 / 38.7).  Ragged rows take the same tiles: 4 x (2056 x 1000 x 4100)
// 49 us with 256 x 256 tiles and 64 us with 544 of 128 x 128, 4096 x 8192 x 4100
// 100 / 137 us (4096 x 8192 x 4096 76 us).
template <class T, bool SUM>
vrc_status_t matmul_typed(MatmulArgs& a, int cus, hipStream_t st)
{
    const bool swap = a.n < a.m;
    const uint32_t few = swap ? a.n : a.m, many = swap ? a.m : a.n;
    const uint64_t products = SUM ? 1 : (uint64_t)a.ranks;
    if (few <= 64) {
        if (few > 32) return launch_few<T, SUM, 32, 2, 8>(a, swap, st);
        const bool by16 = ((many + 15ull) / 16) * products <= (uint64_t)cus;
        if (few <= 16) return by16 ? launch_few<T, SUM, 16, 1, 8>(a, swap, st) : launch_few<T, SUM, 32, 1, 8>(a, swap, st);
        return by16 ? launch_few<T, SUM, 16, 2, 8>(a, swap, st) : launch_few<T, SUM, 32, 1, 8>(a, swap, st);
    }
    // From here an array of scales has 65 bytes, of which a lane of the ragged tiles
    // reads up to 16 at once, or none (kb == 0: zeros, by the 128 x 128 tiles).
    bool even = a.kb && a.kb % (2 * kTileBlocks) == 0;
    for (int r = 0; r < a.ranks; r++) even = even && (uintptr_t)a.as[r] % 16 == 0 && (uintptr_t)a.bs[r] % 16 == 0;
    const auto tiles = [&](uint64_t b) { return ((a.m + b - 1) / b) * ((a.n + b - 1) / b) * products; };
    const uint64_t room = 2 * (uint64_t)cus;
    if (!even) {
        if (tiles(64) <= room) return launch_tiled<T, SUM, false, 64, 64, 1, 2, 2>(a, st);
        // one tile a rank (kb <= 8) would be two in pairs: 8000 x 8000 x 200 34.8 us, 42.6 by pairs
        if (tiles(128) <= room || a.kb <= kTileBlocks) return launch_tiled<T, SUM, false, 128, 128, 2, 2, 2>(a, st);
        return launch_turns<T, SUM, 2, true>(a, st);
    }
    if (tiles(64) <= room) return launch_tiled<T, SUM, true, 64, 64, 1, 2, 4>(a, st);
    if (tiles(128) <= room) return launch_tiled<T, SUM, true, 128, 128, 2, 2, 2>(a, st);
    return a.kb % (4 * kTileBlocks) == 0 ? launch_turns<T, SUM, 4, false>(a, st) : launch_turns<T, SUM, 2, false>(a, st);
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
