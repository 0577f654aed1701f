// vrc_dropout.hip -- dropout inside the collectives: the all-reduce and the
// reduce-scatter with a residual, and the masked all-gather that is the
// reduce-scatter's gradient.
//
// y = res + mask * scale * (x_0 + x_1 + ... ) per element, in fp32, rounded
// once.  The mask comes from Philox-4x32-10 by the element's index, so no call
// stores or reads it: a kernel moves the collective's bytes and the residual's.
// They are streams, bounded by memory; the generator's integer
// multiplications (20 of 32 x 32 bits for four elements) run beside them.
#include <hip/hip_runtime.h>

#include "vrc_ops_host.hpp"

namespace vrc {
namespace {

using host::MaskArgs;

// a ^ b ^ c in one instruction (the compiler makes two).
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c)
{
    return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96);
}

// One Philox-4x32 bijection of ten rounds: counter (block, offset), key seed.
__device__ __forceinline__ void philox(uint64_t block, uint64_t offset, uint64_t seed, uint32_t w[4])
{
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
    uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; r++) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = xor3((uint32_t)(p1 >> 32), c1, k0);
        c2 = xor3((uint32_t)(p0 >> 32), c3, k1);
        c1 = (uint32_t)p1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}

struct Mask {
    uint64_t seed, offset;
    float scale;
    uint32_t thr, kind;

    __device__ explicit Mask(const MaskArgs& a)
        : seed(a.seed), offset(a.offset), scale(a.scale), thr(a.thr), kind(a.kind)
    {
        if (a.offset_dev) offset += *(global_ptr<const uint64_t>)a.offset_dev;
    }

    // Bit j: element 4 * block + j is kept.
    __device__ __forceinline__ uint32_t keep4(uint64_t block) const
    {
        uint32_t w[4];
        philox(block, offset, seed, w);
        return (uint32_t)(w[0] >= thr) | (uint32_t)(w[1] >= thr) << 1 | (uint32_t)(w[2] >= thr) << 2 |
               (uint32_t)(w[3] >= thr) << 3;
    }

    // Bit j: element i + j is kept, j < V.  A vector whose first index is no
    // multiple of four reaches into one block more.
    template <int V>
    __device__ __forceinline__ uint32_t keep(uint64_t i) const
    {
        if (kind != 1) return kind == 0 ? ~0u : 0u;
        const uint64_t b = i >> 2;
        const uint32_t ph = (uint32_t)i & 3;
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < (V + 3) / 4; j++) bits |= keep4(b + j) << (4 * j);
        if constexpr (V > 1) {
            if (ph) bits |= keep4(b + V / 4) << V;
        }
        return bits >> ph;
    }

    // mask * scale * a, with +0 for a dropped element.
    __device__ __forceinline__ float apply(float a, uint32_t bits, int j) const
    {
        return (bits >> j & 1u) ? a * scale : 0.0f;
    }
};

// The N inputs' vectors, folded in rank order in fp32.
template <class T, int N>
__device__ __forceinline__ void fold_f32(const u32x4* in, float* acc)
{
    T::unpack(in[0], acc);
#pragma unroll
    for (int r = 1; r < N; r++) {
        float x[T::VEC];
        T::unpack(in[r], x);
#pragma unroll
        for (int i = 0; i < T::VEC; i++) acc[i] += x[i];
    }
}

template <class T>
__device__ __forceinline__ u32x4 add_residual(const float* acc, u32x4 res)
{
    float x[T::VEC];
    T::unpack(res, x);
#pragma unroll
    for (int i = 0; i < T::VEC; i++) x[i] = acc[i] + x[i];
    return T::pack(x);
}

// ---------------------------------------------------------------------------
// All-reduce.  One-wave workgroups, a 1 KiB tile of every buffer an iteration
// with all its loads in flight (2, 4 or 8 tiles at once, with fewer waves, came to
// within 3 % of the best either way).  A lane reads its elements of every input and
// residual before it writes any output, so an output may be its own input or
// residual.
// RES: 0 none, 1 one residual for all ranks, 2 one for each.
// ---------------------------------------------------------------------------
struct DropArArgs {
    const char* src[kMaxRanks];
    const char* res[kMaxRanks];
    char* dst[kMaxRanks];
    RowSplit g;
    MaskArgs m;
};

template <class T, int N, int RES>
__global__ __launch_bounds__(64) void k_dropout_allreduce(DropArArgs a)
{
    constexpr uint64_t W = 64, E = T::ESZ;
    constexpr int NR = RES == 2 ? N : RES;
    const Mask mask(a.m);
    const uint64_t body = a.g.head * E, nv = a.g.nvb, lane = threadIdx.x;
    for (uint64_t v = blockIdx.x * W + lane; v < nv; v += (uint64_t)gridDim.x * W) {
        u32x4 in[N], res[NR ? NR : 1];
#pragma unroll
        for (int r = 0; r < N; r++) in[r] = ld16<true>(a.src[r] + body + v * 16);
#pragma unroll
        for (int r = 0; r < NR; r++) res[r] = ld16<true>(a.res[r] + body + v * 16);
        issue_loads_first();
        float acc[T::VEC];
        fold_f32<T, N>(in, acc);
        const uint32_t bits = mask.keep<T::VEC>(a.g.head + v * T::VEC);
#pragma unroll
        for (int i = 0; i < T::VEC; i++) acc[i] = mask.apply(acc[i], bits, i);
        u32x4 out = RES == 0 ? T::pack(acc) : u32x4{};
        if constexpr (RES == 1) out = add_residual<T>(acc, res[0]);
#pragma unroll
        for (int r = 0; r < N; r++) {
            if constexpr (RES == 2) out = add_residual<T>(acc, res[r]);
            st16<true>(a.dst[r] + body + v * 16, out);
        }
    }

    const uint64_t ns = a.g.head + a.g.tail;
    for (uint64_t k = blockIdx.x * W + lane; k < ns; k += (uint64_t)gridDim.x * W) {
        const uint64_t i = k < a.g.head ? k : a.g.nvb * T::VEC + k;
        float acc = T::widen(load_s<T>(a.src[0] + i * E));
#pragma unroll
        for (int r = 1; r < N; r++) acc += T::widen(load_s<T>(a.src[r] + i * E));
        acc = mask.apply(acc, mask.keep<1>(i), 0);
        float x[NR ? NR : 1];
#pragma unroll
        for (int r = 0; r < NR; r++) x[r] = T::widen(load_s<T>(a.res[r] + i * E));
#pragma unroll
        for (int r = 0; r < N; r++)
            store_s<T>(a.dst[r] + i * E, T::narrow(RES == 0 ? acc : acc + x[RES == 2 ? r : 0]));
    }
}

// ---------------------------------------------------------------------------
// Chunks of the whole tensor: chunk c is `rows` rows of g[c]'s width at element
// off[c] of the tensor, its rows `stride` elements apart there and packed in
// the rank's own buffer.
// ---------------------------------------------------------------------------
struct ChunkArgs {
    uint64_t off[kMaxRanks];
    uint64_t width[kMaxRanks];
    RowSplit g[kMaxRanks];
    FastDiv by_nvb[kMaxRanks];
    uint64_t rows, stride;
    uint64_t tiles;  // wave tiles per chunk (the largest chunk's)
    uint64_t slots[kMaxRanks];  // scalar slots of each chunk
    FastDiv by_tile;            // division of a tile's number, and of a vector's by by_nvb
    int n;
    bool small;    // those numbers are below 2^31
    bool scalars;  // some chunk has slots
    // Each row's vectors start at its first element whose index is a multiple of four
    // (else the chunk's split g puts them on the grid of its stores).  A vector off
    // the generator's blocks of four needs one block more: twice the work in fp32.
    bool on_blocks;
};

// Elements of a row before its vectors, on_blocks.
__device__ __forceinline__ uint64_t before_block(const ChunkArgs& a, int c, uint64_t row)
{
    return (0 - (a.off[c] + row * a.stride)) & 3;
}

// Wave tile t: chunk and tile within it.  A flat split (rows == 1) walks the
// tensor in address order; a split by columns takes the chunks in turn, so that
// the workgroups at work read neighbouring columns of the same rows.
__device__ __forceinline__ void tile_chunk(const ChunkArgs& a, uint64_t t, int& c, uint64_t& j)
{
    const uint64_t by = a.rows == 1 ? a.tiles : (uint64_t)a.n;
    const uint64_t q = a.small ? a.by_tile.div((uint32_t)t) : t / by;
    const uint64_t r = t - q * by;
    c = __builtin_amdgcn_readfirstlane((int)(a.rows == 1 ? q : r));
    j = a.rows == 1 ? r : q;
}

// Vector v of chunk c: its row and first column; false past the row's end.
template <class T>
__device__ __forceinline__ bool vector_place(const ChunkArgs& a, int c, uint64_t v, uint64_t& row, uint64_t& col)
{
    const RowSplit& g = a.g[c];
    if (v >= a.rows * g.nvb) return false;
    row = 0;
    if (a.rows != 1) row = a.small ? a.by_nvb[c].div((uint32_t)v) : v / g.nvb;
    col = (v - row * g.nvb) * T::VEC;
    if (!a.on_blocks) {
        col += g.head;
        return true;
    }
    col += before_block(a, c, row);
    return col + T::VEC <= a.width[c];
}

// Slot k's element of chunk c's scalars; false where it has none.
template <class T>
__device__ __forceinline__ bool scalar_place(const ChunkArgs& a, int c, uint64_t k, uint64_t& row, uint64_t& col)
{
    if (!a.on_blocks) {
        scalar_slot(k, a.g[c], T::VEC, row, col);
        return true;
    }
    constexpr uint64_t S = T::VEC + 2;
    row = k / S;
    const uint64_t j = k - row * S, head = before_block(a, c, row), width = a.width[c];
    const uint64_t vectors = width > head ? (width - head) / T::VEC : 0;
    col = j < head ? j : vectors * T::VEC + j;
    return col < width;
}

struct DropRsArgs {
    const char* src[kMaxRanks];
    const char* res[kMaxRanks];
    char* dst[kMaxRanks];
    ChunkArgs ch;
    MaskArgs m;
};

template <class T, int N, bool RES>
__global__ __launch_bounds__(64) void k_dropout_reduce_scatter(DropRsArgs a)
{
    constexpr uint64_t W = 64, E = T::ESZ;
    const Mask mask(a.m);
    const uint64_t lane = threadIdx.x;
    const ChunkArgs& ch = a.ch;
    for (uint64_t t = blockIdx.x; t < ch.tiles * N; t += gridDim.x) {
        int c;
        uint64_t j;
        tile_chunk(ch, t, c, j);
        uint64_t row, col;
        if (!vector_place<T>(ch, c, j * W + lane, row, col)) continue;
        const uint64_t i = ch.off[c] + row * ch.stride + col;
        const uint64_t o = (row * ch.width[c] + col) * E;
        u32x4 in[N], res = {};
#pragma unroll
        for (int r = 0; r < N; r++) in[r] = ld16<true>(a.src[r] + i * E);
        if constexpr (RES) res = ld16<true>(a.res[c] + o);
        issue_loads_first();
        float acc[T::VEC];
        fold_f32<T, N>(in, acc);
        const uint32_t bits = mask.keep<T::VEC>(i);
#pragma unroll
        for (int k = 0; k < T::VEC; k++) acc[k] = mask.apply(acc[k], bits, k);
        st16<true>(a.dst[c] + o, RES ? add_residual<T>(acc, res) : T::pack(acc));
    }
    if (!ch.scalars) return;
    for (int c = 0; c < N; c++) {
        const uint64_t ns = ch.slots[c];
        for (uint64_t k = blockIdx.x * W + lane; k < ns; k += (uint64_t)gridDim.x * W) {
            uint64_t row, col;
            if (!scalar_place<T>(ch, c, k, row, col)) continue;
            const uint64_t i = ch.off[c] + row * ch.stride + col;
            const uint64_t o = (row * ch.width[c] + col) * E;
            float acc = T::widen(load_s<T>(a.src[0] + i * E));
#pragma unroll
            for (int r = 1; r < N; r++) acc += T::widen(load_s<T>(a.src[r] + i * E));
            acc = mask.apply(acc, mask.keep<1>(i), 0);
            if constexpr (RES) acc += T::widen(load_s<T>(a.res[c] + o));
            store_s<T>(a.dst[c] + o, T::narrow(acc));
        }
    }
}

struct DropAgArgs {
    const char* src[kMaxRanks];
    char* dst[kMaxRanks];
    ChunkArgs ch;
    MaskArgs m;
};

template <class T>
__global__ __launch_bounds__(64) void k_dropout_all_gather(DropAgArgs a)
{
    constexpr uint64_t W = 64, E = T::ESZ;
    const Mask mask(a.m);
    const uint64_t lane = threadIdx.x;
    const ChunkArgs& ch = a.ch;
    for (uint64_t t = blockIdx.x; t < ch.tiles * (uint64_t)ch.n; t += gridDim.x) {
        int c;
        uint64_t j;
        tile_chunk(ch, t, c, j);
        uint64_t row, col;
        if (!vector_place<T>(ch, c, j * W + lane, row, col)) continue;
        const uint64_t i = ch.off[c] + row * ch.stride + col;
        const u32x4 in = ld16<true>(a.src[c] + (row * ch.width[c] + col) * E);
        const uint32_t bits = mask.keep<T::VEC>(i);
        float x[T::VEC];
        T::unpack(in, x);
#pragma unroll
        for (int k = 0; k < T::VEC; k++) x[k] = mask.apply(x[k], bits, k);
        const u32x4 out = T::pack(x);
        for (int r = 0; r < ch.n; r++) st16<true>(a.dst[r] + i * E, out);
    }
    if (!ch.scalars) return;
    for (int c = 0; c < ch.n; c++) {
        const uint64_t ns = ch.slots[c];
        for (uint64_t k = blockIdx.x * W + lane; k < ns; k += (uint64_t)gridDim.x * W) {
            uint64_t row, col;
            if (!scalar_place<T>(ch, c, k, row, col)) continue;
            const uint64_t i = ch.off[c] + row * ch.stride + col;
            const float x = T::widen(load_s<T>(a.src[c] + (row * ch.width[c] + col) * E));
            const typename T::S s = T::narrow(mask.apply(x, mask.keep<1>(i), 0));
            for (int r = 0; r < ch.n; r++) store_s<T>(a.dst[r] + i * E, s);
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
using namespace host;

// Workgroups: one per wave tile, up to `per_cu` per CU; tails and heads need
// at least one.
unsigned wave_grid(uint64_t tiles, int cus, int per_cu)
{
    const uint64_t cap = (uint64_t)cus * (uint64_t)per_cu;
    const uint64_t g = tiles < cap ? tiles : cap;
    return (unsigned)(g < 1 ? 1 : g);
}

// Waves per CU, by the 16-byte loads that a lane has in flight and the bytes that
// the call moves.  Measured on MI355X, bf16, 2 GB moved (TB/s):
//   all-reduce, ranks (+ residuals): 1: 16 waves 5.2, 8 waves 4.8; 1 + 1: 8 6.0,
//   16 5.7; 2: 8 6.0, 16 5.3; 4: 4 6.0, 8 5.8; 8: 4 5.85, 8 5.5; 8 + 1: 4 5.8, 2 5.75;
//   6 + 6: 2 6.1, 4 5.75; 8 + 8: 2 5.9, 4 5.8, 16 5.4; 16: 2 5.6, 4 5.5;
//   reduce-scatter: 1: 16 4.8, 8 3.8; 2: 16 5.4, 8 5.2; 2 + 1: 8 5.9, 16 5.6; 4: 8 6.0,
//   4 4.9; 8: 4 5.6, 8 5.2; 16: 4 5.4, 8 5.2.
// A call that the 256 MB Infinity Cache holds is better off with more (100 MB,
// all-reduce of 2: 16 waves 5.6, 4 4.3; of 8 + 8: 16 6.1, 2 5.6).
constexpr uint64_t kCached = 256ull << 20;

int allreduce_waves(int loads, uint64_t bytes)
{
    if (bytes <= kCached) return loads <= 1 ? 32 : 16;
    return loads <= 1 ? 16 : loads <= 3 ? 8 : loads <= 9 ? 4 : 2;
}

int reduce_scatter_waves(int loads, uint64_t bytes)
{
    if (bytes <= kCached) return loads <= 1 ? 32 : 16;
    return loads <= 2 ? 16 : loads <= 5 ? 8 : 4;
}

// The all-gather reads one vector per lane and stores it to every rank: 64 waves per
// CU (one rank 4.6 TB/s, 16 waves 4.2; 8 ranks 4.8 with 8 to 64, and 1 store in
// flight per wave 4.4-4.8).
constexpr int kGatherWaves = 64;

template <class T, int N, int RES>
vrc_status_t launch_ar(const DropArArgs& a, int cus, hipStream_t st)
{
    const uint64_t tiles = (a.g.nvb + 63) / 64;
    constexpr int loads = RES == 2 ? 2 * N : N + RES;
    const int waves = allreduce_waves(loads, (loads + N) * a.g.nvb * 16);
    k_dropout_allreduce<T, N, RES><<<wave_grid(tiles, cus, waves), 64, 0, st>>>(a);
    return check_launch();
}

template <class T, int N>
vrc_status_t launch_ar_res(const DropArArgs& a, int res, int cus, hipStream_t st)
{
    switch (res) {
    case 0: return launch_ar<T, N, 0>(a, cus, st);
    case 1: return launch_ar<T, N, 1>(a, cus, st);
    }
    return launch_ar<T, N, 2>(a, cus, st);
}

template <class T>
vrc_status_t allreduce_typed(const char* const* x, const char* const* res, char* const* y, int n, uint64_t count,
                             const MaskArgs& m, int cus, hipStream_t st)
{
    DropArArgs a = {};
    int kind = res ? 1 : 0;
    uintptr_t dst[kMaxRanks];
    for (int r = 0; r < n; r++) {
        a.src[r] = x[r];
        a.dst[r] = y[r];
        dst[r] = (uintptr_t)y[r];
        if (res) {
            a.res[r] = res[r];
            if (res[r] != res[0]) kind = 2;
        }
    }
    a.g = split_rows(write_ref(dst, n), count, T::ESZ);
    a.m = m;
    switch (n) {
    case 1: return launch_ar_res<T, 1>(a, kind, cus, st);
#define VRC_CASE(N) \
    case N: return launch_ar_res<T, N>(a, kind, cus, st);
        VRC_FOR_N(VRC_CASE)
#undef VRC_CASE
    }
    return VRC_ERR_INVALID_ARG;
}

// The chunks of a tensor of `total` elements split over n ranks: flat for
// outer == 1, by columns otherwise.  `ref` gives the address that chunk c's
// vector grid follows, unless `blocks` and the generator's blocks of four lie
// otherwise.
template <class T, class Ref>
ChunkArgs make_chunks(int n, uint64_t total, uint64_t outer, bool blocks, Ref ref)
{
    ChunkArgs a = {};
    a.n = n;
    a.rows = outer;
    a.stride = total / outer;
    for (int c = 0; c < n; c++) {
        if (outer == 1) {
            chunk_range(total, n, c, &a.off[c], &a.width[c]);
        } else {
            a.width[c] = a.stride / (uint64_t)n;
            a.off[c] = (uint64_t)c * a.width[c];
        }
        a.on_blocks = a.on_blocks || (blocks && ((outer > 1 && a.stride % 4 != 0) || a.off[c] % 4 != 0));
    }
    for (int c = 0; c < n; c++) {
        a.g[c] = a.on_blocks ? RowSplit{0, a.width[c] / T::VEC, 0} : split_rows(ref(c, a.off[c]), a.width[c], T::ESZ);
        a.by_nvb[c] = FastDiv::of(a.g[c].nvb);
        const uint64_t tiles = (a.rows * a.g[c].nvb + 63) / 64;
        if (tiles > a.tiles) a.tiles = tiles;
        a.slots[c] = a.rows * (a.on_blocks ? T::VEC + 2 : a.g[c].head + a.g[c].tail);
        a.scalars = a.scalars || a.slots[c];
    }
    // a chunk's vectors are at most 64 of each of its tiles
    a.small = a.tiles * 64 < 1ull << 31 && a.tiles * (uint64_t)n < 1ull << 31;
    a.by_tile = FastDiv::of(outer == 1 ? a.tiles : (uint64_t)n);
    return a;
}

template <class T>
vrc_status_t reduce_scatter_typed(const char* const* x, const char* const* res, char* const* y, int n, uint64_t count,
                                  uint64_t outer, const MaskArgs& m, int cus, hipStream_t st)
{
    DropRsArgs a = {};
    for (int r = 0; r < n; r++) {
        a.src[r] = x[r];
        a.dst[r] = y[r];
        a.res[r] = res ? res[r] : nullptr;
    }
    a.ch = make_chunks<T>(n, count, outer, true, [&](int c, uint64_t) { return (uintptr_t)y[c]; });
    a.m = m;
    const unsigned grid = wave_grid(a.ch.tiles * (uint64_t)n, cus, reduce_scatter_waves(n + (res ? 1 : 0), n * count * T::ESZ));
    switch (n) {
#define VRC_CASE(N)                                                                  \
    case N:                                                                          \
        if (res) k_dropout_reduce_scatter<T, N, true><<<grid, 64, 0, st>>>(a);       \
        else k_dropout_reduce_scatter<T, N, false><<<grid, 64, 0, st>>>(a);          \
        return check_launch();
        VRC_CASE(1)
        VRC_FOR_N(VRC_CASE)
#undef VRC_CASE
    }
    return VRC_ERR_INVALID_ARG;
}

template <class T>
vrc_status_t all_gather_typed(const char* const* x, char* const* y, int n, uint64_t total, uint64_t outer,
                              const MaskArgs& m, int cus, hipStream_t st)
{
    DropAgArgs a = {};
    uintptr_t dst[kMaxRanks];
    for (int r = 0; r < n; r++) {
        a.src[r] = x[r];
        a.dst[r] = y[r];
        dst[r] = (uintptr_t)y[r];
    }
    const uintptr_t at = write_ref(dst, n);
    a.ch = make_chunks<T>(n, total, outer, outer > 1, [&](int, uint64_t off) { return at + off * T::ESZ; });
    a.m = m;
    k_dropout_all_gather<T><<<wave_grid(a.ch.tiles * (uint64_t)n, cus, kGatherWaves), 64, 0, st>>>(a);
    return check_launch();
}

}  // namespace

namespace host {

#define VRC_BY_TYPE(call)                      \
    switch (dt) {                              \
    case VRC_FP32: return call(F32);           \
    case VRC_FP16: return call(F16);           \
    case VRC_BF16: return call(BF16);          \
    default: return VRC_ERR_UNSUPPORTED;       \
    }

vrc_status_t run_allreduce_dropout(const char* const* x, const char* const* res, char* const* y, int n, uint64_t count,
                                   vrc_dtype_t dt, const MaskArgs& m, int cus, hipStream_t st)
{
#define VRC_CALL(T) allreduce_typed<T>(x, res, y, n, count, m, cus, st)
    VRC_BY_TYPE(VRC_CALL)
#undef VRC_CALL
}

vrc_status_t run_reduce_scatter_dropout(const char* const* x, const char* const* res, char* const* y, int n,
                                        uint64_t count, uint64_t outer, vrc_dtype_t dt, const MaskArgs& m, int cus,
                                        hipStream_t st)
{
#define VRC_CALL(T) reduce_scatter_typed<T>(x, res, y, n, count, outer, m, cus, st)
    VRC_BY_TYPE(VRC_CALL)
#undef VRC_CALL
}

vrc_status_t run_all_gather_dropout(const char* const* x, char* const* y, int n, uint64_t total, uint64_t outer,
                                    vrc_dtype_t dt, const MaskArgs& m, int cus, hipStream_t st)
{
#define VRC_CALL(T) all_gather_typed<T>(x, y, n, total, outer, m, cus, st)
    VRC_BY_TYPE(VRC_CALL)
#undef VRC_CALL
}

}  // namespace host
}  // namespace vrc
