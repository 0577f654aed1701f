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

#include <type_traits>

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

    // mask * scale * a, with +0 for a dropped element.  The product is an fp32 value of
    // its own: seeing what becomes of it, the compiler would join it with a conversion to
    // fp16 in one operation, which rounds once and makes -0 a +0.  (It has no such
    // operation for the other types.)
    template <class T>
    __device__ __forceinline__ float apply(float a, uint32_t bits, int j) const
    {
        float y = a * scale;
        if constexpr (std::is_same<T, F16>::value) __asm__("" : "+v"(y));
        return (bits >> j & 1u) ? y : 0.0f;
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
        for (int i = 0; i < T::VEC; i++) acc[i] = mask.apply<T>(acc[i], bits, i);
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
        acc = mask.apply<T>(acc, mask.keep<1>(i), 0);
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
    uint64_t rows, stride, last_width;
    uint64_t tiles;   // wave tiles per chunk (the largest chunk's)
    FastDiv by_tile;  // division of a tile's number, and of a vector's by by_nvb
    int n;
    bool small;  // those numbers are below 2^31
    // The elements that no vector holds: slots, numbered row by row and in a row chunk
    // by chunk, so that neighbouring lanes have neighbouring elements of the whole
    // tensor; chunk c's are from first_slot[c] of a row's row_slots.
    uint64_t slots, row_slots;
    uint32_t first_slot[kMaxRanks];
    FastDiv by_row_slots, by_n;
    bool small_slots;  // their numbers are below 2^31
    // Narrow rows: no vectors, and slot k is elements 4k .. 4k + 3 of the whole tensor, one
    // of the generator's blocks, in whatever chunks and rows they lie.
    bool narrow;
    uint64_t total;
    FastDiv by_width;
    // Each row's vectors start at its first element whose index is a multiple of four
    // (else the chunk's split g puts them on the grid of its stores).  A vector off
    // the generator's blocks of four needs one block more: twice the work in fp32.
    bool on_blocks;
};

// Chunk c's off and width without an array (the last of a flat split has the remainder).
__device__ __forceinline__ uint64_t chunk_off(const ChunkArgs& a, int c) { return (uint64_t)c * a.width[0]; }
__device__ __forceinline__ uint64_t chunk_width(const ChunkArgs& a, int c)
{
    return c == a.n - 1 ? a.last_width : a.width[0];
}

// Elements of a row before its vectors, on_blocks: at most three, and less than a vector
// after them.
template <class T>
constexpr uint32_t kBlockSlots = T::VEC + 2;

__device__ __forceinline__ uint64_t before_block(const ChunkArgs& a, int c, uint64_t row)
{
    return (0 - (chunk_off(a, c) + row * a.stride)) & 3;
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

// What a lane needs of a chunk that it found by its own element, copied into LDS: by a
// lane's own index these would be vector loads of the kernel's arguments (4 x [262144,
// 4 x 63] bf16 166 us, 235 us by such loads).
struct ChunkTable {
    const char* in[kMaxRanks];
    char* out[kMaxRanks];
    uint32_t head[kMaxRanks];
    uint64_t body[kMaxRanks];  // elements in a row's vectors

    __device__ __forceinline__ void put(int c, const char* from, char* to, const RowSplit& g, uint64_t vec)
    {
        in[c] = from;
        out[c] = to;
        head[c] = (uint32_t)g.head;
        body[c] = g.nvb * vec;
    }
};

// Slot k's chunk, row and column; false where it has no element.
template <class T>
__device__ __forceinline__ bool scalar_place(const ChunkArgs& a, const ChunkTable& table, uint64_t k, int& c, uint64_t& row,
                                             uint64_t& col)
{
    row = a.small_slots ? a.by_row_slots.div((uint32_t)k) : k / a.row_slots;
    uint32_t j = (uint32_t)(k - row * a.row_slots);
    if (!a.on_blocks) {
        c = 0;
        uint32_t first = 0;
        for (int d = 1; d < a.n; d++) {
            if (j < a.first_slot[d]) continue;
            c = d;
            first = a.first_slot[d];
        }
        j -= first;
        col = j;
        if (j >= table.head[c]) col += table.body[c];
        return true;
    }
    c = (int)(j / kBlockSlots<T>);
    j -= (uint32_t)c * kBlockSlots<T>;
    col = j;
    const uint64_t head = before_block(a, c, row), width = chunk_width(a, c);
    const uint64_t vectors = width > head ? (width - head) / T::VEC : 0;
    if (j >= head) col += vectors * T::VEC;
    return col < width;
}

// Narrow rows: where the elements 4k .. 4k + 3 of the whole tensor lie.
struct NarrowPlace {
    int c;
    uint64_t row, col;

    __device__ NarrowPlace(const ChunkArgs& a, uint64_t k)
    {
        const uint64_t q = a.small_slots ? a.by_width.div((uint32_t)k * 4) : 4 * k / a.width[0];
        row = a.small_slots ? a.by_n.div((uint32_t)q) : q / (uint64_t)a.n;
        c = (int)(q - row * (uint64_t)a.n);
        col = 4 * k - q * a.width[0];
    }
    // In a chunk's own buffer.
    __device__ uint64_t at(const ChunkArgs& a) const { return row * a.width[0] + col; }
    // The four lie in one row of one chunk.
    __device__ bool together(const ChunkArgs& a) const { return col + 4 <= a.width[0]; }
    __device__ void next(const ChunkArgs& a)
    {
        if (++col < a.width[0]) return;
        col = 0;
        if (++c < a.n) return;
        c = 0;
        row++;
    }
};

// Four consecutive elements as they are stored, at any element.
template <class T>
struct Quad {
    typedef uint32_t Words __attribute__((ext_vector_type(T::ESZ), aligned(1)));
    typename T::S s[4];

    __device__ __forceinline__ void load(const char* p)
    {
        const Words v = __builtin_nontemporal_load((global_ptr<const Words>)p);
#pragma unroll
        for (int e = 0; e < 4; e++) s[e] = T::ESZ == 4 ? v[e % T::ESZ] : (typename T::S)(v[e / 2] >> (16 * (e & 1)));
    }
    __device__ __forceinline__ void store(char* p) const
    {
        Words v;
#pragma unroll
        for (int w = 0; w < T::ESZ; w++)
            v[w] = T::ESZ == 4 ? (uint32_t)s[w] : (uint32_t)s[2 * w % 4] | (uint32_t)s[(2 * w + 1) % 4] << 16;
        __builtin_nontemporal_store(v, (global_ptr<Words>)p);
    }
    // The first `left` of them; the others are zero.
    __device__ __forceinline__ void load_part(const char* p, int left)
    {
#pragma unroll
        for (int e = 0; e < 4; e++) s[e] = e < left ? load_s<T>(p + e * T::ESZ) : (typename T::S)0;
    }
    __device__ __forceinline__ void store_part(char* p, int left) const
    {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (e < left) store_s<T>(p + e * T::ESZ, s[e]);
    }
    // From or to the chunks' own buffers.
    __device__ __forceinline__ void gather(const ChunkArgs& a, const ChunkTable& t, NarrowPlace at, int left)
    {
        if (left == 4 && at.together(a)) {
            load(t.in[at.c] + at.at(a) * T::ESZ);
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            s[e] = e < left ? load_s<T>(t.in[at.c] + at.at(a) * T::ESZ) : (typename T::S)0;
            at.next(a);
        }
    }
    __device__ __forceinline__ void scatter(const ChunkArgs& a, const ChunkTable& t, NarrowPlace at, int left) const
    {
        if (left == 4 && at.together(a)) {
            store(t.out[at.c] + at.at(a) * T::ESZ);
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            if (e < left) store_s<T>(t.out[at.c] + at.at(a) * T::ESZ, s[e]);
            at.next(a);
        }
    }
};

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
        for (int k = 0; k < T::VEC; k++) acc[k] = mask.apply<T>(acc[k], bits, k);
        st16<true>(a.dst[c] + o, RES ? add_residual<T>(acc, res) : T::pack(acc));
    }
    if (ch.slots == 0) return;
    __shared__ ChunkTable table;
    if (lane == 0) {
#pragma unroll
        for (int c = 0; c < N; c++) table.put(c, a.res[c], a.dst[c], ch.g[c], T::VEC);
    }
    __syncthreads();
    for (uint64_t k = blockIdx.x * W + lane; k < ch.slots; k += (uint64_t)gridDim.x * W) {
        int c;
        uint64_t row, col;
        if (!scalar_place<T>(ch, table, k, c, row, col)) continue;
        const uint64_t i = chunk_off(ch, c) + row * ch.stride + col;
        const uint64_t o = (row * chunk_width(ch, c) + col) * E;
        typename T::S in[N], res = 0;
#pragma unroll
        for (int r = 0; r < N; r++) in[r] = load_s<T>(a.src[r] + i * E);
        if constexpr (RES) res = load_s<T>(table.in[c] + o);
        issue_loads_first();
        float acc = T::widen(in[0]);
#pragma unroll
        for (int r = 1; r < N; r++) acc += T::widen(in[r]);
        acc = mask.apply<T>(acc, mask.keep<1>(i), 0);
        if constexpr (RES) acc += T::widen(res);
        store_s<T>(table.out[c] + o, T::narrow(acc));
    }
}

// Narrow rows: a lane folds four elements of the whole tensor's rows, which lie together
// in every input, draws their one block of the mask, and writes them to the chunks that
// they belong to.  8 x [16384, 8 x 7] fp16, a stream of 17 MB, 7.3 us; [131072, 8 x 32]
// 0.6 GB, 130 us, 4.6 TB/s.
template <class T, int N, bool RES>
__global__ __launch_bounds__(64) void k_dropout_reduce_scatter_narrow(DropRsArgs a)
{
    constexpr uint64_t W = 64, E = T::ESZ;
    const Mask mask(a.m);
    const uint64_t lane = threadIdx.x;
    const ChunkArgs& ch = a.ch;
    __shared__ ChunkTable table;
    if (lane == 0) {
#pragma unroll
        for (int c = 0; c < N; c++) table.put(c, a.res[c], a.dst[c], ch.g[c], 0);
    }
    __syncthreads();
    for (uint64_t k = blockIdx.x * W + lane; k < ch.slots; k += (uint64_t)gridDim.x * W) {
        const uint64_t i = 4 * k;
        const int left = ch.total - i < 4 ? (int)(ch.total - i) : 4;
        Quad<T> x[N], res = {};
        if (left == 4) {
#pragma unroll
            for (int r = 0; r < N; r++) x[r].load(a.src[r] + i * E);
        } else {
#pragma unroll
            for (int r = 0; r < N; r++) x[r].load_part(a.src[r] + i * E, left);
        }
        const NarrowPlace to(ch, k);
        if constexpr (RES) res.gather(ch, table, to, left);
        issue_loads_first();
        const uint32_t bits = mask.keep<4>(i);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            float acc = T::widen(x[0].s[e]);
#pragma unroll
            for (int r = 1; r < N; r++) acc += T::widen(x[r].s[e]);
            acc = mask.apply<T>(acc, bits, e);
            if constexpr (RES) acc += T::widen(res.s[e]);
            x[0].s[e] = T::narrow(acc);
        }
        x[0].scatter(ch, table, to, left);
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
        for (int k = 0; k < T::VEC; k++) x[k] = mask.apply<T>(x[k], bits, k);
        const u32x4 out = T::pack(x);
        for (int r = 0; r < ch.n; r++) st16<true>(a.dst[r] + i * E, out);
    }
    if (ch.slots == 0) return;
    __shared__ ChunkTable table;
    if (lane < (uint64_t)ch.n) table.put((int)lane, a.src[lane], nullptr, ch.g[lane], T::VEC);
    __syncthreads();
    for (uint64_t k = blockIdx.x * W + lane; k < ch.slots; k += (uint64_t)gridDim.x * W) {
        int c;
        uint64_t row, col;
        if (!scalar_place<T>(ch, table, k, c, row, col)) continue;
        const uint64_t i = chunk_off(ch, c) + row * ch.stride + col;
        const float x = T::widen(load_s<T>(table.in[c] + (row * chunk_width(ch, c) + col) * E));
        const typename T::S s = T::narrow(mask.apply<T>(x, mask.keep<1>(i), 0));
        for (int r = 0; r < ch.n; r++) store_s<T>(a.dst[r] + i * E, s);
    }
}

// Narrow rows: a lane gathers four elements of the outputs' rows.  8 x [16384, 7] fp16
// 7.7 us; [131072, 56] 1.06 GB, 260 us, 4.1 TB/s (830 us by vectors and single elements).
template <class T>
__global__ __launch_bounds__(64) void k_dropout_all_gather_narrow(DropAgArgs a)
{
    constexpr uint64_t W = 64, E = T::ESZ;
    const Mask mask(a.m);
    const uint64_t lane = threadIdx.x;
    const ChunkArgs& ch = a.ch;
    __shared__ ChunkTable table;
    if (lane < (uint64_t)ch.n) table.put((int)lane, a.src[lane], nullptr, ch.g[lane], 0);
    __syncthreads();
    for (uint64_t k = blockIdx.x * W + lane; k < ch.slots; k += (uint64_t)gridDim.x * W) {
        const uint64_t i = 4 * k;
        const int left = ch.total - i < 4 ? (int)(ch.total - i) : 4;
        Quad<T> x;
        x.gather(ch, table, NarrowPlace(ch, k), left);
        const uint32_t bits = mask.keep<4>(i);
#pragma unroll
        for (int e = 0; e < 4; e++) x.s[e] = T::narrow(mask.apply<T>(T::widen(x.s[e]), bits, e));
        if (left == 4) {
            for (int r = 0; r < ch.n; r++) x.store(a.dst[r] + i * E);
        } else {
            for (int r = 0; r < ch.n; r++) x.store_part(a.dst[r] + i * E, left);
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
using namespace host;

// Workgroups: one per wave tile, up to `per_cu` per CU, and at least one.
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

// The workgroups of a call on chunks.  Where more waves of elements go one by one, or by
// four in narrow rows, than in vectors, the call's time is theirs: up to 64 per CU (us
// with 4 / 16 / 64, reduce-scatter: 8 x [16384, 8 x 47] fp16 50 / 29 / 29, 2 x [524288, 2 x
// 7] bf16 36 / 19 / 16, 8 x [60000, 8 x 65] fp16 270 / 256 / 233, but 16 x [32768, 16 x 40]
// bf16 180 / 169 / 182; all-gather: 52 / 35 / 33, 39 / 20 / 17, 235 / 156 / 156, 189 / 192 / 202).
constexpr int kScalarWaves = 64;

unsigned chunk_grid(const ChunkArgs& a, int cus, int per_cu)
{
    const uint64_t tiles = a.tiles * (uint64_t)a.n, by_slots = (a.slots + 63) / 64;
    return by_slots > tiles ? wave_grid(by_slots, cus, kScalarWaves) : wave_grid(tiles, cus, per_cu);
}

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

// Narrow rows, of `bytes` in a rank's part.  A row's first and last elements go one by
// one where they are no whole vectors, and rows of a few vectors lie on as many memory
// lines as whole lines would.  us by vectors / by blocks of four of the whole tensor, on
// 8 ranks of 16384 rows: fp16 reduce-scatter of 9 elements 31 / 8, 23 44 / 17, 47 61 / 36,
// fp32 of 16 27 / 13; of 8192 rows fp16: of 56 22 / 16, but 64 17 / 18 and, with
// residuals, 120 39 / 41.  2 ranks of 524288 rows, bf16: 8 16.4 / 14.8, 48 87 / 88.
constexpr bool narrow_rs(uint64_t bytes) { return bytes < 128; }

// The all-gather, 8192 rows on 8 ranks, fp16: 100 elements 45 / 33, 136 55 / 42, 200
// 71 / 60, 257 110 / 79, but whole lines 64 18 / 19, 128 31 / 35; 2 ranks of 65536 rows,
// bf16: 136 45 / 29, 257 64 / 63, whole lines 256 41 / 43.
constexpr bool narrow_ag(uint64_t bytes) { return bytes < 512 && bytes % 128 != 0; }

// The chunks of a tensor of `total` elements split over n ranks: flat for
// outer == 1, by columns otherwise.  `ref` gives the address that chunk c's
// vector grid follows, unless `blocks` and the generator's blocks of four lie
// otherwise.
template <class T, class Ref>
ChunkArgs make_chunks(int n, uint64_t total, uint64_t outer, bool blocks, bool narrow, Ref ref)
{
    ChunkArgs a = {};
    a.n = n;
    if (n == 1) outer = 1;  // one chunk is the tensor
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
    a.total = total;
    a.last_width = a.width[n - 1];
    a.narrow = narrow && outer > 1;
    a.by_n = FastDiv::of((uint64_t)n);
    if (a.narrow) {
        a.slots = (total + 3) / 4;
        a.small_slots = total < 1ull << 31;
        a.by_width = FastDiv::of(a.width[0]);
        return a;
    }
    for (int c = 0; c < n; c++) {
        a.g[c] = a.on_blocks ? RowSplit{0, a.width[c] / T::VEC, 0} : split_rows(ref(c, a.off[c]), a.width[c], T::ESZ);
        a.by_nvb[c] = FastDiv::of(a.g[c].nvb);
        const uint64_t tiles = (a.rows * a.g[c].nvb + 63) / 64;
        if (tiles > a.tiles) a.tiles = tiles;
        a.first_slot[c] = (uint32_t)a.row_slots;
        a.row_slots += a.on_blocks ? kBlockSlots<T> : a.g[c].head + a.g[c].tail;
    }
    a.slots = a.rows * a.row_slots;
    a.by_row_slots = FastDiv::of(a.row_slots);
    a.small_slots = a.slots < 1ull << 31;
    // a chunk's vectors are at most 64 of each of its tiles
    a.small = a.tiles * 64 < 1ull << 31 && a.tiles * (uint64_t)n < 1ull << 31;
    a.by_tile = FastDiv::of(outer == 1 ? a.tiles : (uint64_t)n);
    return a;
}

template <class T, int N, bool RES>
vrc_status_t launch_rs(const DropRsArgs& a, unsigned grid, hipStream_t st)
{
    if constexpr (N > 1) {
        if (a.ch.narrow) {
            k_dropout_reduce_scatter_narrow<T, N, RES><<<grid, 64, 0, st>>>(a);
            return check_launch();
        }
    }
    k_dropout_reduce_scatter<T, N, RES><<<grid, 64, 0, st>>>(a);
    return check_launch();
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
    a.ch = make_chunks<T>(n, count, outer, true, narrow_rs(count / outer / (uint64_t)n * T::ESZ), [&](int c, uint64_t) { return (uintptr_t)y[c]; });
    a.m = m;
    const unsigned grid = chunk_grid(a.ch, cus, reduce_scatter_waves(n + (res ? 1 : 0), n * count * T::ESZ));
    switch (n) {
#define VRC_CASE(N) \
    case N: return res ? launch_rs<T, N, true>(a, grid, st) : launch_rs<T, N, false>(a, grid, st);
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
    a.ch = make_chunks<T>(n, total, outer, outer > 1, narrow_ag(total / outer / (uint64_t)n * T::ESZ), [&](int, uint64_t off) { return at + off * T::ESZ; });
    a.m = m;
    const unsigned grid = chunk_grid(a.ch, cus, kGatherWaves);
    if (a.ch.narrow) k_dropout_all_gather_narrow<T><<<grid, 64, 0, st>>>(a);
    else k_dropout_all_gather<T><<<grid, 64, 0, st>>>(a);
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
