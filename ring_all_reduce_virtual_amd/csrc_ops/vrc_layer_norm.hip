// vrc_layer_norm.hip -- layer norm (or RMS norm) in the collective before it, and
// its gradient with the weights' gradients reduced over all ranks' rows.
//
// A row's values stay in registers from the first load to the last store, so
// that every input is read once and every output written once: both passes are
// streams, bound by memory.  LANES lanes have a row, each V vectors of 16 bytes
// of it (vector j * LANES + lane) and one element of the row's end that is no whole
// vector.  The statistics are two passes over those registers (the mean, then the
// squares of the differences from it), not one over sums of squares, which
// loses the variance of rows far from zero.
//
// Measured on MI355X: 8 x [8192, 4096] bf16, summed with the residual, eight outputs, 225 us
// (5.4 TB/s; a large copy 4.9); the gradient of 8 x [2048, 8192] bf16 204 us and 7 us for the
// join of 512 partial sums; 3 x [4003, 1053] fp32, scattered, 20 us (5.0 TB/s).
#include <hip/hip_runtime.h>

#include "vrc_model_host.hpp"

namespace vrc {
namespace {

using host::NormCall;

struct NormArgs {
    const char* src[kMaxRanks];  // the ranks' values (their gradients)
    const char* res[kMaxRanks];  // by part; null where there is none
    const char* sum[kMaxRanks];  // by part: the gradient's h
    char* dst[kMaxRanks];
    char* out[kMaxRanks];        // by part: where h goes, or null
    float* mean[kMaxRanks];      // by part, or null
    float* rstd[kMaxRanks];
    const char* w;
    const char* b;
    float* partial;  // the gradient's: [workgroup][2][width]
    uint64_t rows;   // of every src
    uint32_t width, vectors, tail;  // vectors: whole ones of a row; tail: elements behind them
    float eps, inv_width;
    int n, join, center, wide_weight;
};

// Rank r's rows: `count` of them, from row `first` of its sources.
struct Rows {
    uint64_t first, count;
};

__device__ __forceinline__ Rows rows_of(const NormArgs& a, uint32_t r)
{
    if (a.join != VRC_NORM_SCATTER) return {0, a.rows};
    const uint64_t each = a.rows / (uint64_t)a.n;
    return {r * each, r + 1 == (uint32_t)a.n ? a.rows - r * each : each};
}

// One row's values of one lane: V vectors and one of the row's last elements.
template <class T, int V>
struct Part {
    static constexpr int E = V * T::VEC;
    float v[E], t;
};

// STREAM: rows are read and written past the caches' replacement (non-temporal).
// TAIL: rows may have elements behind their last vector.
template <class T, int LANES, int V, bool STREAM, bool TAIL = true>
struct RowIo {
    uint32_t at[V];    // this lane's vectors in bytes from the row's start; a lane without one has the last
    bool has[V];
    uint32_t tail_at;  // the same of its element of the end
    bool has_tail;
    bool vectors, tail;  // whether the row has any

    __device__ __forceinline__ RowIo(const NormArgs& a, uint32_t lane)
    {
        vectors = a.vectors != 0;
        tail = TAIL && a.tail != 0;
#pragma unroll
        for (int j = 0; j < V; j++) {
            const uint32_t i = j * LANES + lane;
            has[j] = i < a.vectors;
            at[j] = (has[j] ? i : vectors ? a.vectors - 1 : 0) * 16;
        }
        has_tail = TAIL && lane < a.tail;
        tail_at = (a.vectors * T::VEC + (has_tail ? lane : 0)) * T::ESZ;
    }
    struct Raw {
        u32x4 v[V];
        typename T::S t;
    };
    template <bool NT = STREAM>
    __device__ __forceinline__ Raw load(const char* row) const
    {
        Raw x;
        x.t = 0;
        if (tail) x.t = load_s<T>(row + tail_at);
        if (vectors) {
#pragma unroll
            for (int j = 0; j < V; j++) x.v[j] = ld16<NT>(row + at[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; j++) x.v[j] = u32x4{0, 0, 0, 0};
        }
        return x;
    }
    // Values that the lane does not have are zero.
    __device__ __forceinline__ void widen(const Raw& x, Part<T, V>& p) const
    {
#pragma unroll
        for (int j = 0; j < V; j++) {
            float f[T::VEC];
            T::unpack(x.v[j], f);
#pragma unroll
            for (int e = 0; e < T::VEC; e++) p.v[j * T::VEC + e] = has[j] ? f[e] : 0.0f;
        }
        p.t = has_tail ? T::widen(x.t) : 0.0f;
    }
    __device__ __forceinline__ void store(char* row, const Part<T, V>& p) const
    {
#pragma unroll
        for (int j = 0; j < V; j++)
            if (has[j]) st16<STREAM>(row + at[j], T::pack(p.v + j * T::VEC));
        if (has_tail) store_s<T>(row + tail_at, T::narrow(p.t));
    }
    // The same columns of the weight or the bias, of T or (wide) of fp32.
    __device__ __forceinline__ void load_weight(const char* w, bool wide, Part<T, V>& p) const
    {
        if (!wide) {
            widen(load<false>(w), p);
            return;
        }
        constexpr uint32_t UP = 4 / T::ESZ;  // bytes of fp32 per byte of T
#pragma unroll
        for (int j = 0; j < V; j++)
#pragma unroll
            for (int q = 0; q < T::VEC / 4; q++) {
                u32x4 x = {0, 0, 0, 0};
                if (vectors) x = ld16<false>(w + at[j] * UP + q * 16);
                float f[4];
                F32::unpack(x, f);
#pragma unroll
                for (int e = 0; e < 4; e++) p.v[j * T::VEC + q * 4 + e] = has[j] ? f[e] : 0.0f;
            }
        p.t = 0.0f;
        if (tail) p.t = has_tail ? F32::widen(load_s<F32>(w + tail_at * UP)) : 0.0f;
    }
};

// x += the next B sources' rows, all their loads under way at once, folded in order.
template <int B, class T, int LANES, int V, bool STREAM, class Row>
__device__ __forceinline__ void fold(const RowIo<T, LANES, V, STREAM>& io, Row row, int q, Part<T, V>& x)
{
    typename RowIo<T, LANES, V, STREAM>::Raw raw[B];
#pragma unroll
    for (int i = 0; i < B; i++) raw[i] = io.load(row(q + i));
    issue_loads_first();
#pragma unroll
    for (int i = 0; i < B; i++) {
        Part<T, V> p;
        io.widen(raw[i], p);
#pragma unroll
        for (int e = 0; e < p.E; e++) x.v[e] += p.v[e];
        x.t += p.t;
    }
}

// The fold of `n` sources' rows, B at a time; row(q) is where source q's starts.
template <int B, class T, int LANES, int V, bool STREAM, class Row>
__device__ __forceinline__ void fold_all(const RowIo<T, LANES, V, STREAM>& io, Row row, int n, Part<T, V>& x)
{
    // -0, which leaves the first value as it is
#pragma unroll
    for (int e = 0; e < x.E; e++) x.v[e] = -0.0f;
    x.t = -0.0f;
    int q = 0;
    for (; q + B <= n; q += B) fold<B>(io, row, q, x);
    if (B > 2 && n - q == 3) fold<3>(io, row, q, x);
    else if (B > 2 && n - q == 2) fold<2>(io, row, q, x);
    else if (B > 1 && n - q == 1) fold<1>(io, row, q, x);
    // what the lane does not have is zero for the sums
#pragma unroll
    for (int j = 0; j < V; j++)
#pragma unroll
        for (int e = 0; e < T::VEC; e++) x.v[j * T::VEC + e] = io.has[j] ? x.v[j * T::VEC + e] : 0.0f;
    x.t = io.has_tail ? x.t : 0.0f;
}

// Sums of K values each over a row's lanes, the same bits in every lane: a butterfly
// over the wave, then the waves' sums in order from `lds`, which no wave may still
// be reading from the call before the last.
template <int LANES, int K>
__device__ __forceinline__ void row_sums(float (&s)[K], float (*lds)[K], uint32_t wave)
{
#pragma unroll
    for (int k = 0; k < K; k++)
#pragma unroll
        for (int m = 32; m; m >>= 1) s[k] += __shfl_xor(s[k], m, 64);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < K; k++) lds[wave][k] = s[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; k++) s[k] = lds[0][k];
        for (int w = 1; w < LANES / 64; w++)
#pragma unroll
            for (int k = 0; k < K; k++) s[k] += lds[w][k];
    }
}

constexpr int block_of(int lanes) { return lanes < 256 ? 256 : lanes; }

template <class T, int LANES, int V, bool STREAM>
__global__ __launch_bounds__(block_of(LANES)) void k_layer_norm(NormArgs a)
{
    constexpr uint32_t ROWS = block_of(LANES) / LANES;  // of a workgroup at a time
    __shared__ float sums[2][LANES / 64][1];
    // where a workgroup has one row at a time, the compiler is to see that its address is uniform
    const uint32_t lane = ROWS > 1 ? threadIdx.x % LANES : threadIdx.x, group = ROWS > 1 ? threadIdx.x / LANES : 0;
    const uint32_t wave = lane / 64, r = blockIdx.y;
    const Rows mine = rows_of(a, r);
    const RowIo<T, LANES, V, STREAM> io(a, lane);
    const uint64_t pitch = (uint64_t)a.width * T::ESZ;
    const bool each = a.join == VRC_NORM_EACH, all = a.join == VRC_NORM_SUM;
    const int ranks = each ? 1 : a.n, sources = ranks + (a.res[r] != nullptr);
    // where a row is one wave's, no barrier is passed and waves may leave on their own
    for (uint64_t i = blockIdx.x * (uint64_t)ROWS + group; i < mine.count; i += gridDim.x * (uint64_t)ROWS) {
        Part<T, V> x, w, b;
        // 64 to 128 bytes a lane under way
        fold_all<(V <= 2 ? 4 : LANES == 1024 ? 1 : 2)>(io, [&](int q) { return q < ranks ? a.src[each ? r : q] + (mine.first + i) * pitch : a.res[r] + i * pitch; },
                 sources, x);
        io.load_weight(a.w, a.wide_weight, w);
        if (a.b) {
            io.load_weight(a.b, a.wide_weight, b);
        } else {
#pragma unroll
            for (int e = 0; e < b.E; e++) b.v[e] = -0.0f;
            b.t = -0.0f;
        }
        if (a.out[r]) io.store(a.out[r] + i * pitch, x);
        float mean = 0.0f, s[1];
        if (a.center) {
            s[0] = x.t;
#pragma unroll
            for (int e = 0; e < x.E; e++) s[0] += x.v[e];
            row_sums<LANES>(s, sums[0], wave);
            mean = s[0] * a.inv_width;
        }
        s[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < V; j++)
#pragma unroll
            for (int e = 0; e < T::VEC; e++) {
                const float d = io.has[j] ? x.v[j * T::VEC + e] - mean : 0.0f;
                s[0] = fmaf(d, d, s[0]);
            }
        const float d = io.has_tail ? x.t - mean : 0.0f;
        s[0] = fmaf(d, d, s[0]);
        row_sums<LANES>(s, sums[1], wave);
        const float rstd = 1.0f / sqrtf(s[0] * a.inv_width + a.eps);
#pragma unroll
        for (int e = 0; e < x.E; e++) x.v[e] = fmaf((x.v[e] - mean) * rstd, w.v[e], b.v[e]);
        x.t = fmaf((x.t - mean) * rstd, w.t, b.t);
        const int d0 = all ? 0 : (int)r, d1 = all ? a.n : d0 + 1;
        for (int q = d0; q < d1; q++) io.store(a.dst[q] + i * pitch, x);
        if (lane == 0) {
            if (a.mean[r]) a.mean[r][i] = mean;
            if (a.rstd[r]) a.rstd[r][i] = rstd;
        }
        // without a mean there is one sum a row: its place is free for the next row only behind a barrier
        if (LANES > 64 && !a.center) __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// The gradient.  A workgroup walks rows with its columns' sums for dweight and
// dbias in registers and leaves one partial sum of each per column; a second launch
// adds the workgroups' partial sums in order.
// ---------------------------------------------------------------------------
// ONE: each row has one source and is whole vectors; 512 lanes of two vectors then fit 128 registers, so that
// two workgroups, two rows, are on a CU at a time (8 x [2048, 8192] bf16 242 -> 211 us).
template <class T, int LANES, int V, bool STREAM, bool ONE>
__global__ __launch_bounds__(block_of(LANES), ONE && LANES == 512 && V == 2 ? 4 : 1) void k_layer_norm_grad(NormArgs a)
{
    constexpr uint32_t ROWS = block_of(LANES) / LANES, E = V * T::VEC;
    __shared__ float sums[2][LANES / 64][2];
    __shared__ float joined[ROWS > 1 ? ROWS - 1 : 1][ROWS > 1 ? 2 : 1][ROWS > 1 ? (E + 1) * LANES : 1];
    const uint32_t lane = ROWS > 1 ? threadIdx.x % LANES : threadIdx.x, group = ROWS > 1 ? threadIdx.x / LANES : 0;
    const uint32_t wave = lane / 64, r = blockIdx.y;
    const Rows mine = rows_of(a, r);
    const RowIo<T, LANES, V, STREAM, !ONE> io(a, lane);
    const uint64_t pitch = (uint64_t)a.width * T::ESZ;
    const bool each = a.join == VRC_NORM_EACH, all = a.join == VRC_NORM_SUM;
    const int ranks = each ? 1 : a.n;
    const float inv = a.inv_width, c = a.center ? inv : 0.0f;
    Part<T, V> w, dw, db;
    io.load_weight(a.w, a.wide_weight, w);
#pragma unroll
    for (int e = 0; e < w.E; e++) dw.v[e] = db.v[e] = 0.0f;
    dw.t = db.t = 0.0f;
    uint32_t turn = 0;
    for (uint64_t i = blockIdx.x * (uint64_t)ROWS + group; i < mine.count; i += gridDim.x * (uint64_t)ROWS) {
        Part<T, V> dy;
        auto raw_h = io.load(a.sum[r] + i * pitch);
        const float mean = a.center ? a.mean[r][i] : 0.0f, rstd = a.rstd[r][i];
        if constexpr (ONE) io.widen(io.load(a.src[each ? r : 0] + (mine.first + i) * pitch), dy);
        else fold_all<(V <= 2 ? 4 : 2)>(io, [&](int q) { return a.src[each ? r : q] + (mine.first + i) * pitch; }, ranks, dy);
        // x of vector j: computed twice from h, whose 16-bit values take half the registers.  Rows without vectors
        // have zeros there, whose (0 - mean) rstd may be infinite, and NaN times dy = 0
        const float scale = ONE || io.vectors ? rstd : 0.0f;
        const auto x_of = [&](int j, float (&x)[T::VEC]) {
            T::unpack(raw_h.v[j], x);
#pragma unroll
            for (int e = 0; e < T::VEC; e++) x[e] = (x[e] - mean) * scale;  // of lanes without the vector: times dy = 0
        };
        const float xt = io.has_tail ? (T::widen(raw_h.t) - mean) * rstd : 0.0f;
        float s[2] = {0.0f, 0.0f};
        const auto one = [&](float xe, float de, float we, float& dwe, float& dbe) {
            const float g = de * we;
            s[0] += g;
            s[1] = fmaf(g, xe, s[1]);
            dwe = fmaf(de, xe, dwe);
            dbe += de;
        };
#pragma unroll
        for (int j = 0; j < V; j++) {
            float x[T::VEC];
            x_of(j, x);
#pragma unroll
            for (int q = 0, e = j * T::VEC; q < T::VEC; q++, e++) one(x[q], dy.v[e], w.v[e], dw.v[e], db.v[e]);
        }
        one(xt, dy.t, w.t, dw.t, db.t);
        row_sums<LANES>(s, sums[turn], wave);
        turn ^= 1;
        const float level = s[0] * c, along = s[1] * inv;
        // (the compiler would keep the first x)
#pragma unroll
        for (int j = 0; j < V; j++) __asm__ volatile("" : "+v"(raw_h.v[j]));
        const auto two = [&](float xe, float& de, float we) { de = rstd * (fmaf(de, we, -level) - xe * along); };
#pragma unroll
        for (int j = 0; j < V; j++) {
            float x[T::VEC];
            x_of(j, x);
#pragma unroll
            for (int q = 0, e = j * T::VEC; q < T::VEC; q++, e++) two(x[q], dy.v[e], w.v[e]);
        }
        two(xt, dy.t, w.t);
        if (a.res[r]) {
            const auto raw = io.load(a.res[r] + i * pitch);
#pragma unroll
            for (int j = 0; j < V; j++) {
                float d[T::VEC];
                T::unpack(raw.v[j], d);
#pragma unroll
                for (int e = 0; e < T::VEC; e++) dy.v[j * T::VEC + e] += d[e];
            }
            dy.t += T::widen(raw.t);
        }
        const int d0 = all ? 0 : (int)r, d1 = all ? a.n : d0 + 1;
        for (int q = d0; q < d1; q++) io.store(a.dst[q] + i * pitch, dy);
    }
    if constexpr (ROWS > 1) {
        if (group) {
#pragma unroll
            for (int e = 0; e < (int)E; e++) {
                joined[group - 1][0][e * LANES + lane] = dw.v[e];
                joined[group - 1][1][e * LANES + lane] = db.v[e];
            }
            joined[group - 1][0][E * LANES + lane] = dw.t;
            joined[group - 1][1][E * LANES + lane] = db.t;
        }
        __syncthreads();
        if (group) return;
        for (uint32_t g = 0; g + 1 < ROWS; g++) {
#pragma unroll
            for (int e = 0; e < (int)E; e++) {
                dw.v[e] += joined[g][0][e * LANES + lane];
                db.v[e] += joined[g][1][e * LANES + lane];
            }
            dw.t += joined[g][0][E * LANES + lane];
            db.t += joined[g][1][E * LANES + lane];
        }
    }
    float* const to = a.partial + ((uint64_t)r * gridDim.x + blockIdx.x) * 2 * a.width;
    const auto keep = [&](float* row, const Part<T, V>& p) {
#pragma unroll
        for (int j = 0; j < V; j++) {
            if (!io.has[j]) continue;
#pragma unroll
            for (int q = 0; q < T::VEC / 4; q++)
                st16<false>((char*)(row + io.at[j] / T::ESZ + q * 4), F32::pack(p.v + j * T::VEC + q * 4));
        }
        if (io.has_tail) row[io.tail_at / T::ESZ] = p.t;
    };
    keep(to, dw);
    keep(to + a.width, db);
}

// Column sums of the partial sums: out[k][col] = sum over p of partial[p][k][col],
// k = 0 (dweight), 1 (dbias), in the order of p within each of 32 interleaved runs
// and then of the runs.  Eight loads of a lane are under way at once.
template <class T>
__global__ __launch_bounds__(1024) void k_norm_join(const float* partial, uint32_t count, uint32_t width, char* dw, char* db)
{
    __shared__ float part[32][33];
    const uint32_t c = threadIdx.x % 32, run = threadIdx.x / 32, col = blockIdx.x * 32 + c, k = blockIdx.y;
    float s = 0.0f;
    if (col < width) {
        const float* from = partial + (uint64_t)k * width + col;
        const uint64_t pitch = 2 * (uint64_t)width;
        uint32_t p = run;
        for (; p + 7 * 32 < count; p += 8 * 32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = from[(p + i * 32) * pitch];
            issue_loads_first();
#pragma unroll
            for (int i = 0; i < 8; i++) s += v[i];
        }
        for (; p < count; p += 32) s += from[p * pitch];
    }
    part[run][c] = s;
    __syncthreads();
    if (run || col >= width) return;
    for (int q = 1; q < 32; q++) s += part[q][c];
    store_s<T>((k ? db : dw) + (uint64_t)col * T::ESZ, T::narrow(s));
}

// ---------------------------------------------------------------------------
// Rows of more values than a workgroup's registers hold: 1024 lanes walk the row
// element by element, and read its sources again for each pass over it (from the
// caches, mostly).
// ---------------------------------------------------------------------------
template <class T>
struct WideRow {
    const NormArgs& a;
    uint32_t r;
    uint64_t src, own;  // byte offsets of the row in the sources and in what is one per part
    int ranks;
    bool each;
    __device__ __forceinline__ float value(uint32_t col, bool with_res) const
    {
        float s = -0.0f;
        for (int q = 0; q < ranks; q++) s += T::widen(load_s<T>(a.src[each ? r : q] + src + (uint64_t)col * T::ESZ));
        if (with_res) s += T::widen(load_s<T>(a.res[r] + own + (uint64_t)col * T::ESZ));
        return s;
    }
    __device__ __forceinline__ float weight(const char* w, uint32_t col) const
    {
        return a.wide_weight ? F32::widen(load_s<F32>(w + (uint64_t)col * 4)) : T::widen(load_s<T>(w + (uint64_t)col * T::ESZ));
    }
};

template <class T>
__global__ __launch_bounds__(1024) void k_layer_norm_wide(NormArgs a)
{
    __shared__ float sums[2][16][1];
    const uint32_t tid = threadIdx.x, wave = tid / 64, r = blockIdx.y;
    const Rows mine = rows_of(a, r);
    const uint64_t pitch = (uint64_t)a.width * T::ESZ;
    const bool each = a.join == VRC_NORM_EACH, all = a.join == VRC_NORM_SUM, res = a.res[r] != nullptr;
    for (uint64_t i = blockIdx.x; i < mine.count; i += gridDim.x) {
        const WideRow<T> row = {a, r, (mine.first + i) * pitch, i * pitch, each ? 1 : a.n, each};
        float s[1] = {0.0f};
        for (uint32_t col = tid; col < a.width; col += 1024) s[0] += row.value(col, res);
        row_sums<1024>(s, sums[0], wave);
        const float mean = a.center ? s[0] * a.inv_width : 0.0f;
        s[0] = 0.0f;
        for (uint32_t col = tid; col < a.width; col += 1024) {
            const float d = row.value(col, res) - mean;
            s[0] = fmaf(d, d, s[0]);
        }
        row_sums<1024>(s, sums[1], wave);
        const float rstd = 1.0f / sqrtf(s[0] * a.inv_width + a.eps);
        const int d0 = all ? 0 : (int)r, d1 = all ? a.n : d0 + 1;
        // a lane stores its own elements only, behind its loads of them: in place is safe
        for (uint32_t col = tid; col < a.width; col += 1024) {
            const float x = row.value(col, res);
            const uint64_t at = i * pitch + (uint64_t)col * T::ESZ;
            const typename T::S y = T::narrow(fmaf((x - mean) * rstd, row.weight(a.w, col), a.b ? row.weight(a.b, col) : -0.0f));
            if (a.out[r]) store_s<T>(a.out[r] + at, T::narrow(x));
            for (int q = d0; q < d1; q++) store_s<T>(a.dst[q] + at, y);
        }
        if (tid == 0) {
            if (a.mean[r]) a.mean[r][i] = mean;
            if (a.rstd[r]) a.rstd[r][i] = rstd;
        }
    }
}

template <class T>
__global__ __launch_bounds__(1024) void k_layer_norm_grad_wide(NormArgs a)
{
    __shared__ float sums[2][16][2];
    const uint32_t tid = threadIdx.x, wave = tid / 64, r = blockIdx.y;
    const Rows mine = rows_of(a, r);
    const uint64_t pitch = (uint64_t)a.width * T::ESZ;
    const bool each = a.join == VRC_NORM_EACH, all = a.join == VRC_NORM_SUM;
    const float inv = a.inv_width, c = a.center ? inv : 0.0f;
    float* const to = a.partial + ((uint64_t)r * gridDim.x + blockIdx.x) * 2 * a.width;
    for (uint32_t col = tid; col < a.width; col += 1024) to[col] = to[a.width + col] = 0.0f;
    uint32_t turn = 0;
    for (uint64_t i = blockIdx.x; i < mine.count; i += gridDim.x) {
        const WideRow<T> row = {a, r, (mine.first + i) * pitch, i * pitch, each ? 1 : a.n, each};
        const float mean = a.center ? a.mean[r][i] : 0.0f, rstd = a.rstd[r][i];
        const auto x_of = [&](uint32_t col) {
            return (T::widen(load_s<T>(a.sum[r] + i * pitch + (uint64_t)col * T::ESZ)) - mean) * rstd;
        };
        float s[2] = {0.0f, 0.0f};
        for (uint32_t col = tid; col < a.width; col += 1024) {
            const float dy = row.value(col, false), x = x_of(col), g = dy * row.weight(a.w, col);
            s[0] += g;
            s[1] = fmaf(g, x, s[1]);
            to[col] = fmaf(dy, x, to[col]);
            to[a.width + col] += dy;
        }
        row_sums<1024>(s, sums[turn], wave);
        turn ^= 1;
        const float level = s[0] * c, along = s[1] * inv;
        const int d0 = all ? 0 : (int)r, d1 = all ? a.n : d0 + 1;
        for (uint32_t col = tid; col < a.width; col += 1024) {
            const float dy = row.value(col, false), x = x_of(col);
            const uint64_t at = i * pitch + (uint64_t)col * T::ESZ;
            float d = rstd * (fmaf(dy, row.weight(a.w, col), -level) - x * along);
            if (a.res[r]) d += T::widen(load_s<T>(a.res[r] + at));
            for (int q = d0; q < d1; q++) store_s<T>(a.dst[q] + at, T::narrow(d));
        }
    }
}

using namespace host;

template <class T>
NormArgs args_of(const NormCall& c)
{
    NormArgs a = {};
    for (int r = 0; r < c.n; r++) {
        a.src[r] = c.src[r];
        a.dst[r] = c.dst[r];
    }
    for (int p = 0; p < c.parts; p++) {
        a.res[p] = c.res[p];
        a.sum[p] = c.sum[p];
        a.out[p] = c.out[p];
        a.mean[p] = c.mean[p];
        a.rstd[p] = c.rstd[p];
    }
    a.w = c.weight;
    a.b = c.bias;
    a.rows = c.rows;
    a.width = (uint32_t)c.width;
    a.vectors = a.width / T::VEC;
    a.tail = a.width % T::VEC;
    a.eps = (float)c.eps;
    a.inv_width = (float)(1.0 / (double)c.width);
    a.n = c.n;
    a.join = c.join;
    a.center = c.center;
    a.wide_weight = c.wide_weight;
    return a;
}

// The most rows that a rank works on.
uint64_t most_rows(const NormCall& c)
{
    if (c.join != VRC_NORM_SCATTER) return c.rows;
    return c.rows - (c.rows / (uint64_t)c.n) * (uint64_t)(c.n - 1);
}

// Vectors of a row, its last elements counted as one more.
template <class T>
uint64_t row_vectors(uint64_t width) { return (width + T::VEC - 1) / T::VEC; }

// Rows that are read and written once and do not stay in the last-level cache (256 MiB)
// in any case pass by it: 8 x [8192, 4096] bf16, summed, 235 -> 223 us, the gradient of 8 x
// [2048, 8192] 242 -> 234 us; smaller ones stay where their next reader finds them.
bool streams(const NormCall& c, int esz) { return c.rows * c.width * (uint64_t)(c.n * esz) >= 256u << 20; }

template <class T, int LANES, int V>
vrc_status_t launch_norm(const NormArgs& a, uint64_t rows, int parts, bool stream, hipStream_t st)
{
    constexpr uint64_t ROWS = block_of(LANES) / LANES;
    const uint64_t blocks = (rows + ROWS - 1) / ROWS, most = 1u << 20;
    const dim3 grid((unsigned)(blocks < most ? blocks : most), parts);
    if (stream) k_layer_norm<T, LANES, V, true><<<grid, block_of(LANES), 0, st>>>(a);
    else k_layer_norm<T, LANES, V, false><<<grid, block_of(LANES), 0, st>>>(a);
    return check_launch();
}

template <class T>
vrc_status_t norm_typed(const NormCall& c, hipStream_t st)
{
    const NormArgs a = args_of<T>(c);
    const uint64_t v = row_vectors<T>(c.width), rows = most_rows(c);
    // Few rows have four times as many lanes each (256 in place of 64, 1024 in place of 256).  4 ranks' bf16 rows summed with a residual, us with those and with the others: width 1000, 16 rows 4.4
    // and 4.9, 512 5.8 and 6.4, 2,048 12.1 and 10.0; 2048, 16 rows 4.4 and 6.1, 512 7.3 and 8.9, 2,048 17.1 and 15.8;
    // 8192, 16 rows 5.7 and 6.5, 256 10.3 and 11.1, 384 15.6 and 12.8.  One limit for every width is a compromise:
    // rows of 257 to 512 vectors gain nothing (4096, 16 rows 5.5 and 5.1, 256 8.2 and 8.3, 384 12.3 and 9.2).
    const bool few = rows * (uint64_t)c.parts < 512;
#define VRC_NORM(LANES, V) return launch_norm<T, LANES, V>(a, rows, c.parts, streams(c, T::ESZ), st)
    if (v <= 64) VRC_NORM(64, 1);
    if (!few) {
        if (v <= 128) VRC_NORM(64, 2);
        if (v <= 256) VRC_NORM(64, 4);
    }
    if (v <= 256) VRC_NORM(256, 1);
    if (!few) {
        if (v <= 512) VRC_NORM(256, 2);
        if (v <= 1024) VRC_NORM(256, 4);
    }
    if (v <= 1024) VRC_NORM(1024, 1);
    if (v <= 2048) VRC_NORM(1024, 2);
    if constexpr (T::VEC == 4)
        if (v <= 4096) VRC_NORM(1024, 4);
#undef VRC_NORM
    k_layer_norm_wide<T><<<dim3((unsigned)(rows < (1u << 20) ? rows : 1u << 20), c.parts), 1024, 0, st>>>(a);
    return check_launch();
}

// Workgroups that walk the rows of the gradient, for each part.
uint64_t grad_groups(const NormCall& c)
{
    const uint64_t rows = most_rows(c), most = kNormPartials / (uint64_t)c.parts;
    // up to twice as many rows: two for every one, and fewer partial sums
    return rows <= most ? rows : rows <= 2 * most ? (rows + 1) / 2 : most;
}

template <class T, int LANES, int V>
vrc_status_t launch_norm_grad(const NormArgs& a, unsigned groups, int parts, bool stream, hipStream_t st)
{
    const dim3 grid(groups, parts);
    const bool one = (a.join == VRC_NORM_EACH || a.n == 1) && a.tail == 0;
    if (one && stream) k_layer_norm_grad<T, LANES, V, true, true><<<grid, block_of(LANES), 0, st>>>(a);
    else if (one) k_layer_norm_grad<T, LANES, V, false, true><<<grid, block_of(LANES), 0, st>>>(a);
    else if (stream) k_layer_norm_grad<T, LANES, V, true, false><<<grid, block_of(LANES), 0, st>>>(a);
    else k_layer_norm_grad<T, LANES, V, false, false><<<grid, block_of(LANES), 0, st>>>(a);
    return check_launch();
}

template <class T>
vrc_status_t norm_grad_rows(const NormCall& c, const NormArgs& a, unsigned groups, hipStream_t st)
{
    const uint64_t v = row_vectors<T>(c.width);
#define VRC_NORM(LANES, V) return launch_norm_grad<T, LANES, V>(a, groups, c.parts, streams(c, T::ESZ), st)
    if (v <= 64) VRC_NORM(64, 1);
    if (v <= 128) VRC_NORM(64, 2);  // 4 x [2056, 1000] fp16, summed, 14.6 us; 17.5 with 256 lanes a row
    if (v <= 256) VRC_NORM(256, 1);
    if (v <= 512) VRC_NORM(256, 2);
    if (v <= 1024) VRC_NORM(512, 2);
    if (v <= 2048) VRC_NORM(512, 4);
#undef VRC_NORM
    k_layer_norm_grad_wide<T><<<dim3(groups, c.parts), 1024, 0, st>>>(a);
    return check_launch();
}

template <class T>
vrc_status_t norm_grad_typed(const NormCall& c, hipStream_t st)
{
    NormArgs a = args_of<T>(c);
    a.partial = c.partial;
    const unsigned groups = (unsigned)grad_groups(c);
    if (groups) {
        const vrc_status_t rc = norm_grad_rows<T>(c, a, groups, st);
        if (rc) return rc;
    }
    const dim3 grid((unsigned)((c.width + 31) / 32), c.dbias ? 2 : 1);
    const uint32_t count = groups * (unsigned)c.parts;
    if (c.wide_weight) k_norm_join<F32><<<grid, 1024, 0, st>>>(c.partial, count, a.width, c.dweight, c.dbias);
    else k_norm_join<T><<<grid, 1024, 0, st>>>(c.partial, count, a.width, c.dweight, c.dbias);
    return check_launch();
}

}  // namespace

namespace host {

uint64_t norm_grad_workspace(const NormCall& c) { return grad_groups(c) * (uint64_t)c.parts * 2 * c.width * sizeof(float); }

vrc_status_t run_layer_norm(const NormCall& c, vrc_dtype_t dt, hipStream_t st)
{
    switch (dt) {
    case VRC_FP32: return norm_typed<F32>(c, st);
    case VRC_FP16: return norm_typed<F16>(c, st);
    case VRC_BF16: return norm_typed<BF16>(c, st);
    default: return VRC_ERR_UNSUPPORTED;
    }
}

vrc_status_t run_layer_norm_grad(const NormCall& c, vrc_dtype_t dt, hipStream_t st)
{
    switch (dt) {
    case VRC_FP32: return norm_grad_typed<F32>(c, st);
    case VRC_FP16: return norm_grad_typed<F16>(c, st);
    case VRC_BF16: return norm_grad_typed<BF16>(c, st);
    default: return VRC_ERR_UNSUPPORTED;
    }
}

}  // namespace host
}  // namespace vrc
