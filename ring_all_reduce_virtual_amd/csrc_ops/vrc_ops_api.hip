// vrc_ops_api.hip -- the C ABI of include/vrc_ops.h: argument checks, buffer
// sizes and overlaps.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

// The C ABI keeps default visibility; everything else in the library is hidden.
#pragma GCC visibility push(default)
#include "vrc_ops.h"
#pragma GCC visibility pop

#include "vrc_ops_host.hpp"

namespace vrc {
namespace host {
thread_local int g_last_hip_error = 0;
thread_local Plan* g_plan = nullptr;  // vrc_launch.hpp's launches look for one; this library records no plans
}  // namespace host
}  // namespace vrc

namespace {

using namespace vrc::host;
using vrc::kMaxRanks;

// Every pointer of an array of n, none null.
bool pointers(const void* const* p, int n, const char** out)
{
    if (!p) return false;
    for (int r = 0; r < n; r++) {
        if (!p[r]) return false;
        out[r] = static_cast<const char*>(p[r]);
    }
    return true;
}

bool pointers(void* const* p, int n, char** out)
{
    if (!p) return false;
    for (int r = 0; r < n; r++) {
        if (!p[r]) return false;
        out[r] = static_cast<char*>(p[r]);
    }
    return true;
}

vrc_status_t check_dropout(const vrc_dropout_t* d, MaskArgs* m)
{
    if (!d || !(d->p >= 0.0 && d->p <= 1.0)) return VRC_ERR_INVALID_ARG;
    if ((uintptr_t)d->offset_dev % 8 != 0) return VRC_ERR_INVALID_ARG;
    const double thr = std::nearbyint(d->p * 4294967296.0);  // 2^32 at most
    m->seed = d->seed;
    m->offset = d->offset;
    m->offset_dev = reinterpret_cast<const uint64_t*>(d->offset_dev);
    m->kind = thr <= 0.0 ? 0 : thr >= 4294967296.0 ? 2 : 1;
    m->thr = m->kind == 1 ? (uint32_t)thr : 0;
    m->scale = m->kind == 2 ? 0.0f : (float)(1.0 / (1.0 - d->p));
    return VRC_OK;
}

// Ranks, size and type of a call; the size 0 case is left to the caller.
vrc_status_t check_call(int nranks, uint64_t count, int dtype)
{
    if (nranks < 1 || nranks > kMaxRanks || count > kMaxCount) return VRC_ERR_INVALID_ARG;
    if (!dtype_valid(dtype) || !float_dtype(dtype)) return VRC_ERR_UNSUPPORTED;
    return VRC_OK;
}

int bufs(const char* const* p, int n, uint64_t bytes, Buf* out, int at)
{
    for (int r = 0; r < n; r++) out[at++] = {(uintptr_t)p[r], bytes};
    return at;
}

// The mask's offset in device memory among the inputs: no output may hold it.
int offset_buf(const MaskArgs& m, Buf* in, int at)
{
    in[at] = {(uintptr_t)m.offset_dev, m.offset_dev ? sizeof(uint64_t) : 0};
    return at + 1;
}

vrc_status_t allreduce_dropout_impl(const void* const* send, const void* const* residual, void* const* recv, int n,
                                    uint64_t count, int dtype, const vrc_dropout_t* d, hipStream_t st)
{
    vrc_status_t rc = check_call(n, count, dtype);
    if (rc) return rc;
    MaskArgs m;
    rc = check_dropout(d, &m);
    if (rc) return rc;
    if (count == 0) return VRC_OK;
    const char *x[kMaxRanks], *res[kMaxRanks];
    char* y[kMaxRanks];
    if (!pointers(send, n, x) || !pointers(recv, n, y) || (residual && !pointers(residual, n, res)))
        return VRC_ERR_INVALID_ARG;
    const vrc_dtype_t dt = static_cast<vrc_dtype_t>(dtype);
    const uint64_t bytes = count * (uint64_t)esize(dt);
    Buf in[2 * kMaxRanks + 1], out[kMaxRanks];
    int ni = bufs(x, n, bytes, in, 0);
    if (residual) ni = bufs(res, n, bytes, in, ni);
    const int operands = ni;
    ni = offset_buf(m, in, ni);
    bufs(y, n, bytes, out, 0);
    rc = check_outputs(out, n, in, ni, [n, operands](int i, int j) { return j < operands && i == j % n; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    return run_allreduce_dropout(x, residual ? res : nullptr, y, n, count, dt, m, cus, st);
}

// The split of a tensor of `total` elements: chunk c's bytes.
vrc_status_t check_split(int n, uint64_t total, uint64_t outer, int esz, uint64_t* bytes)
{
    if (outer == 0 || total % outer != 0) return VRC_ERR_INVALID_ARG;
    if (outer > 1 && (total / outer) % (uint64_t)n != 0) return VRC_ERR_INVALID_ARG;
    for (int c = 0; c < n; c++) {
        uint64_t off = 0, len = total / (uint64_t)n;
        if (outer == 1) chunk_range(total, n, c, &off, &len);
        bytes[c] = len * (uint64_t)esz;
    }
    return VRC_OK;
}

// As pointers(), but the empty chunks of a flat split may be null.
template <class P, class Q>
bool chunk_pointers(P const* p, int n, const uint64_t* bytes, Q* out)
{
    if (!p) return false;
    for (int c = 0; c < n; c++) {
        if (bytes[c] && !p[c]) return false;
        out[c] = static_cast<Q>(p[c]);
    }
    return true;
}

vrc_status_t reduce_scatter_dropout_impl(const void* const* send, const void* const* residual, void* const* recv, int n,
                                         uint64_t count, uint64_t outer, int dtype, const vrc_dropout_t* d,
                                         hipStream_t st)
{
    vrc_status_t rc = check_call(n, count, dtype);
    if (rc) return rc;
    MaskArgs m;
    rc = check_dropout(d, &m);
    if (rc) return rc;
    const vrc_dtype_t dt = static_cast<vrc_dtype_t>(dtype);
    uint64_t cb[kMaxRanks];
    rc = check_split(n, count, outer, esize(dt), cb);
    if (rc) return rc;
    if (count == 0) return VRC_OK;
    const char *x[kMaxRanks], *res[kMaxRanks];
    char* y[kMaxRanks];
    if (!pointers(send, n, x) || !chunk_pointers(recv, n, cb, y) || (residual && !chunk_pointers(residual, n, cb, res)))
        return VRC_ERR_INVALID_ARG;
    Buf in[2 * kMaxRanks + 1], out[kMaxRanks];
    int ni = bufs(x, n, count * (uint64_t)esize(dt), in, 0);
    for (int c = 0; c < n; c++) {
        if (residual) in[ni++] = {(uintptr_t)res[c], cb[c]};
        out[c] = {(uintptr_t)y[c], cb[c]};
    }
    const int operands = ni;
    ni = offset_buf(m, in, ni);
    rc = check_outputs(out, n, in, ni, [n, operands](int i, int j) { return j < operands && j == n + i; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    return run_reduce_scatter_dropout(x, residual ? res : nullptr, y, n, count, outer, dt, m, cus, st);
}

vrc_status_t all_gather_dropout_impl(const void* const* send, void* const* recv, int n, uint64_t total, uint64_t outer,
                                     int dtype, const vrc_dropout_t* d, hipStream_t st)
{
    vrc_status_t rc = check_call(n, total, dtype);
    if (rc) return rc;
    MaskArgs m;
    rc = check_dropout(d, &m);
    if (rc) return rc;
    const vrc_dtype_t dt = static_cast<vrc_dtype_t>(dtype);
    uint64_t cb[kMaxRanks];
    rc = check_split(n, total, outer, esize(dt), cb);
    if (rc) return rc;
    if (total == 0) return VRC_OK;
    const char* x[kMaxRanks];
    char* y[kMaxRanks];
    if (!chunk_pointers(send, n, cb, x) || !pointers(recv, n, y)) return VRC_ERR_INVALID_ARG;
    Buf in[kMaxRanks + 1], out[kMaxRanks];
    for (int c = 0; c < n; c++) in[c] = {(uintptr_t)x[c], cb[c]};
    const int ni = offset_buf(m, in, n);
    bufs(y, n, total * (uint64_t)esize(dt), out, 0);
    rc = check_outputs(out, n, in, ni, [](int, int) { return false; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    return run_all_gather_dropout(x, y, n, total, outer, dt, m, cus, st);
}

// A matrix's [rows, cols] elements and its blocks, both at most kMaxCount
// bytes' worth, without wrapping.
bool mx4_sizes(uint64_t rows, uint64_t cols, uint64_t* blocks)
{
    if (rows > kMaxCount || cols > kMaxCount) return false;
    const unsigned __int128 v = (unsigned __int128)rows * ((cols + 31) / 32) * 32;
    if (v > kMaxCount) return false;
    *blocks = (uint64_t)(v / 32);
    return true;
}

bool aligned16(const char* const* p, int n)
{
    for (int r = 0; r < n; r++)
        if ((uintptr_t)p[r] % 16 != 0) return false;
    return true;
}

vrc_status_t mx4_quantize_impl(const void* const* x_, void* const* codes_, void* const* scales_, int n, uint64_t rows,
                               uint64_t cols, int dtype, int axis, hipStream_t st)
{
    vrc_status_t rc = check_call(n, 0, dtype);
    if (rc) return rc;
    if (axis != VRC_MX4_ALONG_COLS && axis != VRC_MX4_ALONG_ROWS) return VRC_ERR_UNSUPPORTED;
    const bool along_rows = axis == VRC_MX4_ALONG_ROWS;
    uint64_t blocks;
    if (!mx4_sizes(along_rows ? cols : rows, along_rows ? rows : cols, &blocks)) return VRC_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return VRC_OK;
    const char* x[kMaxRanks];
    char *codes[kMaxRanks], *scales[kMaxRanks];
    if (!pointers(x_, n, x) || !pointers(codes_, n, codes) || !pointers(scales_, n, scales)) return VRC_ERR_INVALID_ARG;
    if (!aligned16(codes, n)) return VRC_ERR_INVALID_ARG;
    const vrc_dtype_t dt = static_cast<vrc_dtype_t>(dtype);
    Buf in[kMaxRanks], out[2 * kMaxRanks];
    bufs(x, n, rows * cols * (uint64_t)esize(dt), in, 0);
    bufs(codes, n, blocks * 16, out, 0);
    bufs(scales, n, blocks, out, n);
    rc = check_outputs(out, 2 * n, in, n, [](int, int) { return false; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    return run_mx4_quantize(x, codes, scales, n, rows, cols, dt, along_rows, cus, st);
}

// gather: every rank's matrix goes to every output, along the columns if by_cols; else
// each to its own.
vrc_status_t mx4_decode_impl(const void* const* codes_, const void* const* scales_, void* const* recv, int n, bool gather,
                             uint64_t rows, uint64_t cols, bool by_cols, int dtype, hipStream_t st)
{
    vrc_status_t rc = check_call(n, 0, dtype);
    if (rc) return rc;
    uint64_t blocks;
    if (!mx4_sizes(rows, cols, &blocks)) return VRC_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return VRC_OK;
    const char *codes[kMaxRanks], *scales[kMaxRanks];
    char* y[kMaxRanks];
    if (!pointers(codes_, n, codes) || !pointers(scales_, n, scales) || !pointers(recv, n, y)) return VRC_ERR_INVALID_ARG;
    if (!aligned16(codes, n)) return VRC_ERR_INVALID_ARG;
    const vrc_dtype_t dt = static_cast<vrc_dtype_t>(dtype);
    Buf in[2 * kMaxRanks], out[kMaxRanks];
    bufs(codes, n, blocks * 16, in, 0);
    bufs(scales, n, blocks, in, n);
    bufs(y, n, rows * cols * (uint64_t)(gather ? n : 1) * (uint64_t)esize(dt), out, 0);
    rc = check_outputs(out, n, in, 2 * n, [](int, int) { return false; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    const uint64_t slab = !gather ? 0 : by_cols ? cols : rows * cols;
    const uint64_t stride = gather && by_cols ? cols * (uint64_t)n : cols;
    return run_mx4_decode(codes, scales, y, n, gather ? n : 0, rows, cols, slab, stride, dt, cus, st);
}

vrc_status_t mx4_matmul_impl(const void* const* ac_, const void* const* as_, const void* const* bc_,
                             const void* const* bs_, void* const* recv, int n, uint64_t m, uint64_t cols,
                             uint64_t kblocks, int dtype, int join, hipStream_t st)
{
    vrc_status_t rc = check_call(n, 0, dtype);
    if (rc) return rc;
    if (join != VRC_MX4_SUM && join != VRC_MX4_EACH) return VRC_ERR_UNSUPPORTED;
    if (m >= 1ull << 31 || cols >= 1ull << 31 || kblocks >= 1ull << 20 || m * cols > kMaxCount) return VRC_ERR_INVALID_ARG;
    if (m == 0 || cols == 0) return VRC_OK;
    const char *ac[kMaxRanks] = {}, *as[kMaxRanks] = {}, *bc[kMaxRanks] = {}, *bs[kMaxRanks] = {};
    char* y[kMaxRanks];
    if (!pointers(recv, n, y)) return VRC_ERR_INVALID_ARG;
    if (kblocks && (!pointers(ac_, n, ac) || !pointers(as_, n, as) || !pointers(bc_, n, bc) || !pointers(bs_, n, bs)))
        return VRC_ERR_INVALID_ARG;
    if (!aligned16(ac, n) || !aligned16(bc, n)) return VRC_ERR_INVALID_ARG;
    const vrc_dtype_t dt = static_cast<vrc_dtype_t>(dtype);
    Buf in[4 * kMaxRanks], out[kMaxRanks];
    bufs(ac, n, m * kblocks * 16, in, 0);
    bufs(as, n, m * kblocks, in, n);
    bufs(bc, n, cols * kblocks * 16, in, 2 * n);
    bufs(bs, n, cols * kblocks, in, 3 * n);
    bufs(y, n, m * cols * (uint64_t)esize(dt), out, 0);
    rc = check_outputs(out, n, in, 4 * n, [](int, int) { return false; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    return run_mx4_matmul(ac, as, bc, bs, y, n, m, cols, kblocks, dt, join == VRC_MX4_SUM, cus, st);
}

}  // namespace

extern "C" {

vrc_status_t vrc_allreduce_dropout(const void* const* send, const void* const* residual, void* const* recv,
                                   int nranks, size_t count, vrc_dtype_t dtype, const vrc_dropout_t* dropout,
                                   vrc_stream_t stream)
{
    return allreduce_dropout_impl(send, residual, recv, nranks, count, raw(dtype), dropout, (hipStream_t)stream);
}

vrc_status_t vrc_reduce_scatter_dropout(const void* const* send, const void* const* residual, void* const* recv,
                                        int nranks, size_t count, size_t outer, vrc_dtype_t dtype,
                                        const vrc_dropout_t* dropout, vrc_stream_t stream)
{
    return reduce_scatter_dropout_impl(send, residual, recv, nranks, count, outer, raw(dtype), dropout,
                                       (hipStream_t)stream);
}

vrc_status_t vrc_all_gather_dropout(const void* const* send, void* const* recv, int nranks, size_t total,
                                    size_t outer, vrc_dtype_t dtype, const vrc_dropout_t* dropout,
                                    vrc_stream_t stream)
{
    return all_gather_dropout_impl(send, recv, nranks, total, outer, raw(dtype), dropout, (hipStream_t)stream);
}

vrc_status_t vrc_mx4_quantize(const void* const* x, void* const* codes, void* const* scales, int nranks, size_t rows,
                              size_t cols, vrc_dtype_t dtype, vrc_mx4_axis_t axis, vrc_stream_t stream)
{
    return mx4_quantize_impl(x, codes, scales, nranks, rows, cols, raw(dtype), raw(axis), (hipStream_t)stream);
}

vrc_status_t vrc_mx4_dequantize(const void* const* codes, const void* const* scales, void* const* recv, int nranks,
                                size_t rows, size_t cols, vrc_dtype_t dtype, vrc_stream_t stream)
{
    return mx4_decode_impl(codes, scales, recv, nranks, false, rows, cols, false, raw(dtype), (hipStream_t)stream);
}

vrc_status_t vrc_mx4_all_gather(const void* const* codes, const void* const* scales, void* const* recv, int nranks,
                                size_t rows, size_t cols, int by_cols, vrc_dtype_t dtype, vrc_stream_t stream)
{
    return mx4_decode_impl(codes, scales, recv, nranks, true, rows, cols, by_cols != 0, raw(dtype),
                           (hipStream_t)stream);
}

vrc_status_t vrc_mx4_matmul(const void* const* a_codes, const void* const* a_scales, const void* const* b_codes,
                            const void* const* b_scales, void* const* recv, int nranks, size_t m, size_t n,
                            size_t kblocks, vrc_dtype_t dtype, vrc_mx4_join_t join, vrc_stream_t stream)
{
    return mx4_matmul_impl(a_codes, a_scales, b_codes, b_scales, recv, nranks, m, n, kblocks, raw(dtype), raw(join),
                           (hipStream_t)stream);
}

int vrc_ops_last_hip_error(void) { return g_last_hip_error; }

int vrc_ops_version(void) { return VRC_OPS_VERSION; }

}  // extern "C"
