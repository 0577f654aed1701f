// vrc_model_api.hip -- the C ABI of include/vrc_model.h: argument checks, buffer
// sizes and overlaps.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

// The C ABI keeps default visibility; everything else in the library is hidden.
#pragma GCC visibility push(default)
#include "vrc_model.h"
#pragma GCC visibility pop

#include "vrc_model_host.hpp"

namespace {

using namespace vrc::host;
using vrc::kMaxRanks;

// A list of one call's buffers.
template <int N>
struct Bufs {
    Buf b[N];
    int n = 0;
    void add(const void* p, uint64_t bytes) { b[n++] = {(uintptr_t)p, p ? bytes : 0}; }
};

bool aligned(const void* p, uintptr_t to) { return (uintptr_t)p % to == 0; }

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------

// The description of a call, without its pointers.
vrc_status_t norm_call(const vrc_layer_norm_t* d, int n, NormCall* c, vrc_dtype_t* dt)
{
    *c = {};
    if (!d || n < 1 || n > kMaxRanks) return VRC_ERR_INVALID_ARG;
    const int dtype = raw(d->dtype), wdtype = raw(d->wdtype), join = raw(d->join);
    if (!float_dtype(dtype) || (wdtype != dtype && wdtype != VRC_FP32)) return VRC_ERR_UNSUPPORTED;
    if (join != VRC_NORM_EACH && join != VRC_NORM_SUM && join != VRC_NORM_SCATTER) return VRC_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.0) || std::isinf(d->eps)) return VRC_ERR_INVALID_ARG;
    if (d->width >= 1ull << 26 || d->rows > kMaxCount || (d->width && d->rows > kMaxCount / d->width)) return VRC_ERR_INVALID_ARG;
    c->rows = d->rows;
    c->width = d->width;
    c->eps = d->eps;
    c->n = n;
    c->parts = join == VRC_NORM_SUM ? 1 : n;
    c->join = join;
    c->center = d->center != 0;
    *dt = static_cast<vrc_dtype_t>(dtype);
    c->wide_weight = wdtype == VRC_FP32 && dtype != VRC_FP32;
    return VRC_OK;
}

uint64_t part_rows(const NormCall& c, int p)
{
    if (c.join != VRC_NORM_SCATTER) return c.rows;
    uint64_t off, len;
    vrc::host::chunk_range(c.rows, c.n, p, &off, &len);
    return len;
}

// One array per part, as `X`s of `bytes` a row; those of parts without rows may be null.
template <class P, class Q, int N>
bool part_pointers(P const* p, const NormCall& c, uint64_t row_bytes, Q* out, Bufs<N>* bufs)
{
    for (int i = 0; i < c.parts; i++) {
        const uint64_t rows = part_rows(c, i);
        if (rows && !p[i]) return false;
        out[i] = (Q)p[i];
        bufs->add(p[i], rows * row_bytes);
    }
    return true;
}

vrc_status_t layer_norm_impl(const vrc_layer_norm_t* d, const void* const* send, const void* const* residual,
                             const void* weight, const void* bias, void* const* recv, void* const* sum,
                             float* const* mean, float* const* rstd, int n, hipStream_t st)
{
    NormCall c;
    vrc_dtype_t dt;
    vrc_status_t rc = norm_call(d, n, &c, &dt);
    if (rc) return rc;
    if (mean && !c.center) return VRC_ERR_INVALID_ARG;
    if (c.rows && c.width == 0 && (mean || rstd)) return VRC_ERR_INVALID_ARG;  // of rows without values there are none
    if (c.rows == 0 || c.width == 0) return VRC_OK;
    const uint64_t row = c.width * (uint64_t)esize(dt), wbytes = c.width * (uint64_t)(c.wide_weight ? 4 : esize(dt));
    Bufs<2 * kMaxRanks + 2> in;
    Bufs<4 * kMaxRanks> out;
    if (!send || !recv || !weight) return VRC_ERR_INVALID_ARG;
    for (int r = 0; r < n; r++) {
        const uint64_t rows = c.join == VRC_NORM_SCATTER ? part_rows(c, r) : c.rows;
        if (!send[r] || (rows && !recv[r])) return VRC_ERR_INVALID_ARG;
        c.src[r] = (const char*)send[r];
        c.dst[r] = (char*)recv[r];
        in.add(send[r], c.rows * row);
        out.add(recv[r], rows * row);
    }
    const int at_res = in.n;
    if (residual && !part_pointers(residual, c, row, c.res, &in)) return VRC_ERR_INVALID_ARG;
    const int at_sum = out.n;
    if (sum && !part_pointers(sum, c, row, c.out, &out)) return VRC_ERR_INVALID_ARG;
    if (mean && !part_pointers(mean, c, sizeof(float), c.mean, &out)) return VRC_ERR_INVALID_ARG;
    if (rstd && !part_pointers(rstd, c, sizeof(float), c.rstd, &out)) return VRC_ERR_INVALID_ARG;
    c.weight = (const char*)weight;
    c.bias = (const char*)bias;
    const int operands = in.n;
    in.add(weight, wbytes);
    in.add(bias, wbytes);
    rc = check_outputs(out.b, out.n, in.b, in.n, [&](int i, int j) {
        if (j < at_res) return i == j && i < n && c.join != VRC_NORM_SCATTER;
        return residual && sum && j < operands && i >= at_sum && i - at_sum == j - at_res;
    });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    return run_layer_norm(c, dt, st);
}

vrc_status_t layer_norm_grad_impl(const vrc_layer_norm_t* d, const void* const* send, const void* const* sum,
                                  const float* const* mean, const float* const* rstd, const void* weight,
                                  const void* const* residual, void* const* recv, void* dweight, void* dbias, int n,
                                  void* workspace, size_t workspace_bytes, hipStream_t st)
{
    NormCall c;
    vrc_dtype_t dt;
    vrc_status_t rc = norm_call(d, n, &c, &dt);
    if (rc) return rc;
    if ((mean != nullptr) != (c.center != 0) && c.rows && c.width) return VRC_ERR_INVALID_ARG;
    if (c.width == 0) return VRC_OK;
    const uint64_t row = c.width * (uint64_t)esize(dt), wbytes = c.width * (uint64_t)(c.wide_weight ? 4 : esize(dt));
    Bufs<5 * kMaxRanks + 1> in;
    Bufs<kMaxRanks + 3> out;
    if (!dweight) return VRC_ERR_INVALID_ARG;
    c.dweight = (char*)dweight;
    c.dbias = (char*)dbias;
    int ranks = 0;
    if (c.rows) {
        if (!send || !sum || !rstd || !recv || !weight) return VRC_ERR_INVALID_ARG;
        for (int r = 0; r < n; r++) {
            const uint64_t rows = c.join == VRC_NORM_SCATTER ? part_rows(c, r) : c.rows;
            if (!send[r] || (rows && !recv[r])) return VRC_ERR_INVALID_ARG;
            c.src[r] = (const char*)send[r];
            c.dst[r] = (char*)recv[r];
            in.add(send[r], c.rows * row);
            out.add(recv[r], rows * row);
        }
        ranks = n;
        if (!part_pointers(sum, c, row, c.sum, &in)) return VRC_ERR_INVALID_ARG;
        if (mean && !part_pointers(mean, c, sizeof(float), c.mean, &in)) return VRC_ERR_INVALID_ARG;
        if (!part_pointers(rstd, c, sizeof(float), c.rstd, &in)) return VRC_ERR_INVALID_ARG;
        if (residual && !part_pointers(residual, c, row, c.res, &in)) return VRC_ERR_INVALID_ARG;
        c.weight = (const char*)weight;
        in.add(weight, wbytes);
    }
    const uint64_t need = norm_grad_workspace(c);
    if (workspace_bytes < need || (need && !workspace) || !aligned(workspace, 16)) return VRC_ERR_INVALID_ARG;
    c.partial = (float*)workspace;
    out.add(dweight, wbytes);
    out.add(dbias, wbytes);
    out.add(workspace, need);
    rc = check_outputs(out.b, out.n, in.b, in.n,
                       [&](int i, int j) { return i == j && i < ranks && c.join != VRC_NORM_SCATTER; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    return run_layer_norm_grad(c, dt, st);
}

// ---------------------------------------------------------------------------
// Cross entropy
// ---------------------------------------------------------------------------

// The description of a call with the pointers that decide what it does.
vrc_status_t entropy_call(const vrc_cross_entropy_t* d, const void* hidden, const void* const* weight, int n,
                          EntropyCall* c, vrc_dtype_t* dt)
{
    *c = {};
    if (!d || n < 1 || n > kMaxRanks || !d->vocab) return VRC_ERR_INVALID_ARG;
    const int dtype = raw(d->dtype);
    if (!float_dtype(dtype)) return VRC_ERR_UNSUPPORTED;
    // what grids and 32-bit offsets within a tile hold
    if (d->tokens >= 1ull << 24 || d->width == 0 || d->width >= 1ull << 20) return VRC_ERR_INVALID_ARG;
    uint64_t total = 0;
    for (int r = 0; r < n; r++) {
        if (d->vocab[r] >= 1ull << 23) return VRC_ERR_INVALID_ARG;
        c->vocab[r] = d->vocab[r];
        total += d->vocab[r];
        if (d->vocab[r] && (!weight || !weight[r])) return VRC_ERR_INVALID_ARG;
        c->weight[r] = weight ? (const char*)weight[r] : nullptr;
    }
    if (total >= 1ull << 23 || (d->tokens && !hidden)) return VRC_ERR_INVALID_ARG;
    if (total * d->width >= 1ull << 37 || d->tokens * d->width >= 1ull << 37) return VRC_ERR_INVALID_ARG;
    c->hidden = (const char*)hidden;
    c->tokens = d->tokens;
    c->width = d->width;
    c->ignore_index = d->ignore_index;
    c->n = n;
    *dt = static_cast<vrc_dtype_t>(dtype);
    return VRC_OK;
}

uint64_t workspace_of(const EntropyCall& c, vrc_dtype_t dt, bool gradient)
{
    switch (dt) {
    case VRC_FP16: return entropy_bytes<vrc::F16>(c, gradient);
    case VRC_BF16: return entropy_bytes<vrc::BF16>(c, gradient);
    default: return entropy_bytes<vrc::F32>(c, gradient);
    }
}

vrc_status_t cross_entropy_impl(const vrc_cross_entropy_t* d, const void* hidden, const void* const* weight,
                                const long long* target, float* loss, float* lse, int n, void* workspace,
                                size_t workspace_bytes, hipStream_t st)
{
    EntropyCall c;
    vrc_dtype_t dt;
    vrc_status_t rc = entropy_call(d, hidden, weight, n, &c, &dt);
    if (rc) return rc;
    if (c.tokens == 0) return VRC_OK;
    if (!lse || (loss && !target) || !aligned(target, 8) || !aligned(lse, 4) || !aligned(loss, 4)) return VRC_ERR_INVALID_ARG;
    const uint64_t need = workspace_of(c, dt, false), esz = (uint64_t)esize(dt);
    if (workspace_bytes < need || (need && !workspace) || !aligned(workspace, 16)) return VRC_ERR_INVALID_ARG;
    c.target = target;
    c.loss = loss;
    c.lse = lse;
    c.workspace = (char*)workspace;
    Bufs<kMaxRanks + 2> in;
    Bufs<3> out;
    in.add(hidden, c.tokens * c.width * esz);
    in.add(target, c.tokens * 8);
    for (int r = 0; r < n; r++) in.add(c.weight[r], c.vocab[r] * c.width * esz);
    out.add(loss, c.tokens * 4);
    out.add(lse, c.tokens * 4);
    out.add(workspace, need);
    rc = check_outputs(out.b, out.n, in.b, in.n, [](int, int) { return false; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    switch (dt) {
    case VRC_FP16: return entropy_loss<vrc::F16>(c, st);
    case VRC_BF16: return entropy_loss<vrc::BF16>(c, st);
    default: return entropy_loss<vrc::F32>(c, st);
    }
}

vrc_status_t cross_entropy_grad_impl(const vrc_cross_entropy_t* d, const void* hidden, const void* const* weight,
                                     const long long* target, const float* lse, const float* dloss, const float* dlse,
                                     void* dhidden, void* const* dweight, int n, void* workspace, size_t workspace_bytes,
                                     hipStream_t st)
{
    EntropyCall c;
    vrc_dtype_t dt;
    vrc_status_t rc = entropy_call(d, hidden, weight, n, &c, &dt);
    if (rc) return rc;
    if (!dhidden && !dweight) return VRC_OK;
    const uint64_t esz = (uint64_t)esize(dt);
    Bufs<kMaxRanks + 5> in;
    Bufs<kMaxRanks + 2> out;
    c.want_dhidden = dhidden != nullptr && c.tokens;
    c.want_dweight = dweight != nullptr;
    c.dhidden = (char*)dhidden;
    in.add(hidden, c.tokens * c.width * esz);
    for (int r = 0; r < n; r++) {
        in.add(c.weight[r], c.vocab[r] * c.width * esz);
        if (!dweight) continue;
        if (c.vocab[r] && !dweight[r]) return VRC_ERR_INVALID_ARG;
        c.dweight[r] = (char*)dweight[r];
        out.add(dweight[r], c.vocab[r] * c.width * esz);
    }
    out.add(dhidden, c.tokens * c.width * esz);
    if (c.tokens && (!target || !lse || !dloss)) return VRC_ERR_INVALID_ARG;
    if (!aligned(target, 8) || !aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dlse, 4)) return VRC_ERR_INVALID_ARG;
    in.add(target, c.tokens * 8);
    in.add(lse, c.tokens * 4);
    in.add(dloss, c.tokens * 4);
    in.add(dlse, c.tokens * 4);
    const uint64_t need = workspace_of(c, dt, true);
    if (workspace_bytes < need || (need && !workspace) || !aligned(workspace, 16)) return VRC_ERR_INVALID_ARG;
    out.add(workspace, need);
    c.target = target;
    c.lse = const_cast<float*>(lse);
    c.dloss = dloss;
    c.dlse = dlse;
    c.workspace = (char*)workspace;
    rc = check_outputs(out.b, out.n, in.b, in.n, [](int, int) { return false; });
    if (rc) return rc;
    int cus;
    rc = begin_launch(&cus);
    if (rc) return rc;
    switch (dt) {
    case VRC_FP16: return entropy_grad<vrc::F16>(c, st);
    case VRC_BF16: return entropy_grad<vrc::BF16>(c, st);
    default: return entropy_grad<vrc::F32>(c, st);
    }
}

}  // namespace

extern "C" {

vrc_status_t vrc_layer_norm(const vrc_layer_norm_t* norm, const void* const* send, const void* const* residual,
                            const void* weight, const void* bias, void* const* recv, void* const* sum,
                            float* const* mean, float* const* rstd, int nranks, vrc_stream_t stream)
{
    return layer_norm_impl(norm, send, residual, weight, bias, recv, sum, mean, rstd, nranks, (hipStream_t)stream);
}

vrc_status_t vrc_layer_norm_grad(const vrc_layer_norm_t* norm, const void* const* send, const void* const* sum,
                                 const float* const* mean, const float* const* rstd, const void* weight,
                                 const void* const* residual, void* const* recv, void* dweight, void* dbias, int nranks,
                                 void* workspace, size_t workspace_bytes, vrc_stream_t stream)
{
    return layer_norm_grad_impl(norm, send, sum, mean, rstd, weight, residual, recv, dweight, dbias, nranks, workspace,
                                workspace_bytes, (hipStream_t)stream);
}

vrc_status_t vrc_layer_norm_grad_workspace(const vrc_layer_norm_t* norm, int nranks, size_t* bytes)
{
    NormCall c;
    vrc_dtype_t dt;
    if (!bytes) return VRC_ERR_INVALID_ARG;
    const vrc_status_t rc = norm_call(norm, nranks, &c, &dt);
    if (rc == VRC_OK) *bytes = norm_grad_workspace(c);
    return rc;
}

vrc_status_t vrc_cross_entropy(const vrc_cross_entropy_t* ce, const void* hidden, const void* const* weight,
                               const long long* target, float* loss, float* lse, int nranks, void* workspace,
                               size_t workspace_bytes, vrc_stream_t stream)
{
    return cross_entropy_impl(ce, hidden, weight, target, loss, lse, nranks, workspace, workspace_bytes, (hipStream_t)stream);
}

vrc_status_t vrc_cross_entropy_workspace(const vrc_cross_entropy_t* ce, const void* hidden, const void* const* weight,
                                         int nranks, size_t* bytes)
{
    EntropyCall c;
    vrc_dtype_t dt;
    if (!bytes) return VRC_ERR_INVALID_ARG;
    const vrc_status_t rc = entropy_call(ce, hidden, weight, nranks, &c, &dt);
    if (rc == VRC_OK) *bytes = workspace_of(c, dt, false);
    return rc;
}

vrc_status_t vrc_cross_entropy_grad(const vrc_cross_entropy_t* ce, const void* hidden, const void* const* weight,
                                    const long long* target, const float* lse, const float* dloss, const float* dlse,
                                    void* dhidden, void* const* dweight, int nranks, void* workspace,
                                    size_t workspace_bytes, vrc_stream_t stream)
{
    return cross_entropy_grad_impl(ce, hidden, weight, target, lse, dloss, dlse, dhidden, dweight, nranks, workspace,
                                   workspace_bytes, (hipStream_t)stream);
}

vrc_status_t vrc_cross_entropy_grad_workspace(const vrc_cross_entropy_t* ce, const void* hidden,
                                              const void* const* weight, int dhidden, int nranks, size_t* bytes)
{
    EntropyCall c;
    vrc_dtype_t dt;
    if (!bytes) return VRC_ERR_INVALID_ARG;
    const vrc_status_t rc = entropy_call(ce, hidden, weight, nranks, &c, &dt);
    if (rc) return rc;
    c.want_dhidden = dhidden != 0 && c.tokens;
    c.want_dweight = true;
    *bytes = workspace_of(c, dt, true);
    return VRC_OK;
}

}  // extern "C"
