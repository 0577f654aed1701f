// vrc_model_host.hpp -- the internal entry points of include/vrc_model.h's
// operators, on checked arguments.  Internal.
#pragma once

#include "vrc_model.h"
#include "vrc_elem.hpp"
#include "vrc_ops_host.hpp"

namespace vrc {
namespace host {

// Workgroups that walk the rows of a layer norm's gradient, each with partial sums
// of its own: two for each CU of the card.
constexpr uint64_t kNormPartials = 512;

struct NormCall {
    const char* src[kMaxRanks];
    const char* res[kMaxRanks];  // by part from here on; null where there is none
    const char* sum[kMaxRanks];
    char* out[kMaxRanks];
    float* mean[kMaxRanks];
    float* rstd[kMaxRanks];
    char* dst[kMaxRanks];
    const char* weight;
    const char* bias;
    char* dweight;
    char* dbias;
    float* partial;
    uint64_t rows, width;
    double eps;
    int n, parts, join, center, wide_weight;
};

uint64_t norm_grad_workspace(const NormCall& c);
vrc_status_t run_layer_norm(const NormCall& c, vrc_dtype_t dt, hipStream_t st);
vrc_status_t run_layer_norm_grad(const NormCall& c, vrc_dtype_t dt, hipStream_t st);

struct EntropyCall {
    const char* hidden;
    const char* weight[kMaxRanks];
    uint64_t vocab[kMaxRanks];
    const long long* target;
    float* loss;
    float* lse;            // the gradient's: read only
    const float* dloss;
    const float* dlse;     // or null
    char* dhidden;         // or null
    char* dweight[kMaxRanks];
    bool want_dhidden, want_dweight;
    uint64_t tokens, width;
    long long ignore_index;
    int n;
    char* workspace;
};

// By element type, each in a unit of its own.
template <class T>
uint64_t entropy_bytes(const EntropyCall& c, bool gradient);
template <class T>
vrc_status_t entropy_loss(const EntropyCall& c, hipStream_t st);
template <class T>
vrc_status_t entropy_grad(const EntropyCall& c, hipStream_t st);

}  // namespace host
}  // namespace vrc
