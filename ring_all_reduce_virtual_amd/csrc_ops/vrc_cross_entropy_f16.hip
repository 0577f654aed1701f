// vrc_cross_entropy_f16.hip -- the cross entropy's kernels of one element type.
#include "vrc_cross_entropy.hpp"

namespace vrc {
namespace host {

template <>
uint64_t entropy_bytes<F16>(const EntropyCall& c, bool gradient) { return EntropyPlan<F16>(c, gradient).bytes; }
template <>
vrc_status_t entropy_loss<F16>(const EntropyCall& c, hipStream_t st) { return cross_entropy_typed<F16>(c, st); }
template <>
vrc_status_t entropy_grad<F16>(const EntropyCall& c, hipStream_t st) { return cross_entropy_grad_typed<F16>(c, st); }

}  // namespace host
}  // namespace vrc
