// vrc_cross_entropy_f32.hip -- the cross entropy's kernels of one element type.
#include "vrc_cross_entropy.hpp"

namespace vrc {
namespace host {

template <>
uint64_t entropy_bytes<F32>(const EntropyCall& c, bool gradient) { return EntropyPlan<F32>(c, gradient).bytes; }
template <>
vrc_status_t entropy_loss<F32>(const EntropyCall& c, hipStream_t st) { return cross_entropy_typed<F32>(c, st); }
template <>
vrc_status_t entropy_grad<F32>(const EntropyCall& c, hipStream_t st) { return cross_entropy_grad_typed<F32>(c, st); }

}  // namespace host
}  // namespace vrc
