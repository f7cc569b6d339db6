// gate_grad_f32.cu - the gradient kernels (gate_grad.cuh) for this type.
#include "gate_grad.cuh"

namespace gmm {
namespace gate {
bool launch_grad_f32(const GradArgs& a, cudaStream_t s) { return grad_impl::launch_grad<float>(a, s); }
}  // namespace gate
}  // namespace gmm
