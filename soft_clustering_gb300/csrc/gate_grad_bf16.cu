// gate_grad_bf16.cu - the gradient kernels (gate_grad.cuh) for this type.
#include "gate_grad.cuh"

namespace gmm {
namespace gate {
bool launch_grad_bf16(const GradArgs& a, cudaStream_t s) { return grad_impl::launch_grad<__nv_bfloat16>(a, s); }
}  // namespace gate
}  // namespace gmm
