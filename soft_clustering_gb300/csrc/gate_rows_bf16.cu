// gate_rows_bf16.cu - the learned gate's kernels (gate_rows.cuh) for this type.
#include "gate_rows.cuh"

namespace gmm {
namespace gate {
GateBlocks launch_gate_bf16(const GateArgs& a, cudaStream_t s) { return rows_impl::launch_gate<__nv_bfloat16>(a, s); }
}  // namespace gate
}  // namespace gmm
