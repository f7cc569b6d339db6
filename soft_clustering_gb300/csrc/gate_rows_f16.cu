// gate_rows_f16.cu - the learned gate's kernels (gate_rows.cuh) for this type.
#include "gate_rows.cuh"

namespace gmm {
namespace gate {
GateBlocks launch_gate_f16(const GateArgs& a, cudaStream_t s) { return rows_impl::launch_gate<__half>(a, s); }
}  // namespace gate
}  // namespace gmm
