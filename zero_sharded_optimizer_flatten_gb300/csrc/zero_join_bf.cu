// The block join's row kernels: activations __nv_bfloat16, residual stream float.
#include "zero_join_rows.cuh"

namespace zero {
template int launch_join_rows<__nv_bfloat16, float>(const JoinArgs&, bool, int*, cudaStream_t);
}  // namespace zero
