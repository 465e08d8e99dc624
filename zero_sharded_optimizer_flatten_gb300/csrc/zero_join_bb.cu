// The block join's row kernels: activations __nv_bfloat16, residual stream __nv_bfloat16.
#include "zero_join_rows.cuh"

namespace zero {
template int launch_join_rows<__nv_bfloat16, __nv_bfloat16>(const JoinArgs&, bool, int*, cudaStream_t);
}  // namespace zero
