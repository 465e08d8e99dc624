// The block join's row kernels: activations __half, residual stream __half.
#include "zero_join_rows.cuh"

namespace zero {
template int launch_join_rows<__half, __half>(const JoinArgs&, bool, int*, cudaStream_t);
}  // namespace zero
