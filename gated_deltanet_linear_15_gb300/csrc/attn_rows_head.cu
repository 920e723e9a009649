// The row kernel of a shared prefix.
#include "attn_rows.cuh"

namespace gdn {
template cudaError_t launch_attn_rows_part<HEAD>(const PagedArgs &, const CUtensorMap &, const CUtensorMap &, bool, int, int, int, cudaStream_t);
}  // namespace gdn
