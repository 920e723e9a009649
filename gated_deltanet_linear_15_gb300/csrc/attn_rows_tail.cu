// The row kernel of the keys behind a shared prefix.
#include "attn_rows.cuh"

namespace gdn {
template cudaError_t launch_attn_rows_part<TAIL>(const PagedArgs &, const CUtensorMap &, const CUtensorMap &, bool, int, int, int, cudaStream_t);
}  // namespace gdn
