// The row kernel of a window with first keys that stay visible.
#include "attn_rows.cuh"

namespace gdn {
template cudaError_t launch_attn_rows_part<SINKS>(const PagedArgs &, const CUtensorMap &, const CUtensorMap &, bool, int, int, int, cudaStream_t);
}  // namespace gdn
