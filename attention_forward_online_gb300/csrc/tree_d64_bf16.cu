// Tree attention at d = 64 in bf16, compiled on its own so that the
// variants build in parallel.
#include "tree_tcgen05.cuh"

namespace osattn {
namespace tree {
template cudaError_t prepare<64, false>();
template cudaError_t launch<64, false>(const TreeArgs&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&);
}  // namespace tree
}  // namespace osattn
