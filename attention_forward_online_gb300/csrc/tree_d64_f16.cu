// Tree attention at d = 64 in fp16, compiled on its own so that the
// variants build in parallel.
#include "tree_tcgen05.cuh"

namespace osattn {
namespace tree {
template cudaError_t prepare<64, true>();
template cudaError_t launch<64, true>(const TreeArgs&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&);
}  // namespace tree
}  // namespace osattn
