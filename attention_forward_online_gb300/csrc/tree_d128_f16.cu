// Tree attention at d = 128 in fp16, compiled on its own so that the
// variants build in parallel.
#include "tree_tcgen05.cuh"

namespace osattn {
namespace tree {
template cudaError_t prepare<128, true>();
template cudaError_t launch<128, true>(const TreeArgs&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&);
}  // namespace tree
}  // namespace osattn
