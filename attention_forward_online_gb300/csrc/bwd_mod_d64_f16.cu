// The modified-score backward at d = 64 in fp16, compiled on its own so
// that the variants build in parallel.
#include "bwd_mod_tcgen05.cuh"

namespace osattn {
namespace bwdmod {
template cudaError_t prepare<64, true>();
template cudaError_t launch<64, true>(const ModArgs&, const BwdModMaps&);
}  // namespace bwdmod
}  // namespace osattn
