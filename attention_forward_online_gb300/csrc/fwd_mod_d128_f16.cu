// The modified-score forward at d = 128 in fp16, compiled on its own so
// that the variants build in parallel.
#include "fwd_mod_tcgen05.cuh"

namespace osattn {
namespace fwdmod {
template cudaError_t prepare<128, true>();
template cudaError_t launch<128, true>(const ModArgs&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&, const CUtensorMap&);
}  // namespace fwdmod
}  // namespace osattn
