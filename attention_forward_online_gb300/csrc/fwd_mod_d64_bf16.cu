// The modified-score forward at d = 64 in bf16, compiled on its own so
// that the variants build in parallel.
#include "fwd_mod_tcgen05.cuh"

namespace osattn {
namespace fwdmod {
template cudaError_t prepare<64, false>();
template cudaError_t launch<64, false>(const ModArgs&, const CUtensorMap&, const CUtensorMap&,
                                    const CUtensorMap&, const CUtensorMap&);
}  // namespace fwdmod
}  // namespace osattn
