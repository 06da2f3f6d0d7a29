// Instantiations of the CTA-pair (cta_group::2) kernel with the general epilogue and
// low-rank adapters appended to every tile.
#include "launch_impl.cuh"

namespace gb300 {

cudaError_t launch_cg2_adapt(const LaunchSpec& s) {
  if (s.bn == 256 && s.stages == 6)
    return by_out<2, 256, 6, false, false, 0, false, false, false, false, false, true>(s);
  return cudaErrorInvalidValue;
}

}  // namespace gb300
