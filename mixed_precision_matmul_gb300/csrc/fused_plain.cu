// The gradients' products of the gated layer and the vocabulary.
#include "fused_gemm.cuh"

namespace mpg {

void fused_lookup_plain(bool pair, FusedKernel* out) {
  *out = pair ? fused_describe<FusedTraits<FusedEpi::kPlain, true>>() : fused_describe<FusedTraits<FusedEpi::kPlain, false>>();
}

}  // namespace mpg
