// Logits: their statistics, and their gradient.
#include "fused_gemm.cuh"

namespace mpg {

void fused_lookup_loss(FusedEpi epi, bool pair, FusedKernel* out) {
  if (epi == FusedEpi::kStats)
    *out = pair ? fused_describe<FusedTraits<FusedEpi::kStats, true>>() : fused_describe<FusedTraits<FusedEpi::kStats, false>>();
  else
    *out = pair ? fused_describe<FusedTraits<FusedEpi::kProb, true>>() : fused_describe<FusedTraits<FusedEpi::kProb, false>>();
}

}  // namespace mpg
