// The gradients of the gated product's projections, computed again: a kernel for each
// activation (three in one are three times the code in every loop).
#include "fused_gemm.cuh"

namespace mpg {
namespace {

template <FusedEpi E, bool kPair>
FusedKernel of_act(int act) {
  switch (act) {
    case kActSilu: return fused_describe<FusedTraits<E, kPair, kActSilu>>();
    case kActGelu: return fused_describe<FusedTraits<E, kPair, kActGelu>>();
    default: return fused_describe<FusedTraits<E, kPair, kActGeluTanh>>();
  }
}

}  // namespace

void fused_lookup_gated_grad(bool pair, int act, FusedKernel* out) {
  *out = pair ? of_act<FusedEpi::kGatedGrad, true>(act) : of_act<FusedEpi::kGatedGrad, false>(act);
}

}  // namespace mpg
