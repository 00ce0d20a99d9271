// The gated product, a kernel for each
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

void fused_lookup_gated(bool pair, int act, FusedKernel* out) {
  *out = pair ? of_act<FusedEpi::kGated, true>(act) : of_act<FusedEpi::kGated, false>(act);
}

}  // namespace mpg
