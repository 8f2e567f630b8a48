// Instantiates every grouped plain MXFP8 quantizer (no activation; see variants.cuh).
#include "variants.cuh"

namespace moeact {
void fill_fwd_plain_grouped(FwdVariant* t) { fill_fwd<kPlain, false, true>(t); }
}  // namespace moeact
