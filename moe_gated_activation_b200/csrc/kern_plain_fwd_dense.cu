// Instantiates every dense plain MXFP8 quantizer (no activation; see variants.cuh).
#include "variants.cuh"

namespace moeact {
void fill_fwd_plain_dense(FwdVariant* t) { fill_fwd<kPlain, false, false>(t); }
}  // namespace moeact
