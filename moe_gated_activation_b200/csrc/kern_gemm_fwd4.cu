// The grouped product's fwd4 kernels (see grouped_gemm_kernel.cuh).
#include "../../include/moeact.h"
#include "grouped_gemm_kernel.cuh"

MOEACT_DEFINE_GEMM_UNIT(fwd4, moeact::kGemmFwd4)
