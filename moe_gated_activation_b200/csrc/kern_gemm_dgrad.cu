// The grouped product's dgrad kernels (see grouped_gemm_kernel.cuh).
#include "../../include/moeact.h"
#include "grouped_gemm_kernel.cuh"

MOEACT_DEFINE_GEMM_UNIT(dgrad, moeact::kGemmDgrad)
