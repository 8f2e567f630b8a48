// The grouped block-scaled products (kern_grouped_gemm_*.cu): the host side's
// view (parameters, tensor-map boxes, launchers).
//
// For the rows of each expert e (a group of consecutive rows, any count):
//   forward   out[i, n]  = sum_k A[i, k] W_e[n, k]
//   dgrad     out[i, n]  = sum_k A[i, k] W_e[k, n]      (A the output gradient)
//   wgrad     dW_e[m, n] = sum_i A[i, m] B[i, n]        (i over the expert's rows)
// with A, B and W block-scaled (E8M0 scales of 32 values along the summed
// index; E4M3 codes, or E2M1 codes in the forward).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace moeact {

enum GemmOp : int { kGemmFwd = 0, kGemmDgrad = 1, kGemmWgrad = 2, kGemmFwd4 = 3 };

// The kernels of an operator: 128 x 128 tiles on single SMs; 256 x 256 tiles on SM
// pairs; single SMs with room in tensor memory for the running totals of bf16 sums
// of more than kGemmLongSum steps (and no others).
enum GemmForm : int { kGemmSingle = 0, kGemmPair = 1, kGemmLong = 2 };

struct GroupedGemmParams {
  const int64_t* row_offs;    // [E + 1]
  const int64_t* cb_offs;     // [E + 1], wgrad only: first block row of each group's scales
  int64_t cb_rows;            // wgrad: rows that the scale arrays hold
  int64_t M;                  // rows of all groups
  int E;
  int K;                      // forward, dgrad: length of the summed index (multiple of 32)
  int R;                      // wgrad: rows of dW_e (A's columns)
  int N;                      // output columns
  const uint8_t* a_scales;
  const uint8_t* b_scales;
  int a_tiled, b_tiled;       // scale layouts: 0 row-major, 1 tiles of 128 x 4
  void* out;
  int64_t ldo;                // output row stride in elements
  int out32;                  // 1: fp32, 0: bf16
  int accumulate;             // 1: add to what out holds (fp32)
  int32_t* status;
  const int32_t* noop;        // nullable
  uint32_t* err;              // device error word
};

// Rows of a tensor-map box: 128 (an SM's share of an operand tile), except 32
// where fewer rows may be wanted: the A rows of the one-SM kernels, whose
// groups can be short, and operands stored with the summed index outermost,
// whose last stage can be short.
constexpr int kGemmBoxRows = 128, kGemmShortBoxRows = 32;
// Output: 32 rows of 128 bytes, 128-byte swizzled, of the [M, N] rows or (wgrad)
// of the [E, R, N] gradients.
constexpr int kGemmOutRows = 32, kGemmOutBytes = 128;

// Steps (of 32 products, E2M1 64) of a bf16 output's sum that may go through one
// accumulator, which drops up to 2^-23 of the sum at each: 2^-9 in all, half of
// what the rounding to bf16 may take.
constexpr int kGemmLongSum = 16384;

// Row-major scales: 32 bytes (8 words) of 128 rows (A of the one-SM kernels:
// of 32), or with the blocks outermost 32 rows of 128 columns.
constexpr int kGemmScaleBytes = 32;

struct GemmMaps {
  CUtensorMap a, b;     // code matrices
  CUtensorMap sa, sb;   // scales, where row-major with steps of 16 bytes
  CUtensorMap out;
  CUtensorMap ra, rb;   // wgrad: the code matrices row by row
};

// Sets the kernels' shared-memory limits (once per device).
cudaError_t grouped_gemm_prepare();
cudaError_t grouped_gemm_launch(int op, GemmForm form, const GroupedGemmParams& p,
                                const GemmMaps& tm, int n_sms, cudaStream_t stream);

// One translation unit per operator.
#define MOEACT_GEMM_UNIT(name)                                                              \
  cudaError_t grouped_gemm_prepare_##name();                                                \
  cudaError_t grouped_gemm_launch_##name(GemmForm form, const GroupedGemmParams& p,         \
                                         const GemmMaps& tm, int n_sms, cudaStream_t stream);
MOEACT_GEMM_UNIT(fwd)
MOEACT_GEMM_UNIT(dgrad)
MOEACT_GEMM_UNIT(wgrad)
MOEACT_GEMM_UNIT(fwd4)
#undef MOEACT_GEMM_UNIT

}  // namespace moeact
