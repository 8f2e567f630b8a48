// Rowwise quantizers of bf16 rows -- MXFP8 (E4M3) and MXFP4 (E2M1), E8M0 scales
// of 32 values -- and the MXFP4 dequantizer: the host side's view of
// kern_mx_rows.cu.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace moeact {

struct MxRowsParams {
  uint16_t* x;              // bf16 [M, ldx]: read by the quantizers, written by the dequantizer
  int64_t ldx;
  int64_t M;
  int K;                    // multiple of 32
  uint8_t* codes;           // E4M3 [M, K]; E2M1 [M, K/2], column 2j in the low half of byte j
  uint8_t* scales;          // [M, K/32], row-major or 128 x 4 tiles
  int tiled;
  // grouped MXFP8: the offsets, checked as the grouped kernels do (a row's
  // blocks lie inside the row, so the groups have no part in the result)
  const int64_t* row_offs;
  const int64_t* cb_offs;
  int E;                    // 0: not grouped
  int32_t* status;
  const int32_t* noop;
};

cudaError_t mxfp8_rows_launch(const MxRowsParams& p, int n_sms, cudaStream_t stream);
cudaError_t mxfp4_rows_launch(const MxRowsParams& p, int n_sms, cudaStream_t stream);
cudaError_t mxfp4_dequantize_launch(const MxRowsParams& p, int n_sms, cudaStream_t stream);

}  // namespace moeact
