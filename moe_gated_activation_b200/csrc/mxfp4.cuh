// MXFP4 (E2M1 codes, E8M0 scales of 32 values) of bf16 rows and back: the
// host side's view of kern_mxfp4.cu.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace moeact {

struct Mxfp4Params {
  uint16_t* x;          // bf16 [M, ldx]: read by the quantizer, written by the dequantizer
  int64_t ldx;
  int64_t M;
  int K;                // multiple of 32
  uint8_t* codes;       // [M, K/2], column 2j in the low half of byte j
  uint8_t* scales;      // [M, K/32], row-major or 128 x 4 tiles
  int tiled;
  const int32_t* noop;
};

cudaError_t mxfp4_quantize_launch(const Mxfp4Params& p, int n_sms, cudaStream_t stream);
cudaError_t mxfp4_dequantize_launch(const Mxfp4Params& p, int n_sms, cudaStream_t stream);

}  // namespace moeact
