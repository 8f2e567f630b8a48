// Rowwise MXFP8 and MXFP4 quantizers and the MXFP4 dequantizer (sm_100a).
//
// A block of 32 values of a row: b = 127 + e, e the smallest integer in
// [-127, 127] with max |x| <= T * 2^e (RCEIL; T = 448 for E4M3, 6 for E2M1);
// code = the nearest-even code of x * 2^(127 - b), saturating, sign of zero
// kept.  NaN in a block: b = 255, every code NaN (E4M3) or 7; infinity: b =
// 254.
//
// All are bound by memory (2 + 33/32 or 17/32 bytes a value).  A lane takes eight
// adjacent values (16 bytes of bf16, 4 bytes of codes), four lanes a block;
// a warp takes the same 256 columns of several rows at a time, so that as many
// 16-byte loads per lane are in flight.  Rows, blocks per SM and the grid are
// the fastest of a sweep (2 - 8 rows, 3 - 8 blocks, grids of 4 - 64 blocks per SM
// and of one pass): at [16384, 7168] the MXFP4 quantizer took 57.2 us (4 rows, 6
// blocks, 12 per SM; 62.7 with 4, 4 and 8), 5.2 TB/s, the MXFP8 one 61.3 us (71.0),
// 5.8 TB/s, and the dequantizer 53.4 us (8 rows, 4 blocks; 60.7 with 4 rows),
// 5.6 TB/s, of 6.5 that a copy reaches.
#include "device_common.cuh"
#include "mx_rows.cuh"

namespace moeact {
namespace {

constexpr int kRowsQ = 4, kRowsD = 8;       // rows a warp works on at a time
constexpr int kBlocksQ = 6, kBlocksD = 4;   // resident blocks per SM
constexpr int kGridR = 12;                  // blocks per SM of a full grid
constexpr int kColsR = 256;      // columns of a warp: 8 per lane
constexpr int kThreadsR = 256;

// b of a block from the magnitude bits of its largest value: with E2M1's
// largest value 6 = 1.5 * 2^2, e = E - 2 - 127, plus one when the mantissa is
// above 1.5 (adding 0x3FFFFF carries exactly then).
__device__ __forceinline__ uint32_t e8m0_from_amax4(uint32_t amag) {
  if (amag >= 0x7F800000u) return amag == 0x7F800000u ? 254u : 255u;
  return (uint32_t)max((int)((amag + 0x3FFFFFu) >> 23) - 2, 0);
}

// Eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float2* v, float mul) {
  const float2 m = make_float2(mul, mul);
  const float2 a = mul2(v[0], m), b = mul2(v[1], m), c = mul2(v[2], m), d = mul2(v[3], m);
  uint32_t r;
  asm("{ .reg .b8 t0, t1, t2, t3; "
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1; cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3; "
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5; cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7; "
      "mov.b32 %0, {t0, t1, t2, t3}; }"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

__device__ __forceinline__ int64_t scale_off(const MxRowsParams& p, int64_t row, int block) {
  const int nb = p.K >> 5;
  if (!p.tiled) return row * nb + block;
  return (((row >> 7) * (nb >> 2) + (block >> 2)) << 9) + ((row & 31) << 4) +
         (((row >> 5) & 3) << 2) + (block & 3);
}

// The grouped offsets' verdict, the same in every block: 0, 3 (not those of
// valid splits) or 4 (tiled scales and a group that is not whole tiles).
__device__ __forceinline__ int check_offsets(const MxRowsParams& p) {
  int bad = 0;
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
    const int64_t r = p.row_offs[e], c = p.cb_offs[e];
    if (e == 0) {
      if (r != 0 || c != 0) bad |= 1;
    } else {
      const int64_t m = r - p.row_offs[e - 1];
      if (m < 0 || r > p.M || c - p.cb_offs[e - 1] != (m + 31) / 32) bad |= 1;
    }
    if (e == p.E && r != p.M) bad |= 1;
    if (p.tiled && (r & 127)) bad |= 2;
  }
  const int b1 = __syncthreads_or(bad & 1), b2 = __syncthreads_or(bad & 2);
  return b1 ? 3 : b2 ? 4 : 0;
}

template <bool F4>
__global__ void __launch_bounds__(kThreadsR, kBlocksQ) mx_rows_kernel(const MxRowsParams p) {
  if (p.noop != nullptr && *p.noop != 0) return;
  if (!F4 && p.E > 0) {
    const int st = check_offsets(p);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = st;
    if (st) return;
  }
  const int lane = threadIdx.x & 31;
  const uint32_t chunks = (uint32_t)(p.K + kColsR - 1) / kColsR;
  const uint32_t items = (uint32_t)((p.M + kRowsQ - 1) / kRowsQ) * chunks;
  const uint32_t stride = gridDim.x * (kThreadsR / 32);
  for (uint32_t i = blockIdx.x * (kThreadsR / 32) + (threadIdx.x >> 5); i < items; i += stride) {
    const uint32_t rg = i / chunks;
    const int col = (int)(i - rg * chunks) * kColsR + 8 * lane;
    const int64_t row0 = (int64_t)rg * kRowsQ;
    const bool in = col < p.K;
    uint4 x[kRowsQ];
#pragma unroll
    for (int r = 0; r < kRowsQ; ++r)
      x[r] = in && row0 + r < p.M
                 ? __ldcs(reinterpret_cast<const uint4*>(p.x + (row0 + r) * p.ldx + col))
                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int r = 0; r < kRowsQ; ++r) {
      // magnitudes as 15-bit integers (NaN above infinity), two to a word
      const uint32_t mask = 0x7FFF7FFFu;
      uint32_t a = __vmaxu2(__vmaxu2(x[r].x & mask, x[r].y & mask),
                            __vmaxu2(x[r].z & mask, x[r].w & mask));
      a = __vmaxu2(a, __shfl_xor_sync(kFull, a, 1));
      a = __vmaxu2(a, __shfl_xor_sync(kFull, a, 2));
      const uint32_t amax = max(a & 0xFFFFu, a >> 16) << 16;
      const uint32_t b = F4 ? e8m0_from_amax4(amax) : e8m0_from_amax(amax);
      const uint32_t mul = scale_multiplier(b);
      const float2 v[4] = {bf16x2_to_f2(x[r].x), bf16x2_to_f2(x[r].y), bf16x2_to_f2(x[r].z),
                           bf16x2_to_f2(x[r].w)};
      if (!in || row0 + r >= p.M) continue;
      const int64_t at = (row0 + r) * (int64_t)p.K + col;
      if constexpr (F4) {
        *reinterpret_cast<uint32_t*>(p.codes + (at >> 1)) = e2m1x8(v, __uint_as_float(mul));
      } else {
        *reinterpret_cast<uint2*>(p.codes + at) =
            make_uint2(e4m3x2_2(v[0], mul, mul) | (e4m3x2_2(v[1], mul, mul) << 16),
                       e4m3x2_2(v[2], mul, mul) | (e4m3x2_2(v[3], mul, mul) << 16));
      }
      if ((lane & 3) == 0) p.scales[scale_off(p, row0 + r, col >> 5)] = (uint8_t)b;
    }
  }
}

// Value of code c times 2^(b - 127); the product is exact in fp32 and (down
// to bf16's subnormals, which hold 0.5 * 2^-127) in bf16.
__global__ void __launch_bounds__(kThreadsR, kBlocksD) mxfp4_dequantize_kernel(const MxRowsParams p) {
  if (p.noop != nullptr && *p.noop != 0) return;
  const int lane = threadIdx.x & 31;
  const uint32_t chunks = (uint32_t)(p.K + kColsR - 1) / kColsR;
  const uint32_t items = (uint32_t)((p.M + kRowsD - 1) / kRowsD) * chunks;
  const uint32_t stride = gridDim.x * (kThreadsR / 32);
  for (uint32_t i = blockIdx.x * (kThreadsR / 32) + (threadIdx.x >> 5); i < items; i += stride) {
    const uint32_t rg = i / chunks;
    const int col = (int)(i - rg * chunks) * kColsR + 8 * lane;
    const int64_t row0 = (int64_t)rg * kRowsD;
    uint32_t q[kRowsD], b[kRowsD];
#pragma unroll
    for (int r = 0; r < kRowsD; ++r) {
      const bool in = col < p.K && row0 + r < p.M;
      q[r] = in ? *reinterpret_cast<const uint32_t*>(
                      p.codes + (row0 + r) * (int64_t)(p.K >> 1) + (col >> 1))
                : 0u;
      b[r] = in ? (uint32_t)p.scales[scale_off(p, row0 + r, col >> 5)] : 0u;
    }
#pragma unroll
    for (int r = 0; r < kRowsD; ++r) {
      if (col >= p.K || row0 + r >= p.M) continue;
      // 2^(b - 127): 2^-127 is subnormal
      const float s = __uint_as_float(b[r] == 255u ? kNanScale : b[r] ? b[r] << 23 : 0x00400000u);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // E2M1: magnitudes 0, 0.5, then (1 + m/2) 2^(x - 1): as fp32 bits,
          // exponent and mantissa bit shifted into place and rebiased by a
          // product (0.5 is a subnormal there), all exact
          const uint32_t c = (q[r] >> (8 * j + 4 * h)) & 15u;
          f[h] = __uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)) * 0x1p126f;
        }
        const float2 y = mul2(make_float2(f[0], f[1]), make_float2(s, s));
        w[j] = pack_bf16x2(y.x, y.y);
      }
      __stcs(reinterpret_cast<uint4*>(p.x + (row0 + r) * p.ldx + col),
             make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

unsigned grid_rows(const MxRowsParams& p, int rows, int n_sms) {
  const int64_t items = (p.M + rows - 1) / rows * ((p.K + kColsR - 1) / kColsR);
  const int64_t blocks = (items + kThreadsR / 32 - 1) / (kThreadsR / 32);
  return (unsigned)(blocks < kGridR * (int64_t)n_sms ? blocks : kGridR * (int64_t)n_sms);
}

}  // namespace

cudaError_t mxfp8_rows_launch(const MxRowsParams& p, int n_sms, cudaStream_t stream) {
  mx_rows_kernel<false><<<grid_rows(p, kRowsQ, n_sms), kThreadsR, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t mxfp4_rows_launch(const MxRowsParams& p, int n_sms, cudaStream_t stream) {
  mx_rows_kernel<true><<<grid_rows(p, kRowsQ, n_sms), kThreadsR, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t mxfp4_dequantize_launch(const MxRowsParams& p, int n_sms, cudaStream_t stream) {
  mxfp4_dequantize_kernel<<<grid_rows(p, kRowsD, n_sms), kThreadsR, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moeact
