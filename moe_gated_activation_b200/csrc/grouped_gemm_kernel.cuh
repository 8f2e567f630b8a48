// The grouped block-scaled products on the fifth-generation tensor cores
// (sm_100a); see grouped_gemm.cuh for what each operator computes.
//
// out tile = 128 rows per SM x BN columns.  PAIR kernels: two SMs work on a
// 256 x 256 tile (cta_group::2: each holds 128 rows of A, 128 of B and its 128
// rows of the result), so that an operand byte brought into shared memory
// serves twice the products of a single SM's 128 x 128 tile; single-SM kernels
// take short groups, whose few rows would leave a 256-row tile mostly empty.
//
// A persistent grid walks the tiles (columns fastest, so that the SMs of a
// wave share the rows of A and one expert's W in L2).  Roles, per SM:
//   warps 0-3  epilogue: accumulator -> registers -> rounding -> shared
//              memory -> whole 128-byte row segments of the output;
//   warps 4-7  scales: E8M0 words from global memory, in either layout, some
//              chunks ahead into shared memory, and each stage's from there
//              into tensor memory (tcgen05.st);
//   warp 8     TMA loads of the code tiles (128 rows x 128 bytes each);
//   warp 9     tensor-memory allocation; in the pair's first SM the MMAs.
// One ring of stages carries codes and scales: `full` collects the TMA bytes
// and the scale warps of both SMs, `empty` comes from the MMAs' commit.
//
// Tensor memory (512 columns): scales at the top; two accumulators below
// them.  Two 256-column accumulators and the scales do not fit, so a pair's
// accumulators overlap by kOverlap columns, which the epilogue drains first:
// the next tile's MMAs start when those columns are free.
//
// Every wait is bounded; on a timeout the kernel sets MOEACT_DEVERR_GEMM_WAIT,
// lets what is in flight finish (bounded) and returns.
#pragma once

#include "grouped_gemm.cuh"
#include "tensor_core.cuh"

namespace moeact {
namespace {

constexpr uint32_t kErrGemmWait = 0x40u;
constexpr int kTileBytes = 16384;         // 128 rows x 128 bytes
constexpr int kEpiWarpBytes = 4096;       // 32 rows x 128 bytes of output
constexpr int kGemmMisc = 1024;           // barriers and small values

template <int OP, bool PAIR>
struct GemmCfg {
  static constexpr bool kF4 = OP == kGemmFwd4;
  static constexpr bool kWgrad = OP == kGemmWgrad;
  static constexpr bool kAmn = OP == kGemmWgrad;                      // A rows = summed index
  static constexpr bool kBmn = OP == kGemmWgrad || OP == kGemmDgrad;  // B rows = summed index
  static constexpr int kCG = PAIR ? 2 : 1;
  static constexpr int kTM = 128 * kCG;
  static constexpr int kBN = PAIR ? 256 : 128;
  static constexpr int kStages = 5;
  static constexpr int kStageK = kF4 ? 256 : 128;      // summed index per stage
  static constexpr int kMmaK = kF4 ? 64 : 32;
  static constexpr int kWords = kF4 ? 2 : 1;           // scale words per row and stage
  static constexpr int kSfbCols = kBN / 32;
  static constexpr int kSfPitch = kWords * (4 + kSfbCols);
  static constexpr int kSfCol = 512 - (kStages * kSfPitch + 15) / 16 * 16;
  static constexpr int kAcc1 = PAIR ? kSfCol - kBN : kBN;   // second accumulator's column
  static constexpr int kOverlap = PAIR ? kBN - kAcc1 : 0;
  static constexpr int kABox = kAmn || !PAIR ? kGemmShortBoxRows : kGemmBoxRows;
  static constexpr int kBBox = kBmn ? kGemmShortBoxRows : kGemmBoxRows;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kGroups = 1 + kBN / 128;        // 128-row groups of scales (and warps)
  static constexpr int kSfBytes = 2 * 8 * kGroups * 512;   // two chunks of 8 words
  static constexpr int kFixed = kStages * kStageBytes + 4 * kEpiWarpBytes + kSfBytes + kGemmMisc;
  static_assert(kAcc1 >= 0 && kAcc1 + kBN <= kSfCol, "tensor-memory columns overlap");
  static_assert(kOverlap % 64 == 0, "the overlap is drained in chunks of 64 columns");
};

struct GemmSmem {
  unsigned char* stages;
  unsigned char* epi;
  unsigned char* sf;   // [2][8 words][A's rows, B's rows by 128][512] scale words
  uint64_t* full;      // [kStages] (first SM of a pair) codes and scales are in
  uint64_t* empty;     // [kStages] the stage's MMAs are done
  uint64_t* d_full;    // [2] an accumulator holds a finished tile
  uint64_t* d_empty;   // [2] (first SM) its columns may be overwritten
  int* misc;           // [0] tensor-memory base, [1] abort
  int* scan;           // [10] warp totals
  int* ro;             // [E + 1] the row offsets (below 2^30)
  int* pre;            // [E + 1] row tiles before each expert (not wgrad)
};

__device__ __forceinline__ bool gemm_aborted(const GemmSmem& m) {
  return __any_sync(kFull, *reinterpret_cast<volatile int*>(m.misc + 1) != 0);
}
__device__ __forceinline__ void gemm_abort(const GroupedGemmParams& p, const GemmSmem& m) {
  *reinterpret_cast<volatile int*>(m.misc + 1) = 1;
  atomicOr(p.err, kErrGemmWait);
}

// One SM's part of an output tile.
struct GemmTile {
  int e;
  int n0;          // first output column
  int rows;        // rows of this SM's part that exist (0 .. 128)
  int64_t row0;    // its first row: of A and the output, or (wgrad) of dW_e
  int64_t k0;      // wgrad: first row of the group
  int kb;          // blocks of 32 of the summed index
  int krows;       // wgrad: rows of the group
};

template <typename C>
__device__ __forceinline__ GemmTile gemm_tile(const GroupedGemmParams& p, const GemmSmem& m,
                                              int t, int rank) {
  GemmTile r;
  const int nt = (p.N + C::kBN - 1) / C::kBN;
  const int mt = t / nt;
  r.n0 = (t - mt * nt) * C::kBN;
  if constexpr (C::kWgrad) {
    const int ht = (p.R + C::kTM - 1) / C::kTM;
    r.e = mt / ht;
    r.row0 = (mt - r.e * ht) * C::kTM + 128 * rank;
    r.rows = max(0, min(128, p.R - (int)r.row0));
    r.k0 = m.ro[r.e];
    r.krows = m.ro[r.e + 1] - (int)r.k0;
    r.kb = (r.krows + 31) >> 5;
  } else {
    int lo = 0, hi = p.E - 1;   // largest e with pre[e] <= mt (then mt < pre[e + 1])
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (m.pre[mid] <= mt) lo = mid; else hi = mid - 1;
    }
    r.e = lo;
    r.row0 = m.ro[lo] + (mt - m.pre[lo]) * C::kTM + 128 * rank;
    r.rows = max(0, min(128, m.ro[lo + 1] - (int)r.row0));
    r.k0 = 0;
    r.krows = 0;
    r.kb = p.K >> 5;
  }
  return r;
}

// ------------------------------------------------------------ scales
// A word holds the scales of four consecutive blocks of one row of an operand
// (rows of the output); a stage needs one word (E4M3) or two (E2M1) per row.
// A loading warp serves 128 rows of one operand: it keeps kChunk words of each
// row in registers, two chunks ahead, and writes them to shared memory in
// pieces of 128 words.
constexpr int kChunk = 8;

// Loads that stay where they are written: a chunk ahead of their use.
__device__ __forceinline__ uint32_t ldg32(const uint8_t* a) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}
__device__ __forceinline__ uint4 ldg128(const uint8_t* a) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(a));
  return v;
}

// How a warp fetches: fixed per operand and launch, so that no load meets
// another path's registers (the loads are unconditional, at addresses clamped
// into the array: what lies outside is never used, and a load under a
// condition was waited for where the paths join, a chunk too early).
enum ScaleMode : int {
  kTiled = 0,       // 128 x 4 tiles
  kRows32 = 1,      // row-major, a row's blocks a multiple of 32 bytes
  kRows16 = 2,      // ... of 16
  kRows4 = 3,       // ... of 4
  kRowsAny = 4,     // ... any: aligned words, shifted into place
  kCols = 5,        // row-major, blocks outermost
};

// Where a warp's scales of a tile come from.
struct ScaleSrc {
  const uint8_t* s;   // the operand's scales
  int64_t r0;         // rows: first row; columns: first scale row of the group
  int64_t rows;       // rows: rows that exist
  int pitch;          // rows: bytes (blocks) of a row; columns: width
  int c0;             // columns: first column
  int nb;             // columns: blocks of the summed index
  int64_t tile0;      // tiled: index of the first 512-byte tile
  int words;          // words of the summed index
};

template <typename C>
__device__ __forceinline__ ScaleSrc scale_src(const GroupedGemmParams& p, const GemmTile& t,
                                              int group) {
  ScaleSrc r;
  const bool a = group == 0;
  r.s = a ? p.a_scales : p.b_scales;
  r.r0 = r.rows = r.tile0 = 0;
  r.pitch = p.K >> 5;
  r.c0 = r.nb = 0;
  if (C::kAmn) {
    r.r0 = p.cb_offs[t.e];
    r.pitch = a ? p.R : p.N;
    r.c0 = a ? (int)t.row0 : t.n0 + 128 * (group - 1);
    r.nb = t.kb;
    // the group's [width, blocks] matrix starts at byte k0 / 32 * width
    r.tile0 = ((t.k0 >> 5) * r.pitch >> 9) +
              (int64_t)(min(r.c0, r.pitch - 1) >> 7) * (t.krows >> 7);
  } else if (a) {
    r.r0 = t.row0;
    r.rows = p.M;
  } else if (C::kBmn) {
    // W quantised as one [E K, N] matrix in blocks of 32 rows
    r.nb = r.pitch;
    r.r0 = (int64_t)t.e * r.nb;
    r.pitch = p.N;
    r.c0 = t.n0 + 128 * (group - 1);
    r.tile0 = (int64_t)(min(r.c0, r.pitch - 1) >> 7) * (((int64_t)p.E * r.nb) >> 2) + (r.r0 >> 2);
  } else {
    r.r0 = (int64_t)t.e * p.N + t.n0 + 128 * (group - 1);
    r.rows = (int64_t)p.E * p.N;
  }
  r.words = (t.kb + 3) >> 2;
  return r;
}

// Words u .. u + kChunk - 1 of the warp's 128 rows.  Tiled, and row-major with
// the summed index inside the rows: w[i][j] is row 32 j + lane's (kRowsAny:
// the aligned words that hold them, one more per row).  kCols: w[i][j] holds
// columns c0 + 4 lane .. + 3 of block 4 (u + i) + j.
template <int MODE, bool OUTER>
__device__ __forceinline__ void fetch_scales(const ScaleSrc& c, int u, int lane,
                                             uint32_t (*w)[4]) {
  const int last = c.words - 1;
  if constexpr (MODE == kTiled && OUTER) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const uint4 v = ldg128(c.s + ((c.tile0 + min(u + i, last)) << 9) + 16 * lane);
      w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
    }
  } else if constexpr (MODE == kTiled) {
    // row by row: a group's first row need not be a tile's
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = min(c.r0 + 32 * j + lane, c.rows - 1);
      const uint8_t* a = c.s + ((r >> 7) * c.words << 9) + ((r & 31) << 4) + (((r >> 5) & 3) << 2);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) w[i][j] = ldg32(a + 512 * min(u + i, last));
    }
  } else if constexpr (MODE == kCols) {
    const uint8_t* a = c.s + c.r0 * c.pitch + min(c.c0 + 4 * lane, c.pitch - 4);
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[i][j] = ldg32(a + (int64_t)min(4 * (u + i) + j, c.nb - 1) * c.pitch);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = min(c.r0 + 32 * j + lane, c.rows - 1);
      const uint8_t* a = c.s + r * c.pitch;
      if constexpr (MODE == kRows32) {
        // a whole sector in one load: the operand tiles' stream leaves few
        // request slots
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0][j]), "=r"(w[1][j]), "=r"(w[2][j]), "=r"(w[3][j]),
                       "=r"(w[4][j]), "=r"(w[5][j]), "=r"(w[6][j]), "=r"(w[7][j])
                     : "l"(a + 4 * u));
      } else if constexpr (MODE == kRows16) {
#pragma unroll
        for (int i = 0; i < kChunk; i += 4) {
          const uint4 v = ldg128(a + 4 * min(u + i, last - 3));
          w[i][j] = v.x, w[i + 1][j] = v.y, w[i + 2][j] = v.z, w[i + 3][j] = v.w;
        }
      } else if constexpr (MODE == kRows4) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) w[i][j] = ldg32(a + 4 * min(u + i, last));
      } else {
        // the array starts on a word; a word that holds one of its bytes is
        // read whole
        const int64_t end = (c.rows * c.pitch - 1) >> 2, at = (r * c.pitch + 4 * u) >> 2;
#pragma unroll
        for (int i = 0; i <= kChunk; ++i) w[i][j] = ldg32(c.s + 4 * min(at + i, end));
      }
    }
  }
}

// A piece of 128 words in shared memory.  A's: row r's word at byte 4 r (each
// warp reads its own 32).  B's: row 32 j + l's at byte 16 l + 4 j (a lane reads
// its four).
template <bool A, int MODE>
__device__ __forceinline__ void put_words(unsigned char* dst, int lane, const uint32_t* x) {
  uint32_t w[4] = {x[0], x[1], x[2], x[3]};
  if constexpr (MODE == kCols) {
    // four blocks of four columns a lane: a 4 x 4 byte transpose
    const uint32_t t0 = __byte_perm(x[0], x[1], 0x5140), t1 = __byte_perm(x[2], x[3], 0x5140);
    const uint32_t t2 = __byte_perm(x[0], x[1], 0x7362), t3 = __byte_perm(x[2], x[3], 0x7362);
    w[0] = __byte_perm(t0, t1, 0x5410), w[1] = __byte_perm(t0, t1, 0x7632);
    w[2] = __byte_perm(t2, t3, 0x5410), w[3] = __byte_perm(t2, t3, 0x7632);
  }
  if constexpr (A != (MODE == kCols)) {
    // A, rows 32 j + lane: word 32 j + lane; B, columns 4 lane + j: stored in
    // the order j = (k + lane / 2) mod 4, so that each store's 32 words fall
    // into different banks
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (A) {
        *reinterpret_cast<uint32_t*>(dst + 4 * (32 * k + lane)) = w[k];
      } else {
        const int j = (k + (lane >> 1)) & 3;
        const uint32_t v = j & 2 ? (j & 1 ? w[3] : w[2]) : (j & 1 ? w[1] : w[0]);
        *reinterpret_cast<uint32_t*>(dst + (4 * (lane & 7) + j) * 16 + (lane >> 3) * 4) = v;
      }
    }
  } else {
    *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// One of warps 4-7.  LOADER: it fetches a group of 128 rows' words (group 0:
// A's) two chunks ahead.  All four write every stage's words from shared into
// tensor memory (tcgen05.st: a tcgen05.cp would take the tensor pipe's time),
// warp q lanes 32 q .. 32 q + 31: lane l's A word, row 32 q + l's, in column q
// of four; B column c, row 32 c + l's word.
template <typename C, bool LOADER, bool OUTER, int MODE, bool A>
__device__ __forceinline__ void gemm_scales(const GroupedGemmParams& p, const GemmSmem& m,
                                            uint32_t tbase, int tiles, int first, int step,
                                            int rank, int group) {
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
  const uint32_t dst0 = tbase + ((uint32_t)(32 * q) << 16) + (uint32_t)C::kSfCol;
  constexpr int kStagesPerChunk = kChunk / C::kWords;
  constexpr int kRegs = kChunk + (MODE == kRowsAny ? 1 : 0);
  constexpr int kChunkBytes = kChunk * C::kGroups * 512;
  int slot = 0, buf = 0;
  uint32_t phase = 1;   // a fresh barrier's preceding phase counts as complete
  // walks the chunks of every tile: chunk `chunk` of tile t
  struct Walk { int t, chunk, left; };
  auto next = [&](Walk& k, GemmTile& tile) {   // the next chunk's stages, 0 at the end
    while (k.left <= 0) {
      k.t += step;
      if (k.t >= tiles) return 0;
      tile = gemm_tile<C>(p, m, k.t, rank);
      k.left = (tile.kb * 32 + C::kStageK - 1) / C::kStageK;
      k.chunk = -1;
    }
    const int n = min(k.left, kStagesPerChunk);
    k.left -= n;
    ++k.chunk;
    return n;
  };
  Walk load = {first - step, 0, 0}, serve = {first - step, 0, 0};
  ScaleSrc src;
  GemmTile load_tile, serve_tile;
  struct Chunk { int word; int64_t r0; };   // what kRowsAny shifts and masks by
  auto fetch = [&](uint32_t (*w)[4], Chunk& ch) {
    if constexpr (LOADER) {
      if (next(load, load_tile) == 0) return;
      if (load.chunk == 0) src = scale_src<C>(p, load_tile, group);
      fetch_scales<MODE, OUTER>(src, load.chunk * kChunk, lane, w);
      ch.word = load.chunk * kChunk;
      ch.r0 = src.r0;
    }
  };
  auto one = [&](uint32_t (*w)[4], Chunk& ch) {
    const int stages = next(serve, serve_tile);
    if (stages == 0) return false;
    unsigned char* sf = m.sf + buf * kChunkBytes;
    if constexpr (LOADER) {
      if constexpr (MODE == kRowsAny) {
        const int pitch = src.pitch;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t r = min(ch.r0 + 32 * j + lane, src.rows - 1);
          const int sh = 8 * (int)((r * pitch) & 3);
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            w[i][j] = __funnelshift_r(w[i][j], w[i + 1][j], sh);
            // (bytes past the row's end are another row's: a NaN scale there
            // would meet the zeros of half an E2M1 step)
            if (4 * (ch.word + i) + 4 > pitch)
              w[i][j] &= (1u << (8 * max(0, pitch - 4 * (ch.word + i)))) - 1u;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i < stages * C::kWords) put_words<A, MODE>(sf + 512 * (C::kGroups * i + group), lane, w[i]);
      fetch(w, ch);
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");   // the chunk is in shared memory
    bool ok = true;
    for (int s = 0; s < stages; ++s) {
      ok = ok && __all_sync(kFull, tc::sleep(m.empty + slot, phase));
      if (ok) {
        tc::fence_after();
        const uint32_t dst = dst0 + slot * C::kSfPitch;
#pragma unroll
        for (int i = 0; i < C::kWords; ++i) {
          const unsigned char* piece = sf + 512 * C::kGroups * (s * C::kWords + i);
          const uint32_t a = *reinterpret_cast<const uint32_t*>(piece + 4 * (32 * q + lane));
          tc::st1(dst + 4 * i + q, a);
#pragma unroll
          for (int k = 1; k < C::kGroups; ++k) {
            const uint4 b = *reinterpret_cast<const uint4*>(piece + 512 * k + 16 * lane);
            tc::st4(dst + 4 * C::kWords + C::kSfbCols * i + 4 * (k - 1), b.x, b.y, b.z, b.w);
          }
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive_cluster(tc::leader_addr(m.full + slot));
      }
      if (++slot == C::kStages) slot = 0, phase ^= 1;
    }
    if (!ok || gemm_aborted(m)) {
      ok = false;
      gemm_abort(p, m);
    }
    buf ^= 1;
    // the four warps leave together after an abort, at a barrier of their own
    int gone;
    asm volatile("{ .reg .pred p, r; setp.ne.s32 p, %1, 0; bar.red.or.pred r, 2, 128, p; "
                 "selp.s32 %0, 1, 0, r; }" : "=r"(gone) : "r"((int)!ok) : "memory");
    return gone == 0;
  };
  uint32_t w0[kRegs][4], w1[kRegs][4];
  Chunk c0, c1;
  fetch(w0, c0);
  fetch(w1, c1);
  while (one(w0, c0) && one(w1, c1)) {
  }
}

// The scale warp's role and loads, fixed for the launch.
template <typename C>
__device__ __forceinline__ void gemm_scales_any(const GroupedGemmParams& p, const GemmSmem& m,
                                                uint32_t tbase, int tiles, int first, int step,
                                                int rank, int group) {
  const bool tiled = group == 0 ? p.a_tiled : p.b_tiled;
  const int pitch = p.K >> 5;
#define MOEACT_SCALES(OUTER, MODE, A) \
  gemm_scales<C, true, OUTER, MODE, A>(p, m, tbase, tiles, first, step, rank, group)
#define MOEACT_SCALES_OF(OUTER, A)                             \
  if constexpr (OUTER) {                                       \
    if (tiled) MOEACT_SCALES(true, kTiled, A);                 \
    else MOEACT_SCALES(true, kCols, A);                        \
  } else {                                                     \
    if (tiled) MOEACT_SCALES(false, kTiled, A);                \
    else if ((pitch & 31) == 0) MOEACT_SCALES(false, kRows32, A); \
    else if ((pitch & 15) == 0) MOEACT_SCALES(false, kRows16, A); \
    else if ((pitch & 3) == 0) MOEACT_SCALES(false, kRows4, A);   \
    else MOEACT_SCALES(false, kRowsAny, A);                    \
  }
  if (group == 0) {
    MOEACT_SCALES_OF(C::kAmn, true)
  } else if (group < C::kGroups) {
    MOEACT_SCALES_OF(C::kBmn, false)
  } else {
    gemm_scales<C, false, false, kRows32, false>(p, m, tbase, tiles, first, step, rank, group);
  }
#undef MOEACT_SCALES_OF
#undef MOEACT_SCALES
}

// ------------------------------------------------------------ code tiles
// Warp 8.  wgrad: the last rows of a group, when they are no multiple of 32,
// are copied with plain loads and zeros after them, for both operands (rows of
// the next group must not meet in the sum, and zeros times its NaNs would
// not be zero).
template <typename C>
__device__ __forceinline__ void copy_tail(unsigned char* dst, const uint8_t* src, int64_t ld,
                                          int64_t row, int rows, int col, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3), c = lane & 7;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && col + 16 * c < ld)
      v = __ldg(reinterpret_cast<const uint4*>(src + (row + r) * ld + col + 16 * c));
    *reinterpret_cast<uint4*>(dst + r * 128 + ((c ^ (r & 7)) << 4)) = v;
  }
}

template <typename C>
__device__ void gemm_producer(const GroupedGemmParams& p, const GemmSmem& m, const void* tm_a,
                              const void* tm_b, int tiles, int first, int step, int rank) {
  const int lane = threadIdx.x & 31;
  const bool leader = tc::elect_one();
  int slot = 0;
  uint32_t phase = 1;
  for (int t = first; t < tiles; t += step) {
    const GemmTile tile = gemm_tile<C>(p, m, t, rank);
    const int stages = (tile.kb * 32 + C::kStageK - 1) / C::kStageK;
    const int col_b = tile.n0 + (C::kCG == 2 ? 128 * rank : 0);   // this SM's rows of B
    for (int s = 0; s < stages; ++s) {
      if (!__all_sync(kFull, tc::spin(m.empty + slot, phase))) {
        if (leader) gemm_abort(p, m);
        return;
      }
      unsigned char* da = m.stages + slot * C::kStageBytes;
      unsigned char* db = da + kTileBytes;
      const uint32_t bar = tc::leader_addr(m.full + slot);
      int na = 0, nb = 1;   // boxes of A and B
      if constexpr (C::kAmn) {
        const int left = tile.krows - 128 * s, full = min(4, left >> 5);
        na = nb = full;
        if (full < 4 && (left & 31) != 0) {
          copy_tail<C>(da + full * 4096, p.a_codes, p.R, tile.k0 + 128 * s + 32 * full, left & 31,
                       (int)tile.row0, lane);
          copy_tail<C>(db + full * 4096, p.b_codes, p.N, tile.k0 + 128 * s + 32 * full, left & 31,
                       col_b, lane);
          tc::fence_proxy_async();
        }
      } else {
        na = (tile.rows + C::kABox - 1) / C::kABox;
        if constexpr (C::kBmn) nb = min(4, tile.kb - 4 * s);
      }
      __syncwarp();
      if (leader) {
        tc::arrive_tx_cluster(bar, (uint32_t)(na * C::kABox + nb * C::kBBox) * 128u);
        for (int i = 0; i < na; ++i) {
          if constexpr (C::kAmn)
            tc::load_2d<C::kCG>(da + i * 4096, tm_a, (int)tile.row0,
                                (int)tile.k0 + 128 * s + 32 * i, bar);
          else
            tc::load_2d<C::kCG>(da + i * C::kABox * 128, tm_a, 128 * s,
                                (int)tile.row0 + C::kABox * i, bar);
        }
        for (int i = 0; i < nb; ++i) {
          if constexpr (C::kAmn)
            tc::load_2d<C::kCG>(db + i * 4096, tm_b, col_b, (int)tile.k0 + 128 * s + 32 * i, bar);
          else if constexpr (C::kBmn)
            tc::load_2d<C::kCG>(db + i * 4096, tm_b, col_b, tile.e * p.K + 128 * s + 32 * i, bar);
          else
            tc::load_2d<C::kCG>(db, tm_b, 128 * s, tile.e * p.N + col_b, bar);
        }
      }
      __syncwarp();
      if (++slot == C::kStages) slot = 0, phase ^= 1;
    }
  }
}

// ------------------------------------------------------------ MMAs
// Warp 9 of the (first) SM, converged, one elected lane issuing, so that the
// descriptors are warp-uniform.
template <typename C>
__device__ void gemm_mma(const GroupedGemmParams& p, const GemmSmem& m, uint32_t tbase, int tiles,
                         int first, int step) {
  const bool leader = tc::elect_one();
  // E4M3 x E4M3 (format 0) or E2M1 x E2M1 (format 1), major bits, E8M0 scales,
  // N / 8 and M / 16
  constexpr uint32_t kIdesc = (C::kF4 ? (1u << 7) | (1u << 10) : 0u) |
                              (C::kAmn ? 1u << 15 : 0u) | (C::kBmn ? 1u << 16 : 0u) |
                              ((uint32_t)(C::kBN / 8) << 17) | (1u << 23) |
                              ((uint32_t)(C::kTM / 16) << 24);
  // one MMA's step along the summed index: 32 bytes of each row, or 32 rows
  constexpr uint64_t kStepA = C::kAmn ? 256 : 2, kStepB = C::kBmn ? 256 : 2;
  const uint64_t a0 = tc::desc_sw128(smem_addr(m.stages));
  const uint64_t b0 = tc::desc_sw128(smem_addr(m.stages + kTileBytes));
  int slot = 0, n = 0;
  uint32_t phase = 0;
  for (int t = first; t < tiles; t += step) {
    const int kb = gemm_tile<C>(p, m, t, 0).kb;
    if (kb == 0) continue;
    const int mmas = (kb * 32 + C::kMmaK - 1) / C::kMmaK;
    // the tile whose columns this one takes: the last but one, or with
    // overlapping accumulators the last
    const int w = n - (C::kOverlap ? 1 : 2);
    if (w >= 0 && !__all_sync(kFull, tc::spin(m.d_empty + (w & 1), (uint32_t)(w >> 1) & 1u))) {
      if (leader) gemm_abort(p, m);
      return;
    }
    tc::fence_after();
    const uint32_t d = tbase + (uint32_t)((n & 1) * C::kAcc1);
    for (int i0 = 0; i0 < mmas; i0 += 4) {
      if (!__all_sync(kFull, tc::spin(m.full + slot, phase))) {
        if (leader) gemm_abort(p, m);
        return;
      }
      tc::fence_after();
      if (leader) {
        const uint64_t ad = a0 + (uint64_t)slot * (C::kStageBytes >> 4);
        const uint64_t bd = b0 + (uint64_t)slot * (C::kStageBytes >> 4);
        const uint32_t sf = tbase + C::kSfCol + slot * C::kSfPitch;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + j < mmas) {
            const uint32_t id = C::kF4 ? (uint32_t)(j & 1) * 2 : (uint32_t)j;   // scale byte
            const int word = C::kF4 ? j >> 1 : 0;
            tc::mma<C::kCG, C::kF4>(d, ad + kStepA * j, bd + kStepB * j,
                                    kIdesc | (id << 4) | (id << 29), sf + 4 * word,
                                    sf + 4 * C::kWords + C::kSfbCols * word,
                                    (i0 | j) != 0 ? 1u : 0u);
          }
        tc::commit<C::kCG>(m.empty + slot);
      }
      __syncwarp();
      if (++slot == C::kStages) slot = 0, phase ^= 1;
    }
    if (leader) tc::commit<C::kCG>(m.d_full + (n & 1));
    __syncwarp();
    ++n;
  }
}

// ------------------------------------------------------------ epilogue
// 32 rows x 128 bytes from registers (thread t: row t, as eight 16-byte
// pieces) through the warp's staging, so that each store writes whole row
// segments.  `cols` output columns of the piece's 128 bytes exist.
template <bool OUT32>
__device__ __forceinline__ void store_piece(const GroupedGemmParams& p, unsigned char* stg,
                                            const uint4* v, int64_t row, int rows, int col,
                                            int lane) {
  constexpr int kPer = OUT32 ? 4 : 8;   // columns in 16 bytes
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) = v[c];
  __syncwarp();
  const int c = lane & 7;
  const bool in = col + kPer * c < p.N;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 4 * k + (lane >> 3);
    uint4 w = *reinterpret_cast<const uint4*>(stg + r * 128 + ((c ^ (r & 7)) << 4));
    if (in && r < rows) {
      if constexpr (OUT32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + (row + r) * p.ldo +
                                                col + kPer * c);
        float4 f = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                               __uint_as_float(w.w));
        if (p.accumulate) {
          const float4 o = *dst;
          f = make_float4(__fadd_rn(o.x, f.x), __fadd_rn(o.y, f.y), __fadd_rn(o.z, f.z),
                          __fadd_rn(o.w, f.w));
        }
        *dst = f;
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (row + r) * p.ldo + col +
                                  kPer * c) = w;
      }
    }
  }
  __syncwarp();
}

template <typename C>
__device__ void gemm_epilogue(const GroupedGemmParams& p, const GemmSmem& m, uint32_t tbase,
                              int tiles, int first, int step, int rank) {
  const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  unsigned char* stg = m.epi + q * kEpiWarpBytes;
  int n = 0;
  for (int t = first; t < tiles; t += step) {
    const GemmTile tile = gemm_tile<C>(p, m, t, rank);
    const int rows = max(0, min(32, tile.rows - 32 * q));
    const int64_t row = (C::kWgrad ? (int64_t)tile.e * p.R : 0) + tile.row0 + 32 * q;
    if (tile.kb == 0) {   // wgrad of an expert without rows: zeros
      if (p.accumulate) continue;
      uint4 z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int c = 0; c < C::kBN; c += p.out32 ? 32 : 64) {
        if (p.out32) store_piece<true>(p, stg, z, row, rows, tile.n0 + c, lane);
        else store_piece<false>(p, stg, z, row, rows, tile.n0 + c, lane);
      }
      continue;
    }
    const int b = n & 1;
    if (!__all_sync(kFull, tc::sleep(m.d_full + b, (uint32_t)(n >> 1) & 1u)) || gemm_aborted(m)) {
      gemm_abort(p, m);
      return;
    }
    tc::fence_after();
    const uint32_t src = tbase + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * C::kAcc1);
    constexpr int kChunks = C::kBN / 64, kOver = C::kOverlap / 64;
#pragma unroll 1
    for (int i = 0; i < kChunks; ++i) {
      // the overlapping columns first: the first accumulator's last chunks,
      // the second one's first
      const int c = kOver && b == 0 ? (i + kChunks - kOver) % kChunks : i;
      uint32_t v[64];
      tc::ld32(src + 64 * c, v);
      tc::ld32(src + 64 * c + 32, v + 32);
      tc::wait_ld();
      if (i == (kOver ? kOver : kChunks) - 1) {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive_cluster(tc::leader_addr(m.d_empty + b));
      }
      const int col = tile.n0 + 64 * c;
      if (col >= p.N || rows == 0) continue;
      if (p.out32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[j] = make_uint4(v[32 * h + 4 * j], v[32 * h + 4 * j + 1], v[32 * h + 4 * j + 2],
                              v[32 * h + 4 * j + 3]);
          store_piece<true>(p, stg, w, row, rows, col + 32 * h, lane);
        }
      } else {
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t* x = v + 8 * j;
          w[j] = make_uint4(pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                            pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                            pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                            pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7])));
        }
        store_piece<false>(p, stg, w, row, rows, col, lane);
      }
    }
    ++n;
  }
}

// ------------------------------------------------------------ kernel
template <int OP, bool PAIR>
__global__ void __launch_bounds__(kGemmThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,
                        const __grid_constant__ CUtensorMap tm_b, const GroupedGemmParams p) {
  using C = GemmCfg<OP, PAIR>;
  if (p.noop != nullptr && *p.noop != 0) return;
  extern __shared__ __align__(1024) unsigned char gemm_smem[];
  unsigned char* base = gemm_smem + ((1024u - (smem_addr(gemm_smem) & 1023u)) & 1023u);
  GemmSmem m;
  m.stages = base;
  m.epi = base + C::kStages * C::kStageBytes;
  m.sf = m.epi + 4 * kEpiWarpBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(m.epi + 4 * kEpiWarpBytes + C::kSfBytes);
  m.full = bars;
  m.empty = m.full + C::kStages;
  m.d_full = m.empty + C::kStages;
  m.d_empty = m.d_full + 2;
  m.misc = reinterpret_cast<int*>(bars + 64);
  m.scan = m.misc + 16;
  m.ro = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(bars) + kGemmMisc);
  m.pre = m.ro + p.E + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = PAIR ? (int)tc::cluster_rank() : 0;

  // ---- the groups: offsets checked, row tiles before each expert
  const int E = p.E;
  const int per = (E + kGemmThreads - 1) / kGemmThreads;
  const int e_lo = min(E, tid * per), e_hi = min(E, e_lo + per);
  int local = 0, bad = 0;
  for (int e = e_lo; e < e_hi; ++e) {
    const int64_t r0 = p.row_offs[e], r1 = p.row_offs[e + 1];
    m.ro[e] = (int)r0;
    m.ro[e + 1] = (int)r1;   // (the next thread's first writes the same)
    if (r1 < r0 || r0 < 0 || r1 > p.M) bad |= 1;
    else local += (int)((r1 - r0 + C::kTM - 1) / C::kTM);
    if constexpr (C::kWgrad) {
      if (p.cb_offs[e + 1] - p.cb_offs[e] != (r1 - r0 + 31) >> 5) bad |= 1;
      if ((p.a_tiled || p.b_tiled) && ((r1 - r0) & 127) != 0) bad |= 2;
    }
  }
  if (tid == 0 && (p.row_offs[0] != 0 || p.row_offs[E] != p.M)) bad |= 1;
  if (C::kWgrad && tid == 0 && (p.cb_offs[0] != 0 || p.cb_offs[E] > p.cb_rows)) bad |= 1;
  int incl = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) m.scan[warp] = incl;
  const int bad1 = __syncthreads_or(bad & 1);
  const int bad2 = __syncthreads_or(bad & 2);
  if (blockIdx.x == 0 && tid == 0) *p.status = bad1 ? 3 : bad2 ? 4 : 0;
  if (bad1 || bad2) return;
  int before = incl - local, total = 0;
  for (int w = 0; w < kGemmThreads / 32; ++w) {
    const int v = m.scan[w];
    if (w < warp) before += v;
    total += v;
  }
  if constexpr (!C::kWgrad) {
    for (int e = e_lo; e < e_hi; ++e) {
      m.pre[e] = before;
      before += (m.ro[e + 1] - m.ro[e] + C::kTM - 1) / C::kTM;
    }
    if (tid == 0) m.pre[E] = total;
  } else {
    total = E * ((p.R + C::kTM - 1) / C::kTM);
  }
  const int tiles = total * ((p.N + C::kBN - 1) / C::kBN);
  const int first = blockIdx.x / C::kCG, step = gridDim.x / C::kCG;

  // ---- barriers and tensor memory
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(m.full + i, 5 * C::kCG);   // per SM: the TMA warp and four scale warps
      mbar_init(m.empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(m.d_full + i, 1);
      mbar_init(m.d_empty + i, 4 * C::kCG);
    }
    m.misc[1] = 0;
    mbar_init_fence();
  }
  if (warp == 9) {
    tc::tmem_alloc<C::kCG>(reinterpret_cast<uint32_t*>(m.misc), 512);
    tc::tmem_relinquish<C::kCG>();
  }
  tc::fence_before();
  __syncthreads();
  if (PAIR) tc::cluster_sync();   // the pair's barriers exist before either arrives on them
  tc::fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(m.misc);

  if (warp < 4) gemm_epilogue<C>(p, m, tbase, tiles, first, step, rank);
  else if (warp < 8) gemm_scales_any<C>(p, m, tbase, tiles, first, step, rank, warp - 4);
  else if (warp == 8) gemm_producer<C>(p, m, &tm_a, &tm_b, tiles, first, step, rank);
  else if (rank == 0) gemm_mma<C>(p, m, tbase, tiles, first, step);

  tc::fence_before();
  __syncthreads();
  // after an abort, copies and MMAs may still be in flight: each ends by
  // itself in microseconds, and nothing may take the memory before
  if (*reinterpret_cast<volatile int*>(m.misc + 1)) {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 2000000ull) {
    }
    __syncthreads();
  }
  if (PAIR) tc::cluster_sync();   // no arrival or MMA of the pair reaches an SM that has left
  if (warp == 9) {
    tc::fence_after();
    tc::tmem_dealloc<C::kCG>(tbase, 512);
  }
}

template <int OP, bool PAIR>
int gemm_smem_bytes(int E) {
  using C = GemmCfg<OP, PAIR>;
  return 1024 + C::kFixed + (E + 1) * (C::kWgrad ? 4 : 8);
}

template <int OP, bool PAIR>
cudaError_t gemm_prepare_one(int max_groups) {
  return cudaFuncSetAttribute(grouped_gemm_kernel<OP, PAIR>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              gemm_smem_bytes<OP, PAIR>(max_groups));
}

template <int OP, bool PAIR>
cudaError_t gemm_launch_one(const GroupedGemmParams& p, const CUtensorMap& tm_a,
                            const CUtensorMap& tm_b, int n_sms, cudaStream_t stream) {
  using C = GemmCfg<OP, PAIR>;
  // at most as many row tiles as full ones and one more per group
  const int64_t row_tiles = C::kWgrad ? (int64_t)p.E * ((p.R + C::kTM - 1) / C::kTM)
                                      : p.M / C::kTM + (p.E < p.M ? p.E : p.M);
  const int64_t tiles = row_tiles * ((p.N + C::kBN - 1) / C::kBN);
  const int64_t most = n_sms / C::kCG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * C::kCG));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = gemm_smem_bytes<OP, PAIR>(p.E);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C::kCG;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, grouped_gemm_kernel<OP, PAIR>, tm_a, tm_b, p);
}

}  // namespace
}  // namespace moeact

// Defines one operator's prepare and launch functions.
#define MOEACT_DEFINE_GEMM_UNIT(name, OP)                                                       \
  namespace moeact {                                                                            \
  cudaError_t grouped_gemm_prepare_##name() {                                                   \
    cudaError_t e = gemm_prepare_one<OP, false>(MOEACT_MAX_GROUPS);                             \
    return e != cudaSuccess ? e : gemm_prepare_one<OP, true>(MOEACT_MAX_GROUPS);                \
  }                                                                                             \
  cudaError_t grouped_gemm_launch_##name(bool pair, const GroupedGemmParams& p,                 \
                                         const CUtensorMap& tm_a, const CUtensorMap& tm_b,      \
                                         int n_sms, cudaStream_t stream) {                      \
    return pair ? gemm_launch_one<OP, true>(p, tm_a, tm_b, n_sms, stream)                       \
                : gemm_launch_one<OP, false>(p, tm_a, tm_b, n_sms, stream);                     \
  }                                                                                             \
  }
