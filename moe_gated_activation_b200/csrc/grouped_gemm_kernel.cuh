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
//              memory -> bulk tensor stores of 32 rows x 128 bytes;
//   warps 4-7  scales: E8M0 words from shared memory, as they came, into the
//              order of tensor memory and each stage's there (tcgen05.st);
//   warp 8     TMA loads of the code tiles (128 rows x 128 bytes each);
//   warp 9     tensor-memory allocation; in the pair's first SM the MMAs;
//   warp 10    the scales' copies into shared memory, some chunks ahead;
//   warps 12-15  wgrad on pairs: a second set of epilogue warps (warp 11 does
//              nothing: the sets are groups of four).
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

#include <algorithm>
#include <type_traits>

#include "grouped_gemm.cuh"
#include "tensor_core.cuh"

namespace moeact {
namespace {

constexpr uint32_t kErrGemmWait = 0x40u;
constexpr int kTileBytes = 16384;         // 128 rows x 128 bytes
constexpr int kPieceBytes = 4096;         // 32 rows x 128 bytes of output
constexpr int kGemmMisc = 1024;           // barriers and small values
constexpr int kChunk = 8;                 // scale words of a row fetched together
constexpr int kRawDepth = 2;              // chunks on their way
constexpr int kRawBytes = 128 * 36;       // a chunk of 128 rows as it arrives

// The groups' tables: two words a group, one (`pre`) above kGroupsInSmem groups,
// whose row offsets are read from global memory.
constexpr int kGroupsInSmem = 1200;
constexpr int group_bytes_gemm(int E) { return (E + 1) * (E <= kGroupsInSmem ? 8 : 4); }

// The tensor cores drop what falls below an accumulator's last bit instead of
// rounding it: one sum over 65,536 rows of 2^23 and then 2^-5 a step lost every
// later step, 64 in all, and wgrad of random codes was off by 1.1e-10 times the
// rows relative to the norm (6.8e-6 at 62,348).  fp32 outputs therefore take a
// sum in segments of this many steps, which the epilogue adds with rounding
// (at most 6.7e-7 there; shorter sums keep their time, one group of 65,536
// rows, 2048 x 1536, takes 203 us for 186).  bf16 ones, whose own rounding is
// 2^-8, take one sum of up to kGemmLongSum steps, and longer ones in segments too
// (kGemmLong; wgrad's by a second launch, which leaves the short groups to the
// first: on single SMs 2^20 rows on 128 experts, 2048 x 1536, took 3,680 us for
// 2,380).  A multiple of a stage's 4 steps.
constexpr int kSegment = 256;

template <int OP, GemmForm FORM>
struct GemmCfg {
  static constexpr bool PAIR = FORM == kGemmPair;
  static constexpr bool kLong = FORM == kGemmLong;
  static constexpr bool kF4 = OP == kGemmFwd4;
  static constexpr bool kWgrad = OP == kGemmWgrad;
  static constexpr bool kAmn = OP == kGemmWgrad;                      // A rows = summed index
  static constexpr bool kBmn = OP == kGemmWgrad || OP == kGemmDgrad;  // B rows = summed index
  // wgrad on pairs: short sums, so a second set of epilogue warps (12-15) takes
  // half of the columns
  static constexpr int kSets = PAIR && kWgrad ? 2 : 1;
  static constexpr int kThreads = kSets == 2 ? 512 : 352;
  static constexpr int kCG = PAIR ? 2 : 1;
  // Of the handovers between a pair's SMs only that of a stage to the MMAs has
  // shared memory behind it, which the copies write.
  static constexpr tc::Order kOrder = PAIR ? tc::kPair : tc::kSm;
  static constexpr tc::Order kDataOrder = PAIR ? tc::kPairData : tc::kSm;
  static constexpr int kTM = 128 * kCG;
  static constexpr int kBN = PAIR ? 256 : 128;
  // (the second set's staging takes the place of a fifth stage)
  static constexpr int kStages = kSets == 2 ? 4 : 5;
  static constexpr int kStageK = kF4 ? 256 : 128;      // summed index per stage
  static constexpr int kMmaK = kF4 ? 64 : 32;
  static constexpr int kWords = kF4 ? 2 : 1;           // scale words per row and stage
  static constexpr int kSfbCols = kBN / 32;
  static constexpr int kSfPitch = kWords * (4 + kSfbCols);
  static constexpr int kSfCol = 512 - (kStages * kSfPitch + 63) / 64 * 64;
  static constexpr int kAcc1 = PAIR ? kSfCol - kBN : kBN;   // second accumulator's column
  static constexpr int kOverlap = PAIR ? kBN - kAcc1 : 0;
  static constexpr int kTotal = 2 * kBN;   // kLong: the running totals
  static constexpr int kABox = kAmn || !PAIR ? kGemmShortBoxRows : kGemmBoxRows;
  static constexpr int kBBox = kBmn ? kGemmShortBoxRows : kGemmBoxRows;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kGroups = 1 + kBN / 128;        // 128-row groups of scales (and warps)
  static constexpr int kSfBytes = kChunk * kGroups * 512;   // a chunk, ready for tensor memory
  static constexpr int kRawGroupBytes = kRawDepth * kRawBytes;
  static constexpr int kFixed = kStages * kStageBytes + 4 * kSets * kPieceBytes + kSfBytes +
                                kGroups * kRawGroupBytes + kGemmMisc;
  static_assert(kFixed + 1024 + group_bytes_gemm(2040) <= 232448 &&
                    kFixed + 1024 + group_bytes_gemm(kGroupsInSmem) <= 232448,
                "shared memory of a block");
  static_assert(kAcc1 >= 0 && kAcc1 + kBN <= kSfCol, "tensor-memory columns overlap");
  static_assert(!kLong || kTotal + kBN <= kSfCol, "tensor-memory columns overlap");
  static_assert(kOverlap % 64 == 0, "the overlap is drained in chunks of 64 columns");
};

struct GemmSmem {
  unsigned char* stages;
  unsigned char* epi;
  unsigned char* sf;   // [kChunk][A's rows, B's rows by 128][512] scale words
  unsigned char* raw;  // [groups][kRawDepth][kRawBytes] the same as they arrive
  uint64_t* full;      // [kStages] (first SM of a pair) codes and scales are in
  uint64_t* empty;     // [kStages] the stage's MMAs are done
  uint64_t* raw_full;  // [groups][kRawDepth] a chunk of scales has arrived
  uint64_t* raw_empty; // [kRawDepth] ... and is in its pieces
  uint64_t* d_full;    // [2] an accumulator holds a finished tile
  uint64_t* d_empty;   // [2] (first SM) its columns may be overwritten
  int* head;           // [kRawDepth][4] of a raw chunk: its stages, the groups' places (ScaleHead)
  int* misc;           // [0] tensor-memory base, [1] abort
  int* scan;           // [16] warp totals
  int* ro;             // [E + 1] the row offsets (below 2^30); null: too many
  int* pre;            // [E + 1] row tiles before each expert; wgrad: scale rows before it
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

// Walks the tiles first, first + step, ...: columns fastest, then rows.
// (Splitting the tiles of a last, partial wave by columns over idle SMs cost the
// copying thread more in every stage than the shorter wave gave: 64 rows on 50
// experts, 2048 -> 1536, 36.9 -> 40 us.)
template <typename C>
struct GemmWalk {
  int t, tiles, step;
  int nt, ni, dn;      // column tiles; this one; the step's
  int mt, dm;          // row tile over all groups; the step's
  int e;

  __device__ __forceinline__ GemmWalk(const GroupedGemmParams& p, int first, int step_, int tiles_)
      : t(first), tiles(tiles_), step(step_), e(0) {
    nt = (p.N + C::kBN - 1) / C::kBN;
    mt = first / nt;
    ni = first - mt * nt;
    dm = step / nt;
    dn = step - dm * nt;
  }
  __device__ __forceinline__ bool done() const { return t >= tiles; }
  __device__ __forceinline__ int row_off(const GroupedGemmParams& p, const GemmSmem& m, int g) {
    return m.ro != nullptr ? m.ro[g] : (int)p.row_offs[g];
  }
  __device__ __forceinline__ void next() {
    t += step;
    mt += dm;
    ni += dn;
    if (ni >= nt) ni -= nt, ++mt;
  }
  __device__ __forceinline__ GemmTile tile(const GroupedGemmParams& p, const GemmSmem& m,
                                           int rank) {
    GemmTile r;
    r.n0 = ni * C::kBN;
    if constexpr (C::kWgrad) {
      const int ht = (p.R + C::kTM - 1) / C::kTM;
      e = mt / ht;
      r.row0 = (mt - e * ht) * C::kTM + 128 * rank;
      r.rows = max(0, min(128, p.R - (int)r.row0));
      r.k0 = row_off(p, m, e);
      r.krows = row_off(p, m, e + 1) - (int)r.k0;
      r.kb = (r.krows + 31) >> 5;
      // long bf16 sums are the kLong kernel's: nothing to do here, or only these
      if (C::kLong ? r.kb <= kGemmLongSum : !p.out32 && r.kb > kGemmLongSum)
        r.kb = r.krows = r.rows = 0;
    } else {
      int hi = p.E - 1;   // largest e with pre[e] <= mt (then mt < pre[e + 1])
      while (e < hi) {
        const int mid = (e + hi + 1) >> 1;
        if (m.pre[mid] <= mt) e = mid; else hi = mid - 1;
      }
      r.row0 = row_off(p, m, e) + (mt - m.pre[e]) * C::kTM + 128 * rank;
      r.rows = max(0, min(128, row_off(p, m, e + 1) - (int)r.row0));
      r.k0 = 0;
      r.krows = 0;
      r.kb = p.K >> 5;
    }
    r.e = e;
    return r;
  }
};

// ------------------------------------------------------------ scales
// A word holds the scales of four consecutive blocks of one row of an operand
// (rows of the output); a stage needs one word (E4M3) or two (E2M1) per row.
// They go in chunks of kChunk words: bulk copies (where the layout has no
// 16-byte steps, cp.async) bring a chunk to shared memory kRawDepth chunks
// ahead; warps 4, 5 (and 6) each put one group of 128 rows' words into pieces
// of 128, in the order in which tensor memory takes them; warps 4-7 then write
// each stage's words there.  (Plain
// loads into registers ahead of their use waited for one another, and their
// unrolled code missed the instruction cache: 3 - 6 thousand cycles a chunk.)
enum ScaleMode : int {
  kTiled = 0,       // 128 x 4 tiles
  kRows16 = 1,      // row-major, a row's blocks a multiple of 16 bytes
  kRows4 = 2,       // ... of 4
  kRowsAny = 3,     // ... any: aligned words, shifted into place
  kCols = 4,        // row-major, blocks outermost
  kFlat = 5,        // row-major, a row's blocks in one chunk: 128 rows in one piece
};

// Where a warp's scales of a tile come from.
struct ScaleSrc {
  const uint8_t* s;   // the operand's scales
  int64_t r0;         // rows: first row; columns: first scale row of the group
  int n;              // rows or columns of the 128 that the tile uses (may be <= 0)
  int64_t bytes;      // rows: the array's length
  int pitch;          // rows: bytes (blocks) of a row; columns: width
  int c0;             // columns: first column
  int nb;             // blocks of the summed index
  int64_t tile0;      // tiled: index of the first 512-byte tile
  int words;          // words of the summed index
};

template <typename C>
__device__ __forceinline__ ScaleSrc scale_src(const GroupedGemmParams& p, const GemmSmem& m,
                                              const GemmTile& t, int group) {
  ScaleSrc r;
  const bool a = group == 0;
  r.s = a ? p.a_scales : p.b_scales;
  r.r0 = r.tile0 = r.bytes = 0;
  r.pitch = p.K >> 5;
  r.c0 = 0;
  r.nb = t.kb;
  if (C::kAmn) {
    r.r0 = m.pre[t.e];   // (wgrad: the scale rows before each group)
    r.pitch = a ? p.R : p.N;
    r.c0 = a ? (int)t.row0 : t.n0 + 128 * (group - 1);
    r.n = r.pitch - r.c0;
    // the group's [width, blocks] matrix starts at byte k0 / 32 * width
    r.tile0 = ((t.k0 >> 5) * r.pitch >> 9) +
              (int64_t)(min(r.c0, r.pitch - 1) >> 7) * (t.krows >> 7);
  } else if (a) {
    r.r0 = t.row0;
    r.n = t.rows;
    r.bytes = p.M * r.pitch;
  } else if (C::kBmn) {
    // W quantised as one [E K, N] matrix in blocks of 32 rows
    r.r0 = (int64_t)t.e * r.pitch;
    r.tile0 = r.r0 >> 2;
    r.c0 = t.n0 + 128 * (group - 1);
    r.tile0 += (int64_t)(min(r.c0, p.N - 1) >> 7) * (((int64_t)p.E * r.pitch) >> 2);
    r.pitch = p.N;
    r.n = p.N - r.c0;
  } else {
    r.r0 = (int64_t)t.e * p.N + t.n0 + 128 * (group - 1);
    r.n = p.N - t.n0 - 128 * (group - 1);
    r.bytes = (int64_t)p.E * p.N * r.pitch;
  }
  r.words = (t.kb + 3) >> 2;
  return r;
}

// `have` bytes (1 .. 4; 1 .. 16) and zeros to 4 (16).
__device__ __forceinline__ void copy4(uint32_t dst, const uint8_t* src, int have = 4) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(have)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have)
               : "memory");
}

// Starts the copies of words u .. of the warp's 128 rows into `raw` (those of
// the chunk that exist; rows that the tile does not use are left out as far as
// that is cheap: with every SM of a decoding step reading the scales of a few
// rows' neighbours too, the weights arrived a third slower).  Every lane
// arrives once on `bar`, with or after its copies.
template <int MODE, bool OUTER>
__device__ __forceinline__ void start_chunk(const ScaleSrc& c, const void* tmap, int box_rows,
                                            int u, int lane, unsigned char* raw, uint64_t* bar) {
  const int n = c.n > 0 ? min(kChunk, c.words - u) : 0;
  const uint32_t dst = smem_addr(raw);
  if constexpr (MODE == kCols || MODE == kRows16) {
    if (lane == 0) {
      // 32 block rows of 128 columns, or 32 bytes of up to 128 rows
      const int boxes = n == 0 ? 0
                        : MODE == kCols || box_rows == 128 ? 1 : (min(128, c.n) + 31) / 32;
      mbar_expect_tx(bar, boxes * (MODE == kCols ? 4096 : 32 * box_rows));
      for (int i = 0; i < boxes; ++i)
        tc::load_2d<1>(raw + 1024 * i, tmap, MODE == kCols ? c.c0 : 4 * u,
                       MODE == kCols ? (int)c.r0 + 4 * u : (int)c.r0 + 32 * i, smem_addr(bar));
      return;
    }
  } else if (MODE == kTiled && (OUTER || (c.r0 & 127) == 0)) {
    if (lane == 0) {   // the rows are a tile's: its words lie one after another
      const int64_t tile = OUTER ? c.tile0 : (c.r0 >> 7) * c.words;
      mbar_expect_tx(bar, 512 * n);
      // the buffer's last chunk may have come by cp.async (another group's rows)
      if constexpr (!OUTER) tc::fence_proxy_async();
      if (n > 0) bulk_load(raw, c.s + ((tile + u) << 9), 512 * n, bar);
      return;
    }
  } else {
    const int rows = n == 0 ? 0 : min(128, c.n);
    if constexpr (MODE == kFlat) {
      const int64_t at = c.r0 * c.pitch & ~(int64_t)15;
      const int all = (int)(c.r0 * c.pitch - at) + rows * c.pitch;
      const int64_t left = c.bytes - at;
      if (rows > 0)
        for (int t = 16 * lane; t < all; t += 512)
          copy16(dst + t, c.s + at + t, (int)min((int64_t)16, left - t));
    } else if constexpr (MODE == kTiled) {
      for (int i = lane; i < rows; i += 32) {
        const int64_t r = c.r0 + i;
        const uint8_t* a = c.s + (((r >> 7) * c.words + u) << 9) + ((r & 31) << 4) +
                           (((r >> 5) & 3) << 2);
        for (int k = 0; k < n; ++k)
          copy4(dst + 512 * k + 16 * (i & 31) + 4 * (i >> 5), a + 512 * k);
      }
    } else {
      // up to nine words a row, neighbouring lanes a row's (kRowsAny: aligned
      // words that hold its eight; of the array's last word the bytes that are
      // the array's)
      constexpr int kPer = MODE == kRowsAny ? 9 : 8;
      for (int t = lane; t < kPer * rows; t += 32) {
        const int r = t / kPer, i = t - kPer * r;
        const int64_t at = (((c.r0 + r) * c.pitch + 4 * u) & ~(int64_t)3) + 4 * i;
        if (i < n + kPer - 8 && at < c.bytes)
          copy4(dst + 36 * r + 4 * i, c.s + at, (int)min((int64_t)4, c.bytes - at));
      }
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
    return;
  }
  tc::arrive(bar);
}

// A piece of 128 words.  A's: row r's at byte 4 r (each warp reads its own
// 32).  B's: row 32 j + l's at byte 16 l + 4 j (a lane reads its four).
template <bool A>
__device__ __forceinline__ void put_rows(unsigned char* dst, int lane, uint32_t w0, uint32_t w1,
                                         uint32_t w2, uint32_t w3) {
  if constexpr (A) {
    uint32_t* d = reinterpret_cast<uint32_t*>(dst) + lane;
    d[0] = w0, d[32] = w1, d[64] = w2, d[96] = w3;
  } else {
    *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w0, w1, w2, w3);
  }
}
// The same from four blocks of columns 4 lane .. + 3: a 4 x 4 byte transpose;
// for B the words are stored in the order (k + lane / 2) mod 4, so that each
// store's 32 fall into different banks.
template <bool A>
__device__ __forceinline__ void put_cols(unsigned char* dst, int lane, uint32_t x0, uint32_t x1,
                                         uint32_t x2, uint32_t x3) {
  const uint32_t t0 = __byte_perm(x0, x1, 0x5140), t1 = __byte_perm(x2, x3, 0x5140);
  const uint32_t t2 = __byte_perm(x0, x1, 0x7362), t3 = __byte_perm(x2, x3, 0x7362);
  const uint32_t w0 = __byte_perm(t0, t1, 0x5410), w1 = __byte_perm(t0, t1, 0x7632);
  const uint32_t w2 = __byte_perm(t2, t3, 0x5410), w3 = __byte_perm(t2, t3, 0x7632);
  if constexpr (A) {
    *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w0, w1, w2, w3);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = (k + (lane >> 1)) & 3;
      const uint32_t v = j & 2 ? (j & 1 ? w3 : w2) : (j & 1 ? w1 : w0);
      *reinterpret_cast<uint32_t*>(dst + (4 * (lane & 7) + j) * 16 + (lane >> 3) * 4) = v;
    }
  }
}

// A chunk that has arrived: its words into the warp's pieces.
template <int MODE, bool A, int STRIDE>
__device__ __forceinline__ void put_chunk(int head, int pitch, int lane, const unsigned char* raw,
                                          unsigned char* sf) {
  const int n = head & 15, first = (head >> 4) & 15, left = (head >> 8) & 63;
  if constexpr (MODE == kTiled) {
    for (int i = 0; i < n; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(raw + 512 * i + 16 * lane);
      put_rows<A>(sf + STRIDE * i, lane, v.x, v.y, v.z, v.w);
    }
  } else if constexpr (MODE == kCols) {
    for (int i = 0; i < n; ++i) {
      const uint32_t* x = reinterpret_cast<const uint32_t*>(raw + 512 * i) + lane;
      put_cols<A>(sf + STRIDE * i, lane, x[0], x[32], x[64], x[96]);
    }
  } else if constexpr (MODE == kRowsAny || MODE == kFlat) {   // (and kRows4)
    int sh[4], at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 32 * j + lane;
      at[j] = MODE == kFlat ? first + r * pitch : 36 * r + ((first + r * pitch) & 3);
      sh[j] = 8 * (at[j] & 3);
      at[j] >>= 2;
    }
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      // bytes past the row's end are another row's: a NaN scale there would
      // meet the zeros of half an E2M1 step
      const int have = min(4, left - 4 * i);
      const uint32_t mask = have < 4 ? (1u << (8 * have)) - 1u : ~0u;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t* x = reinterpret_cast<const uint32_t*>(raw) + at[j] + i;
        w[j] = __funnelshift_r(x[0], x[1], sh[j]) & mask;
      }
      put_rows<A>(sf + STRIDE * i, lane, w[0], w[1], w[2], w[3]);
    }
  } else {
    for (int h = 0; 4 * h < n; ++h) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *reinterpret_cast<const uint4*>(raw + 32 * (32 * j + lane) + 16 * h);
      unsigned char* d = sf + STRIDE * 4 * h;
      put_rows<A>(d, lane, v[0].x, v[1].x, v[2].x, v[3].x);
      if (4 * h + 1 < n) put_rows<A>(d + STRIDE, lane, v[0].y, v[1].y, v[2].y, v[3].y);
      if (4 * h + 2 < n) put_rows<A>(d + 2 * STRIDE, lane, v[0].z, v[1].z, v[2].z, v[3].z);
      if (4 * h + 3 < n) put_rows<A>(d + 3 * STRIDE, lane, v[0].w, v[1].w, v[2].w, v[3].w);
    }
  }
}

__device__ __forceinline__ int scale_mode(bool outer, bool tiled, int pitch) {
  return tiled ? kTiled
         : outer ? kCols
         : (pitch & 15) == 0 ? kRows16
         : pitch <= 4 * kChunk ? kFlat
         : (pitch & 3) == 0 ? kRows4 : kRowsAny;
}
// Whether the copies go by a tensor map (else there is none).
__device__ __forceinline__ bool scales_by_map(int mode) { return mode == kRows16 || mode == kCols; }

// What put_chunk needs of a chunk of a group: its words (4 bits), the place of
// its first byte in the 16 or 4 bytes copied first (4 bits), the bytes of a row
// left from its first word on (kRowsAny, kFlat; at most 63).
template <typename C>
__device__ __forceinline__ int scale_head(const ScaleSrc& c, int u) {
  const int n = c.n > 0 ? min(kChunk, c.words - u) : 0;
  return n | ((int)(c.r0 * c.pitch & 15) << 4) | (min(63, c.pitch - 4 * u) << 8);
}

// Warp 10: the copies of every chunk of every group, kRawDepth ahead, with what
// the warps that take them need to know (so that they look up no tile).  (In a
// warp of its own: the setting up of a tile's copies -- a search for the
// group, 64-bit addresses, cold code -- took one to three thousand cycles out
// of the warps that feed tensor memory.)
template <typename C>
__device__ void gemm_scale_loader(const GroupedGemmParams& p, const GemmSmem& m,
                                  const void* tm_sa, const void* tm_sb, int tiles, int first,
                                  int step, int rank) {
  const int lane = threadIdx.x & 31;
  const int mode_a = scale_mode(C::kAmn, p.a_tiled, p.K >> 5);
  const int mode_b = scale_mode(C::kBmn, p.b_tiled, p.K >> 5);
  int buf = 0;
  uint32_t phase = 1;
  for (GemmWalk<C> w(p, first, step, tiles); !w.done(); w.next()) {
    const GemmTile t = w.tile(p, m, rank);
    const int words = (t.kb + 3) >> 2;
    for (int u = 0; u < words; u += kChunk) {
      if (!__all_sync(kFull, tc::sleep<tc::kSm>(m.raw_empty + buf, phase)) || gemm_aborted(m)) {
        gemm_abort(p, m);
        return;
      }
      if (lane == 0)
        m.head[4 * buf] = min(kChunk / C::kWords, (t.kb * 32 + C::kStageK - 1) / C::kStageK -
                                                      u / C::kWords);
#pragma unroll 1
      for (int g = 0; g < C::kGroups; ++g) {
        const ScaleSrc src = scale_src<C>(p, m, t, g);
        if (lane == 0) {
          m.head[4 * buf + 1 + g] = scale_head<C>(src, u);
          __threadfence_block();   // (an arrival by cp.async does not order it)
        }
        unsigned char* raw = m.raw + g * C::kRawGroupBytes + buf * kRawBytes;
        uint64_t* bar = m.raw_full + g * kRawDepth + buf;
        const int mode = g == 0 ? mode_a : mode_b;
        const void* tmap = g == 0 ? tm_sa : tm_sb;
        const int box = g == 0 ? C::kABox : 128;
        if constexpr (C::kBmn) {
          if (g > 0 || C::kAmn) {
            if (mode == kCols) start_chunk<kCols, true>(src, tmap, box, u, lane, raw, bar);
            else start_chunk<kTiled, true>(src, tmap, box, u, lane, raw, bar);
            continue;
          }
        }
        if constexpr (!C::kAmn) {
          switch (mode) {
            case kTiled: start_chunk<kTiled, false>(src, tmap, box, u, lane, raw, bar); break;
            case kRows16: start_chunk<kRows16, false>(src, tmap, box, u, lane, raw, bar); break;
            case kFlat: start_chunk<kFlat, false>(src, tmap, box, u, lane, raw, bar); break;
            case kRows4: start_chunk<kRows4, false>(src, tmap, box, u, lane, raw, bar); break;
            default: start_chunk<kRowsAny, false>(src, tmap, box, u, lane, raw, bar);
          }
        }
      }
      __syncwarp();
      if (++buf == kRawDepth) buf = 0, phase ^= 1;
    }
  }
  // the end: a chunk without stages
  if (!__all_sync(kFull, tc::sleep<tc::kSm>(m.raw_empty + buf, phase)) || gemm_aborted(m)) {
    gemm_abort(p, m);
    return;
  }
  if (lane == 0) m.head[4 * buf] = 0;
  for (int g = 0; g < C::kGroups; ++g) tc::arrive(m.raw_full + g * kRawDepth + buf);
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One of warps 4-7.  PUT: it puts group `group`'s (0: A's rows) words into
// pieces.  Tensor memory: lane l of quarter q, A's word of row 32 q + l in
// column q of four; B's column c, row 32 c + l's word in lane l of every
// quarter.
template <typename C, bool PUT, int MODE, bool A>
__device__ __forceinline__ void gemm_scales(const GroupedGemmParams& p, const GemmSmem& m,
                                            uint32_t tbase, int group) {
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
  const uint32_t dst0 = tbase + ((uint32_t)(32 * q) << 16) + (uint32_t)C::kSfCol;
  const uint32_t full0 = tc::leader_addr(m.full);
  constexpr int kStagesPerChunk = kChunk / C::kWords;
  constexpr int kStride = C::kGroups * 512;
  unsigned char* raw = m.raw + group * C::kRawGroupBytes;
  uint64_t* raw_full = m.raw_full + group * kRawDepth;
  int slot = 0;
  uint32_t phase = 1;   // a fresh barrier's preceding phase counts as complete
  uint32_t raw_phase = 0;
  const int pitch = p.K >> 5;
  auto serve = [&](int buf) {
    bool ok = __all_sync(kFull, tc::sleep<tc::kSm>(raw_full + buf, raw_phase));
    int stages = 0;
    if (ok) {
      stages = *reinterpret_cast<volatile int*>(m.head + 4 * buf);
      if constexpr (PUT)
        if (stages > 0)
          put_chunk<MODE, A, kStride>(*reinterpret_cast<volatile int*>(m.head + 4 * buf + 1 + group),
                                      pitch, lane, raw + buf * kRawBytes, m.sf + 512 * group);
    }
    __syncwarp();
    if (lane == 0) tc::arrive(m.raw_empty + buf);
    if (buf == kRawDepth - 1) raw_phase ^= 1;
    asm volatile("bar.sync 1, 128;" ::: "memory");   // the chunk is in its pieces
    // a stage's words are read before the wait for its slot, and the waits
    // spin: the chain from a free slot to its scales in tensor memory bounds
    // the rate of stages
    uint32_t wa[C::kWords];
    uint4 wb[C::kWords][C::kGroups - 1];
    auto read = [&](int s) {
#pragma unroll
      for (int i = 0; i < C::kWords; ++i) {
        const unsigned char* piece = m.sf + kStride * (s * C::kWords + i);
        wa[i] = *reinterpret_cast<const uint32_t*>(piece + 4 * (32 * q + lane));
#pragma unroll
        for (int k = 1; k < C::kGroups; ++k)
          wb[i][k - 1] = *reinterpret_cast<const uint4*>(piece + 512 * k + 16 * lane);
      }
    };
    if (stages > 0) read(0);
    for (int s = 0; s < stages; ++s) {
      ok = ok && __all_sync(kFull, tc::spin<C::kOrder>(m.empty + slot, phase));
      if (ok) {
        tc::fence_after();
        const uint32_t dst = dst0 + slot * C::kSfPitch;
#pragma unroll
        for (int i = 0; i < C::kWords; ++i) {
          tc::st1(dst + 4 * i + q, wa[i]);
#pragma unroll
          for (int k = 0; k < C::kGroups - 1; ++k)
            tc::st4(dst + 4 * C::kWords + C::kSfbCols * i + 4 * k, wb[i][k].x, wb[i][k].y,
                    wb[i][k].z, wb[i][k].w);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive_leader<C::kOrder>(full0 + 8 * slot);
      }
      if (s + 1 < stages) read(s + 1);
      if (++slot == C::kStages) slot = 0, phase ^= 1;
    }
    if (!ok || gemm_aborted(m)) {
      ok = false;
      gemm_abort(p, m);
    }
    // every warp has read the pieces; after an abort they leave together
    int gone;
    asm volatile("{ .reg .pred p, r; setp.ne.s32 p, %1, 0; bar.red.or.pred r, 2, 128, p; "
                 "selp.s32 %0, 1, 0, r; }" : "=r"(gone) : "r"((int)!ok) : "memory");
    return gone == 0 && stages > 0;
  };
  for (int buf = 0; serve(buf);)
    if (++buf == kRawDepth) buf = 0;
}

// The scale warp's role, fixed for the launch.
template <typename C>
__device__ __forceinline__ void gemm_scales_any(const GroupedGemmParams& p, const GemmSmem& m,
                                                uint32_t tbase, int group) {
#define MOEACT_SCALES(MODE, A) \
  gemm_scales<C, true, MODE, A>(p, m, tbase, group)
#define MOEACT_SCALES_OF(OUTER, TILED, A)                      \
  if constexpr (OUTER) {                                       \
    if (TILED) MOEACT_SCALES(kTiled, A);                       \
    else MOEACT_SCALES(kCols, A);                              \
  } else {                                                     \
    switch (scale_mode(false, TILED, p.K >> 5)) {              \
      case kTiled: MOEACT_SCALES(kTiled, A); break;            \
      case kRows16: MOEACT_SCALES(kRows16, A); break;          \
      case kFlat: MOEACT_SCALES(kFlat, A); break;              \
      default: MOEACT_SCALES(kRowsAny, A);                     \
    }                                                          \
  }
  if (group == 0) {
    MOEACT_SCALES_OF(C::kAmn, p.a_tiled, true)
  } else if (group < C::kGroups) {
    MOEACT_SCALES_OF(C::kBmn, p.b_tiled, false)
  } else {
    gemm_scales<C, false, kRows16, false>(p, m, tbase, 0);
  }
#undef MOEACT_SCALES_OF
#undef MOEACT_SCALES
}

// ------------------------------------------------------------ code tiles
// Warp 8.  wgrad: blocks of 32 rows of a group at any row.  The rows past the
// group's end are the next group's: they must not meet in the sum, and a zero
// times a NaN of theirs would not be zero, so they are zeros in both operands.
// A group's last block is therefore copied row by row, the rows past its end
// from past the array's, which read as zeros.  (A warp that cleared them after
// the copies had to release its stores to the other SM of a pair, which takes
// as long as all that the SM has under way: wgrad short 32.7 us for 28.8, wgrad
// train 443 for 441.  That block first of a tile's, on its way while the tile
// before is summed: 429 for 434, short 30 for 29.)
template <typename C>
__device__ __forceinline__ void gemm_copy_codes(const GroupedGemmParams& p, const GemmSmem& m,
                                                const void* tm_a, const void* tm_b,
                                                const void* tm_ra, const void* tm_rb, int tiles,
                                                int first, int step, int rank) {
  const uint32_t full0 = tc::leader_addr(m.full);
  int slot = 0;
  uint32_t phase = 1;
  for (GemmWalk<C> walk(p, first, step, tiles); !walk.done(); walk.next()) {
    const GemmTile tile = walk.tile(p, m, rank);
    const int stages = (tile.kb * 32 + C::kStageK - 1) / C::kStageK;
    const int col_b = tile.n0 + (C::kCG == 2 ? 128 * rank : 0);   // this SM's rows of B
    // B's first box row: of the summed index where that is outermost
    const int yb = C::kBmn ? tile.e * p.K : tile.e * p.N + col_b;
    const int rows_a = (tile.rows + C::kABox - 1) / C::kABox;
    for (int s = 0; s < stages; ++s) {
      if (!tc::spin<C::kOrder>(m.empty + slot, phase)) {
        gemm_abort(p, m);
        return;
      }
      unsigned char* da = m.stages + slot * C::kStageBytes;
      unsigned char* db = da + kTileBytes;
      const uint32_t bar = full0 + 8 * slot;
      const int blocks = min(4, tile.kb - 4 * s);
      const int na = C::kAmn ? blocks : rows_a, nb = C::kBmn ? blocks : 1;
      const uint32_t bytes = (uint32_t)(na * C::kABox + nb * C::kBBox) * 128u;
      if constexpr (C::kCG == 1)
        tc::arrive_tx(bar, bytes);
      else
        tc::arrive_tx_leader(bar, bytes);
      if constexpr (C::kWgrad) {
        const int row = (int)tile.k0 + 128 * s, left = tile.krows - 128 * s;
        for (int i = 0; 32 * (i + 1) <= left && i < 4; ++i) {
          tc::load_2d<C::kCG>(da + 4096 * i, tm_a, (int)tile.row0, row + 32 * i, bar);
          tc::load_2d<C::kCG>(db + 4096 * i, tm_b, col_b, row + 32 * i, bar);
        }
        if (left < 128 && (left & 31) != 0) {
          for (int j = left & ~31; j < ((left + 31) & ~31); ++j) {
            const int y = j < left ? row + j : (int)p.M;
            tc::load_2d<C::kCG>(da + 128 * j, tm_ra, (int)tile.row0, y, bar);
            tc::load_2d<C::kCG>(db + 128 * j, tm_rb, col_b, y, bar);
          }
        }
      } else {
        for (int i = 0; i < na; ++i)
          tc::load_2d<C::kCG>(da + i * C::kABox * 128, tm_a, 128 * s,
                              (int)tile.row0 + C::kABox * i, bar);
        for (int i = 0; i < nb; ++i)
          tc::load_2d<C::kCG>(db + i * C::kBBox * 128, tm_b, C::kBmn ? col_b : 128 * s,
                              yb + (C::kBmn ? 128 * s : 0) + C::kBBox * i, bar);
      }
      if (++slot == C::kStages) slot = 0, phase ^= 1;
    }
  }
}

// (One thread runs the loop: warp-wide votes and barriers in every stage cost 1 to
// 7% of products over short sums.)
template <typename C>
__device__ void gemm_producer(const GroupedGemmParams& p, const GemmSmem& m, const void* tm_a,
                              const void* tm_b, const void* tm_ra, const void* tm_rb, int tiles,
                              int first, int step, int rank) {
  if (tc::elect_one())
    gemm_copy_codes<C>(p, m, tm_a, tm_b, tm_ra, tm_rb, tiles, first, step, rank);
  __syncwarp();
}

// Steps of a sum of `mmas` that one accumulator takes.
template <typename C>
__device__ __forceinline__ int segment_steps(const GroupedGemmParams& p, int mmas) {
  return C::kLong || p.out32 ? kSegment : mmas;
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
  for (GemmWalk<C> walk(p, first, step, tiles); !walk.done(); walk.next()) {
    const int kb = C::kWgrad ? walk.tile(p, m, 0).kb : p.K >> 5;
    if (kb == 0) continue;
    const int mmas = (kb * 32 + C::kMmaK - 1) / C::kMmaK;
    const int segment = segment_steps<C>(p, mmas);
    for (int i1 = 0; i1 < mmas; i1 += segment, ++n) {
      // the tile (or segment) whose columns this one takes: the last but one,
      // or with overlapping accumulators the last
      const int w = n - (C::kOverlap ? 1 : 2);
      if (w >= 0 && !__all_sync(kFull, tc::spin<C::kOrder>(m.d_empty + (w & 1),
                                                              (uint32_t)(w >> 1) & 1u))) {
        if (leader) gemm_abort(p, m);
        return;
      }
      tc::fence_after();
      const uint32_t d = tbase + (uint32_t)((n & 1) * C::kAcc1);
      const int end = min(mmas, i1 + segment);
      for (int i0 = i1; i0 < end; i0 += 4) {
        if (!__all_sync(kFull, tc::spin<C::kDataOrder>(m.full + slot, phase))) {
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
            if (i0 + j < end) {
              const uint32_t id = C::kF4 ? (uint32_t)(j & 1) * 2 : (uint32_t)j;   // scale byte
              const int word = C::kF4 ? j >> 1 : 0;
              tc::mma<C::kCG, C::kF4>(d, ad + kStepA * j, bd + kStepB * j,
                                      kIdesc | (id << 4) | (id << 29), sf + 4 * word,
                                      sf + 4 * C::kWords + C::kSfbCols * word,
                                      i0 + j != i1 ? 1u : 0u);
            }
          tc::commit<C::kCG>(m.empty + slot);
        }
        __syncwarp();
        if (++slot == C::kStages) slot = 0, phase ^= 1;
      }
      if (leader) tc::commit<C::kCG>(m.d_full + (n & 1));
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------ epilogue
// 32 rows x 128 bytes from registers (thread t: row t, as eight 16-byte
// pieces) into the warp's staging, swizzled (piece c of row r at c ^ (r mod
// 8)), and from there to the output: whole pieces by one bulk tensor store,
// which clips rows and columns past the output's and leaves the warp free; a
// product's pieces with fewer rows by plain stores of whole row segments.
// `add` (fp32): to what the output holds, by a bulk tensor addition in the
// memory's own units, which gives the bits of the warps' additions
// (accumulating wgrad of 128 groups of 512 rows, 2048 x 1536: 682 us, floor
// 528; loads, adds and plain stores by the warps: 1,050).
template <bool WGRAD, bool OUT32>
__device__ __forceinline__ void store_piece(const GroupedGemmParams& p, const void* tm_out,
                                            unsigned char* stg, const uint4* v,
                                            int64_t row, int rows, int col, int e, int e_row,
                                            bool add, int lane) {
  constexpr int kPer = OUT32 ? 4 : 8;   // columns in 16 bytes
  if (lane == 0) tc::bulk_wait_read();   // the last store has read the staging
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) = v[c];
  if (WGRAD || rows == 32) {
    tc::fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      if constexpr (WGRAD) {
        if (OUT32 && add) tc::add_3d(tm_out, stg, col, e_row, e);
        else tc::store_3d(tm_out, stg, col, e_row, e);
      } else {
        if (OUT32 && add) tc::add_2d(tm_out, stg, col, (int)row);
        else tc::store_2d(tm_out, stg, col, (int)row);
      }
      tc::bulk_commit();
    }
    __syncwarp();
    return;
  }
  __syncwarp();
  const int c = lane & 7;
  const bool in = col + kPer * c < p.N;
  float4 o[OUT32 ? 8 : 1];   // what the output holds: one wait for all of it
  if constexpr (OUT32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = 4 * k + (lane >> 3);
      if (add && in && r < rows)
        o[k] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.out) +
                                                (row + r) * p.ldo + col + kPer * c);
    }
  }
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
        if (add)
          f = make_float4(__fadd_rn(o[k].x, f.x), __fadd_rn(o[k].y, f.y),
                          __fadd_rn(o[k].z, f.z), __fadd_rn(o[k].w, f.w));
        *dst = f;
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (row + r) * p.ldo + col +
                                  kPer * c) = w;
      }
    }
  }
  __syncwarp();
}

// A tile whose bf16 sums are in segments: adds each to the totals in tensor memory
// and gives the last's, rounded, to put(values, column).  n: the accumulators
// used so far.  (Kernels of their own have it: in those for short sums it cost
// every call, gemm4 decode 22.6 -> 24.6 us.)
template <typename C, typename Put>
__device__ __forceinline__ bool gemm_long_tile(const GroupedGemmParams& p, const GemmSmem& m,
                                               uint32_t tbase, int mmas, int& n, const Put& put) {
  const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t quarter = tbase + ((uint32_t)(32 * q) << 16);
  for (int i = 0; i < mmas; i += kSegment, ++n) {
    const int b = n & 1;
    if (!__all_sync(kFull, tc::sleep<C::kOrder>(m.d_full + b, (uint32_t)(n >> 1) & 1u)) ||
        gemm_aborted(m)) {
      gemm_abort(p, m);
      return false;
    }
    tc::fence_after();
    const bool first = i == 0, last = i + kSegment >= mmas;
#pragma unroll 1
    for (int c = 0; c < C::kBN; c += 64) {
      uint4 w[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32], t[32];
        tc::ld32(quarter + b * C::kAcc1 + c + 32 * h, v);
        if (!first) tc::ld32(quarter + C::kTotal + c + 32 * h, t);
        tc::wait_ld();
        tc::tie(v);
        if (!first) {
          tc::tie(t);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j] = __float_as_uint(__fadd_rn(__uint_as_float(t[j]), __uint_as_float(v[j])));
        }
        if (!last) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            tc::st4(quarter + C::kTotal + c + 32 * h + j, v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        uint32_t* x = reinterpret_cast<uint32_t*>(w) + 16 * h;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          x[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
      }
      tc::wait_st();
      if (last) put(w, c);
    }
    tc::fence_before();
    __syncwarp();
    if (lane == 0) tc::arrive_leader<C::kOrder>(tc::leader_addr(m.d_empty) + 8 * b);
  }
  return true;
}

template <typename C>
__device__ void gemm_epilogue(const GroupedGemmParams& p, const GemmSmem& m, const void* tm_out,
                              uint32_t tbase, int tiles, int first, int step, int rank,
                              int set) {
  const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  unsigned char* stg = m.epi + (4 * set + q) * kPieceBytes;
  constexpr int kChunks = C::kBN / 64 / C::kSets;   // of 64 columns, of this set
  const uint32_t d_empty = tc::leader_addr(m.d_empty);
  int n = 0;
  for (GemmWalk<C> walk(p, first, step, tiles); !walk.done(); walk.next()) {
    const GemmTile tile = walk.tile(p, m, rank);
    const int rows = max(0, min(32, tile.rows - 32 * q));
    const int e_row = (int)tile.row0 + 32 * q;   // row of A, or (wgrad) of dW_e
    const int64_t row = (C::kWgrad ? (int64_t)tile.e * p.R : 0) + e_row;
    const int mmas = (tile.kb * 32 + C::kMmaK - 1) / C::kMmaK;
    const int segments = p.out32 ? (mmas + kSegment - 1) / kSegment : 1;
    bool add = p.accumulate;
    auto put = [&](auto out32, const uint4* v, int col) {
      store_piece<C::kWgrad, decltype(out32)::value>(p, tm_out, stg, v, row, rows, col, tile.e,
                                                     e_row, add, lane);
    };
    using Bf16 = std::integral_constant<bool, false>;
    using Fp32 = std::integral_constant<bool, true>;
    if (tile.kb == 0) {   // wgrad of an expert without rows: zeros
      if (p.accumulate || rows == 0) continue;
      uint4 z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = make_uint4(0u, 0u, 0u, 0u);
      const int per = p.out32 ? 32 : 64;
      const int c0 = tile.n0 + 64 * kChunks * set;
      for (int c = c0; c < min(c0 + 64 * kChunks, p.N); c += per) {
        if (p.out32) put(Fp32(), z, c);
        else put(Bf16(), z, c);
      }
      continue;
    }
    if constexpr (C::kLong) {
      if (!gemm_long_tile<C>(p, m, tbase, mmas, n, [&](const uint4* w, int c) {
            if (tile.n0 + c < p.N && rows > 0) put(Bf16(), w, tile.n0 + c);
          }))
        return;
    } else for (int seg = 0; seg < segments; ++seg, ++n, add = true) {   // (not compiled otherwise)
      if (seg && lane == 0) tc::bulk_wait();   // the stores that it adds to are done
      const int b = n & 1;
      if (!__all_sync(kFull, tc::sleep<C::kOrder>(m.d_full + b, (uint32_t)(n >> 1) & 1u)) ||
          gemm_aborted(m)) {
        gemm_abort(p, m);
        return;
      }
      tc::fence_after();
      const uint32_t src = tbase + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * C::kAcc1);
      // The overlapping columns first: the first accumulator's last chunks, the
      // second one's first.  The columns may be overwritten by the tile after the
      // next once they are read here, and by the next one's where they overlap: a
      // set without overlapping columns only says that it is through with the
      // tile before this one.
      constexpr int kOver = C::kOverlap / 64;
      const bool over = C::kSets == 1 || (b == 0) == (set == 1);
      auto release = [&]() {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive_leader<C::kOrder>(d_empty + 8 * b);
      };
      if (!over) release();
#pragma unroll 1
      for (int i = 0; i < kChunks; ++i) {
        const int c = kChunks * set +
                      (kOver && b == 0 && over ? (i + kChunks - kOver) % kChunks : i);
        uint32_t v[64];
        tc::ld32(src + 64 * c, v);
        tc::ld32(src + 64 * c + 32, v + 32);
        tc::wait_ld();
        tc::tie(v);
        tc::tie(v + 32);
        if (over && i == (kOver ? kOver : kChunks) - 1) release();
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
            if (col + 32 * h < p.N) put(Fp32(), w, col + 32 * h);
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
          put(Bf16(), w, col);
        }
      }
    }
  }
  if (lane == 0) tc::bulk_wait();   // the stores are out before the memory is given up
  __syncwarp();
}

// ------------------------------------------------------------ kernel
template <int OP, GemmForm FORM>
__global__ void __launch_bounds__(GemmCfg<OP, FORM>::kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,
                        const __grid_constant__ CUtensorMap tm_b,
                        const __grid_constant__ CUtensorMap tm_sa,
                        const __grid_constant__ CUtensorMap tm_sb,
                        const __grid_constant__ CUtensorMap tm_out,
                        const __grid_constant__ CUtensorMap tm_ra,
                        const __grid_constant__ CUtensorMap tm_rb, const GroupedGemmParams p) {
  using C = GemmCfg<OP, FORM>;
  constexpr bool PAIR = C::PAIR;
  if (p.noop != nullptr && *p.noop != 0) return;
  extern __shared__ __align__(1024) unsigned char gemm_smem[];
  unsigned char* base = gemm_smem + ((1024u - (smem_addr(gemm_smem) & 1023u)) & 1023u);
  GemmSmem m;
  m.stages = base;
  m.epi = base + C::kStages * C::kStageBytes;
  m.sf = m.epi + 4 * C::kSets * kPieceBytes;
  m.raw = m.sf + C::kSfBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(m.raw + C::kGroups * C::kRawGroupBytes);
  m.full = bars;
  m.empty = m.full + C::kStages;
  m.raw_full = m.empty + C::kStages;
  m.raw_empty = m.raw_full + C::kGroups * kRawDepth;
  m.d_full = m.raw_empty + kRawDepth;
  m.d_empty = m.d_full + 2;
  m.misc = reinterpret_cast<int*>(bars + 64);
  m.head = m.misc + 4;
  m.scan = m.misc + 16;
  m.pre = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(bars) + kGemmMisc);
  m.ro = p.E <= kGroupsInSmem ? m.pre + p.E + 1 : nullptr;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {   // only the maps that the host has encoded: those that copies will use
    if (p.M > 0) {
      tc::prefetch_map(&tm_a);
      tc::prefetch_map(&tm_b);
      if (C::kWgrad) tc::prefetch_map(&tm_ra), tc::prefetch_map(&tm_rb);
      if (scales_by_map(scale_mode(C::kAmn, p.a_tiled, p.K >> 5))) tc::prefetch_map(&tm_sa);
      if (scales_by_map(scale_mode(C::kBmn, p.b_tiled, p.K >> 5))) tc::prefetch_map(&tm_sb);
    }
    tc::prefetch_map(&tm_out);
  }
  const int rank = PAIR ? (int)tc::cluster_rank() : 0;

  // ---- the groups: offsets checked, row tiles before each expert
  const int E = p.E;
  const int per = (E + C::kThreads - 1) / C::kThreads;
  const int e_lo = min(E, tid * per), e_hi = min(E, e_lo + per);
  int local = 0, bad = 0;
  for (int e = e_lo; e < e_hi; ++e) {
    const int64_t r0 = p.row_offs[e], r1 = p.row_offs[e + 1];
    if (m.ro != nullptr) {
      m.ro[e] = (int)r0;
      m.ro[e + 1] = (int)r1;   // (the next thread's first writes the same)
    }
    if (r1 < r0 || r0 < 0 || r1 > p.M) bad |= 1;
    else local += (int)((r1 - r0 + C::kTM - 1) / C::kTM);
    if constexpr (C::kWgrad) {
      m.pre[e] = (int)p.cb_offs[e];
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
  for (int w = 0; w < C::kThreads / 32; ++w) {
    const int v = m.scan[w];
    if (w < warp) before += v;
    total += v;
  }
  if constexpr (!C::kWgrad) {
    for (int e = e_lo; e < e_hi; ++e) {
      m.pre[e] = before;
      before += (int)((p.row_offs[e + 1] - p.row_offs[e] + C::kTM - 1) / C::kTM);
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
      mbar_init(m.full + i, 5 * C::kCG);   // per SM: warp 8 and four scale warps
      mbar_init(m.empty + i, 1);
    }
    for (int i = 0; i < C::kGroups * kRawDepth; ++i) mbar_init(m.raw_full + i, 32);
    for (int i = 0; i < kRawDepth; ++i) mbar_init(m.raw_empty + i, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(m.d_full + i, 1);
      mbar_init(m.d_empty + i, 4 * C::kSets * C::kCG);
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

  if (warp < 4 || warp >= 12)
    gemm_epilogue<C>(p, m, &tm_out, tbase, tiles, first, step, rank, warp >= 12);
  else if (warp < 8) gemm_scales_any<C>(p, m, tbase, warp - 4);
  else if (warp == 8) gemm_producer<C>(p, m, &tm_a, &tm_b, &tm_ra, &tm_rb, tiles, first, step, rank);
  else if (warp == 10) gemm_scale_loader<C>(p, m, &tm_sa, &tm_sb, tiles, first, step, rank);
  else if (warp == 9 && rank == 0) gemm_mma<C>(p, m, tbase, tiles, first, step);

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

template <int OP, GemmForm FORM>
int gemm_smem_bytes(int E) {
  using C = GemmCfg<OP, FORM>;
  return 1024 + C::kFixed + group_bytes_gemm(E);
}

template <int OP, GemmForm FORM>
cudaError_t gemm_prepare_one(int max_groups) {
  return cudaFuncSetAttribute(grouped_gemm_kernel<OP, FORM>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              std::max(gemm_smem_bytes<OP, FORM>(max_groups),
                                       gemm_smem_bytes<OP, FORM>(kGroupsInSmem)));
}

template <int OP, GemmForm FORM>
cudaError_t gemm_launch_one(const GroupedGemmParams& p, const GemmMaps& tm, int n_sms,
                            cudaStream_t stream) {
  using C = GemmCfg<OP, FORM>;
  // at most as many row tiles as full ones and one more per group
  const int64_t row_tiles = C::kWgrad ? (int64_t)p.E * ((p.R + C::kTM - 1) / C::kTM)
                                      : p.M / C::kTM + (p.E < p.M ? p.E : p.M);
  const int64_t tiles = row_tiles * ((p.N + C::kBN - 1) / C::kBN);
  const int64_t most = n_sms / C::kCG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * C::kCG));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = gemm_smem_bytes<OP, FORM>(p.E);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C::kCG;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, grouped_gemm_kernel<OP, FORM>, tm.a, tm.b, tm.sa, tm.sb, tm.out,
                            tm.ra, tm.rb, p);
}

}  // namespace
}  // namespace moeact

// Defines one operator's prepare and launch functions.
#define MOEACT_DEFINE_GEMM_UNIT(name, OP)                                                       \
  namespace moeact {                                                                            \
  cudaError_t grouped_gemm_prepare_##name() {                                                   \
    cudaError_t e = gemm_prepare_one<OP, kGemmSingle>(MOEACT_MAX_GROUPS);                       \
    if (e == cudaSuccess) e = gemm_prepare_one<OP, kGemmPair>(MOEACT_MAX_GROUPS);               \
    return e != cudaSuccess ? e : gemm_prepare_one<OP, kGemmLong>(MOEACT_MAX_GROUPS);           \
  }                                                                                             \
  cudaError_t grouped_gemm_launch_##name(GemmForm form, const GroupedGemmParams& p,             \
                                         const GemmMaps& tm, int n_sms, cudaStream_t stream) {  \
    return form == kGemmPair   ? gemm_launch_one<OP, kGemmPair>(p, tm, n_sms, stream)           \
           : form == kGemmLong ? gemm_launch_one<OP, kGemmLong>(p, tm, n_sms, stream)           \
                               : gemm_launch_one<OP, kGemmSingle>(p, tm, n_sms, stream);        \
  }                                                                                             \
  }
