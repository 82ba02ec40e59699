// Attention over a 4-bit KV block store (nosa_quant_dense_attend, nosa_quant_attend).
//
// With K^ = n s + m (codes n, a scale s and a minimum m per token and group of 32 dims; quant_core.cuh),
//   q . K^_t = sum_gr s_{t,gr} (q_gr . n_{t,gr}) + sum_gr m_{t,gr} sum(q_gr)
//   sum_t p_t V^_t = sum_t (p_t s_{t,gr}) n_{t,gr} + sum_t p_t m_{t,gr}
// so codes enter the tensor cores without being turned into values: a masked code in the low mantissa bits of
// an f16 is the subnormal n 2^-24 (n 2^-20 four bits further up, which the other operand or the result makes
// good by an exact 2^-4): five instructions for eight codes.  The other terms are one more MMA each: the row
// sums of q, split into two f16, against the K minima, and a 16-row operand of V's minima with a row of ones that
// yields the softmax sum too.
//
// grid (quant_plan): one wave of CTAs; the units' blocks in one line are cut into equal pieces, one per CTA, so that
// ragged lengths balance, or a cluster of CTAs takes a unit.  A warp takes half (two tiles of 16 tokens) of every
// second block or so through a ring of its own of bulk copies to shared memory, so that no warp waits for another;
// per tile (mma.sync m16n8k16, f16 in, fp32 accumulate; with at most 32 rows a unit tcgen05's tiles of 64 rows and
// more would be mostly empty, and the codes would have to be written out as f16 to shared memory first):
//   S^T (16 tokens x 8 rows) = K codes . q^T        8 MMAs, one accumulator per group, + 1 for m
//   P^T by movmatrix of the f16-packed weights, times s per group
//   O^T (128 dims x 8 rows) += V codes^T . P^T       8 MMAs, + 1 for m and the sum
// The query rows of a unit (q heads x query tokens, at most 32) are NT tiles of 8.  Weights are 2^(logit - R): R
// follows a row's maximum only when that would get a weight above 2^14, so the usual tile needs no rescaling; where a
// scale of 2 or more could take weight x s out of f16, all of a warp's weights shrink by a power of two for good.  A CTA
// merges its warps in shared memory; a unit's parts, where several CTAs share it, merge through the cluster or in a
// second kernel.  Weights, their products with s and the maxima of every second tile are f16 because the tensor cores
// take them so; scores, sums and references are float32.  Against 64 bits results are off by 0.0017 to 0.0018 (root mean
// square, relative), by 0.0016 to 0.0017 with everything in float32: the rest is the result's rounding to bf16.
//
// Bound by HBM where a call is long: 256 units of 32,768 tokens and 4 rows (1.34 GB) in 199 us, 1.00 of measured HBM.
// A tile takes 276 instructions with one row tile, at 16 warps an SM about the time of its 2,560 bytes, so shorter calls
// pay for their start and end: 256 units listing 81 blocks (212 MB) 43.0 us, 0.74.  With two row tiles 317 instructions:
// 16 units of 65,521 tokens and 16 rows 45.8 us against 25 of HBM.  With four 566, 76 of them MMAs: the same and 32 rows
// 85.0 us against 25 of HBM and 33 of the tensor pipe.
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "host.h"
#include "quant_core.cuh"

namespace nosa {

namespace cg = cooperative_groups;

constexpr int kMergeWarps = 8;
constexpr int kStageTokens = 32, kStageBytes4 = 2 * kTileBytes;
constexpr int kQaSplitUnits = 2048;   // beyond, one CTA per unit
constexpr int kQaList = 256;          // listed blocks looked up at a time
constexpr int kQaMaxRows = 32;
constexpr int kQaRowStride = 132;     // floats per row of a warp's partial in shared memory (no bank conflicts)
constexpr size_t kQaErrBytes = 256;   // the scratch starts with the device error word
constexpr float kNoRef = -3e38f;      // reference of a row that has seen no token

// Half blocks in flight per worker.  A pair of warps frees a stage one late.
__host__ __device__ constexpr int stages(int nt) { return nt == 4 ? 3 : 2; }

// Shared memory of the rings of n workers, which their partials (nt row tiles) reuse.
__host__ __device__ constexpr int quant_ring_bytes(int nt, int n) {
  const int ring = n * stages(nt) * kStageBytes4, partials = n * 8 * nt * kQaRowStride * 4;
  return ring > partials ? ring : partials;
}

enum { kWhole, kPieces, kCluster };

struct QuantArgs {
  const uint16_t* q;
  const uint8_t* store;
  const int32_t* sel;       // null: every block (dense)
  const int32_t* sel_slot;  // null: row b holds block b
  const int32_t* lens;
  uint16_t* out;
  int* err;
  int2* meta;     // [unit]: its first part and how many there are (1: the output is written already)
  float2* stats;  // [part][row]: reference and softmax sum
  float* part;    // [part][row][128]
  int units, nq, rows, max_blocks, max_sel, max_len;
  int split;      // kWhole: one CTA per unit, kPieces: equal pieces of all units' blocks, kCluster: a cluster per unit
  float scale;    // softmax scale x log2(e)
  long long wait_limit;  // SM cycles a wait for a staged half block may take before it gives up (< 0: none)
};

// D (16 x 8, f32) += A (16 x 16, row) . B (16 x 8, col), f16 inputs.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with D = A . B: a zero operand costs nothing, a zeroed accumulator four moves.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D (16 x 8, f32) = A (16 x 8, row) . B (8 x 8, col), f16 inputs.
__device__ __forceinline__ void mma_f16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};\n"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {
  const __half2 v = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t at_least_2(uint32_t a) {  // a mask of the halves that are 2 or more
  return __hge2_mask(*reinterpret_cast<const __half2*>(&a), __half2half2(__ushort_as_half((unsigned short)0x4000)));
}
__device__ __forceinline__ float half_lo(uint32_t a) { return __low2float(*reinterpret_cast<const __half2*>(&a)); }
__device__ __forceinline__ float half_hi(uint32_t a) { return __high2float(*reinterpret_cast<const __half2*>(&a)); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// The query rows of one tile of 8 as MMA operands, and the factors that undo their scaling.
struct QueryTile {
  uint32_t b[8][2];  // [2 group + half]: dims 32 gr + 8 t + {0,4}, {1,5} 2^-4 | {2,6}, {3,7} 2^-4 of row g
  uint32_t sums;     // t = 0, 1: high halves of the sums of groups 2t, 2t + 1; t = 2, 3: the low halves
};

// Rows 8 nt + g of q: scaled by a power of two that brings the row's largest magnitude into [2^9, 2^10)
// (bf16 values down to 2^-22 of it stay exact in f16, those of odd dims a sixteenth of their size among its subnormals,
// and a group's sum stays in range).
// alpha: the factors that turn the scores of rows 2t, 2t + 1, which are counted in 2^-24 / unit, into logits in base 2.
__device__ __forceinline__ void load_query(QueryTile& Q, float (&alpha)[2], const uint16_t* q, int row, int rows, int lane,
                                           float scale, float unit) {
  const int t = lane & 3;
  uint4 x[4];
  uint32_t big = 0;  // the largest magnitude's bf16 bits
#pragma unroll
  for (int gr = 0; gr < 4; ++gr) {
    x[gr] = row < rows ? *reinterpret_cast<const uint4*>(q + (size_t)row * kHeadDim + 32 * gr + 8 * t) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {x[gr].x, x[gr].y, x[gr].z, x[gr].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) big = max(big, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  }
  big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
  // 2^(9 - e) for the exponent e of the largest value; 1 where the row is zero or not finite
  const int e = (int)(big >> 7) - 127;
  const int shift = big == 0 || big >= 0x7f80u ? 0 : min(9 - e, 126);
  const float f = __uint_as_float((uint32_t)(127 + shift) << 23), inv = __uint_as_float((uint32_t)(127 - shift) << 23);
  float sum[4];
#pragma unroll
  for (int gr = 0; gr < 4; ++gr) {
    const uint32_t w[4] = {x[gr].x, x[gr].y, x[gr].z, x[gr].w};
    float v[8];
    sum[gr] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = bf16_to_float((uint16_t)(w[i >> 1] >> (16 * (i & 1)))) * f;
      sum[gr] += v[i];
    }
    Q.b[2 * gr][0] = pack_half2(v[0], v[4]);
    Q.b[2 * gr][1] = pack_half2(v[1] * 0.0625f, v[5] * 0.0625f);
    Q.b[2 * gr + 1][0] = pack_half2(v[2], v[6]);
    Q.b[2 * gr + 1][1] = pack_half2(v[3] * 0.0625f, v[7] * 0.0625f);
    sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
    sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
  }
  const uint32_t h01 = pack_half2(sum[0], sum[1]), h23 = pack_half2(sum[2], sum[3]);
  const uint32_t l01 = pack_half2(sum[0] - half_lo(h01), sum[1] - half_hi(h01));
  const uint32_t l23 = pack_half2(sum[2] - half_lo(h23), sum[3] - half_hi(h23));
  Q.sums = t == 0 ? h01 : t == 1 ? h23 : t == 2 ? l01 : l23;
  // Kept away from zero and infinity.  128 products of a q below 2^10 and an x^ below 2^20 make a score below 2^37, and
  // any two differ by 2^-48 (f16's smallest steps) or not at all: below 2^-100 all weights are equal, and from 2^77 on any
  // score but the largest has none, while score x alpha stays within float32.
  const float most = 0x1p77f * (0x1p24f / unit);
  scale *= 0x1p24f / unit;
  alpha[0] = fminf(fmaxf(scale * __shfl_sync(0xffffffffu, inv, 8 * t), 0x1p-100f), most);  // row 2t's lanes: 8t ..
  alpha[1] = fminf(fmaxf(scale * __shfl_sync(0xffffffffu, inv, 8 * t + 4), 0x1p-100f), most);
}

// One warp's running state for a tile of 8 rows: of rows 2t, 2t + 1 the score that has the largest weight allowed, 2^lift
// (a score z has 2^((z - top) alpha + lift), so that a huge score less itself is zero; lift is the warp's, 14 until a V
// scale of 2 or more calls for less, and no part of top, where a huge score would swallow it); O^T (codes' part, in
// units of 2^-24, or 2^-20 for odd dims); and the minima's part: rows 0..3 the groups, row 4 the softmax sum,
// rows 8..11 the groups' maxima that enter as sixteenths.  A warp of a pair (process_pair) holds half the dims: GR = 2 groups.
constexpr float kTopWeight = 14.f;  // lift at the start
template <int GR>
struct RowTile {
  float top[2];
  float o[2 * GR][4];
  float c[4];
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The V side of a tile as a lane holds it, GR groups from group g0 on: codes and scales of token pairs t, t + 4, and the
// rows of the operand that goes with the weights alone: row g group g0 + g's minimum (g < GR), row 4 ones (the softmax
// sum).
//
// flip (all ones in a stage's second tile, else zero): the tile enters as -(15 - n) s and m + 15 s, its codes
// complemented, its products negated and its maxima in the place of the minima.  Sums over codes of 0 .. 15 and over
// minima alone would each be far larger than their total, and so would the rounding of long sums, which the tensor
// cores cut off rather than round; with tiles taken from either end the sums stay near their totals.  (Taking 8 off each
// code did the same for 3 to 7 % more time.)  A maximum with a scale of 2 or more, which may lie beyond f16, enters as its
// sixteenth in row 8 + g instead (there the subnormals' step, 2^-24, is nothing against s; for smaller scales it could be
// as large as the values).  large: the stage may have such a scale.  The single warps ask first, which saves them 1 %; the
// pairs, which that branch would cost 4 %, always say yes.
template <int GR>
struct ValueRegs {
  uint32_t c[2][GR], s[2][GR], m[2], m16[2];
};
template <int GR>
__device__ __forceinline__ void load_words(uint32_t (&w)[GR], const unsigned char* p) {
  if constexpr (GR == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}
template <int GR>
__device__ __forceinline__ void load_values(ValueRegs<GR>& V, const unsigned char* tile, int g0, uint32_t flip, bool large,
                                            int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_words<GR>(V.c[h], tile + kTileV + 512 * h + 16 * lane + 4 * g0);
    load_words<GR>(V.s[h], tile + kTileVs + 16 * (4 * h + t) + 4 * g0);
    const unsigned char* w = tile + kTileVs + 16 * (4 * h + t) + 4 * (g0 + (g & (GR - 1)));
    uint32_t m = *reinterpret_cast<const uint32_t*>(w + kTileVm - kTileVs);
    const uint32_t keep = g < GR ? 0xffffffffu : 0u, ones = g == 4 ? 0x3C003C00u : 0u;
    uint32_t m16 = 0;
    if (flip) {
      const uint32_t s = *reinterpret_cast<const uint32_t*>(w);
      if (large) {
        const uint32_t big = at_least_2(s);
        m16 = fma_half2(s, 0x3B803B80u, mul_half2(m, 0x2C002C00u)) & big;  // 15 s / 16 + m / 16
        m = fma_half2(s, 0x4B804B80u, m) & ~big;
      } else {
        m = fma_half2(s, 0x4B804B80u, m);
      }
    }
    V.m[h] = (m & keep) | ones;
    V.m16[h] = m16 & keep;
  }
}

// O^T += V^T . P^T for NT row tiles; p[nt][h] = weights of row g, token pair t + 4 h, as f16x2.
template <int NT, int GR>
__device__ __forceinline__ void add_values(RowTile<GR> (&A)[NT], const ValueRegs<GR>& V, uint32_t flip, const uint32_t (&p)[NT][2]) {
  const uint32_t sign = flip & 0x80008000u;
#pragma unroll
  for (int gr = 0; gr < GR; ++gr) {
    const uint32_t w0 = V.c[0][gr], w1 = V.c[1][gr], x0 = w0 >> 8, x1 = w1 >> 8;
    const uint32_t a[8] = {(w0 ^ flip) & 0x000F000Fu, (w0 ^ flip) & 0x00F000F0u, (w1 ^ flip) & 0x000F000Fu, (w1 ^ flip) & 0x00F000F0u,
                           (x0 ^ flip) & 0x000F000Fu, (x0 ^ flip) & 0x00F000F0u, (x1 ^ flip) & 0x000F000Fu, (x1 ^ flip) & 0x00F000F0u};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t b0 = mul_half2(p[nt][0] ^ sign, V.s[0][gr]), b1 = mul_half2(p[nt][1] ^ sign, V.s[1][gr]);
      mma_f16(A[nt].o[2 * gr], a[0], a[1], a[2], a[3], b0, b1);
      mma_f16(A[nt].o[2 * gr + 1], a[4], a[5], a[6], a[7], b0, b1);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) mma_f16(A[nt].c, V.m[0], V.m16[0], V.m[1], V.m16[1], p[nt][0], p[nt][1]);
}

// Prepares a tile that not every row sees as a whole (left: tokens of the context from its first on, possibly none).
// Behind the context the store may hold anything, and 0 x NaN is a NaN, so those tokens' V scales and minima are
// cleared (codes are finite as they stand).  So is a NaN group of a token that only some rows see: the rows that see
// it get a bit of `poison`, and their dims of that group a NaN in the end.
__device__ __forceinline__ void clear_tail(unsigned char* tile, int* poison, int left, int nq, int rows, int lane) {
#pragma unroll 1
  for (int i = lane; i < kTileTokens / 2 * 8; i += 32) {  // [s, m][token pair][group] words of two tokens
    uint32_t* w = reinterpret_cast<uint32_t*>(tile + kTileVs) + i;
    uint32_t x = *w;
#pragma unroll 1
    for (int par = 0; par < 2; ++par) {
      const int late = 2 * ((i >> 2) & 7) + par - (left - nq);  // rows of query tokens from `late` on see the token
      const uint32_t mask = par ? 0xffff0000u : 0x0000ffffu;
      if (late >= nq) {
        x &= ~mask;
      } else if (late > 0 && (x & mask & 0x7c007c00u) == (mask & 0x7c007c00u)) {
        x &= ~mask;
        for (int row = 0; row < rows; ++row)
          if (row % nq >= late) atomicOr(&poison[row], 1 << (i & 3));
      }
    }
    *w = x;
  }
  fence_proxy_async_smem();  // the next bulk copy into the stage comes after these writes
  __syncwarp();
}

// The query side in shared memory, for more than one row tile (registers hold it for one).
struct QueryShared {
  uint4 b[4][32];    // [group][lane]: QueryTile::b of the group
  uint32_t sums[32];
  float2 alpha[32];
};

// The 2^24 that the codes lack go into the K scales (8 products a tile), or for one row tile into alpha and, the
// other way, into the m part (4).
__host__ __device__ constexpr float code_unit(int nt) { return nt == 1 ? 1.f : 0x1p24f; }

// Scores of kTiles tiles from `tile0` on for all row tiles: z[tile][row tile] of tokens g, g + 8 and rows 2t, 2t + 1.
// A token that a row does not see (left: tokens of the context from the first tile's first on) gets -inf.
template <int NT, int kTiles>
__device__ __forceinline__ void score_tiles(float (&z)[kTiles][NT][4], const QueryTile& Q, const QueryShared* qs,
                                            const unsigned char* tile0, bool tail, int left, int nq, int rows, int lane) {
  constexpr float kCodeUnit = code_unit(NT);
  const int g = lane >> 2, t = lane & 3;
  float ks[kTiles][2][4];
  uint4 kc[kTiles][2];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const unsigned char* tile = tile0 + i * kTileBytes;
    uint32_t km[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kc[i][h] = *reinterpret_cast<const uint4*>(tile + 64 * (g + 8 * h) + 16 * t);
      const uint2 s = *reinterpret_cast<const uint2*>(tile + kTileKs + 16 * (g + 8 * h));
      km[h] = *reinterpret_cast<const uint32_t*>(tile + kTileKs + 16 * (g + 8 * h) + 8 + 4 * (t & 1));
      ks[i][h][0] = half_lo(s.x) * kCodeUnit;
      ks[i][h][1] = half_hi(s.x) * kCodeUnit;
      ks[i][h][2] = half_lo(s.y) * kCodeUnit;
      ks[i][h][3] = half_hi(s.y) * kCodeUnit;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_f16_k8(z[i][nt], km[0], km[1], NT == 1 ? Q.sums : qs[nt].sums[lane]);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[i][nt][e] *= 0x1p-24f * kCodeUnit;
    }
  }
#pragma unroll
  for (int gr = 0; gr < 4; ++gr) {
    uint32_t a[kTiles][8];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint32_t w0 = word(kc[i][0], gr), w1 = word(kc[i][1], gr), x0 = w0 >> 8, x1 = w1 >> 8;
      a[i][0] = w0 & 0x000F000Fu;
      a[i][1] = w1 & 0x000F000Fu;
      a[i][2] = w0 & 0x00F000F0u;
      a[i][3] = w1 & 0x00F000F0u;
      a[i][4] = x0 & 0x000F000Fu;
      a[i][5] = x1 & 0x000F000Fu;
      a[i][6] = x0 & 0x00F000F0u;
      a[i][7] = x1 & 0x00F000F0u;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint4 b;
      if constexpr (NT == 1)
        b = make_uint4(Q.b[2 * gr][0], Q.b[2 * gr][1], Q.b[2 * gr + 1][0], Q.b[2 * gr + 1][1]);
      else
        b = qs[nt].b[gr][lane];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        float acc[4];
        mma_f16_first(acc, a[i][0], a[i][1], a[i][2], a[i][3], b.x, b.y);
        mma_f16(acc, a[i][4], a[i][5], a[i][6], a[i][7], b.z, b.w);
        z[i][nt][0] = fmaf(acc[0], ks[i][0][gr], z[i][nt][0]);
        z[i][nt][1] = fmaf(acc[1], ks[i][0][gr], z[i][nt][1]);
        z[i][nt][2] = fmaf(acc[2], ks[i][1][gr], z[i][nt][2]);
        z[i][nt][3] = fmaf(acc[3], ks[i][1][gr], z[i][nt][3]);
      }
    }
  }
  if (tail) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 8 * nt + 2 * t + (e & 1), token = kTileTokens * i + g + 8 * (e >> 1);
          if (row >= rows || token >= left - (nq - 1) + row % nq) z[i][nt][e] = -INFINITY;
        }
  }
}

// The lane's best score of row 2t + e over its tokens.
template <int NT, int kTiles>
__device__ __forceinline__ float lane_best(const float (&z)[kTiles][NT][4], int nt, int e) {
  float best = fmaxf(z[0][nt][e], z[0][nt][e + 2]);
  if constexpr (kTiles == 2) best = fmaxf(best, fmaxf(z[1][nt][e], z[1][nt][e + 2]));
  return best;
}

// The weight (as a power of two) up to which weights x V scales up to vmax stay within f16: products below 2^15.
__device__ __forceinline__ float weight_limit(float vmax) {
  if (!(vmax <= 65504.f)) vmax = 0.f;  // a NaN scale sets no limit
  return kTopWeight - (float)max((int)(__float_as_uint(vmax) >> 23) - 127, 0);
}

template <int GR>
__device__ __forceinline__ void rescale_row(RowTile<GR>& S, int e, float f) {
#pragma unroll
  for (int mt = 0; mt < 2 * GR; ++mt) {
    S.o[mt][e] *= f;
    S.o[mt][e + 2] *= f;
  }
  S.c[e] *= f;
  S.c[e + 2] *= f;
}

// Raises row 2t + e's top so that `best`, its best score, weighs 2^(lift - 4), where it would weigh more than 2^lift.
// Returns whether it still weighs more than 2^limit.
template <int GR>
__device__ __forceinline__ bool raise_top(RowTile<GR>& S, int e, float best, float al, float lift, float limit) {
  const float old = S.top[e];
  if (best > old) {  // the row's lanes agree; rows differ
    S.top[e] = best + 4.f / al;
    rescale_row(S, e, ex2((old - S.top[e]) * al));
  }
  return fmaf(best - S.top[e], al, lift) > limit;
}

// Shrinks the weights of all rows from 2^lift at most to 2^limit.
template <int NT, int GR>
__device__ __forceinline__ void lower_lift(RowTile<GR> (&A)[NT], float& lift, float limit) {
  const float f = ex2(limit - lift);
  lift = limit;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) rescale_row(A[nt], e, f);
}

// Weights of tokens g, g + 8 and rows 2t, 2t + 1 as f16, transposed: of row g and token pairs t, t + 4.
__device__ __forceinline__ void weights(uint32_t (&p)[2], const float (&z)[4], const float (&top)[2], float al0, float al1,
                                        float lift) {
  float w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = ex2(fmaf(z[e] - top[e & 1], e & 1 ? al1 : al0, lift));
  p[0] = movmatrix_trans(pack_half2(w[0], w[1]));
  p[1] = movmatrix_trans(pack_half2(w[2], w[3]));
}

// One or two row tiles: a warp takes a stage (two tiles, 32 tokens) by itself, both tiles at once so that their chains
// of dependent operations overlap.  left: tokens of the context from the stage's first on.
template <int NT>
__device__ __forceinline__ void process_stage(RowTile<4> (&A)[NT], float& lift, const QueryTile& Q, const float (&alpha1)[2],
                                              const QueryShared* qs, unsigned char* stage, int* poison, int left, int nq,
                                              int rows, int lane) {
  const bool tail = left - (nq - 1) < kStageTokens;  // some row does not see the whole stage
  if (tail) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) clear_tail(stage + i * kTileBytes, poison, left - i * kTileTokens, nq, rows, lane);
  }
  // the largest V scale of the stage: below 2, weights up to 2^14 times scales stay within f16
  const uint4 vs = *reinterpret_cast<const uint4*>(stage + (lane >> 3 & 1) * kTileBytes + kTileVs + 16 * (lane & 7));
  const uint32_t vmax2 = max_half2(max_half2(vs.x, vs.y), max_half2(vs.z, vs.w));
  bool raise = (vmax2 & 0x40004000u) != 0;  // 2 or more
  float z[2][NT][4];
  score_tiles<NT, 2>(z, Q, qs, stage, tail, left, nq, rows, lane);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) raise |= lane_best<NT, 2>(z, nt, e) > A[nt].top[e];
  bool large = false;
  if (__any_sync(0xffffffffu, raise)) {
    float vmax = fmaxf(half_lo(vmax2), half_hi(vmax2));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
    const float limit = weight_limit(vmax);
    large = limit < kTopWeight;
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 al = NT == 1 ? make_float2(alpha1[0], alpha1[1]) : qs[nt].alpha[lane];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float best = lane_best<NT, 2>(z, nt, e);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
        over |= raise_top(A[nt], e, best, e ? al.y : al.x, lift, limit);
      }
    }
    if (__any_sync(0xffffffffu, over)) lower_lift(A, lift, limit);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 al = NT == 1 ? make_float2(alpha1[0], alpha1[1]) : qs[nt].alpha[lane];
      weights(p[nt], z[i][nt], A[nt].top, al.x, al.y, lift);
    }
    ValueRegs<4> V;
    load_values(V, stage + i * kTileBytes, 0, i ? ~0u : 0u, large, lane);
    add_values(A, V, i ? ~0u : 0u, p);
  }
}

// Four row tiles: their accumulators would take half a thread's registers, and a stage's chain of operations is long, so
// two warps share a stage.  Each scores one of its two tiles for all rows and hands its weights to the other through shared memory; then
// each adds both tiles' values for its half of the dims.  The two keep the same tops: a warp that wants one raised says
// so with its weights, and then both take the better of their rows' best scores and weigh again.
template <int NT>
struct PairShared {
  uint4 p[2][2][(NT + 1) / 2][32];  // [turn][warp of the pair]: the weights, two row tiles each
  int flags[2][2];            // [turn][warp]: kRaise, kLate
  float best[2][8 * NT];      // [warp]: the rows' best scores, and the largest V scale, when a top is raised
  float vmax[2];
};
enum { kRaise = 1, kLate = 2 };

__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;\n" ::"r"(pair + 1) : "memory"); }

// Returns whether the stage has arrived (late: this warp has seen that it has not; then the other is told).
template <int NT>
__device__ __forceinline__ bool process_pair(RowTile<2> (&A)[NT], float& lift, const QueryShared* qs, PairShared<NT>& X, int turn, int pair,
                                             int role, bool late, unsigned char* stage, int* poison, int left, int nq,
                                             int rows, int lane) {
  const int g = lane >> 2, t = lane & 3;
  unsigned char* tile = stage + role * kTileBytes;
  float z[1][NT][4];
  uint32_t p[NT][2], vmax2 = 0;
  auto weigh = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 al = qs[nt].alpha[lane];
      weights(p[nt], z[0][nt], A[nt].top, al.x, al.y, lift);
    }
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) X.p[turn][role][i][lane] = make_uint4(p[2 * i][0], p[2 * i][1], p[2 * i + 1][0], p[2 * i + 1][1]);
  };
  int flags = late ? kLate : 0;
  if (!late) {
    left -= role * kTileTokens;
    const bool tail = left - (nq - 1) < kTileTokens;
    if (tail) clear_tail(tile, poison, left, nq, rows, lane);
    const uint4 vs = *reinterpret_cast<const uint4*>(tile + kTileVs + 16 * (lane & 7));
    vmax2 = max_half2(max_half2(vs.x, vs.y), max_half2(vs.z, vs.w));
    bool raise = (vmax2 & 0x40004000u) != 0;  // as in process_stage
    score_tiles<NT, 1>(z, QueryTile(), qs, tile, tail, left, nq, rows, lane);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) raise |= lane_best<NT, 1>(z, nt, e) > A[nt].top[e];
    if (__any_sync(0xffffffffu, raise)) flags = kRaise;
    weigh();
  }
  if (lane == 0) X.flags[turn][role] = flags;
  pair_sync(pair);
  flags = X.flags[turn][0] | X.flags[turn][1];
  if (flags & kLate) return false;
  if (flags) {
    float vmax = fmaxf(half_lo(vmax2), half_hi(vmax2));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
    if (lane == 0) X.vmax[role] = vmax;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float best = lane_best<NT, 1>(z, nt, e);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (g == 0) X.best[role][8 * nt + 2 * t + e] = best;
      }
    pair_sync(pair);
    const float limit = weight_limit(fmaxf(X.vmax[0], X.vmax[1]));
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 al = qs[nt].alpha[lane];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * nt + 2 * t + e;
        over |= raise_top(A[nt], e, fmaxf(X.best[0][row], X.best[1][row]), e ? al.y : al.x, lift, limit);
      }
    }
    if (__any_sync(0xffffffffu, over)) lower_lift(A, lift, limit);  // the pair's warps see the same
    weigh();
    pair_sync(pair);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // (the warp's own weights too come back from there: fewer registers in between)
#pragma unroll
    for (int k = 0; k < NT / 2; ++k) {
      const uint4 v = X.p[turn][i][k][lane];
      p[2 * k][0] = v.x, p[2 * k][1] = v.y, p[2 * k + 1][0] = v.z, p[2 * k + 1][1] = v.w;
    }
    ValueRegs<2> V;
    load_values(V, stage + i * kTileBytes, 2 * role, i ? ~0u : 0u, true, lane);
    add_values(A, V, i ? ~0u : 0u, p);
  }
  return true;
}

// Waits for a staged half block.  Returns whether it came within `limit` cycles; waits on for those that did not, as long
// again as the longest limit, so that the copy has landed before the ring has another use or the CTA ends.
__device__ __forceinline__ bool stage_wait(uint64_t* bar, uint32_t phase, long long limit) {
  if (mbar_try_wait(bar, phase)) return limit >= 0;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, phase)) {
    if (clock64() - t0 > 2 * kWaitCycles) return false;
  }
  return clock64() - t0 <= limit;
}

// Adds a part (reference r, sum l, four dims o) to a running one.
__device__ __forceinline__ void merge_part(float& R, float& L, float4& O, float r, float l, const float4& o) {
  const float top = fmaxf(R, r), f = ex2(R - top), h = ex2(r - top);
  R = top;
  L = L * f + l * h;
  O.x = O.x * f + o.x * h;
  O.y = O.y * f + o.y * h;
  O.z = O.z * f + o.z * h;
  O.w = O.w * f + o.w * h;
}

// Four dims of an output row: zeros where no token was seen.
__device__ __forceinline__ void store_out(uint16_t* out, const float4& o, float l) {
  uint2 v = make_uint2(0, 0);
  if (l != 0.f) v = make_uint2(pack_bf16x2(o.x / l, o.y / l), pack_bf16x2(o.z / l, o.w / l));
  *reinterpret_cast<uint2*>(out) = v;
}

// The blocks that CTA i of n takes of `total`: [first(i), first(i + 1)), and the CTA that takes block b.
// (total is at most kQaSplitUnits x 16384.)
__device__ __forceinline__ int cta_first(int total, int i, int n) { return (int)((long long)total * i / n); }
__device__ __forceinline__ int cta_of(int total, int b, int n) { return (int)(((long long)(b + 1) * n - 1) / total); }

// Workers of a CTA: warps, or pairs of them for four row tiles.
__host__ __device__ constexpr int workers(int nt, int warps) { return nt == 4 ? warps / 2 : warps; }
// Warps an SM by registers: 128 a thread for one row tile (where the compiler spills 84 bytes a thread), 255 for more.
__host__ __device__ constexpr int warps_per_sm(int nt) { return nt == 1 ? 16 : 8; }

template <int NT, int W>
__global__ void __launch_bounds__(W * 32, warps_per_sm(NT) / W) quant_attend_kernel(const __grid_constant__ QuantArgs a) {
  constexpr int kThreads = W * 32, N = workers(NT, W), S = stages(NT);
  constexpr bool kPair = NT == 4;
  static_assert(W >= NT, "a warp per row tile loads the queries");
  static_assert(N % 2 == 0 && N <= 15, "halves of blocks are dealt to the workers; a named barrier per pair");
  // the workers' rings, then [worker][8 NT rows][kQaRowStride], their partials; behind them, for pairs, the query
  // operands and what the warps of a pair exchange
  extern __shared__ __align__(16) float smem[];
  __shared__ __align__(8) uint64_t bars[N][S];
  __shared__ int2 list[kQaList];  // (row of the store, tokens of the context from the block on)
  __shared__ float wr[N][8 * NT], wl[N][8 * NT];
  __shared__ int scan[32], found[2];
  __shared__ int poison[kQaMaxRows];  // [row]: groups that end as NaN
  __shared__ float2 merged[8 * NT];  // a cluster CTA's references and sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int me = kPair ? warp >> 1 : warp, role = kPair ? warp & 1 : 0;  // the warp's worker, and its part in the pair
  if (lane == 0 && role == 0) {
#pragma unroll
    for (int st = 0; st < S; ++st) mbar_init(&bars[me][st], 1);
    fence_mbar_init();
  }
  if (kPair)
    __syncthreads();
  else
    __syncwarp();
  pdl_wait();
  pdl_launch_dependents();

  auto length = [&](int u) { return a.sel ? max(a.lens[u], 0) : min(max(a.lens[u], 0), a.max_len); };
  // blocks of a unit's work; an empty unit counts as one, so that somebody writes its zeros
  auto blocks_of = [&](int u) { return a.sel ? a.max_sel : max((length(u) + kBlock - 1) / kBlock, 1); };

  // The units' blocks in one line, cut into one piece per CTA: this CTA's are `todo` blocks from block `at` of
  // unit u on, and unit u's begin at `begin` of `total`.
  const int ranks = a.split == kCluster ? (int)cg::this_cluster().num_blocks() : 1;
  const int rank = a.split == kCluster ? (int)cg::this_cluster().block_rank() : 0;
  int u = blockIdx.x / ranks, at = 0, pieces = gridDim.x;
  int todo = 1, total = 1, begin = 0;
  auto cut = [&]() {  // a stage per worker at least; further CTAs have nothing to do
    pieces = min((int)gridDim.x, (total + N / 2 - 1) / (N / 2));
    const int lo = blockIdx.x < pieces ? cta_first(total, blockIdx.x, pieces) : total;
    todo = blockIdx.x < pieces ? cta_first(total, blockIdx.x + 1, pieces) - lo : 0;
    return lo;
  };
  if (a.split == kPieces) {
    if (a.sel) {
      total = a.units * a.max_sel;
      begin = cut();
      u = begin / a.max_sel;
      at = begin % a.max_sel;
    } else {
      const int per = (a.units + kThreads - 1) / kThreads, u0 = threadIdx.x * per, u1 = min(u0 + per, a.units);
      int mine = 0, sum;
      for (int i = u0; i < u1; ++i) mine += blocks_of(i);
      int before = block_scan_excl(mine, scan, &sum);
      total = sum;
      const int lo = begin = cut();
      for (int i = u0; i < u1; ++i) {  // the one thread whose units hold block lo
        const int n = blocks_of(i);
        if (before <= lo && lo < before + n) {
          found[0] = i;
          found[1] = before;
        }
        before += n;
      }
      __syncthreads();
      if (todo == 0) return;
      u = found[0];
      at = lo - found[1];
    }
    begin -= at;
  }

  QueryShared* qs = reinterpret_cast<QueryShared*>(reinterpret_cast<unsigned char*>(smem) + quant_ring_bytes(NT, N));
  PairShared<NT>* pairs = reinterpret_cast<PairShared<NT>*>(qs + (NT > 1 ? NT : 0));
  unsigned char* ring = reinterpret_cast<unsigned char*>(smem) + me * S * kStageBytes4;
  int in = 0, out = 0, phase = 0, turn = 0;  // the ring's next stage to fill and to use, and that one's phase
  bool late = false;
  for (; todo > 0; ++u, at = 0) {
    const int len = length(u), whole = blocks_of(u);
    int first = at, end = whole;
    if (a.split == kPieces) {
      end = min(whole, at + todo);
      todo -= end - first;
    } else {
      first = cta_first(whole, rank, ranks);
      end = cta_first(whole, rank + 1, ranks);
      todo = 0;
    }
    if (threadIdx.x == 0 && first == 0 && rank == 0 && len != a.lens[u]) atomicOr(a.err, kErrBounds);
    if (threadIdx.x < kQaMaxRows) poison[threadIdx.x] = 0;
    if (a.nq > 1) __syncthreads();
    QueryTile Q;
    RowTile<kPair ? 2 : 4> A[NT];
    float alpha1[2], lift = kTopWeight;
    auto load_queries = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (NT == 1 || warp == nt) {
          load_query(Q, alpha1, a.q + (size_t)u * a.rows * kHeadDim, 8 * nt + g, a.rows, lane, a.scale, code_unit(NT));
          if (NT > 1) {
#pragma unroll
            for (int gr = 0; gr < 4; ++gr)
              qs[nt].b[gr][lane] = make_uint4(Q.b[2 * gr][0], Q.b[2 * gr][1], Q.b[2 * gr + 1][0], Q.b[2 * gr + 1][1]);
            qs[nt].sums[lane] = Q.sums;
            qs[nt].alpha[lane] = make_float2(alpha1[0], alpha1[1]);
          }
        }
        A[nt].top[0] = A[nt].top[1] = kNoRef;
#pragma unroll
        for (int mt = 0; mt < (kPair ? 4 : 8); ++mt) A[nt].o[mt][0] = A[nt].o[mt][1] = A[nt].o[mt][2] = A[nt].o[mt][3] = 0.f;
        A[nt].c[0] = A[nt].c[1] = A[nt].c[2] = A[nt].c[3] = 0.f;
      }
      if (NT > 1) __syncthreads();
    };

    // The blocks, listed ones looked up kQaList at a time and those without a token left out.  Worker w takes half
    // w % 2 of the blocks w / 2, w / 2 + N / 2, ...  (an empty second half of the last block too: it adds nothing).
    const int batch = a.sel ? kQaList : max(end - first, 1), half = (me & 1) * kStageTokens;
    const uint8_t* base = a.store + (size_t)u * a.max_blocks * kQuantBlockBytes + (me & 1) * kStageBytes4;
    for (int b0 = first; b0 < end || b0 == first; b0 += batch) {
      int n = max(min(batch, end - b0), 0);
      if (a.sel) {
        if (b0 > first) __syncthreads();  // the list before is used up
        int kept = 0;
        for (int j0 = 0; j0 < n; j0 += kThreads) {
          int2 e = make_int2(0, 0);
          if (j0 + (int)threadIdx.x < n) {
            const size_t i = (size_t)u * a.max_sel + b0 + j0 + threadIdx.x;
            const int block = a.sel[i];
            const int slot = block < 0 ? 0 : a.sel_slot ? a.sel_slot[i] : block;
            const bool held = slot >= 0 && slot < a.max_blocks;
            if (!held) atomicOr(a.err, kErrBounds);
            const long long left = block < 0 || !held ? 0 : (long long)len - (long long)block * kBlock;
            e = make_int2(slot, (int)min(max(left, 0ll), 2ll * kBlock));  // 128 or more: every row sees the whole block
          }
          int sum;
          const int at = block_scan_excl(e.y > 0, scan, &sum);
          if (e.y > 0) list[kept + at] = e;
          kept += sum;
        }
        n = kept;
        __syncthreads();
      } else if (len == 0) {
        n = 0;
      }
      const int step = N / 2, mine = (n - (me >> 1) + step - 1) / step;  // the worker's halves
      int started = 0;
      auto issue = [&]() {  // the next half into the stage whose turn it is
        if (started >= mine || late) return;
        if (lane == 0 && role == 0) {
          const int j = (me >> 1) + started * step, row = a.sel ? list[j].x : b0 + j;
          mbar_arrive_expect_tx(&bars[me][in], kStageBytes4);
          bulk_copy_g2s(smem_u32(ring + in * kStageBytes4), base + (size_t)row * kQuantBlockBytes, kStageBytes4, &bars[me][in]);
        }
        in = in + 1 == S ? 0 : in + 1;
        ++started;
      };
#pragma unroll
      for (int i = 0; i < S; ++i) issue();
      if (b0 == first) load_queries();  // while the first stages arrive
      for (int done = 0; done < started; ++done) {
        late |= !__all_sync(0xffffffffu, stage_wait(&bars[me][out], phase, a.wait_limit));
        unsigned char* stage = ring + out * kStageBytes4;
        const int j = (me >> 1) + done * step, left = (a.sel ? list[j].y : len - (b0 + j) * kBlock) - half;
        if constexpr (kPair) {
          // beyond the sync inside, both warps are through with the stage before, and its place is free
          late = !process_pair<NT>(A, lift, qs, pairs[me], turn, me, role, late, stage, poison, left, a.nq, a.rows, lane);
          turn ^= 1;
          if (started - done < S) issue();
        } else if (!late) {  // otherwise wait for what is in flight, and start no more
          process_stage<NT>(A, lift, Q, alpha1, qs, stage, poison, left, a.nq, a.rows, lane);
          __syncwarp();  // the stage is read
          issue();
        }
        out = out + 1 == S ? 0 : out + 1;
        if (out == 0) phase ^= 1;
      }
    }
    if (late) {  // a wait gave up: poison the outputs
      if (lane == 0) atomicOr(a.err, kErrTimeout);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) A[nt].c[0] = A[nt].c[1] = __int_as_float(0x7fc00000);
    }
    __syncthreads();  // the rings become the warps' partials

    // the worker's partial: O of rows 2t, 2t + 1, dims 32 gr + 4 g .. + 3 of the warp's groups, without the lift (a huge
    // reference would swallow it)
    const float unit = ex2(-lift);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const auto& T = A[nt];
      const float2 al = NT > 1 ? qs[nt].alpha[lane] : make_float2(alpha1[0], alpha1[1]);
      float* w = smem + (me * 8 * NT + 8 * nt + 2 * t) * kQaRowStride + 64 * role;
#pragma unroll
      for (int gr = 0; gr < (kPair ? 2 : 4); ++gr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m =
              fmaf(__shfl_sync(0xffffffffu, T.c[i + 2], 4 * gr + t), 16.f, __shfl_sync(0xffffffffu, T.c[i], 4 * gr + t)) * unit;
          const float even = 0x1p24f * unit, odd = 0x1p20f * unit;
          *reinterpret_cast<float4*>(w + i * kQaRowStride + 32 * gr + 4 * g) =
              make_float4(fmaf(T.o[2 * gr][i], even, m), fmaf(T.o[2 * gr][i + 2], odd, m),
                          fmaf(T.o[2 * gr + 1][i], even, m), fmaf(T.o[2 * gr + 1][i + 2], odd, m));
        }
      }
      if (g == 4 && role == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          wr[me][8 * nt + 2 * t + i] = fmaxf(T.top[i] * (i ? al.y : al.x), kNoRef);  // in base-2 logits
          wl[me][8 * nt + 2 * t + i] = T.c[i] * unit;
        }
      }
    }
    __syncthreads();
    const bool complete = first == 0 && end == whole;
    const int part = blockIdx.x + u;  // a piece's end and a unit's each move on by one: no two segments share a part
    for (int idx = threadIdx.x; idx < a.rows * (kHeadDim / 4); idx += kThreads) {
      const int row = idx >> 5, x = 4 * (idx & 31);
      float R = wr[0][row];
#pragma unroll
      for (int w = 1; w < N; ++w) R = fmaxf(R, wr[w][row]);
      float L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < N; ++w) {
        const float f = ex2(wr[w][row] - R);
        const float4 o = *reinterpret_cast<const float4*>(smem + (w * 8 * NT + row) * kQaRowStride + x);
        L = fmaf(wl[w][row], f, L);
        O.x = fmaf(o.x, f, O.x);
        O.y = fmaf(o.y, f, O.y);
        O.z = fmaf(o.z, f, O.z);
        O.w = fmaf(o.w, f, O.w);
      }
      if (poison[row] >> (x >> 5) & 1) O.x = O.y = O.z = O.w = __int_as_float(0x7fc00000);
      if (ranks > 1) {  // in the place of worker 0's, which this thread alone has read
        *reinterpret_cast<float4*>(smem + row * kQaRowStride + x) = O;
        if (x == 0) merged[row] = make_float2(R, L);
      } else if (complete) {
        store_out(a.out + ((size_t)u * a.rows + row) * kHeadDim + x, O, L);
      } else {
        const size_t i = (size_t)part * a.rows + row;
        if (x == 0) a.stats[i] = make_float2(R, L);
        *reinterpret_cast<float4*>(a.part + i * kHeadDim + x) = O;
      }
    }
    if (ranks > 1) {  // each CTA of the cluster merges its share of the outputs through distributed shared memory
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      for (int idx = rank * kThreads + threadIdx.x; idx < a.rows * (kHeadDim / 4); idx += ranks * kThreads) {
        const int row = idx >> 5, x = 4 * (idx & 31);
        float R = kNoRef, L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int r = 0; r < ranks; ++r) {
          const float2 m = *cluster.map_shared_rank(&merged[row], r);
          merge_part(R, L, O, m.x, m.y, *reinterpret_cast<const float4*>(cluster.map_shared_rank(smem + row * kQaRowStride + x, r)));
        }
        store_out(a.out + ((size_t)u * a.rows + row) * kHeadDim + x, O, L);
      }
      cluster.sync();  // keep every CTA's shared memory until all have read it
      return;
    }
    if (a.split == kPieces && first == 0 && threadIdx.x == 0)
      a.meta[u] = make_int2(part, cta_of(total, begin + whole - 1, pieces) - blockIdx.x + 1);
    begin += whole;
    if (todo > 0) {
      fence_proxy_async_smem();  // the next segment's copies come after these reads and writes
      __syncthreads();
    }
  }
}

// Merges the parts of a unit's row, where there are several: one CTA of eight warps per (unit, row), each warp
// every eighth part, each lane four dims.
__global__ void __launch_bounds__(kMergeWarps * 32) quant_merge_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ float4 so[kMergeWarps][32];
  __shared__ float2 ss[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = blockIdx.x / a.rows, row = blockIdx.x % a.rows;
  pdl_wait();
  pdl_launch_dependents();
  const int2 m = a.meta[u];
  if (m.y == 1) return;
  float R = kNoRef, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = warp; c < m.y; c += kMergeWarps) {
    const size_t i = (size_t)(m.x + c) * a.rows + row;
    const float2 s = a.stats[i];
    merge_part(R, L, O, s.x, s.y, *reinterpret_cast<const float4*>(a.part + i * kHeadDim + 4 * lane));
  }
  so[warp][lane] = O;
  if (lane == 0) ss[warp] = make_float2(R, L);
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) merge_part(R, L, O, ss[w].x, ss[w].y, so[w][lane]);
    store_out(a.out + ((size_t)u * a.rows + row) * kHeadDim + 4 * lane, O, L);
  }
}

template <int NT, int W>
constexpr int quant_smem_bytes() {
  return quant_ring_bytes(NT, workers(NT, W)) +
         (NT > 1 ? NT * (int)sizeof(QueryShared) : 0) + (NT == 4 ? workers(NT, W) * (int)sizeof(PairShared<NT>) : 0);
}

// The kernel's forms: row tiles and warps.  One row tile: eight warps a CTA (fewer parts to merge), or four for small
// calls (a shorter merge); more row tiles take the registers of eight warps an SM, two CTAs of four.
enum { kForm1x8, kForm1x4, kForm2x4, kForm4x4, kForms };

// What the launches need of a device, looked up once (a call costs more in look-ups than in launching otherwise).
struct QuantDevice {
  int sms, ctas[kForms];  // resident CTAs of each form on the whole device
};
static std::mutex g_quant_mutex;
static QuantDevice g_quant_device[64] = {};

template <int NT, int W>
static cudaError_t set_up_quant_attend(int sms, int* ctas) {
  const int smem = quant_smem_bytes<NT, W>();
  cudaError_t e = cudaFuncSetAttribute(quant_attend_kernel<NT, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(quant_attend_kernel<NT, W>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, quant_attend_kernel<NT, W>, W * 32, smem);
  if (e == cudaSuccess && *ctas < 1) e = cudaErrorInvalidConfiguration;
  *ctas *= sms;
  return e;
}

static bool quant_device(QuantDevice* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return false;
  }
  std::lock_guard<std::mutex> lock(g_quant_mutex);
  QuantDevice& d = g_quant_device[dev];
  if (!d.sms) {
    QuantDevice n = {};
    if (cudaDeviceGetAttribute(&n.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n.sms < 1 ||
        set_up_quant_attend<1, 8>(n.sms, &n.ctas[kForm1x8]) != cudaSuccess ||
        set_up_quant_attend<1, 4>(n.sms, &n.ctas[kForm1x4]) != cudaSuccess ||
        set_up_quant_attend<2, 4>(n.sms, &n.ctas[kForm2x4]) != cudaSuccess ||
        set_up_quant_attend<4, 4>(n.sms, &n.ctas[kForm4x4]) != cudaSuccess) {
      (void)cudaGetLastError();
      return false;
    }
    d = n;
  }
  *out = d;
  return true;
}

// How many CTAs a call takes, and how they share it.
struct QuantPlan {
  int form, split, ctas, cluster;
};

// Query rows' form, its workers a CTA and its CTAs in one wave.
static int row_form(int rows) { return rows <= 8 ? kForm1x8 : rows <= 16 ? kForm2x4 : kForm4x4; }
static int form_workers(int form) { return form == kForm1x8 ? 8 : form == kForm2x4 ? 4 : 2; }
static int form_wave(const QuantDevice& d, int form) { return std::min(d.ctas[form], 8 * d.sms); }

// Bytes of `parts` parts of `units` units behind the error word.
static size_t parts_bytes(size_t units, size_t parts, int rows) {
  return kQaErrBytes + units * sizeof(int2) + parts * rows * (kHeadDim + 2) * sizeof(float) + 16;
}

// What a call wants for its scratch: enough for pieces whether it takes them or not, so that more units, rows or blocks never
// want less, and a scratch made for the largest call serves them all.  More units than a wave take pieces only where a
// round's empty places, fewer than a wave, times the blocks are above 24 units (quant_plan).
static size_t quant_bytes(const QuantDevice& d, int units, int rows, int blocks) {
  const int form = row_form(rows), n = form_workers(form);
  const long long wave = std::max({form_wave(d, kForm1x8), form_wave(d, kForm2x4), form_wave(d, kForm4x4)});
  const long long u = std::min<long long>({units, kQaSplitUnits, std::max(wave, wave * blocks / 24)});
  return parts_bytes(u, std::min(wave, (u * blocks + n / 2 - 1) / (n / 2)) + u, rows);
}

// The largest power of two of CTAs per unit, `most` at most, that fits all units into one wave and leaves each worker
// a stage (clusters of 3, 6 or 12 pack badly).
static int cluster_size(int units, int blocks, int wave, int n, int most) {
  int cl = most;
  while (cl > 1 && ((long long)units * cl > wave || (cl - 1) * (n / 2) >= blocks)) cl /= 2;
  return cl;
}

// Three ways, by what a call pays (microseconds on GB300, back to back in a graph, all units of one length):
//  * a cluster per unit, merged through distributed shared memory: no second kernel (about 5), but a unit cannot
//    spread further, and ragged lengths do not balance.
//  * equal pieces of all units' blocks over one wave, merged by a second kernel.
//  * one CTA per unit, where they are more than a wave and the last round is not too empty for their length: 512 units
//    of 64 blocks 64.7 against 67.6 in pieces, of 8 blocks 15.9 against 24.2; 1024 of 64 114 against 124.
// 8 rows a unit:               cluster, 4 warps   cluster, 8 warps   pieces, 8 warps
//    2 units of 64 blocks            7.0                 7.5               7.9
//    8 units of 256                 14.0                14.0              12.3
//   16 units of 64                   9.1                 9.4              10.0
//   16 units of 256                 17.1                19.3              14.8
//   64 units of 64                  13.9                13.3              17.3
//  256 units of 32                  21.6                20.7              27.4
//  256 units listing 81             44.7                43.0              46.9
// So clusters (of eight warps a CTA) where they fill most of a wave and the units are not long (listed blocks balance,
// lengths may not; the border of 100 listed blocks a CTA has no measurement of its own but the 81 below it), clusters of
// four warps a CTA for small calls.  16 and 32 rows: the same where clusters fill a wave (64 units of 64 blocks 18.8
// against 23.3 and 31.8 against 35.9, 256 of 32 29.5 against 36.6 and 53.4 against 61.5), pieces from a few blocks a CTA on
// where they do not (16 units of 64 blocks, 32 rows 19.6 against 17.8), and 16 CTAs for very few units (2 of 32 blocks,
// 16 rows 9.2 against 10.2 in pieces).
static QuantPlan quant_plan(const QuantDevice& d, int units, int rows, int blocks, bool listed) {
  const int form = row_form(rows), n = form_workers(form), wave = form_wave(d, form);
  const int rounds = (units + wave - 1) / wave;
  if (units > kQaSplitUnits || (units > wave && (long long)(rounds * wave - units) * blocks <= 24ll * units))
    return {form, kWhole, units, 0};
  const int cl = cluster_size(units, blocks, wave, n, form != kForm1x8 && 64 * units <= wave ? 16 : 8);
  if (units * cl <= wave && 2 * units * cl > wave && blocks <= (listed ? 100 : 32) * cl)
    return {form, kCluster, units * cl, cl};
  if (form == kForm1x8) {
    const int wave4 = form_wave(d, kForm1x4), cl4 = cluster_size(units, blocks, wave4, 4, 16);
    if (units * cl4 <= wave4 && blocks <= 6 * cl4) return {kForm1x4, kCluster, units * cl4, cl4};
  } else if (units * cl <= wave && blocks <= 4 * cl) {
    return {form, kCluster, units * cl, cl};
  }
  const long long pieces = ((long long)units * blocks + n / 2 - 1) / (n / 2);
  return {form, kPieces, (int)std::min<long long>(wave, pieces), 0};
}

template <int NT, int W>
static cudaError_t launch_quant_attend(const QuantArgs& a, const QuantPlan& p, cudaStream_t st) {
  return launch_ex(quant_attend_kernel<NT, W>, dim3((unsigned)p.ctas), dim3(W * 32), quant_smem_bytes<NT, W>(), st, true,
                   p.cluster, a);
}

static thread_local long long g_wait_limit = kWaitCycles;

static nosa_status quant_attend(QuantArgs& a, int blocks, void* scratch, size_t scratch_bytes, cudaStream_t st) {
  QuantDevice d;
  if (!quant_device(&d)) return NOSA_ERR_CUDA;
  const QuantPlan plan = quant_plan(d, a.units, a.rows, blocks, a.sel != nullptr);
  if (scratch_bytes < quant_bytes(d, a.units, a.rows, blocks)) return NOSA_ERR_CAPACITY;
  const size_t parts = (size_t)plan.ctas + a.units;
  unsigned char* p = static_cast<unsigned char*>(scratch);
  a.split = plan.split;
  a.wait_limit = g_wait_limit;
  a.err = reinterpret_cast<int*>(p);
  a.part = reinterpret_cast<float*>(p + kQaErrBytes);
  a.stats = reinterpret_cast<float2*>(a.part + parts * a.rows * kHeadDim);
  a.meta = reinterpret_cast<int2*>(a.stats + parts * a.rows);
  cudaError_t e = plan.form == kForm1x8   ? launch_quant_attend<1, 8>(a, plan, st)
                  : plan.form == kForm1x4 ? launch_quant_attend<1, 4>(a, plan, st)
                  : plan.form == kForm2x4 ? launch_quant_attend<2, 4>(a, plan, st)
                                          : launch_quant_attend<4, 4>(a, plan, st);
  if (e == cudaSuccess && plan.split == kPieces)
    e = launch_ex(quant_merge_kernel, dim3((unsigned)(a.units * a.rows)), dim3(kMergeWarps * 32), 0, st, true, 0, a);
  if (e == cudaSuccess) return NOSA_OK;
  (void)cudaGetLastError();
  return NOSA_ERR_CUDA;
}

// The checks both calls share; units x rows stays below 2^31 with units <= 2^20.
static bool bad_args(const void* q, const void* store, const void* lens, const void* out, const void* scratch, int units,
                     int group, int nq, int max_blocks, float scale) {
  if (!q || !store || !lens || !out || !scratch) return true;
  if (units < 1 || units > (1 << 20) || group < 1 || group > kMaxGroup || nq < 1 || nq > kQaMaxRows ||
      group * nq > kQaMaxRows || max_blocks < 1 || !(scale >= 0.f) || isinf(scale))
    return true;
  if ((long long)units * max_blocks >= (1ll << 31)) return true;
  auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  return off(q, 16) || off(store, 16) || off(lens, 4) || off(out, 16) || off(scratch, 256);
}

}  // namespace nosa

using namespace nosa;

extern "C" nosa_status nosa_debug_quant_wait(long long cycles) {
  g_wait_limit = cycles == 0 ? kWaitCycles : std::min(cycles, kWaitCycles);
  return NOSA_OK;
}

extern "C" size_t nosa_quant_scratch_bytes(int units, int rows, int blocks) {
  QuantDevice d;
  if (units < 1 || units > (1 << 20) || rows < 1 || rows > kQaMaxRows || blocks < 1 || blocks > 16384 || !quant_device(&d))
    return 0;
  return quant_bytes(d, units, rows, blocks);
}

extern "C" nosa_status nosa_quant_dense_attend(const uint16_t* q, const uint8_t* store, int units, int group,
                                               int n_queries, int max_blocks, const int32_t* lens, int max_len,
                                               float softmax_scale, uint16_t* out, void* scratch, size_t scratch_bytes,
                                               void* stream) {
  if (bad_args(q, store, lens, out, scratch, units, group, n_queries, max_blocks, softmax_scale)) return NOSA_ERR_INVALID_ARG;
  if (max_len < 1 || max_len > (1 << 20) || max_len > (long long)max_blocks * kBlock) return NOSA_ERR_INVALID_ARG;
  QuantArgs a{};
  a.q = q;
  a.store = store;
  a.lens = lens;
  a.out = out;
  a.units = units;
  a.nq = n_queries;
  a.rows = group * n_queries;
  a.max_blocks = max_blocks;
  a.max_len = max_len;
  a.scale = (softmax_scale > 0.f ? softmax_scale : 1.f / sqrtf((float)kHeadDim)) * 1.4426950408889634f;
  return quant_attend(a, (max_len + kBlock - 1) / kBlock, scratch, scratch_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" nosa_status nosa_quant_attend(const uint16_t* q, const uint8_t* store, const int32_t* sel,
                                         const int32_t* sel_slot, int units, int group, int n_queries, int max_blocks,
                                         int max_sel, const int32_t* lens, float softmax_scale, uint16_t* out,
                                         void* scratch, size_t scratch_bytes, void* stream) {
  if (bad_args(q, store, lens, out, scratch, units, group, n_queries, max_blocks, softmax_scale)) return NOSA_ERR_INVALID_ARG;
  if (!sel || max_sel < 1 || max_sel > 16384 || reinterpret_cast<uintptr_t>(sel) % 4 || reinterpret_cast<uintptr_t>(sel_slot) % 4)
    return NOSA_ERR_INVALID_ARG;
  QuantArgs a{};
  a.q = q;
  a.store = store;
  a.sel = sel;
  a.sel_slot = sel_slot;
  a.lens = lens;
  a.out = out;
  a.units = units;
  a.nq = n_queries;
  a.rows = group * n_queries;
  a.max_blocks = max_blocks;
  a.max_sel = max_sel;
  a.scale = (softmax_scale > 0.f ? softmax_scale : 1.f / sqrtf((float)kHeadDim)) * 1.4426950408889634f;
  return quant_attend(a, max_sel, scratch, scratch_bytes, static_cast<cudaStream_t>(stream));
}
