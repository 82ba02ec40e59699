// Attention over a 4-bit KV block store (nosa_quant_dense_attend, nosa_quant_attend).
//
// With K^ = n s + m (codes n, a scale s and a minimum m per token and group of 32 dims; quant_core.cuh),
//   q . K^_t = sum_gr s_{t,gr} (q_gr . n_{t,gr}) + sum_gr m_{t,gr} sum(q_gr)
//   sum_t p_t V^_t = sum_t (p_t s_{t,gr}) n_{t,gr} + sum_t p_t m_{t,gr}
// so codes enter the tensor cores as they are and are never turned into values: a masked code in the
// low mantissa bits of an f16 is the subnormal n 2^-24 (n 2^-20 four bits further up, which the other
// operand or the result makes good by an exact 2^-4), two instructions' worth of masking per four
// codes.  The terms in m are one more MMA each: the row sums of q, split into two f16 against the
// K minima, and a 16-row operand of the V minima with a row of ones that yields the softmax sum too.
//
// grid: one CTA per (unit, chunk of tiles), four warps.  A warp takes every fourth tile of 16 tokens
// of the chunk on its own (mma.sync m16n8k16, f16 in, fp32 accumulate):
//   S^T (16 tokens x 8 rows) = K codes . q^T       8 MMAs, one accumulator per group, + 1 for m
//   P^T by movmatrix of the f16-packed weights, times s per group
//   O^T (128 dims x 8 rows) += V codes^T . P^T      8 MMAs, + 1 for m and the sum
// The query rows of a unit (q heads x query tokens, at most 32) are NT tiles of 8.  Weights are
// exp2(logit - R): R follows a row's maximum only when that outgrows it by 2^14, so the usual tile needs
// no rescaling, and is set so that weight x s stays within f16 (R rises with a scale of 2 or more).
// The CTA merges its warps in shared memory; chunks merge in a second kernel.
#include <algorithm>

#include "host.h"
#include "quant_core.cuh"

namespace nosa {

constexpr int kQaWarps = 4;
constexpr int kQaThreads = kQaWarps * 32;
constexpr int kQaMaxRows = 32;
constexpr int kQaRowStride = 132;     // floats per row of a warp's partial in shared memory (no bank conflicts)
constexpr size_t kQaErrBytes = 256;   // the scratch starts with the device error word
constexpr float kNoRef = -3e38f;      // R of a row that has seen no token

struct QuantArgs {
  const uint16_t* q;
  const uint8_t* store;
  const int32_t* sel;       // null: every block (dense)
  const int32_t* sel_slot;  // null: row b holds block b
  const int32_t* lens;
  uint16_t* out;
  float* part;  // [unit][chunk][row][2 + 128]
  int* err;
  int group, nq, rows, max_blocks, max_sel, max_len;
  int chunk_tiles, chunks;
  float scale;  // softmax scale x log2(e)
};

// D (16 x 8, f32) += A (16 x 16, row) . B (16 x 8, col), f16 inputs.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D (16 x 8, f32) += A (16 x 8, row) . B (8 x 8, col), f16 inputs.
__device__ __forceinline__ void mma_f16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};\n"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(b0));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {
  const __half2 v = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float half_lo(uint32_t a) { return half_bits_to_float(a & 0xffffu); }
__device__ __forceinline__ float half_hi(uint32_t a) { return half_bits_to_float(a >> 16); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// The query rows of one tile of 8 as MMA operands, and the factors that undo their scaling.
struct QueryTile {
  uint32_t b[8][2];  // [2 group + half]: dims 32 gr + 8 t + {0,4}, {1,5} 2^-4 | {2,6}, {3,7} 2^-4 of row g
  uint32_t sums;     // t = 0, 1: high halves of the sums of groups 2t, 2t + 1; t = 2, 3: the low halves
  float alpha[2];    // logit factor of rows 2t, 2t + 1 (softmax scale, log2 e, the row's power of two)
};

// Rows 8 nt + g of q: scaled by a power of two that brings the row's largest magnitude into [2^9, 2^10)
// (bf16 values down to 2^-23 of it stay exact in f16, and a group's sum stays in range).
__device__ __forceinline__ void load_query(QueryTile& Q, const uint16_t* q, int row, int rows, int lane, float scale) {
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
  Q.alpha[0] = scale * __shfl_sync(0xffffffffu, inv, 8 * t);      // row 2t's lanes are 8t .. 8t + 3
  Q.alpha[1] = scale * __shfl_sync(0xffffffffu, inv, 8 * t + 4);
}

// One warp's running state for a tile of 8 rows: references of rows 2t, 2t + 1, O^T (codes' part, in units
// of 2^-24, or 2^-20 for odd dims), and the m part: rows 0..3 the groups, row 4 the softmax sum.
struct RowTile {
  float r[2];
  float o[8][4];
  float c[4];
};

// A tile's operands as a lane holds them.
struct TileRegs {
  uint4 kc[2], vc[2];  // codes: tokens g, g + 8; token pairs t, t + 4
  uint2 ks[2];         // K scales of tokens g, g + 8
  uint32_t km[2];      // K minima of groups 2 (t % 2), + 1 of tokens g, g + 8
  uint4 vs[2];         // V scales of the four groups, token pairs t, t + 4
  uint32_t vm[2];      // rows of the m operand: group g's minima (g < 4), ones (g = 4), zeros
};

__device__ __forceinline__ void load_tile(TileRegs& T, const uint8_t* src, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    T.kc[h] = *reinterpret_cast<const uint4*>(src + 64 * (g + 8 * h) + 16 * t);
    T.vc[h] = *reinterpret_cast<const uint4*>(src + kTileV + 512 * h + 16 * lane);
    T.ks[h] = *reinterpret_cast<const uint2*>(src + kTileKs + 16 * (g + 8 * h));
    T.km[h] = *reinterpret_cast<const uint32_t*>(src + kTileKs + 16 * (g + 8 * h) + 8 + 4 * (t & 1));
    T.vs[h] = *reinterpret_cast<const uint4*>(src + kTileVs + 16 * (4 * h + t));
    const uint32_t m = *reinterpret_cast<const uint32_t*>(src + kTileVm + 16 * (4 * h + t) + 4 * (g & 3));
    T.vm[h] = g < 4 ? m : g == 4 ? 0x3C003C00u : 0u;
  }
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Keeps the halves of w whose token (2 pair, 2 pair + 1) is below `n`.
__device__ __forceinline__ uint32_t keep_tokens(uint32_t w, int first, int n) {
  return first + 1 < n ? w : first < n ? w & 0xffffu : 0u;
}

// Adds the V side of a tile to one row tile: p[h] = weights of token pairs t + 4 h as f16x2.
__device__ __forceinline__ void add_values(RowTile& A, const TileRegs& T, const uint32_t (&p)[2]) {
#pragma unroll
  for (int gr = 0; gr < 4; ++gr) {
    const uint32_t b0 = mul_half2(p[0], word(T.vs[0], gr)), b1 = mul_half2(p[1], word(T.vs[1], gr));
    const uint32_t w0 = word(T.vc[0], gr), w1 = word(T.vc[1], gr), x0 = w0 >> 8, x1 = w1 >> 8;
    mma_f16(A.o[2 * gr], w0 & 0x000F000Fu, w0 & 0x00F000F0u, w1 & 0x000F000Fu, w1 & 0x00F000F0u, b0, b1);
    mma_f16(A.o[2 * gr + 1], x0 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x000F000Fu, x1 & 0x00F000F0u, b0, b1);
  }
  mma_f16(A.c, T.vm[0], 0u, T.vm[1], 0u, p[0], p[1]);
}

// The rare tile at the end of a context with several query tokens where a token that only some of the
// rows see has a NaN group: 0 x NaN must not reach the others, so each token from `from` on is added
// alone, into the rows that gave it a weight.  p as above, zero for the tokens a row does not see.
__device__ __noinline__ void add_values_by_token(RowTile& A, const TileRegs& T, const uint32_t (&p)[2], int from) {
  const int lane = threadIdx.x & 31, t = lane & 3;
  for (int tok = from; tok < kTileTokens; ++tok) {
    const int h = tok >> 3, owner = (tok & 7) >> 1, par = tok & 1;
    TileRegs S = T;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t keep = i == h && t == owner ? (par ? 0xffff0000u : 0x0000ffffu) : 0u;
      w[i] = p[i] & keep;
      S.vs[i] = make_uint4(T.vs[i].x & keep, T.vs[i].y & keep, T.vs[i].z & keep, T.vs[i].w & keep);
      S.vm[i] = T.vm[i] & keep;
    }
    RowTile D;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) D.o[mt][0] = D.o[mt][1] = D.o[mt][2] = D.o[mt][3] = 0.f;
    D.c[0] = D.c[1] = D.c[2] = D.c[3] = 0.f;
    add_values(D, S, w);
    // the token's weight for rows 2t, 2t + 1: held by lane (row, owner)
    const uint32_t mine = h ? w[1] : w[0];
    const uint32_t p0 = __shfl_sync(0xffffffffu, mine, 8 * t + owner), p1 = __shfl_sync(0xffffffffu, mine, 8 * t + 4 + owner);
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      A.o[mt][0] += p0 ? D.o[mt][0] : 0.f;
      A.o[mt][1] += p1 ? D.o[mt][1] : 0.f;
      A.o[mt][2] += p0 ? D.o[mt][2] : 0.f;
      A.o[mt][3] += p1 ? D.o[mt][3] : 0.f;
    }
    A.c[0] += p0 ? D.c[0] : 0.f;
    A.c[1] += p1 ? D.c[1] : 0.f;
    A.c[2] += p0 ? D.c[2] : 0.f;
    A.c[3] += p1 ? D.c[3] : 0.f;
  }
}

// A half that is infinite or NaN, in either position.
__device__ __forceinline__ bool not_finite2(uint32_t w) {
  return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}

// One tile of 16 tokens for all row tiles.  left: tokens of the context from the tile's first on (may exceed 16).
template <int NT>
__device__ __forceinline__ void process_tile(RowTile (&A)[NT], const QueryTile (&Q)[NT], TileRegs& T, int left, int nq,
                                             int rows, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const bool tail = left - (nq - 1) < kTileTokens;  // some row does not see the whole tile
  int odd_from = kTileTokens;                       // first token that has to be added alone
  if (tail) {
    // behind the context the store may hold anything: its codes are finite as they stand, its scales go
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int first = 2 * t + 8 * h;
      T.vs[h].x = keep_tokens(T.vs[h].x, first, left);
      T.vs[h].y = keep_tokens(T.vs[h].y, first, left);
      T.vs[h].z = keep_tokens(T.vs[h].z, first, left);
      T.vs[h].w = keep_tokens(T.vs[h].w, first, left);
      if (g < 4) T.vm[h] = keep_tokens(T.vm[h], first, left);
    }
    if (nq > 1) {
      bool odd = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t late = ~keep_tokens(0xffffffffu, 2 * t + 8 * h, left - (nq - 1));
        odd |= not_finite2(T.vs[h].x & late) || not_finite2(T.vs[h].y & late) || not_finite2(T.vs[h].z & late) ||
               not_finite2(T.vs[h].w & late);
      }
      if (__any_sync(0xffffffffu, odd)) odd_from = max(left - (nq - 1), 0);
    }
  }
  // the largest V scale of the lane's tokens (the lanes of one t agree)
  const uint32_t vmax2 = max_half2(max_half2(max_half2(T.vs[0].x, T.vs[0].y), max_half2(T.vs[0].z, T.vs[0].w)),
                                   max_half2(max_half2(T.vs[1].x, T.vs[1].y), max_half2(T.vs[1].z, T.vs[1].w)));
  const bool large = (vmax2 & 0x7fffu) >= 0x4000u || (vmax2 >> 16 & 0x7fffu) >= 0x4000u;  // 2 or more

  // K scales as floats, times the 2^24 that the codes lack
  float ks[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    ks[h][0] = half_lo(T.ks[h].x) * 16777216.f;
    ks[h][1] = half_hi(T.ks[h].x) * 16777216.f;
    ks[h][2] = half_lo(T.ks[h].y) * 16777216.f;
    ks[h][3] = half_hi(T.ks[h].y) * 16777216.f;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float z[4] = {0.f, 0.f, 0.f, 0.f};
    mma_f16_k8(z, T.km[0], T.km[1], Q[nt].sums);
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      const uint32_t w0 = word(T.kc[0], gr), w1 = word(T.kc[1], gr), x0 = w0 >> 8, x1 = w1 >> 8;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      mma_f16(acc, w0 & 0x000F000Fu, w1 & 0x000F000Fu, w0 & 0x00F000F0u, w1 & 0x00F000F0u, Q[nt].b[2 * gr][0], Q[nt].b[2 * gr][1]);
      mma_f16(acc, x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x00F000F0u, Q[nt].b[2 * gr + 1][0],
              Q[nt].b[2 * gr + 1][1]);
      z[0] = fmaf(acc[0], ks[0][gr], z[0]);
      z[1] = fmaf(acc[1], ks[0][gr], z[1]);
      z[2] = fmaf(acc[2], ks[1][gr], z[2]);
      z[3] = fmaf(acc[3], ks[1][gr], z[3]);
    }
    z[0] *= Q[nt].alpha[0];
    z[1] *= Q[nt].alpha[1];
    z[2] *= Q[nt].alpha[0];
    z[3] *= Q[nt].alpha[1];
    if (tail) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * nt + 2 * t + (i & 1), token = g + 8 * (i >> 1);
        if (row >= rows || token >= left - (nq - 1) + row % nq) z[i] = -INFINITY;
      }
    }
    RowTile& S = A[nt];
    const float mx0 = fmaxf(z[0], z[2]), mx1 = fmaxf(z[1], z[3]);
    if (__any_sync(0xffffffffu, mx0 - S.r[0] > 14.f || mx1 - S.r[1] > 14.f || large)) {
      // a row's maximum has outgrown its reference, or weight x scale might leave f16
      float top[2] = {mx0, mx1}, vmax = fmaxf(half_lo(vmax2), half_hi(vmax2));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
        top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
      }
      vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 1));
      vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
      // vmax < 2^e: weights up to 2^limit keep the products below 2^15 (a NaN scale sets no limit)
      if (!(vmax <= 65504.f)) vmax = 0.f;
      const int e = (int)(__float_as_uint(vmax) >> 23) - 126;
      const float limit = (float)(14 - max(e - 1, 0));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (top[i] - S.r[i] > limit) {
          const float r = top[i] - (limit - 4.f), f = ex2(S.r[i] - r);
          S.r[i] = r;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            S.o[mt][i] *= f;
            S.o[mt][i + 2] *= f;
          }
          S.c[i] *= f;
          S.c[i + 2] *= f;
        }
      }
    }
    // weights of tokens g (+ 8), rows 2t, 2t + 1; transposed: of row g, token pairs t, t + 4
    uint32_t p[2] = {movmatrix_trans(pack_half2(ex2(z[0] - S.r[0]), ex2(z[1] - S.r[1]))),
                     movmatrix_trans(pack_half2(ex2(z[2] - S.r[0]), ex2(z[3] - S.r[1])))};
    if (odd_from < kTileTokens) {
      RowTile B = S;  // a copy, so that S itself stays in registers
      add_values_by_token(B, T, p, odd_from);
      S = B;
      TileRegs U = T;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int first = 2 * t + 8 * h;
        U.vs[h].x = keep_tokens(T.vs[h].x, first, odd_from);
        U.vs[h].y = keep_tokens(T.vs[h].y, first, odd_from);
        U.vs[h].z = keep_tokens(T.vs[h].z, first, odd_from);
        U.vs[h].w = keep_tokens(T.vs[h].w, first, odd_from);
        U.vm[h] = keep_tokens(T.vm[h], first, odd_from);  // the row of ones too: those tokens are counted
        p[h] = keep_tokens(p[h], first, odd_from);
      }
      add_values(S, U, p);
    } else {
      add_values(S, T, p);
    }
  }
}

// Stores output element x of a unit's row: zero where no token was seen.
__device__ __forceinline__ uint16_t finish(float o, float l) {
  const __nv_bfloat16 v = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
  return __bfloat16_as_ushort(v);
}

template <int NT>
__global__ void __launch_bounds__(kQaThreads) quant_attend_kernel(const __grid_constant__ QuantArgs a) {
  extern __shared__ __align__(16) float smem[];  // [warp][8 NT rows][kQaRowStride], the merge's
  __shared__ float wr[kQaWarps][8 * NT], wl[kQaWarps][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  pdl_wait();
  pdl_launch_dependents();
  const int len0 = a.lens[u];
  const int len = a.sel ? max(len0, 0) : min(max(len0, 0), a.max_len);
  if (len != len0 && threadIdx.x == 0 && chunk == 0) atomicOr(a.err, kErrBounds);
  QueryTile Q[NT];
  RowTile A[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    load_query(Q[nt], a.q + (size_t)u * a.rows * kHeadDim, 8 * nt + g, a.rows, lane, a.scale);
    A[nt].r[0] = A[nt].r[1] = kNoRef;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) A[nt].o[mt][0] = A[nt].o[mt][1] = A[nt].o[mt][2] = A[nt].o[mt][3] = 0.f;
    A[nt].c[0] = A[nt].c[1] = A[nt].c[2] = A[nt].c[3] = 0.f;
  }
  const int tiles = a.sel ? 4 * a.max_sel : (len + kTileTokens - 1) / kTileTokens;
  const int end = min((chunk + 1) * a.chunk_tiles, tiles);
  for (int i = chunk * a.chunk_tiles + warp; i < end; i += kQaWarps) {
    int block = i >> 2, slot = block;
    if (a.sel) {
      block = a.sel[(size_t)u * a.max_sel + (i >> 2)];
      if (block < 0) continue;
      slot = a.sel_slot ? a.sel_slot[(size_t)u * a.max_sel + (i >> 2)] : block;
      if (slot < 0 || slot >= a.max_blocks) {
        if (lane == 0) atomicOr(a.err, kErrBounds);
        continue;
      }
    }
    const long long left = (long long)len - ((long long)block * kBlock + (i & 3) * kTileTokens);
    if (left <= 0) continue;
    TileRegs T;
    load_tile(T, a.store + ((size_t)u * a.max_blocks + slot) * kQuantBlockBytes + (i & 3) * kTileBytes, lane);
    process_tile<NT>(A, Q, T, (int)min(left, 1ll << 20), a.nq, a.rows, lane);
  }

  // the warp's partial: O of rows 2t, 2t + 1, dims 32 gr + 4 g .. + 3
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const RowTile& S = A[nt];
    float* w = smem + (warp * 8 * NT + 8 * nt + 2 * t) * kQaRowStride;
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float m = __shfl_sync(0xffffffffu, S.c[i], 4 * gr + t);
        *reinterpret_cast<float4*>(w + i * kQaRowStride + 32 * gr + 4 * g) =
            make_float4(fmaf(S.o[2 * gr][i], 0x1p24f, m), fmaf(S.o[2 * gr][i + 2], 0x1p20f, m),
                        fmaf(S.o[2 * gr + 1][i], 0x1p24f, m), fmaf(S.o[2 * gr + 1][i + 2], 0x1p20f, m));
      }
    }
    if (g == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        wr[warp][8 * nt + 2 * t + i] = S.r[i];
        wl[warp][8 * nt + 2 * t + i] = S.c[i];
      }
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < a.rows * (kHeadDim / 4); idx += kQaThreads) {
    const int row = idx >> 5, x = 4 * (idx & 31);
    float R = wr[0][row];
#pragma unroll
    for (int w = 1; w < kQaWarps; ++w) R = fmaxf(R, wr[w][row]);
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kQaWarps; ++w) {
      const float f = ex2(wr[w][row] - R);
      const float4 o = *reinterpret_cast<const float4*>(smem + (w * 8 * NT + row) * kQaRowStride + x);
      L = fmaf(wl[w][row], f, L);
      O.x = fmaf(o.x, f, O.x);
      O.y = fmaf(o.y, f, O.y);
      O.z = fmaf(o.z, f, O.z);
      O.w = fmaf(o.w, f, O.w);
    }
    if (a.chunks == 1) {
      uint2 v;
      v.x = finish(O.x, L) | (uint32_t)finish(O.y, L) << 16;
      v.y = finish(O.z, L) | (uint32_t)finish(O.w, L) << 16;
      *reinterpret_cast<uint2*>(a.out + ((size_t)u * a.rows + row) * kHeadDim + x) = v;
    } else {
      float* part = a.part + ((size_t)blockIdx.x * a.rows + row) * kPartStride;
      if (x == 0) {
        part[0] = R;
        part[1] = L;
      }
      *reinterpret_cast<float2*>(part + 2 + x) = make_float2(O.x, O.y);
      *reinterpret_cast<float2*>(part + 4 + x) = make_float2(O.z, O.w);
    }
  }
}

// Merges a unit row's chunks: one CTA of 128 threads per (unit, row), thread x its dim x.
__global__ void __launch_bounds__(kHeadDim) quant_merge_kernel(const float* __restrict__ part, uint16_t* __restrict__ out,
                                                               int rows, int chunks) {
  pdl_wait();
  pdl_launch_dependents();
  const int u = blockIdx.x / rows, row = blockIdx.x % rows, x = threadIdx.x;
  const float* p = part + ((size_t)u * chunks * rows + row) * kPartStride;
  const size_t step = (size_t)rows * kPartStride;
  float R = kNoRef;
  for (int c = 0; c < chunks; ++c) R = fmaxf(R, p[c * step]);
  float L = 0.f, O = 0.f;
  for (int c = 0; c < chunks; ++c) {
    const float f = ex2(p[c * step] - R);
    L = fmaf(p[c * step + 1], f, L);
    O = fmaf(p[c * step + 2 + x], f, O);
  }
  out[((size_t)u * rows + row) * kHeadDim + x] = finish(O, L);
}

// How a call is split: about four CTAs of at least four tiles per SM and unit's share.
struct QuantPlan {
  int chunk_tiles, chunks;
};
static QuantPlan quant_plan(int units, int tiles, int sms) {
  const long long most = 1 + 16ll * sms / units;  // units x chunks <= units + 16 SMs
  const long long want = std::min<long long>(most, std::max<long long>(1, (4ll * sms + units - 1) / units));
  const int chunk = std::max<int>(kQaWarps, (int)((tiles + want - 1) / want));
  return {chunk, (tiles + chunk - 1) / chunk};
}

static int quant_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  return sms;
}

template <int NT>
static cudaError_t launch_quant_attend(const QuantArgs& a, int units, cudaStream_t st) {
  const int smem = kQaWarps * 8 * NT * kQaRowStride * (int)sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(quant_attend_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_ex(quant_attend_kernel<NT>, dim3((unsigned)(units * a.chunks)), dim3(kQaThreads), smem, st, true, 0, a);
}

static nosa_status quant_attend(QuantArgs& a, int units, int blocks, void* scratch, size_t scratch_bytes, cudaStream_t st) {
  const int sms = quant_sms();
  if (sms <= 0) return NOSA_ERR_CUDA;
  const QuantPlan plan = quant_plan(units, 4 * blocks, sms);
  if (scratch_bytes < nosa_quant_scratch_bytes(units, a.rows, blocks)) return NOSA_ERR_CAPACITY;
  a.chunk_tiles = plan.chunk_tiles;
  a.chunks = plan.chunks;
  a.err = reinterpret_cast<int*>(scratch);
  a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(scratch) + kQaErrBytes);
  cudaError_t e = a.rows <= 8    ? launch_quant_attend<1>(a, units, st)
                  : a.rows <= 16 ? launch_quant_attend<2>(a, units, st)
                                 : launch_quant_attend<4>(a, units, st);
  if (e == cudaSuccess && plan.chunks > 1)
    e = launch_ex(quant_merge_kernel, dim3((unsigned)(units * a.rows)), dim3(kHeadDim), 0, st, true, 0,
                  (const float*)a.part, a.out, a.rows, plan.chunks);
  if (e == cudaSuccess) return NOSA_OK;
  (void)cudaGetLastError();
  return NOSA_ERR_CUDA;
}

// The checks both calls share; units x rows and units x chunks stay below 2^31 with units <= 2^20.
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

extern "C" size_t nosa_quant_scratch_bytes(int units, int rows, int blocks) {
  const int sms = quant_sms();
  if (sms <= 0 || units < 1 || units > (1 << 20) || rows < 1 || rows > kQaMaxRows || blocks < 1 || blocks > 16384) return 0;
  return kQaErrBytes + (size_t)units * quant_plan(units, 4 * blocks, sms).chunks * rows * kPartStride * sizeof(float);
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
  a.group = group;
  a.nq = n_queries;
  a.rows = group * n_queries;
  a.max_blocks = max_blocks;
  a.max_len = max_len;
  a.scale = (softmax_scale > 0.f ? softmax_scale : 1.f / sqrtf((float)kHeadDim)) * 1.4426950408889634f;
  return quant_attend(a, units, (max_len + kBlock - 1) / kBlock, scratch, scratch_bytes, static_cast<cudaStream_t>(stream));
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
  a.group = group;
  a.nq = n_queries;
  a.rows = group * n_queries;
  a.max_blocks = max_blocks;
  a.max_sel = max_sel;
  a.scale = (softmax_scale > 0.f ? softmax_scale : 1.f / sqrtf((float)kHeadDim)) * 1.4426950408889634f;
  return quant_attend(a, units, max_sel, scratch, scratch_bytes, static_cast<cudaStream_t>(stream));
}
