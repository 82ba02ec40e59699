// Attention over an 8-bit KV block store (nosa_byte_dense_attend, nosa_byte_attend).
//
// With codes c and one scale each for a block's K and V, the scores are s_K (q . c_t) and a block adds
// s_V sum_t p_t c_t to the result: e4m3 codes are exact in f16, two in a conversion, so they go to mma.sync m16n8k16 with f16
// operands and float32 accumulators, and the scales are one float32 factor each per block.  (mma.sync takes e4m3 too, but
// sm_103a converts it inside: 7.9 cycles an MMA with new operands against 2.7 of f16.  With at most 32 rows a unit
// tcgen05's tiles of 64 rows and more would be mostly empty.)
//
// As for the 4-bit store, CTAs share the units' blocks in equal pieces, or a cluster of CTAs takes a unit (byte_plan), and a
// warp takes half a block (two tiles of 16 tokens) at a time through a ring of its own of bulk copies.  Per half block
// and 8 query rows:
//   S^T (2 x 16 tokens x 8 rows) = K codes . q^T       16 MMAs in two chains
//   P^T by movmatrix of the f16-packed weights
//   O^T (128 dims x 8 rows) += s_V (V codes^T . P^T)    16 MMAs into fresh accumulators, 32 FMAs: results stay in true
//                                                  units whatever the blocks' scales
// Weights are 2^(logit - R), R within 14 of the row's maximum, their sum float32.  Where masses are wanted a half block
// stores its (R, sum) per row; the rows' final references and sums turn these into masses in the end (in a kernel of their own after pieces).
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "byte_core.cuh"
#include "host.h"
#include "store_core.cuh"

namespace nosa {

namespace cg = cooperative_groups;

constexpr int kHalfTokens = 32, kHalfBytes = 2 * kByteTile;
constexpr int kHalfStage = kHalfBytes + 128;  // a stage: half a block and, behind it, the block's scales
constexpr int kWarps = 4, kStages = 2, kThreads = kWarps * 32, kCtasPerSm = 2;
constexpr int kMassThreads = 128;
constexpr float kTopLead = 10.f, kTopWeight = 14.f;  // a new reference weighs the best score 2^10; up to 2^14 it stays

struct ByteArgs {
  const uint16_t* q;
  const uint8_t* store;
  const int32_t* sel;       // null: every block (dense)
  const int32_t* sel_slot;  // null: row b holds block b
  const int32_t* lens;
  uint16_t* out;
  float* mass;    // null: not wanted
  int* err;
  int2* meta;     // [unit]: its first part and how many there are (1: the output is written already)
  float2* stats;  // [part][row]: reference and softmax sum
  float* part;    // [part][row][128]
  float2* total;  // [unit][row]: final reference and sum, where masses are wanted
  float2* half;   // [unit][block][half][mass_rows]: reference and sum of a half block
  int units, nq, rows, mass_rows, max_blocks, max_sel, max_len, blocks;  // blocks: per unit, listed or up to max_len
  int split;
  float scale;    // softmax scale x log2(e)
  long long wait_limit;  // SM cycles a wait for a staged half block may take before it gives up (< 0: none)
};

// Eight query rows as MMA operands: of row g, dims 32 t + 16 c + 4 w .. + 3 in [4 c + w].
struct ByteQuery {
  uint32_t b[8][2];
};

// Rows 8 nt + g of q, scaled by a power of two that brings the row's largest magnitude into [2^9, 2^10) (bf16 values
// down to 2^-22 of it stay exact in f16).  alpha: the factors that turn rows 2t, 2t + 1 of q . c into logits in base 2
// for a K scale of 1.
__device__ __forceinline__ void load_byte_query(ByteQuery& Q, float (&alpha)[2], const uint16_t* q, int row, int rows,
                                                int lane, float scale) {
  const int t = lane & 3;
  uint4 x[4];
  uint32_t big = 0;  // the largest magnitude's bf16 bits
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = row < rows ? *reinterpret_cast<const uint4*>(q + (size_t)row * kHeadDim + 32 * t + 8 * i) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) big = max(big, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
  }
  big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
  // 2^(9 - e) for the exponent e of the largest value; 1 where the row is zero or not finite
  const int e = (int)(big >> 7) - 127;
  const int shift = big == 0 || big >= 0x7f80u ? 0 : min(9 - e, 126);
  const float f = __uint_as_float((uint32_t)(127 + shift) << 23);
  float inv = __uint_as_float((uint32_t)(127 - shift) << 23);
  if (big >= 0x7f80u) inv = __int_as_float(0x7fc00000);  // then every logit is a NaN
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      Q.b[2 * i + (k >> 1)][k & 1] = pack_half2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float al = scale * __shfl_sync(0xffffffffu, inv, 8 * t + 4 * i);  // row 2t's lanes: 8t ..
    alpha[i] = al > 0x1p127f ? 0x1p127f : al;  // finite: it may meet a zero s_K (a NaN stays)
  }
}

// Logits per score: alpha x s_K, kept where logits are finite (scores are below 2^26: 128 products of a q below 2^10 and a
// code of at most 448).
__device__ __forceinline__ float logit_factor(float alpha, float sk) {
  const float c = alpha * sk;
  return c > 0x1p100f ? 0x1p100f : c;  // (a NaN stays)
}

// The query side in shared memory, for more than one row tile (registers hold it for one).
struct ByteQueryShared {
  uint4 b[4][32];  // [two operands][lane]
  float2 alpha[32];
};

// A warp's running state for a tile of 8 rows: of rows 2t, 2t + 1 the reference (a logit in base 2), the lane's part of
// the softmax sum, and O^T: dims 16 g + 2 j and + 1 of those rows.
struct ByteRows {
  float top[2], l[2];
  float o[8][4];
};

// Prepares a half block that not every row sees as a whole (left: tokens of the context from its first on, possibly
// none).  Behind the context the store may hold anything, and 0 x NaN is a NaN, so those tokens' V codes are cleared.  So
// is a NaN of a token that only some rows see: the rows that see it get a bit of `poison`, and a NaN in that dim in the
// end.
__device__ __noinline__ void clear_byte_tail(unsigned char* stage, uint32_t (*poison)[4], int left, int nq, int rows, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int tile = 0; tile < 2; ++tile) {
    const int late0 = kByteTileTokens * tile + 2 * t - (left - nq);  // rows of query tokens from there on see token 2t
    // per half of the tile, the bytes of words (two dims of two tokens) that some row sees, and that not every row sees
    uint32_t keep[2], part[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int late = late0 + 8 * h;
      keep[h] = (late < nq ? 0x00ff00ffu : 0u) | (late + 1 < nq ? 0xff00ff00u : 0u);
      part[h] = keep[h] & ((late > 0 ? 0x00ff00ffu : 0u) | (late >= 0 ? 0xff00ff00u : 0u));
    }
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint4* at = reinterpret_cast<uint4*>(stage + tile * kByteTile + kByteV + 512 * c + 16 * lane);
      const uint4 v = *at;
      uint32_t w[4] = {v.x & keep[0], v.y & keep[1], v.z & keep[0], v.w & keep[1]};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t nan = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u & part[e & 1];
        while (nan) {
          const int b = (__ffs(nan) - 1) >> 3, d = 16 * g + 4 * c + 2 * (e >> 1) + (b >> 1);
          const int late = late0 + 8 * (e & 1) + (b & 1);
          for (int row = 0; row < rows; ++row)
            if (row % nq >= late) atomicOr(&poison[row][d >> 5], 1u << (d & 31));
          w[e] &= ~(0xffu << (8 * b));
          nan &= nan - 1;
        }
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  fence_proxy_async_smem();  // the next bulk copy into the stage comes after these writes
  __syncwarp();
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// One half block, two tiles, for all row tiles.  left: tokens of the context from its first on; mass: where its sums
// go, or null.
template <int NT>
__device__ __forceinline__ void process_half(ByteRows (&A)[NT], const ByteQuery& Q, const float (&alpha1)[2],
                                             const ByteQueryShared* qs, unsigned char* stage, uint32_t (*poison)[4], int left,
                                             int rows, int nq, float2* mass, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const bool tail = left - (nq - 1) < kHalfTokens;  // some row does not see the whole half
  if (tail) clear_byte_tail(stage, poison, left, nq, rows, lane);
  const float2 s = *reinterpret_cast<const float2*>(stage + kHalfBytes);  // s_K, s_V
  float z[2][NT][4];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint4 k[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        k[i][h] = *reinterpret_cast<const uint4*>(stage + i * kByteTile + 1024 * h + 512 * c + 16 * lane);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t f[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        codes_to_half2(word_of(k[i][0], w), f[i][0], f[i][2]);
        codes_to_half2(word_of(k[i][1], w), f[i][1], f[i][3]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint2 b;
        if constexpr (NT == 1)
          b = make_uint2(Q.b[4 * c + w][0], Q.b[4 * c + w][1]);
        else
          b = *(reinterpret_cast<const uint2*>(&qs[nt].b[2 * c + (w >> 1)][lane]) + (w & 1));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (c == 0 && w == 0)
            mma_f16_first(z[i][nt], f[i][0], f[i][1], f[i][2], f[i][3], b.x, b.y);
          else
            mma_f16(z[i][nt], f[i][0], f[i][1], f[i][2], f[i][3], b.x, b.y);
        }
      }
    }
  }
  // logits, and whether a row's best would weigh more than its reference allows
  bool raise = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2 al = NT == 1 ? make_float2(alpha1[0], alpha1[1]) : qs[nt].alpha[lane];
    const float f0 = logit_factor(al.x, s.x), f1 = logit_factor(al.y, s.x);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[i][nt][e] *= e & 1 ? f1 : f0;
        if (tail) {
          const int row = 8 * nt + 2 * t + (e & 1), token = kByteTileTokens * i + g + 8 * (e >> 1);
          if (row >= rows || token >= left - (nq - 1) + row % nq) z[i][nt][e] = -INFINITY;
        }
      }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      raise |= fmaxf(fmaxf(z[0][nt][e], z[0][nt][e + 2]), fmaxf(z[1][nt][e], z[1][nt][e + 2])) - A[nt].top[e] > kTopWeight;
  }
  if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float best = fmaxf(fmaxf(z[0][nt][e], z[0][nt][e + 2]), fmaxf(z[1][nt][e], z[1][nt][e + 2]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (best - A[nt].top[e] > kTopWeight) {  // the row's lanes agree; rows differ
          // (the best itself where it is so large that the difference would not be what it should)
          const float top = best - (best - kTopLead) > kTopWeight ? best : best - kTopLead;
          const float f = ex2(A[nt].top[e] - top);
          A[nt].top[e] = top;
          A[nt].l[e] *= f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            A[nt].o[j][e] *= f;
            A[nt].o[j][e + 2] *= f;
          }
        }
      }
  }
  // weights of tokens g, g + 8 and rows 2t, 2t + 1; as f16, transposed: of row g and token pairs t, t + 4
  uint32_t p[2][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = ex2(z[i][nt][e] - A[nt].top[e & 1]);
        sum[e & 1] += w[e];
      }
      p[i][nt][0] = movmatrix_trans(pack_half2(w[0], w[1]));
      p[i][nt][1] = movmatrix_trans(pack_half2(w[2], w[3]));
    }
    A[nt].l[0] += sum[0];
    A[nt].l[1] += sum[1];
    if (mass) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
        sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
      }
      const int row = 8 * nt + 2 * t;
      if (g == 0 && row < rows)
        *reinterpret_cast<float4*>(mass + row) = make_float4(A[nt].top[0], sum[0], A[nt].top[1], sum[1]);
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = *reinterpret_cast<const uint4*>(stage + i * kByteTile + kByteV + 512 * c + 16 * lane);
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      uint32_t f[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        codes_to_half2(jj ? v[i].z : v[i].x, f[i][0], f[i][1]);
        codes_to_half2(jj ? v[i].w : v[i].y, f[i][2], f[i][3]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float d[4];
        mma_f16_first(d, f[0][0], f[0][1], f[0][2], f[0][3], p[0][nt][0], p[0][nt][1]);
        mma_f16(d, f[1][0], f[1][1], f[1][2], f[1][3], p[1][nt][0], p[1][nt][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) A[nt].o[2 * c + jj][e] = fmaf(d[e], s.y, A[nt].o[2 * c + jj][e]);
      }
    }
  }
}

__host__ __device__ constexpr int byte_ring_bytes(int nt) {
  const int ring = kWarps * kStages * kHalfStage, partials = kWarps * 8 * nt * kQaRowStride * 4;
  return ring > partials ? ring : partials;
}
// Two CTAs an SM, by registers or by shared memory: a third with one row tile left 512 units of 64 blocks a round that was
// nearly empty (102 us against 85).  Two stages a warp: with three, HBM is slower (256 units of 512 blocks 331 us against
// 307), with one 364.
template <int NT>
constexpr int byte_smem_bytes() {
  const int need = byte_ring_bytes(NT) + (NT > 1 ? NT * (int)sizeof(ByteQueryShared) : 0);
  return need > 80 * 1024 ? need : 80 * 1024;
}

// The mass of entry i of unit u: per row, the sums of the block's halves at the row's final reference, over its final sum
// (final: of each row the reference, and 1 / the sum, 0 where no token was seen).
__device__ __forceinline__ float block_mass(const ByteArgs& a, int u, int i, const float2* final) {
  const size_t at = (size_t)u * a.blocks + i;
  const int len = a.sel ? max(a.lens[u], 0) : min(max(a.lens[u], 0), a.max_len);
  int block = i;
  if (a.sel) {
    block = a.sel[at];
    const int slot = block < 0 ? -1 : a.sel_slot ? a.sel_slot[at] : block;
    if (slot < 0 || slot >= a.max_blocks) return 0.f;
  }
  float sum = 0.f;
  if ((long long)block * kBlock < len) {
    const float2* half = a.half + at * 2 * a.mass_rows;
    for (int h = 0; h < 2; ++h)
      for (int row = 0; row < a.rows; ++row) {
        const float2 s = half[h * a.mass_rows + row], r = final[row];
        if (r.y != 0.f) sum = fmaf(s.y * ex2(s.x - r.x), r.y, sum);
      }
  }
  return sum;
}
__device__ __forceinline__ float2 final_of(float R, float L) { return make_float2(R, L == 0.f ? 0.f : 1.f / L); }

template <int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) byte_attend_kernel(const __grid_constant__ ByteArgs a) {
  // the warps' rings, then [warp][8 NT rows][kQaRowStride], their partials; behind them the query operands
  extern __shared__ __align__(128) float smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ int4 list[kQaList];  // (row of the store, tokens of the context from the block on, the entry's index)
  __shared__ float wr[kWarps][8 * NT], wl[kWarps][8 * NT];
  __shared__ int scan[32], found[2];
  __shared__ uint32_t poison[kQaMaxRows][4];  // [row]: dims that end as NaN
  __shared__ float2 merged[8 * NT];           // a cluster CTA's references and sums
  __shared__ float2 final[8 * NT];            // the unit's, for its masses
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (lane == 0) {
#pragma unroll
    for (int st = 0; st < kStages; ++st) mbar_init(&bars[warp][st], 1);
    fence_mbar_init();
  }
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
  const int me = blockIdx.x / ranks;
  int u = me, at = 0, pieces = gridDim.x;
  int todo = 1, total = 1, begin = 0;
  auto cut = [&]() {  // a half block per warp at least; further CTAs have nothing to do
    pieces = min(pieces, (total + kWarps / 2 - 1) / (kWarps / 2));
    const int lo = me < pieces ? cta_first(total, me, pieces) : total;
    todo = me < pieces ? cta_first(total, me + 1, pieces) - lo : 0;
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

  ByteQueryShared* qs = reinterpret_cast<ByteQueryShared*>(reinterpret_cast<unsigned char*>(smem) + byte_ring_bytes(NT));
  unsigned char* ring = reinterpret_cast<unsigned char*>(smem) + warp * kStages * kHalfStage;
  int in = 0, out = 0, phase = 0;  // the ring's next stage to fill and to use, and that one's phase
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
    if (a.nq > 1) {
      for (int i = threadIdx.x; i < kQaMaxRows * 4; i += kThreads) poison[i >> 2][i & 3] = 0;
      __syncthreads();
    }
    ByteQuery Q;
    ByteRows A[NT];
    float alpha1[2];
    auto load_queries = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (NT == 1 || warp == nt) {
          load_byte_query(Q, alpha1, a.q + (size_t)u * a.rows * kHeadDim, 8 * nt + g, a.rows, lane, a.scale);
          if (NT > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              qs[nt].b[i][lane] = make_uint4(Q.b[2 * i][0], Q.b[2 * i][1], Q.b[2 * i + 1][0], Q.b[2 * i + 1][1]);
            qs[nt].alpha[lane] = make_float2(alpha1[0], alpha1[1]);
          }
        }
        A[nt].top[0] = A[nt].top[1] = kNoRef;
        A[nt].l[0] = A[nt].l[1] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) A[nt].o[j][0] = A[nt].o[j][1] = A[nt].o[j][2] = A[nt].o[j][3] = 0.f;
      }
      if (NT > 1) __syncthreads();
    };

    // The blocks, listed ones looked up kQaList at a time and those without a token left out.  Warp w takes half
    // w % 2 of the blocks w / 2, w / 2 + kWarps / 2, ...  (an empty half of the last block too: it adds nothing).
    const int batch = a.sel ? kQaList : max(end - first, 1), half = warp & 1;
    const uint8_t* base = a.store + (size_t)u * a.max_blocks * kByteBlockBytes;
    for (int b0 = first; b0 < end || b0 == first; b0 += batch) {
      int n = max(min(batch, end - b0), 0);
      if (a.sel) {
        if (b0 > first) __syncthreads();  // the list before is used up
        int kept = 0;
        for (int j0 = 0; j0 < n; j0 += kThreads) {
          int4 e = make_int4(0, 0, b0 + j0 + threadIdx.x, 0);
          if (j0 + (int)threadIdx.x < n) {
            const size_t i = (size_t)u * a.max_sel + e.z;
            const int block = a.sel[i];
            const int slot = block < 0 ? 0 : a.sel_slot ? a.sel_slot[i] : block;
            const bool held = slot >= 0 && slot < a.max_blocks;
            if (!held) atomicOr(a.err, kErrBounds);
            const long long left = block < 0 || !held ? 0 : (long long)len - (long long)block * kBlock;
            e.x = slot;
            e.y = (int)min(max(left, 0ll), 2ll * kBlock);  // 128 or more: every row sees the whole block
          }
          int sum;
          const int to = block_scan_excl(e.y > 0, scan, &sum);
          if (e.y > 0) list[kept + to] = e;
          kept += sum;
        }
        n = kept;
        __syncthreads();
      } else if (len == 0) {
        n = 0;
      }
      constexpr int step = kWarps / 2;
      const int mine = (n - warp / 2 + step - 1) / step;  // the warp's halves
      int started = 0;
      auto issue = [&]() {  // the next half into the stage whose turn it is
        if (started >= mine || late) return;
        if (lane == 0) {
          const int j = warp / 2 + started * step, row = a.sel ? list[j].x : b0 + j;
          const uint8_t* src = base + (size_t)row * kByteBlockBytes;
          const uint32_t to = smem_u32(ring + in * kHalfStage);
          mbar_arrive_expect_tx(&bars[warp][in], kHalfBytes + 16);
          bulk_copy_g2s(to, src + half * kHalfBytes, kHalfBytes, &bars[warp][in]);
          bulk_copy_g2s(to + kHalfBytes, src + kByteScales, 16, &bars[warp][in]);
        }
        in = in + 1 == kStages ? 0 : in + 1;
        ++started;
      };
#pragma unroll
      for (int i = 0; i < kStages; ++i) issue();
      if (b0 == first) load_queries();  // while the first stages arrive
      for (int done = 0; done < started; ++done) {
        late |= !__all_sync(0xffffffffu, stage_wait(&bars[warp][out], phase, a.wait_limit));
        if (!late) {  // otherwise wait for what is in flight, and start no more
          const int j = warp / 2 + done * step;
          const int left = (a.sel ? list[j].y : len - (b0 + j) * kBlock) - half * kHalfTokens;
          float2* mass = nullptr;
          if (a.mass)
            mass = a.half + (((size_t)u * a.blocks + (a.sel ? list[j].z : b0 + j)) * 2 + half) * a.mass_rows;
          process_half<NT>(A, Q, alpha1, qs, ring + out * kHalfStage, poison, left, a.rows, a.nq, mass, lane);
          __syncwarp();  // the stage is read
          issue();
        }
        out = out + 1 == kStages ? 0 : out + 1;
        if (out == 0) phase ^= 1;
      }
    }
    if (late) {  // a wait gave up: poison the outputs
      if (lane == 0) atomicOr(a.err, kErrTimeout);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) A[nt].l[0] = A[nt].l[1] = __int_as_float(0x7fc00000);
    }
    __syncthreads();  // the rings become the warps' partials

    // the warp's partial: of rows 2t, 2t + 1, dims 16 g .. + 15
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float* w = smem + (warp * 8 * NT + 8 * nt + 2 * t) * kQaRowStride + 16 * g;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(w + i * kQaRowStride + 4 * j) = make_float4(
              A[nt].o[2 * j][i], A[nt].o[2 * j][i + 2], A[nt].o[2 * j + 1][i], A[nt].o[2 * j + 1][i + 2]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) A[nt].l[i] += __shfl_xor_sync(0xffffffffu, A[nt].l[i], o);
        if (g == 0) {
          wr[warp][8 * nt + 2 * t + i] = A[nt].top[i];
          wl[warp][8 * nt + 2 * t + i] = A[nt].l[i];
        }
      }
    }
    __syncthreads();
    const bool complete = first == 0 && end == whole;
    const int part = me + u;  // a piece's end and a unit's each move on by one: no two segments share a part
    const size_t out0 = (size_t)u * a.rows;  // the unit's first row of the result
    for (int idx = threadIdx.x; idx < a.rows * (kHeadDim / 4); idx += kThreads) {
      const int row = idx >> 5, x = 4 * (idx & 31);
      float R = wr[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) R = fmaxf(R, wr[w][row]);
      float L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(wr[w][row] - R);
        const float4 o = *reinterpret_cast<const float4*>(smem + (w * 8 * NT + row) * kQaRowStride + x);
        L = fmaf(wl[w][row], f, L);
        O.x = fmaf(o.x, f, O.x);
        O.y = fmaf(o.y, f, O.y);
        O.z = fmaf(o.z, f, O.z);
        O.w = fmaf(o.w, f, O.w);
      }
      if (a.nq > 1) {
        const uint32_t bad = poison[row][x >> 5] >> (x & 31) & 15u;
        const float nan = __int_as_float(0x7fc00000);
        if (bad & 1u) O.x = nan;
        if (bad & 2u) O.y = nan;
        if (bad & 4u) O.z = nan;
        if (bad & 8u) O.w = nan;
      }
      if (ranks > 1) {  // in the place of warp 0's, which this thread alone has read
        *reinterpret_cast<float4*>(smem + row * kQaRowStride + x) = O;
        if (x == 0) merged[row] = make_float2(R, L);
      } else if (complete) {
        store_out(a.out + (out0 + row) * kHeadDim + x, O, L);
        if (x == 0) {
          final[row] = final_of(R, L);
          if (a.mass && a.split == kPieces) a.total[out0 + row] = make_float2(R, L);
        }
      } else {
        const size_t i = (size_t)part * a.rows + row;
        if (x == 0) a.stats[i] = make_float2(R, L);
        *reinterpret_cast<float4*>(a.part + i * kHeadDim + x) = O;
      }
    }
    if (ranks > 1) {  // each CTA of the cluster merges its share of the outputs through distributed shared memory
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      if (a.mass) {
        if (threadIdx.x < a.rows) {
          float R = kNoRef, L = 0.f;
          for (int r = 0; r < ranks; ++r) R = fmaxf(R, cluster.map_shared_rank(&merged[threadIdx.x], r)->x);
          for (int r = 0; r < ranks; ++r) {
            const float2 m = *cluster.map_shared_rank(&merged[threadIdx.x], r);
            L = fmaf(m.y, ex2(m.x - R), L);
          }
          final[threadIdx.x] = final_of(R, L);
        }
        __syncthreads();
        for (int i = cta_first(a.blocks, rank, ranks) + threadIdx.x; i < cta_first(a.blocks, rank + 1, ranks); i += kThreads)
          a.mass[(size_t)u * a.blocks + i] = block_mass(a, u, i, final);
      }
      for (int idx = rank * kThreads + threadIdx.x; idx < a.rows * (kHeadDim / 4); idx += ranks * kThreads) {
        const int row = idx >> 5, x = 4 * (idx & 31);
        float R = kNoRef, L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int r = 0; r < ranks; ++r) {
          const float2 m = *cluster.map_shared_rank(&merged[row], r);
          merge_part(R, L, O, m.x, m.y, *reinterpret_cast<const float4*>(cluster.map_shared_rank(smem + row * kQaRowStride + x, r)));
        }
        store_out(a.out + (out0 + row) * kHeadDim + x, O, L);
      }
      cluster.sync();  // keep every CTA's shared memory until all have read it
      return;
    }
    if (a.split != kPieces && a.mass) {
      __syncthreads();  // the warps' sums are written, and final
      for (int i = threadIdx.x; i < a.blocks; i += kThreads) a.mass[(size_t)u * a.blocks + i] = block_mass(a, u, i, final);
    }
    if (a.split == kPieces && first == 0 && threadIdx.x == 0)
      a.meta[u] = make_int2(part, cta_of(total, begin + whole - 1, pieces) - me + 1);
    begin += whole;
    if (todo > 0) {
      fence_proxy_async_smem();  // the next segment's copies come after these reads and writes
      __syncthreads();
    }
  }
}

// Merges the parts of a unit's row, where there are several: one CTA of eight warps per (unit, row), each warp
// every eighth part, each lane four dims.
__global__ void __launch_bounds__(kMergeWarps * 32) byte_merge_kernel(const __grid_constant__ ByteArgs a) {
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
    if (lane == 0 && a.mass) a.total[(size_t)u * a.rows + row] = make_float2(R, L);
  }
}

// The blocks' masses, where the units were cut into pieces.
__global__ void __launch_bounds__(kMassThreads) byte_mass_kernel(const __grid_constant__ ByteArgs a) {
  __shared__ float2 final[kQaMaxRows];
  const int ctas = (a.blocks + kMassThreads - 1) / kMassThreads, u = blockIdx.x / ctas;
  const int i = blockIdx.x % ctas * kMassThreads + threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < a.rows) {
    const float2 s = a.total[(size_t)u * a.rows + threadIdx.x];
    final[threadIdx.x] = final_of(s.x, s.y);
  }
  __syncthreads();
  if (i < a.blocks) a.mass[(size_t)u * a.blocks + i] = block_mass(a, u, i, final);
}

// What the launches need of a device, looked up once (a call costs more in look-ups than in launching otherwise).
struct ByteDevice {
  int sms;
  int wave;  // CTAs that are resident at once
};
static std::mutex g_byte_mutex;
static ByteDevice g_byte_device[64] = {};

template <int NT>
static cudaError_t set_up_byte_attend(int sms, int* wave) {
  const int smem = byte_smem_bytes<NT>();
  int ctas = 0;
  cudaError_t e = cudaFuncSetAttribute(byte_attend_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(byte_attend_kernel<NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, byte_attend_kernel<NT>, kThreads, smem);
  if (e == cudaSuccess && ctas < 1) e = cudaErrorInvalidConfiguration;
  *wave = std::min(*wave, ctas * sms);
  return e;
}

static bool byte_device(ByteDevice* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return false;
  }
  std::lock_guard<std::mutex> lock(g_byte_mutex);
  ByteDevice& d = g_byte_device[dev];
  if (!d.sms) {
    ByteDevice n = {0, 1 << 30};
    if (cudaDeviceGetAttribute(&n.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n.sms < 1 ||
        set_up_byte_attend<1>(n.sms, &n.wave) != cudaSuccess || set_up_byte_attend<2>(n.sms, &n.wave) != cudaSuccess ||
        set_up_byte_attend<4>(n.sms, &n.wave) != cudaSuccess) {
      (void)cudaGetLastError();
      return false;
    }
    n.wave = std::min(n.wave, 8 * n.sms);
    d = n;
  }
  *out = d;
  return true;
}

// How many CTAs a call takes, and how they share it.
struct BytePlan {
  int split, ctas, cluster;
};

static int mass_rows(int rows) { return (rows + 1) & ~1; }

// Bytes behind the error word: `parts` parts of `units` units, the units' places among them and their rows' totals, and
// the half blocks' sums where masses are wanted.
static size_t byte_parts_bytes(size_t units, size_t parts, int rows, size_t blocks, bool mass) {
  return kQaErrBytes + parts * rows * (kHeadDim + 2) * sizeof(float) + units * sizeof(int2) + units * rows * sizeof(float2) +
         (mass ? units * blocks * 2 * mass_rows(rows) * sizeof(float2) : 0) + 16;
}

// What a call wants for its scratch: enough for pieces whether it takes them or not, so that more units, rows or blocks never
// want less, and a scratch made for the largest call serves them all.
static size_t byte_bytes(const ByteDevice& d, int units, int rows, int blocks, bool mass) {
  return byte_parts_bytes(units, (size_t)d.wave + units, rows, blocks, mass);
}

// The largest power of two of CTAs per unit, `most` at most, that fits all units into one wave and leaves each warp a half
// block.
static int byte_cluster_size(int units, int blocks, int wave, int most) {
  int cl = most;
  while (cl > 1 && ((long long)units * cl > wave || (cl - 1) * (kWarps / 2) >= blocks)) cl /= 2;
  return cl;
}

static BytePlan byte_plan(const ByteDevice& d, int units, int blocks, bool listed) {
  const int wave = d.wave, rounds = (units + wave - 1) / wave;
  if (units > kQaSplitUnits || (units > wave && (long long)(rounds * wave - units) * blocks <= 24ll * units))
    return {kWhole, units, 0};
  const int cl = byte_cluster_size(units, blocks, wave, 32 * units <= wave ? 16 : 8);
  if (units * cl <= wave && 2 * units * cl > wave && blocks <= (listed ? 160 : 32) * cl) return {kCluster, units * cl, cl};
  if (units * cl <= wave && blocks <= 6 * cl) return {kCluster, units * cl, cl};
  const long long pieces = ((long long)units * blocks + kWarps / 2 - 1) / (kWarps / 2);
  return {kPieces, (int)std::min<long long>(wave, pieces), 0};
}

template <int NT>
static cudaError_t launch_byte_attend(const ByteArgs& a, const BytePlan& p, cudaStream_t st) {
  return launch_ex(byte_attend_kernel<NT>, dim3((unsigned)p.ctas), dim3(kThreads), byte_smem_bytes<NT>(), st, true,
                   p.cluster, a);
}

static nosa_status byte_attend(ByteArgs& a, void* scratch, size_t scratch_bytes, cudaStream_t st) {
  ByteDevice d;
  if (!byte_device(&d)) return NOSA_ERR_CUDA;
  const BytePlan plan = byte_plan(d, a.units, a.blocks, a.sel != nullptr);
  if (scratch_bytes < byte_bytes(d, a.units, a.rows, a.blocks, a.mass != nullptr)) return NOSA_ERR_CAPACITY;
  const size_t parts = (size_t)plan.ctas + a.units;
  unsigned char* p = static_cast<unsigned char*>(scratch);
  a.split = plan.split;
  a.wait_limit = g_wait_limit;
  a.mass_rows = mass_rows(a.rows);
  a.err = reinterpret_cast<int*>(p);
  a.half = reinterpret_cast<float2*>(p + kQaErrBytes);
  a.part = reinterpret_cast<float*>(a.half + (a.mass ? (size_t)a.units * a.blocks * 2 * a.mass_rows : 0));
  a.total = reinterpret_cast<float2*>(a.part + (plan.split == kPieces ? parts * a.rows * kHeadDim : 0));
  a.stats = a.total + (size_t)a.units * a.rows;
  a.meta = reinterpret_cast<int2*>(a.stats + (plan.split == kPieces ? parts * a.rows : 0));
  cudaError_t e = a.rows <= 8    ? launch_byte_attend<1>(a, plan, st)
                  : a.rows <= 16 ? launch_byte_attend<2>(a, plan, st)
                                 : launch_byte_attend<4>(a, plan, st);
  if (e == cudaSuccess && plan.split == kPieces)
    e = launch_ex(byte_merge_kernel, dim3((unsigned)(a.units * a.rows)), dim3(kMergeWarps * 32), 0, st, true, 0, a);
  if (e == cudaSuccess && plan.split == kPieces && a.mass)
    e = launch_ex(byte_mass_kernel, dim3((unsigned)(a.units * ((a.blocks + kMassThreads - 1) / kMassThreads))),
                  dim3(kMassThreads), 0, st, true, 0, a);
  if (e == cudaSuccess) return NOSA_OK;
  (void)cudaGetLastError();
  return NOSA_ERR_CUDA;
}

// The checks both calls share; units x rows stays below 2^31 with units <= 2^20.
static bool bad_byte_args(const void* q, const void* store, const void* lens, const void* out, const void* mass,
                          const void* scratch, int units, int group, int nq, int max_blocks, float scale) {
  if (!q || !store || !lens || !out || !scratch) return true;
  if (units < 1 || units > (1 << 20) || group < 1 || group > kMaxGroup || nq < 1 || nq > kQaMaxRows ||
      group * nq > kQaMaxRows || max_blocks < 1 || !(scale >= 0.f) || isinf(scale))
    return true;
  if ((long long)units * max_blocks >= (1ll << 31)) return true;
  auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  return off(q, 16) || off(store, 16) || off(lens, 4) || off(out, 16) || off(mass, 4) || off(scratch, 256);
}

}  // namespace nosa

using namespace nosa;

extern "C" size_t nosa_byte_scratch_bytes(int units, int rows, int blocks, int mass) {
  ByteDevice d;
  if (units < 1 || units > (1 << 20) || rows < 1 || rows > kQaMaxRows || blocks < 1 || blocks > 16384 ||
      (long long)units * blocks >= (1ll << 31) || !byte_device(&d))
    return 0;
  return byte_bytes(d, units, rows, blocks, mass != 0);
}

extern "C" nosa_status nosa_byte_dense_attend(const uint16_t* q, const uint8_t* store, int units, int group,
                                              int n_queries, int max_blocks, const int32_t* lens, int max_len,
                                              float softmax_scale, uint16_t* out, float* mass, void* scratch,
                                              size_t scratch_bytes, void* stream) {
  if (bad_byte_args(q, store, lens, out, mass, scratch, units, group, n_queries, max_blocks, softmax_scale))
    return NOSA_ERR_INVALID_ARG;
  if (max_len < 1 || max_len > (1 << 20) || max_len > (long long)max_blocks * kBlock) return NOSA_ERR_INVALID_ARG;
  ByteArgs a{};
  a.q = q;
  a.store = store;
  a.lens = lens;
  a.out = out;
  a.mass = mass;
  a.units = units;
  a.nq = n_queries;
  a.rows = group * n_queries;
  a.max_blocks = max_blocks;
  a.max_len = max_len;
  a.blocks = (max_len + kBlock - 1) / kBlock;
  a.scale = (softmax_scale > 0.f ? softmax_scale : 1.f / sqrtf((float)kHeadDim)) * 1.4426950408889634f;
  return byte_attend(a, scratch, scratch_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" nosa_status nosa_byte_attend(const uint16_t* q, const uint8_t* store, const int32_t* sel,
                                        const int32_t* sel_slot, int units, int group, int n_queries, int max_blocks,
                                        int max_sel, const int32_t* lens, float softmax_scale, uint16_t* out,
                                        float* mass, void* scratch, size_t scratch_bytes, void* stream) {
  if (bad_byte_args(q, store, lens, out, mass, scratch, units, group, n_queries, max_blocks, softmax_scale))
    return NOSA_ERR_INVALID_ARG;
  if (!sel || max_sel < 1 || max_sel > 16384 || (long long)units * max_sel >= (1ll << 31) ||
      reinterpret_cast<uintptr_t>(sel) % 4 || reinterpret_cast<uintptr_t>(sel_slot) % 4)
    return NOSA_ERR_INVALID_ARG;
  ByteArgs a{};
  a.q = q;
  a.store = store;
  a.sel = sel;
  a.sel_slot = sel_slot;
  a.lens = lens;
  a.out = out;
  a.mass = mass;
  a.units = units;
  a.nq = n_queries;
  a.rows = group * n_queries;
  a.max_blocks = max_blocks;
  a.max_sel = a.blocks = max_sel;
  a.scale = (softmax_scale > 0.f ? softmax_scale : 1.f / sqrtf((float)kHeadDim)) * 1.4426950408889634f;
  return byte_attend(a, scratch, scratch_bytes, static_cast<cudaStream_t>(stream));
}
