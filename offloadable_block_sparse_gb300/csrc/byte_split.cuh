// What the two attention kernels over an 8-bit store share (byte_attend.cu: up to 8 query rows a unit, byte_attend_tc.cu: up
// to 32): their arguments, how CTAs share the units' blocks, the lists of blocks, and what becomes of a CTA's part of a
// unit's result.
#pragma once

#include <cooperative_groups.h>

#include "byte_core.cuh"
#include "store_core.cuh"

namespace nosa {

namespace cg = cooperative_groups;

constexpr int kByteThreads = 128;
constexpr float kTopLead = 10.f, kTopWeight = 14.f;  // a new reference weighs the best score 2^10; up to 2^14 it stays

// Results are kept in true units as long as no block's s_V is above kLargeScale: of 2^20 tokens with weights of up to 2^14
// and codes of up to 448 their sum is below 2^123.  From the first such block on a part's are kept in units of 2^40, below
// 2^122 with the largest scale of 2^119; a step then loses up to 2^-110 of a result (half of float32's 2^-149 in those units,
// over a sum of weights of at least 1).  The sign bit of a part's softmax sum says so (large_sum).
constexpr float kLargeScale = 0x1p80f, kLargeUnit = 0x1p40f;

__device__ __forceinline__ float large_sum(float l, bool large) { return large ? -l : l; }

// Adds a part (reference and marked sum s, four dims o) to a running one in units that `large` tells.
__device__ __forceinline__ void merge_byte_part(float& R, float& L, float4& O, bool& large, const float2& s, const float4& o) {
  const bool part = __float_as_int(s.y) < 0;
  const float top = fmaxf(R, s.x), f = ex2(R - top), h = ex2(s.x - top);
  const float fo = part && !large ? f / kLargeUnit : f, ho = large && !part ? h / kLargeUnit : h;
  R = top;
  L = L * f + fabsf(s.y) * h;
  O.x = O.x * fo + o.x * ho;
  O.y = O.y * fo + o.y * ho;
  O.z = O.z * fo + o.z * ho;
  O.w = O.w * fo + o.w * ho;
  large |= part;
}

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
  float2* stats;  // [part][row]: reference and softmax sum (large_sum)
  float* part;    // [part][row][128]
  float2* total;  // [unit][row]: final reference and sum, where masses are wanted
  float2* half;   // [unit][block][half][mass_rows]: reference and sum of a half block
  int units, nq, rows, mass_rows, max_blocks, max_sel, max_len, blocks;  // blocks: per unit, listed or up to max_len
  int split;
  float scale;    // softmax scale x log2(e); infinite where float32's normal range does not hold it
  float scale_m;  // the same as scale_m 2^scale_e, in any case
  int scale_e;
  long long wait_limit;  // SM cycles a wait for staged blocks may take before it gives up (< 0: none)
  bool products_late;    // count those for products as given up
};

// A logit is a score (below 2^26: 128 products of a q below 2^10 and a code of at most 448) x alpha x s_K, alpha = scale x inv
// being what turns the row's scores into logits in base 2, inv a power of two.  alpha is one float32 where that neither
// overflows nor loses bits, infinity elsewhere.  A factor alpha s_K above kWideFactor, infinity among them, is a NaN to the
// kernels; where they raise references they look for these and take wide_logit with the factor's own exponent.
constexpr float kWideFactor = 0x1p64f;
__device__ __forceinline__ float row_factor(float scale, float inv) {
  const float alpha = scale * inv;
  return alpha != alpha || (alpha >= 0x1p-100f && alpha <= 0x1p100f) ? alpha : INFINITY;
}
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23 & 0xff) - 127; }
// x 2^e for x = score x (scale's mantissa).  Sizes from 2^90 on, which the others stay below, are drawn together, sixteen powers
// of two to one and evenly between them: below 2^110 then, in the same order and with differences as far beyond any softmax's
// reach.  (Cut at a largest factor or logit, unequal ones would be equal or change places.)
__device__ __forceinline__ float wide_logit(float x, int e) {
  const uint32_t bits = __float_as_uint(x), size = bits & 0x7fffffffu;
  if (size == 0 || size > 0x7f800000u) return x;
  const int to = (int)(size >> 23) - 127 + e;
  if (to < -126) return 0.f;
  const uint32_t drawn = ((uint32_t)(90 + 127) << 23) + (((uint32_t)(to - 90) << 23 | (size & 0x7fffffu)) >> 4);
  return __uint_as_float((bits & 0x80000000u) | (to < 90 ? size + ((uint32_t)e << 23) : drawn));
}
// The larger, or a NaN if one is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// A row's new reference for its best logit: the best itself where it is so large that the difference would not be what
// it should.
__device__ __forceinline__ float reference(float best) {
  return best - (best - kTopLead) > kTopWeight ? best : best - kTopLead;
}

__device__ __forceinline__ int unit_length(const ByteArgs& a, int u) {
  return a.sel ? max(a.lens[u], 0) : min(max(a.lens[u], 0), a.max_len);
}
// Blocks of a unit's work; an empty unit counts as one, so that somebody writes its zeros.
__device__ __forceinline__ int unit_blocks(const ByteArgs& a, int u) {
  return a.sel ? a.max_sel : max((unit_length(a, u) + kBlock - 1) / kBlock, 1);
}

// A CTA's share of the work: `todo` blocks from block `at` of unit u on, where unit u's begin at `begin` of all units' in
// one line, `total`, that is cut into `pieces`; or (whole units, clusters) its rank's part of unit u.
struct ByteShare {
  int u, at, todo, total, begin, pieces, ranks, rank;
};
// step: the fewest blocks of a piece.
__device__ __forceinline__ ByteShare byte_share(const ByteArgs& a, int step, int* scan, int* found) {
  ByteShare s;
  s.ranks = a.split == kCluster ? (int)cg::this_cluster().num_blocks() : 1;
  s.rank = a.split == kCluster ? (int)cg::this_cluster().block_rank() : 0;
  s.u = blockIdx.x / s.ranks;
  s.at = s.begin = 0;
  s.todo = s.total = 1;
  s.pieces = gridDim.x;
  if (a.split != kPieces) return s;
  auto cut = [&]() {  // further CTAs have nothing to do
    s.pieces = min((int)gridDim.x, (s.total + step - 1) / step);
    const int lo = (int)blockIdx.x < s.pieces ? cta_first(s.total, blockIdx.x, s.pieces) : s.total;
    s.todo = (int)blockIdx.x < s.pieces ? cta_first(s.total, blockIdx.x + 1, s.pieces) - lo : 0;
    return lo;
  };
  if (a.sel) {
    s.total = a.units * a.max_sel;
    s.begin = cut();
    s.u = s.begin / a.max_sel;
    s.at = s.begin % a.max_sel;
  } else {
    const int per = (a.units + (int)blockDim.x - 1) / (int)blockDim.x, u0 = threadIdx.x * per, u1 = min(u0 + per, a.units);
    int mine = 0, sum;
    for (int i = u0; i < u1; ++i) mine += unit_blocks(a, i);
    int before = block_scan_excl(mine, scan, &sum);
    s.total = sum;
    s.begin = cut();
    for (int i = u0; i < u1; ++i) {  // the one thread whose units hold block s.begin
      const int n = unit_blocks(a, i);
      if (before <= s.begin && s.begin < before + n) {
        found[0] = i;
        found[1] = before;
      }
      before += n;
    }
    __syncthreads();
    if (s.todo > 0) {
      s.u = found[0];
      s.at = s.begin - found[1];
    }
  }
  s.begin -= s.at;
  return s;
}

// The share's part of unit s.u: blocks [first, end) of `whole`, of a context of len tokens.
struct ByteSegment {
  int len, whole, first, end;
  __device__ __forceinline__ bool complete() const { return first == 0 && end == whole; }
};
__device__ __forceinline__ ByteSegment next_segment(const ByteArgs& a, ByteShare& s) {
  ByteSegment g;
  g.len = unit_length(a, s.u);
  g.whole = unit_blocks(a, s.u);
  if (a.split == kPieces) {
    g.first = s.at;
    g.end = min(g.whole, s.at + s.todo);
    s.todo -= g.end - g.first;
  } else {
    g.first = cta_first(g.whole, s.rank, s.ranks);
    g.end = cta_first(g.whole, s.rank + 1, s.ranks);
    s.todo = 0;
  }
  if (threadIdx.x == 0 && g.first == 0 && s.rank == 0 && g.len != a.lens[s.u]) atomicOr(a.err, kErrBounds);
  return g;
}

// Looks up n listed blocks of unit u from entry b0 on, and leaves those without a token out: the list of (row of the store,
// tokens of the context from the block on, entry), and how many there are.  Contains barriers, the last behind the list.
__device__ __forceinline__ int byte_list(const ByteArgs& a, int u, int len, int b0, int n, int* scan, int4* list) {
  int kept = 0;
  for (int j0 = 0; j0 < n; j0 += (int)blockDim.x) {
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
  __syncthreads();
  return kept;
}

// Prepares a staged tile that not every row sees as a whole (left: tokens of the context from its first on, possibly
// none).  Behind the context the store may hold anything, and 0 x NaN is a NaN, so those tokens' V codes are cleared.  So
// is a NaN of a token that only some rows see: the rows that see it get a bit of `poison`, and a NaN in that dim in the
// end.
static __device__ __noinline__ void clear_byte_tail(unsigned char* tile, uint32_t (*poison)[4], int left, int nq, int rows, int lane) {
  const int g = lane >> 2, t = lane & 3, late0 = 2 * t - (left - nq);  // rows of query tokens from there on see token 2t
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
    uint4* at = reinterpret_cast<uint4*>(tile + kByteV + 512 * c + 16 * lane);
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
  fence_proxy_async_smem();  // the next bulk copy into the stage comes after these writes
  __syncwarp();
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

// What becomes of a CTA's part of unit s.u: part[worker][rows_alloc][kQaRowStride] holds N workers' results, wr and wl
// [worker][rows_alloc] their references and sums, poison the dims that end as NaN (where there is more than one query
// token), large whether they are in units of kLargeUnit.  They go into the result where the CTA has the whole unit, through the cluster, or to the merge kernel.
template <int N, int kRows>
__device__ __forceinline__ void finish_segment(const ByteArgs& a, ByteShare& s, const ByteSegment& g, float* part,
                                               const float (*wr)[kRows], const float (*wl)[kRows], const uint32_t (*poison)[4],
                                               float2* merged, float2* final, bool large) {
  const int p = blockIdx.x + s.u;  // a piece's end and a unit's each move on by one: no two segments share a part
  const size_t out0 = (size_t)s.u * a.rows;  // the unit's first row of the result
  for (int idx = threadIdx.x; idx < a.rows * (kHeadDim / 4); idx += (int)blockDim.x) {
    const int row = idx >> 5, x = 4 * (idx & 31);
    float R = wr[0][row];
#pragma unroll
    for (int w = 1; w < N; ++w) R = fmaxf(R, wr[w][row]);
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < N; ++w) {
      const float f = ex2(wr[w][row] - R);
      const float4 o = *reinterpret_cast<const float4*>(part + (w * kRows + row) * kQaRowStride + x);
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
    if (s.ranks > 1) {  // in the place of worker 0's, which this thread alone has read
      *reinterpret_cast<float4*>(part + row * kQaRowStride + x) = O;
      if (x == 0) merged[row] = make_float2(R, large_sum(L, large));
    } else if (g.complete()) {
      store_out(a.out + (out0 + row) * kHeadDim + x, O, L, large ? kLargeUnit : 1.f);
      if (x == 0) {
        final[row] = final_of(R, L);
        if (a.mass && a.split == kPieces) a.total[out0 + row] = make_float2(R, L);
      }
    } else {
      const size_t i = (size_t)p * a.rows + row;
      if (x == 0) a.stats[i] = make_float2(R, large_sum(L, large));
      *reinterpret_cast<float4*>(a.part + i * kHeadDim + x) = O;
    }
  }
  if (s.ranks > 1) {  // each CTA of the cluster merges its share of the outputs through distributed shared memory
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (a.mass) {
      if (threadIdx.x < a.rows) {
        float R = kNoRef, L = 0.f;
        for (int r = 0; r < s.ranks; ++r) R = fmaxf(R, cluster.map_shared_rank(&merged[threadIdx.x], r)->x);
        for (int r = 0; r < s.ranks; ++r) {
          const float2 m = *cluster.map_shared_rank(&merged[threadIdx.x], r);
          L = fmaf(fabsf(m.y), ex2(m.x - R), L);
        }
        final[threadIdx.x] = final_of(R, L);
      }
      __syncthreads();
      for (int i = cta_first(a.blocks, s.rank, s.ranks) + threadIdx.x; i < cta_first(a.blocks, s.rank + 1, s.ranks); i += (int)blockDim.x)
        a.mass[(size_t)s.u * a.blocks + i] = block_mass(a, s.u, i, final);
    }
    for (int idx = s.rank * (int)blockDim.x + threadIdx.x; idx < a.rows * (kHeadDim / 4); idx += s.ranks * (int)blockDim.x) {
      const int row = idx >> 5, x = 4 * (idx & 31);
      float R = kNoRef, L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
      bool any_large = false;
#pragma unroll 4
      for (int r = 0; r < s.ranks; ++r) {
        const float2 m = *cluster.map_shared_rank(&merged[row], r);
        merge_byte_part(R, L, O, any_large, m, *reinterpret_cast<const float4*>(cluster.map_shared_rank(part + row * kQaRowStride + x, r)));
      }
      store_out(a.out + (out0 + row) * kHeadDim + x, O, L, any_large ? kLargeUnit : 1.f);
    }
    cluster.sync();  // keep every CTA's shared memory until all have read it
    return;
  }
  if (a.split != kPieces && a.mass) {
    __syncthreads();  // the warps' sums are written, and final
    for (int i = threadIdx.x; i < a.blocks; i += (int)blockDim.x) a.mass[(size_t)s.u * a.blocks + i] = block_mass(a, s.u, i, final);
  }
  if (a.split == kPieces && g.first == 0 && threadIdx.x == 0)
    a.meta[s.u] = make_int2(p, cta_of(s.total, s.begin + g.whole - 1, s.pieces) - blockIdx.x + 1);
  s.begin += g.whole;
  ++s.u;
  s.at = 0;
}

// In byte_attend_tc.cu: the kernel for 9 to 32 rows a unit, its set-up (and how many of its CTAs are resident at once).
cudaError_t launch_byte_attend_tc(const ByteArgs& a, int ctas, int cluster, cudaStream_t st);
cudaError_t set_up_byte_attend_tc(int sms, int* wave);
constexpr int kTcChunkBlocks = 2;  // blocks that it takes at a time

}  // namespace nosa
