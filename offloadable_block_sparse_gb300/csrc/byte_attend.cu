// Attention over an 8-bit KV block store (nosa_byte_dense_attend, nosa_byte_attend).
//
// With codes c and one scale each for a block's K and V, the scores are s_K (q . c_t) and a block adds
// s_V sum_t p_t c_t to the result: e4m3 codes are exact in f16, two in a conversion, so they go to mma.sync m16n8k16 with f16
// operands and float32 accumulators, and the scales are one float32 factor each per block.  (mma.sync takes e4m3 too, at 7.9
// cycles an MMA with new operands against 2.7 of f16.)  For up to 8 query rows a unit; byte_attend_tc.cu, on tcgen05, takes
// more.
//
// As for the 4-bit store, CTAs share the units' blocks in equal pieces, or a cluster of CTAs takes a unit (byte_plan), and a
// warp takes half a block (two tiles of 16 tokens) at a time through a ring of its own of bulk copies.  Per half block:
//   S^T (2 x 16 tokens x 8 rows) = K codes . q^T       16 MMAs in two chains
//   P^T by movmatrix of the f16-packed weights
//   O^T (128 dims x 8 rows) += s_V (V codes^T . P^T)    16 MMAs into fresh accumulators, 32 FMAs: results stay in true
//                                                  units whatever the blocks' scales (or in units of 2^40: byte_split.cuh)
// Weights are 2^(logit - R), R within 14 of the row's maximum, their sum float32.  Where masses are wanted a half block
// stores its (R, sum) per row; the rows' final references and sums turn these into masses in the end (in a kernel of their
// own after pieces).
//
// Bound by HBM where a call is long: 256 units of 32,768 tokens and 4 rows (2.15 GB) in 306 us, 1.05 of measured HBM (a copy);
// ragged 196 us, 1.02.  400 instructions a half block (423 with masses), of which 128 conversions and 32 MMAs, leave the issue
// slots 70 % empty.  Shorter calls pay for their start and end: 256 units listing 81 blocks 54.5 us, 0.94, with the masses of
// 128 87 us, 0.92.  (With the copies by a thread that the compiler does not know to be one, 57.4 and 90.)
#include <algorithm>
#include <cmath>
#include <mutex>

#include "byte_split.cuh"
#include "host.h"
#include "tc.cuh"

namespace nosa {

constexpr int kHalfTokens = 32, kHalfBytes = 2 * kByteTile;
constexpr int kHalfStage = kHalfBytes + 128;  // a stage: half a block and, behind it, the block's scales
constexpr int kWarps = kByteThreads / 32, kStages = 2, kCtasPerSm = 2;
constexpr int kByteRows = 8;  // query rows a unit at most
constexpr int kMassThreads = 128;

// Eight query rows as MMA operands: of row g, dims 32 t + 16 c + 4 w .. + 3 in [4 c + w].
struct ByteQuery {
  uint32_t b[8][2];
};

// What turns the scores q . c of rows 2t, 2t + 1 into logits: row_factor, the row's own power of two in it, and the largest
// factor of all eight rows.
struct ByteFactors {
  float alpha[2], inv[2], most;
};

// Row g of q, scaled by a power of two that brings the row's largest magnitude into [2^9, 2^10) (bf16 values
// down to 2^-22 of it stay exact in f16).
__device__ __forceinline__ void load_byte_query(ByteQuery& Q, ByteFactors& F, const uint16_t* q, int rows, int lane,
                                                float scale) {
  const int row = lane >> 2, t = lane & 3;
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
  const float al = row_factor(scale, inv);
  F.most = __uint_as_float(__reduce_max_sync(0xffffffffu, al == al ? __float_as_uint(al) : 0u));
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // row 2t's lanes: 8t ..
    F.alpha[i] = __shfl_sync(0xffffffffu, al, 8 * t + 4 * i);
    F.inv[i] = __shfl_sync(0xffffffffu, inv, 8 * t + 4 * i);
  }
}

// A warp's running state: of rows 2t, 2t + 1 the reference (a logit in base 2), the lane's part of the softmax sum, and O^T:
// dims 16 g + 2 j and + 1 of those rows, in units of 1 / per.
struct ByteRows {
  float top[2], l[2], per;
  float o[8][4];

  __device__ __forceinline__ void to_large() {
    per = 1.f / kLargeUnit;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] *= 1.f / kLargeUnit;
  }
};

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// A score x to a logit where the block's factor is beyond kWideFactor for some row.  (Eight in line made the shortest calls 2 %
// slower.)
static __device__ __noinline__ float wide_one(float x, float inv, float sk, float scale_m, int scale_e) {
  const float y = wide_logit(sk == 0.f ? 0.f : x * scale_m, scale_e + exponent_of(inv) + exponent_of(sk));
  return inv != inv ? inv : y;
}
// One half block: both tiles of tokens at once, so that their chains of dependent operations overlap.
// left: tokens of the context from its first on; mass: where its sums go, or null.
__device__ __forceinline__ void process_half(ByteRows& A, const ByteQuery& Q, const ByteFactors& F, float scale_m, int scale_e,
                                             unsigned char* stage, uint32_t (*poison)[4], int left, int rows, int nq,
                                             float2* mass, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const bool tail = left - (nq - 1) < kHalfTokens;  // some row does not see the whole half
  if (tail) {
    clear_byte_tail(stage, poison, left, nq, rows, lane);
    clear_byte_tail(stage + kByteTile, poison, left - kByteTileTokens, nq, rows, lane);
  }
  const float2 s = *reinterpret_cast<const float2*>(stage + kHalfBytes);  // s_K, s_V
  float z[2][4];
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
      const uint32_t b0 = Q.b[4 * c + w][0], b1 = Q.b[4 * c + w][1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t f[4];
        codes_to_half2(word_of(k[i][0], w), f[0], f[2]);
        codes_to_half2(word_of(k[i][1], w), f[1], f[3]);
        if (c == 0 && w == 0)
          mma_f16_first(z[i], f[0], f[1], f[2], f[3], b0, b1);
        else
          mma_f16(z[i], f[0], f[1], f[2], f[3], b0, b1);
      }
    }
  }
  // logits; whether a row's best would weigh more than its reference allows, or something else wants care
  float y[2][4];
  const float sk = F.most * s.x <= kWideFactor ? s.x : __int_as_float(0x7fc00000), f0 = F.alpha[0] * sk, f1 = F.alpha[1] * sk;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[i][e] = z[i][e] * (e & 1 ? f1 : f0);
  auto hide = [&]() {  // what a row does not see
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 2 * t + (e & 1), token = kByteTileTokens * i + g + 8 * (e >> 1);
        if (row >= rows || token >= left - (nq - 1) + row % nq) y[i][e] = -INFINITY;
      }
  };
  if (tail) hide();
  bool raise = s.y * A.per > kLargeScale;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    raise |= !(max_or_nan(max_or_nan(y[0][e], y[0][e + 2]), max_or_nan(y[1][e], y[1][e + 2])) - A.top[e] <= kTopWeight);
  if (__any_sync(0xffffffffu, raise)) {
    if (s.y * A.per > kLargeScale) A.to_large();
    if (!(F.most * s.x <= kWideFactor)) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = wide_one(z[i][e], F.inv[e & 1], s.x, scale_m, scale_e);
      if (tail) hide();
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float b = fmaxf(fmaxf(y[0][e], y[0][e + 2]), fmaxf(y[1][e], y[1][e + 2]));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
      if (b - A.top[e] > kTopWeight) {  // the row's lanes agree; rows differ
        const float top = reference(b), f = ex2(A.top[e] - top);
        A.top[e] = top;
        A.l[e] *= f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          A.o[j][e] *= f;
          A.o[j][e + 2] *= f;
        }
      }
    }
  }
  // weights of tokens g, g + 8 and rows 2t, 2t + 1; as f16, transposed: of row g and token pairs t, t + 4
  uint32_t p[2][2];
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = ex2(y[i][e] - A.top[e & 1]);
      sum[e & 1] += w[e];
    }
    p[i][0] = movmatrix_trans(pack_half2(w[0], w[1]));
    p[i][1] = movmatrix_trans(pack_half2(w[2], w[3]));
  }
  A.l[0] += sum[0];
  A.l[1] += sum[1];
  if (mass) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
      sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
    }
    if (g == 0 && 2 * t < rows) *reinterpret_cast<float4*>(mass + 2 * t) = make_float4(A.top[0], sum[0], A.top[1], sum[1]);
  }
  const float sv = s.y * A.per;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = *reinterpret_cast<const uint4*>(stage + i * kByteTile + kByteV + 512 * c + 16 * lane);
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      float d[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t f[4];
        codes_to_half2(jj ? v[i].z : v[i].x, f[0], f[1]);
        codes_to_half2(jj ? v[i].w : v[i].y, f[2], f[3]);
        if (i == 0)
          mma_f16_first(d, f[0], f[1], f[2], f[3], p[0][0], p[0][1]);
        else
          mma_f16(d, f[0], f[1], f[2], f[3], p[1][0], p[1][1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) A.o[2 * c + jj][e] = fmaf(d[e], sv, A.o[2 * c + jj][e]);
    }
  }
}

// Two CTAs an SM by shared memory: a third left 512 units of 64 blocks a round that was nearly empty (102 us against 85).
// Two stages a warp: with three, HBM is slower (256 units of 512 blocks 331 us against 307), with one 364.
constexpr int kByteSmem = 80 * 1024, kRingBytes = kWarps * kStages * kHalfStage;
static_assert(kRingBytes <= kByteSmem && kWarps * kByteRows * kQaRowStride * 4 <= kRingBytes, "");

__global__ void __launch_bounds__(kByteThreads, kCtasPerSm) byte_attend_kernel(const __grid_constant__ ByteArgs a) {
  // the warps' rings, then [warp][row][kQaRowStride], their partials
  extern __shared__ __align__(128) float smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ int4 list[kQaList];
  __shared__ float wr[kWarps][kByteRows], wl[kWarps][kByteRows];
  __shared__ int scan[32], found[2];
  __shared__ uint32_t poison[kByteRows][4];  // [row]: dims that end as NaN
  __shared__ float2 merged[kByteRows];       // a cluster CTA's references and sums
  __shared__ float2 final[kByteRows];        // the unit's, for its masses
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (lane == 0) {
#pragma unroll
    for (int st = 0; st < kStages; ++st) mbar_init(&bars[warp][st], 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();
  ByteShare share = byte_share(a, kWarps / 2, scan, found);

  unsigned char* ring = reinterpret_cast<unsigned char*>(smem) + warp * kStages * kHalfStage;
  int in = 0, out = 0, phase = 0;  // the ring's next stage to fill and to use, and that one's phase
  bool late = false;
  while (share.todo > 0) {
    const int u = share.u;
    const ByteSegment seg = next_segment(a, share);
    if (a.nq > 1) {
      if (threadIdx.x < 4 * kByteRows) poison[threadIdx.x >> 2][threadIdx.x & 3] = 0;
      __syncthreads();
    }
    ByteQuery Q;
    ByteRows A;
    ByteFactors F;

    // The blocks, listed ones looked up kQaList at a time and those without a token left out.  Warp w takes half
    // w % 2 of the blocks w / 2, w / 2 + kWarps / 2, ...  (an empty half of the last block too: it adds nothing).
    const int batch = a.sel ? kQaList : max(seg.end - seg.first, 1), half = warp & 1;
    const uint8_t* base = a.store + (size_t)u * a.max_blocks * kByteBlockBytes;
    for (int b0 = seg.first; b0 < seg.end || b0 == seg.first; b0 += batch) {
      int n = max(min(batch, seg.end - b0), 0);
      if (a.sel) {
        if (b0 > seg.first) __syncthreads();  // the list before is used up
        n = byte_list(a, u, seg.len, b0, n, scan, list);
      } else if (seg.len == 0) {
        n = 0;
      }
      constexpr int step = kWarps / 2;
      const int mine = (n - warp / 2 + step - 1) / step;  // the warp's halves
      int started = 0;
      auto issue = [&]() {  // the next half into the stage whose turn it is
        if (started >= mine || late) return;
        if (tc::elect()) {
          const int j = warp / 2 + started * step, row = a.sel ? list[j].x : b0 + j;
          const uint8_t* src = base + (size_t)row * kByteBlockBytes;
          const uint32_t to = smem_u32(ring + in * kHalfStage);
          mbar_arrive_expect_tx(&bars[warp][in], kHalfBytes + 16);
          // (a half block's codes, and the scales, which lie behind the second half)
          bulk_copy_g2s(to, src + half * kHalfBytes, kHalfBytes + 16 * half, &bars[warp][in]);
          if (!half) bulk_copy_g2s(to + kHalfBytes, src + kByteScales, 16, &bars[warp][in]);
        }
        in = in + 1 == kStages ? 0 : in + 1;
        ++started;
      };
#pragma unroll
      for (int i = 0; i < kStages; ++i) issue();
      if (b0 == seg.first) {  // while the first stages arrive
        load_byte_query(Q, F, a.q + (size_t)u * a.rows * kHeadDim, a.rows, lane, a.scale);
        A.top[0] = A.top[1] = kNoRef;
        A.l[0] = A.l[1] = 0.f;
        A.per = 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) A.o[j][0] = A.o[j][1] = A.o[j][2] = A.o[j][3] = 0.f;
      }
      for (int done = 0; done < started; ++done) {
        late |= !__all_sync(0xffffffffu, stage_wait(&bars[warp][out], phase, a.wait_limit));
        if (!late) {  // otherwise wait for what is in flight, and start no more
          const int j = warp / 2 + done * step;
          const int left = (a.sel ? list[j].y : seg.len - (b0 + j) * kBlock) - half * kHalfTokens;
          float2* mass = nullptr;
          if (a.mass) mass = a.half + (((size_t)u * a.blocks + (a.sel ? list[j].z : b0 + j)) * 2 + half) * a.mass_rows;
          process_half(A, Q, F, a.scale_m, a.scale_e, ring + out * kHalfStage, poison, left, a.rows, a.nq, mass, lane);
          __syncwarp();  // the stage is read
          issue();
        }
        out = out + 1 == kStages ? 0 : out + 1;
        if (out == 0) phase ^= 1;
      }
    }
    if (late) {  // a wait gave up: poison the outputs
      if (lane == 0) atomicOr(a.err, kErrTimeout);
      A.l[0] = A.l[1] = __int_as_float(0x7fc00000);
    }
    const bool large = __syncthreads_or(A.per != 1.f);  // also: the rings become the warps' partials
    if (large && A.per == 1.f) A.to_large();

    // the warp's partial: of rows 2t, 2t + 1, dims 16 g .. + 15
    float* w = smem + (warp * kByteRows + 2 * t) * kQaRowStride + 16 * g;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(w + i * kQaRowStride + 4 * j) =
            make_float4(A.o[2 * j][i], A.o[2 * j][i + 2], A.o[2 * j + 1][i], A.o[2 * j + 1][i + 2]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) A.l[i] += __shfl_xor_sync(0xffffffffu, A.l[i], o);
      if (g == 0) {
        wr[warp][2 * t + i] = A.top[i];
        wl[warp][2 * t + i] = A.l[i];
      }
    }
    __syncthreads();
    finish_segment<kWarps, kByteRows>(a, share, seg, smem, wr, wl, poison, merged, final, large);
    if (share.todo > 0) {
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
  bool large = false;
#pragma unroll 4
  for (int c = warp; c < m.y; c += kMergeWarps) {
    const size_t i = (size_t)(m.x + c) * a.rows + row;
    merge_byte_part(R, L, O, large, a.stats[i], *reinterpret_cast<const float4*>(a.part + i * kHeadDim + 4 * lane));
  }
  so[warp][lane] = O;
  if (lane == 0) ss[warp] = make_float2(R, large_sum(L, large));
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) merge_byte_part(R, L, O, large, ss[w], so[w][lane]);
    store_out(a.out + ((size_t)u * a.rows + row) * kHeadDim + 4 * lane, O, L, large ? kLargeUnit : 1.f);
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
  int wave[2];  // CTAs that are resident at once: of this kernel, of byte_attend_tc.cu's
};
static std::mutex g_byte_mutex;
static ByteDevice g_byte_device[64] = {};

static cudaError_t set_up_byte_attend(int sms, int* wave) {
  int ctas = 0;
  cudaError_t e = cudaFuncSetAttribute(byte_attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kByteSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(byte_attend_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, byte_attend_kernel, kByteThreads, kByteSmem);
  if (e == cudaSuccess && ctas < 1) e = cudaErrorInvalidConfiguration;
  *wave = std::min(ctas, 8) * sms;
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
    ByteDevice n = {};
    if (cudaDeviceGetAttribute(&n.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n.sms < 1 ||
        set_up_byte_attend(n.sms, &n.wave[0]) != cudaSuccess || set_up_byte_attend_tc(n.sms, &n.wave[1]) != cudaSuccess) {
      (void)cudaGetLastError();
      return false;
    }
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

// What a call wants for its scratch: enough for pieces whether it takes them or not (of the most units that pieces are made
// of, where there are more), so that more units, rows or blocks never want less, and a scratch made for the largest call serves
// them all.
static size_t byte_bytes(const ByteDevice& d, int units, int rows, int blocks, bool mass) {
  const int wave = std::max(d.wave[0], d.wave[1]);
  return byte_parts_bytes(units, (size_t)wave + std::min(units, kQaSplitUnits), rows, blocks, mass);
}

// The fewest blocks that keep a CTA of the kernel for so many rows busy: half a block a warp, or a chunk.
static int byte_step(int rows) { return rows <= kByteRows ? kWarps / 2 : kTcChunkBlocks; }

// The largest power of two of CTAs per unit, `most` at most, that fits all units into one wave and leaves each something to do.
static int byte_cluster_size(int units, int blocks, int wave, int step, int most) {
  int cl = most;
  while (cl > 1 && ((long long)units * cl > wave || (cl - 1) * step >= blocks)) cl /= 2;
  return cl;
}

// Three ways, by what a call pays (microseconds on GB300, back to back in a graph, all units of one length, one store: up to
// 64 units of 64 blocks partly from L2, without which they take 2 to 3 more):
//  * a cluster per unit, merged through distributed shared memory: no second kernel, but a unit cannot spread further, and
//    ragged lengths do not balance.  Clusters of 16 fit an eighth of the device or so: 16 units of 64 blocks 15.4 with 16,
//    9.6 with 8.
//  * equal pieces of all units' blocks over one wave, merged by a second kernel (3 to 5).
//  * one CTA per unit, where they are more than a wave and the last round is not too empty for their length.
// 4 or 8 rows a unit:          cluster   whole   pieces     32 rows (16):   cluster        whole          pieces
//    2 units of 64 blocks         6.8               7.6        2 of 32        9.8 ( 8.1)                  10.4 ( 9.2)
//    8 units of 256              14.6              12.8        8 of 64       12.8 (10.5)                  13.5 (10.8)
//   16 units of 64                9.6               9.7       16 of 64       14.8 (12.1)                  14.8 (12.2)
//   16 units of 256              21.7              15.2       16 of 256      33.7 (27.5)                  23.3 (19.1)
//   32 units of 64               10.2              13.4       32 of 64       16.0 (13.0)                  22.3 (18.5)
//   64 units of 64               14.0              17.3       64 of 64       21.9 (17.9)                  30.3 (23.6)
//  128 units of 64               26.4              30.8
//  256 units of 32               25.2              29.1      256 of 32       36.5 (30.0)                  49.9 (39.1)
//  256 units listing 128         86                90        256 listing 81  80.3 (65.5)                  87.7 (70.7)
//  512 units of 64                        83       91        512 of 16                     44.3 (36.3)    64.2 (47.2)
// So clusters where they fill most of a wave and the units are not long (listed blocks balance, lengths may not), and for
// small calls; pieces otherwise.
static BytePlan byte_plan(const ByteDevice& d, int units, int rows, int blocks, bool listed) {
  const int wave = d.wave[rows > kByteRows], rounds = (units + wave - 1) / wave, step = byte_step(rows);
  if (units > kQaSplitUnits || (units > wave && (long long)(rounds * wave - units) * blocks <= 24ll * units))
    return {kWhole, units, 0};
  const int cl = byte_cluster_size(units, blocks, wave, step, 32 * units <= wave ? 16 : 8);
  if (units * cl <= wave && 2 * units * cl > wave && blocks <= (listed ? 160 : 32) * cl) return {kCluster, units * cl, cl};
  if (units * cl <= wave && blocks <= 6 * cl) return {kCluster, units * cl, cl};
  return {kPieces, (int)std::min<long long>(wave, ((long long)units * blocks + step - 1) / step), 0};
}

static void set_scale(ByteArgs& a, float softmax_scale) {
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.f / sqrtf((float)kHeadDim);
  const double exact = scale * 1.4426950408889634;
  const bool normal = exact >= 0x1p-126 && exact <= 0x1p127;
  a.scale = normal ? scale * 1.4426950408889634f : INFINITY;
  a.scale_m = (float)std::frexp(normal ? (double)a.scale : exact, &a.scale_e);
}

static nosa_status byte_attend(ByteArgs& a, void* scratch, size_t scratch_bytes, cudaStream_t st) {
  ByteDevice d;
  if (!byte_device(&d)) return NOSA_ERR_CUDA;
  const BytePlan plan = byte_plan(d, a.units, a.rows, a.blocks, a.sel != nullptr);
  if (scratch_bytes < byte_bytes(d, a.units, a.rows, a.blocks, a.mass != nullptr)) return NOSA_ERR_CAPACITY;
  const size_t parts = (size_t)plan.ctas + a.units;
  unsigned char* p = static_cast<unsigned char*>(scratch);
  a.split = plan.split;
  a.wait_limit = g_wait_limit == kProductsGiveUp ? kWaitCycles : g_wait_limit;
  a.products_late = g_wait_limit < 0;
  a.mass_rows = mass_rows(a.rows);
  a.err = reinterpret_cast<int*>(p);
  a.half = reinterpret_cast<float2*>(p + kQaErrBytes);
  a.part = reinterpret_cast<float*>(a.half + (a.mass ? (size_t)a.units * a.blocks * 2 * a.mass_rows : 0));
  a.total = reinterpret_cast<float2*>(a.part + (plan.split == kPieces ? parts * a.rows * kHeadDim : 0));
  a.stats = a.total + (size_t)a.units * a.rows;
  a.meta = reinterpret_cast<int2*>(a.stats + (plan.split == kPieces ? parts * a.rows : 0));
  cudaError_t e = a.rows > kByteRows ? launch_byte_attend_tc(a, plan.ctas, plan.cluster, st)
                                     : launch_ex(byte_attend_kernel, dim3((unsigned)plan.ctas), dim3(kByteThreads), kByteSmem,
                                                 st, true, plan.cluster, a);
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
  set_scale(a, softmax_scale);
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
  set_scale(a, softmax_scale);
  return byte_attend(a, scratch, scratch_bytes, static_cast<cudaStream_t>(stream));
}
