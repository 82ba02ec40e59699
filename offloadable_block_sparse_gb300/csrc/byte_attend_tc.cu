// Attention over an 8-bit KV block store for 9 to 32 query rows a unit (several drafted tokens of a group of q heads): the same
// sums as byte_attend.cu on the fifth-generation tensor cores.
//
// With so many rows mma.sync spends its time on fragments, and a warp's operands, accumulators and weights do not fit its
// registers (32 rows of 16 units of 65,521 tokens: 961 instructions for 32 tokens, 91 us; 16 rows 54).  Here a CTA of 256
// threads takes a chunk of two blocks, 128 tokens; two threads, with half the rows each, are a token and later a dim:
//   S (128 tokens x 2 x NR) = K . q^T   tcgen05 kind::f8f6f4: K's codes as they are, moved into tensor memory; q as two e4m3
//                                      codes a value (its columns twice), exact to 2^-21 of the row's largest
//   weights of the thread's token: as f16 into shared memory, their sums float32 in registers
//   O^T (128 dims x NR) += s_V (V^T . P)   kind::f16: V's codes converted to f16 and moved into tensor memory, one product per
//                                      block, read back and added in float32 with the block's scale
// The store's order is that of 8 x 4 words' fragments, which tcgen05.st 16x128b takes: both operands reach tensor memory
// without a shuffle, and shared memory only sees the codes arrive and leave (with operands in its 128-byte swizzle, by plain
// stores and stmatrix, 69.5 us where it was then 62.8).  The copies of two chunks, the products with V and the next chunk's
// keys overlap, and the two CTAs of an SM.  Row references are the CTA's: a thread whose score would weigh more than 2^14
// says so at the barrier before the second product, and then all raise theirs and weigh again.
//
// 16 units of 65,521 tokens take 56.2 us with 32 rows and 51.4 with 16, against 40 of HBM: a chunk's chain of waits and two
// barriers, 2,750 cycles of a CTA alone, 3,200 of two on an SM, and some 12,000 cycles before and after the 27 chunks.
// Instructions for one thread (products, copies) take it a hundred cycles each, so they are spread over the warps (all
// products by one warp and all copies by another: 62.8).  64 units of 64 blocks 22.1 us with 32 rows, 18.0 with 16 (mma.sync 36.7 and
// 21.8; 23.7 and 19.8 where the store is not in L2), 256 of 32 35.4 and 29.7 (59.7 and 34.1), 256 listing 81 75.9 and 65.0, 2 of 32
// 9.8 and 8.1 (15.2 and 10.2).  Tried without gain: 128 threads;
// one barrier a chunk, with the next chunk's keys and scores before this one's products (69); prefetching into L2.
#include <type_traits>

#include "byte_split.cuh"
#include "host.h"
#include "tc.cuh"

namespace nosa {

constexpr int kTcTokens = kTcChunkBlocks * kBlock;
constexpr int kTcThreads = 256;
static_assert(2 * kTcTokens == kTcThreads && kTcTokens == kHeadDim, "two threads a token, and a dim");
// shared memory: P (128 tokens x 64 f16, of which the rows' are used) and q (rows twice x 128 codes), both in the 128-byte
// swizzle, and two stages, each the codes of a chunk's blocks
constexpr int kTcP = 0, kTcQ = kTcP + 16384, kTcStage = kTcQ + 8192, kTcStageBytes = kTcChunkBlocks * kByteScales;
constexpr int kTcSmem = kTcStage + 2 * kTcStageBytes + 1024;
static_assert(32 * kQaRowStride * 4 <= kTcStage, "the partial result takes the operands' place");
// tensor memory: scores of both codes of q; a block's result twice; V^T of both blocks (128 dims x 64 f16 each); K (128 tokens
// x 128 codes)
constexpr uint32_t kTcO = 64, kTcV = 128, kTcK = kTcV + kTcChunkBlocks * kBlock / 2, kTcCols = 256;
static_assert(kTcChunkBlocks == 2 && kTcK + kHeadDim / 4 <= kTcCols, "two CTAs share an SM's 512 columns");

// The unit's query rows as operands: row r's codes in rows r (the values') and NR + r (16 times what these leave) of sq, and
// row_factor and the row's own power of two in it.  A warp takes every eighth row, a lane four
// dims.  The largest magnitude of a row is brought into [2^7, 2^8), so that bf16's eight bits are two codes of four down to
// 2^-13 of it.
template <int NR>
__device__ __forceinline__ void load_tc_queries(uint2 (&x)[NR / 8], const ByteArgs& a, int u, int warp, int lane) {
#pragma unroll
  for (int i = 0; i < NR / 8; ++i) {
    const int row = warp + 8 * i;
    x[i] = row < a.rows ? *reinterpret_cast<const uint2*>(a.q + ((size_t)u * a.rows + row) * kHeadDim + 4 * lane) : make_uint2(0, 0);
  }
}
template <int NR>
__device__ __forceinline__ void place_tc_queries(const uint2 (&x)[NR / 8], const ByteArgs& a, unsigned char* sq, float* alpha, float* invs,
                                                 int warp, int lane) {
#pragma unroll
  for (int i = 0; i < NR / 8; ++i) {
    const int row = warp + 8 * i;
    uint32_t big = max(max(x[i].x & 0x7fffu, (x[i].x >> 16) & 0x7fffu), max(x[i].y & 0x7fffu, (x[i].y >> 16) & 0x7fffu));
    big = __reduce_max_sync(0xffffffffu, big);
    const int shift = big == 0 || big >= 0x7f80u ? 0 : min(7 - ((int)(big >> 7) - 127), 126);
    const float f = __uint_as_float((uint32_t)(127 + shift) << 23);
    const float inv = big >= 0x7f80u ? __int_as_float(0x7fc00000) : __uint_as_float((uint32_t)(127 - shift) << 23);
    const float v[4] = {__uint_as_float(x[i].x << 16) * f, __uint_as_float(x[i].x & 0xffff0000u) * f,
                        __uint_as_float(x[i].y << 16) * f, __uint_as_float(x[i].y & 0xffff0000u) * f};
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t c = to_codes(v[2 * k], v[2 * k + 1]), h = codes_to_half2(c);
      const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&h));
      hi |= c << (16 * k);
      lo |= to_codes((v[2 * k] - got.x) * 16.f, (v[2 * k + 1] - got.y) * 16.f) << (16 * k);
    }
    const int at = 16 * ((lane & 7) ^ (row & 7)) + 4 * (lane >> 3);  // K's order of dims (NR is a multiple of 8)
    *reinterpret_cast<uint32_t*>(sq + row * 128 + at) = hi;
    *reinterpret_cast<uint32_t*>(sq + (NR + row) * 128 + at) = lo;
    if (lane == 0) {
      alpha[row] = row_factor(a.scale, inv);
      invs[row] = inv;
    }
  }
}

// A warp moves a tile's K codes into tensor memory: lane i of its 16 is token i, column 16 c + 4 w + t the codes of dims
// 32 t + 16 c + 4 w .. + 3.
__device__ __forceinline__ void place_keys(uint32_t tk, const unsigned char* tile, int lane) {
  uint32_t k[16];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // tokens g + 8 h
      const uint4 x = *reinterpret_cast<const uint4*>(tile + 1024 * h + 512 * c + 16 * lane);
      k[8 * c + h] = x.x, k[8 * c + 2 + h] = x.y, k[8 * c + 4 + h] = x.z, k[8 * c + 6 + h] = x.w;
    }
  tc::st_rows16(tk, k);
}

// A warp converts its quarter of the dims of a block's V codes to f16 and moves them, transposed, into tensor memory:
// lane 8 k + g of the quarter q is dim 16 g + 4 q + k, a column two tokens.
__device__ __forceinline__ void place_values(uint32_t tv, const uint4 (&v)[kByteTiles]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // dims 4 q + 2 i, + 1
    uint32_t f[16];
#pragma unroll
    for (int tile = 0; tile < kByteTiles; ++tile) {
      codes_to_half2(i ? v[tile].z : v[tile].x, f[4 * tile], f[4 * tile + 1]);
      codes_to_half2(i ? v[tile].w : v[tile].y, f[4 * tile + 2], f[4 * tile + 3]);
    }
    tc::st_rows16(tv + ((uint32_t)(16 * i) << 16), f);
  }
}

// Sums of R values over a warp: lane r (mod R) gets value r's.
template <int R>
__device__ __forceinline__ float sum_rows(const float (&v)[R], int lane) {
  float x[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    x[r] = v[r];
#pragma unroll
    for (int o = 16; o >= R; o >>= 1) x[r] += __shfl_xor_sync(0xffffffffu, x[r], o);
  }
#pragma unroll
  for (int n = R / 2; n > 0; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int r = 0; r < n; ++r) {
      const float keep = up ? x[r + n] : x[r], give = up ? x[r] : x[r + n];
      x[r] = keep + __shfl_xor_sync(0xffffffffu, give, n);
    }
  }
  return x[0];
}

// Four consecutive floats of shared memory that all lanes read.
__device__ __forceinline__ void read4(float (&v)[4], const float* p) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}

// NR: rows a unit at most, 16 or 32.
template <int NR>
__global__ void __launch_bounds__(kTcThreads, 2) byte_attend_tc_kernel(const __grid_constant__ ByteArgs a) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bar_raw[2], bar_s, bar_o;  // a stage's copies, a chunk's scores, its products with V
  __shared__ __align__(16) float scales[2][kTcChunkBlocks][4];  // [stage][block]: s_K, s_V
  __shared__ int4 list[kQaList];
  __shared__ int scan[32], found[2];
  __shared__ uint32_t tbase;
  __shared__ __align__(16) float alpha[NR], invs[NR], top[NR], raised[NR], factor[kTcChunkBlocks][NR];
  __shared__ uint32_t best[4][NR];
  __shared__ float sums[4][NR], wr[1][NR], wl[1][NR];
  __shared__ uint32_t poison[NR][4];
  __shared__ float2 merged[NR], final[NR];
  constexpr int R = NR / 2;           // a thread's rows
  constexpr uint32_t idS = tc::plain_idesc(128, 2 * NR, 0), idO = tc::plain_idesc(128, NR, 1);
  unsigned char* sm = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset, so that it stays a shared-memory address)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int quarter = warp & 3, r0 = warp >> 2 ? R : 0, at = 32 * quarter + lane;  // the thread's rows, token and dim's place
  if (tid == 0) {
    mbar_init(&bar_raw[0], kTcChunkBlocks);
    mbar_init(&bar_raw[1], kTcChunkBlocks);
    mbar_init(&bar_s, 1);
    mbar_init(&bar_o, 2);
    fence_mbar_init();
  }
  if (warp == 0) tc::alloc(&tbase, kTcCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_wait();
  pdl_launch_dependents();
  ByteShare share = byte_share(a, kTcChunkBlocks, scan, found);
  const uint32_t tm = tbase, tlane = tm + ((uint32_t)(32 * quarter) << 16), trow = tlane + r0, sa = smem_u32(sm);

  // The stage of the chunk in work, which is also its phase of bar_s (and of bar_o, whose chunk before has the other), and the
  // phases of the stages' copies (a bit each; there too, for want of a register, kLargeBit: o is in units of kLargeUnit).
  int st = 0, ph_raw = 0;
  constexpr int kLargeBit = 4, kOddBias = 1024;
  bool late = false, stuck = false;  // a wait gave up: known to all behind the next barrier; of this warp, for products
  while (share.todo > 0) {
    const int u = share.u;
    const ByteSegment seg = next_segment(a, share);
    float o[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) o[r] = l[r] = 0.f;
    if (tid < NR) {
      top[tid] = kNoRef;
      poison[tid][0] = poison[tid][1] = poison[tid][2] = poison[tid][3] = 0;
    }
    float sv[kTcChunkBlocks] = {};  // the V scales of the chunk whose products are in flight, in the units of o
    bool flying = false;
    // waits are decided for the whole warp: the tensor-memory accesses behind them are warp-collective
    auto wait_for = [&](uint64_t* bar, int phase) {
      stuck |= !__all_sync(0xffffffffu, mbar_wait_bounded(bar, phase, kWaitCycles));
      tc::fence_after();
    };
    auto add_products = [&]() {  // O += s_V of the chunk before: the thread's dim, its rows
      wait_for(&bar_o, st ^ 1);
      uint32_t d[kTcChunkBlocks][R];
#pragma unroll
      for (int b = 0; b < kTcChunkBlocks; ++b) tc::ld(trow + kTcO + b * NR, d[b]);
      tc::wait_ld();
#pragma unroll
      for (int b = 0; b < kTcChunkBlocks; ++b) tc::landed(d[b]);
#pragma unroll
      for (int b = 0; b < kTcChunkBlocks; ++b)
#pragma unroll
        for (int r = 0; r < R; ++r) o[r] = fmaf(__uint_as_float(d[b][r]), sv[b], o[r]);
    };

    uint2 q[NR / 8];
    load_tc_queries<NR>(q, a, u, warp, lane);
    const int batch = a.sel ? kQaList : max(seg.end - seg.first, 1);
    const uint8_t* base = a.store + (size_t)u * a.max_blocks * kByteBlockBytes;
    for (int b0 = seg.first; b0 < seg.end || b0 == seg.first; b0 += batch) {
      int n = max(min(batch, seg.end - b0), 0);
      if (a.sel) {
        if (b0 > seg.first) __syncthreads();  // the list before is used up
        n = byte_list(a, u, seg.len, b0, n, scan, list);
      } else if (seg.len == 0) {
        n = 0;
      }
      const int chunks = late ? 0 : (n + 1) / kTcChunkBlocks;
      // The copies of chunk c into stage `to`: a warp a block, as such an instruction takes a warp a hundred cycles or more, and
      // several lanes of a warp take them one after the other.
      auto issue = [&](int c, int to) {
        if (c >= chunks || !(warp == 1 || warp == 2) || !tc::elect()) return;
        const int b = warp - 1, j = kTcChunkBlocks * c + b;
        if (j >= n) {
          mbar_arrive(&bar_raw[to]);
          return;
        }
        const uint8_t* src = base + (size_t)(a.sel ? list[j].x : b0 + j) * kByteBlockBytes;
        mbar_arrive_expect_tx(&bar_raw[to], kByteScales + 16);
        bulk_copy_g2s(sa + kTcStage + to * kTcStageBytes + b * kByteScales, src, kByteScales, &bar_raw[to]);
        bulk_copy_g2s(smem_u32(scales[to][b]), src + kByteScales, 16, &bar_raw[to]);
      };
      // tokens of the context from block j (of the list) on
      auto left_of = [&](int j) { return j >= n ? 0 : a.sel ? list[j].y : seg.len - (b0 + j) * kBlock; };
      issue(0, st);
      issue(1, st ^ 1);
      if (b0 == seg.first) {  // while the first chunk arrives
        place_tc_queries<NR>(q, a, sm + kTcQ, alpha, invs, warp, lane);
        __syncthreads();
      }
      for (int c = 0; c < chunks; ++c) {
        auto wait_raw = [&](int stage) {
          late |= !__all_sync(0xffffffffu, stage_wait(&bar_raw[stage], ph_raw >> stage & 1, a.wait_limit));
          ph_raw ^= 1 << stage;
        };
        wait_raw(st);
        // a warp takes one of the chunk's eight tiles, whose tokens are its lanes: of K all, of V what must not be looked at
        const int own = 2 * quarter + (warp >> 2), half = warp >> 2;
        unsigned char* stage = sm + kTcStage + st * kTcStageBytes;
        unsigned char* codes = stage + own / kByteTiles * kByteScales + own % kByteTiles * kByteTile;
        const int left = left_of(kTcChunkBlocks * c + own / kByteTiles) - kByteTileTokens * (own % kByteTiles);
        if (left - (a.nq - 1) < kByteTileTokens) clear_byte_tail(codes, poison, left, a.nq, a.rows, lane);
        place_keys(tlane + ((uint32_t)(16 * half) << 16) + kTcK, codes, lane);
        float scale[kTcChunkBlocks];  // V's
#pragma unroll
        for (int b = 0; b < kTcChunkBlocks; ++b) {
          const bool there = kTcChunkBlocks * c + b < n;
          const float2 s = there ? *reinterpret_cast<const float2*>(scales[st][b]) : make_float2(0.f, 0.f);
          scale[b] = s.y;
          if (warp == 6 + b && lane < NR) {  // (a large V scale makes its block's factors odd too, so that it is looked at)
            float f = alpha[lane] * s.x;
            if (!(f <= kWideFactor && s.y <= kLargeScale)) {
              uint32_t odd = 0x7fffffffu;  // a NaN whose low bits are the exponent and kOddBias (0: no scale), or all set
              if (!isnan(alpha[lane])) odd = 0x7fc00000u + (s.x == 0.f ? 0 : kOddBias + a.scale_e + exponent_of(invs[lane]) + exponent_of(s.x));
              f = __uint_as_float(odd);
            }
            factor[b][lane] = f;
          }
        }
        tc::wait_st();
        fence_proxy_async_smem();  // q (generic stores) is read by the tensor core
        tc::fence_before();
        late = __syncthreads_or(late || stuck);
        tc::fence_after();
        if (late) {
          if (c + 1 < chunks) wait_raw(st ^ 1);  // it is in flight
          break;
        }
        if (warp == 0 && tc::elect()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 dims each
            tc::mma_f8_ta(tm, tm + kTcK + 8 * k, tc::sw128_desc(sa + kTcQ + 32 * k), idS, k > 0);
          tc::commit(&bar_s);
        }
        __syncwarp();
        if (flying) add_products();  // then V^T's place and P are free
        // a quarter of the dims of block `half` of V
        uint4 v[kByteTiles];
#pragma unroll
        for (int i = 0; i < kByteTiles; ++i)
          v[i] = *reinterpret_cast<const uint4*>(stage + half * kByteScales + i * kByteTile + kByteV + 512 * quarter + 16 * lane);
        place_values(tlane + kTcV + half * (kBlock / 2), v);
#pragma unroll
        for (int b = 0; b < kTcChunkBlocks; ++b) sv[b] = ph_raw & kLargeBit ? scale[b] * (1.f / kLargeUnit) : scale[b];

        // the thread's token: the logits of its rows
        const int block = at / kBlock, j = kTcChunkBlocks * c + block, mine = left_of(j) - at % kBlock;  // rows of query tokens from nq - mine on see it
        wait_for(&bar_s, st);
        // Weights 2^(logit - top), as f16 into P.  Where one is more than its reference allows (or a factor or a V scale wants
        // care), all raise theirs and weigh again.
        float y[R];
        auto weigh = [&](auto again) {
          const bool pass = again;
          if (pass) {
            stuck |= a.products_late;  // (here it costs nothing; every unit's first chunk comes by)
            // Where a factor is odd, but for rows of q that hold a NaN, all scores become logits in their place first.
            uint32_t odd = __float_as_uint(factor[0][tid % (kTcChunkBlocks * NR)]);
            if (__syncthreads_or(odd > 0x7f800000u && odd != 0x7fffffffu)) {
#pragma unroll 1
              for (int r = 0; r < R; ++r) {
                uint32_t v[2] = {tc::ld1(trow + r), tc::ld1(trow + NR + r)};
                tc::wait_ld();
                tc::landed(v);
                float x = fmaf(__uint_as_float(v[1]), 0.0625f, __uint_as_float(v[0]));
                const float f = factor[block][r0 + r];
                odd = __float_as_uint(f);
                const bool wide = odd > 0x7f800000u && odd != 0x7fffffffu;
                x = wide ? wide_logit(x * a.scale_m, (int)(odd - 0x7fc00000u) - kOddBias) : x * f;
                tc::st1(trow + r, __float_as_uint(x));
                tc::st1(trow + NR + r, 0u);
              }
              tc::wait_st();
              __syncthreads();
              if (tid < kTcChunkBlocks * NR) factor[0][tid] = 1.f;
              __syncthreads();
            }
          }
          uint32_t d[R], e[R];
          tc::ld(trow, d);
          tc::ld(trow + NR, e);
          tc::wait_ld();
          tc::landed(d);
          tc::landed(e);
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            float f[4];
            read4(f, &factor[block][r0 + r]);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[r + i] = fmaf(__uint_as_float(e[r + i]), 0.0625f, __uint_as_float(d[r + i])) * f[i];
          }
          if (mine < a.nq) {
            int query = r0 % a.nq;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              if (query < a.nq - mine) y[r] = -INFINITY;
              query = query + 1 == a.nq ? 0 : query + 1;
            }
          }
          if (pass) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const uint32_t m = __reduce_max_sync(0xffffffffu, orderable(y[r]));
              if (lane == 0) best[quarter][r0 + r] = m;
            }
            __syncthreads();
            if (tid < NR) {
              const uint32_t m = max(max(best[0][tid], best[1][tid]), max(best[2][tid], best[3][tid]));
              const float b = __uint_as_float(m & 0x80000000u ? m ^ 0x80000000u : ~m);
              float f = 1.f;
              if (b - top[tid] > kTopWeight) {
                const float ref = reference(b);
                f = ex2(top[tid] - ref);
                top[tid] = ref;
              }
              raised[tid] = f;
            }
            __syncthreads();
            float unit = 1.f;
            if (!(ph_raw & kLargeBit) && fmaxf(sv[0], sv[1]) > kLargeScale) {  // (the products of the chunks before are in o)
              ph_raw |= kLargeBit;
              unit = 1.f / kLargeUnit;
              sv[0] *= unit;
              sv[1] *= unit;
            }
#pragma unroll
            for (int r = 0; r < R; r += 4) {
              float f[4];
              read4(f, &raised[r0 + r]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[r + i] *= f[i] * unit;
                l[r + i] *= f[i];
              }
            }
          }
          float over = -INFINITY;
          uint32_t p[R / 2];
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            float ref[4];
            read4(ref, &top[r0 + r]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = y[r + i] - ref[i];
              over = max_or_nan(over, x);
              y[r + i] = ex2(x);
            }
            p[r / 2] = pack_half2(y[r], y[r + 1]);
            p[r / 2 + 1] = pack_half2(y[r + 2], y[r + 3]);
          }
#pragma unroll
          for (int i = 0; i < R / 8; ++i)
            *reinterpret_cast<uint4*>(sm + kTcP + at * 128 + 16 * ((r0 / 8 + i) ^ (at & 7))) =
                make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
          tc::wait_st();             // V^T
          fence_proxy_async_smem();  // P is read by the tensor core
          tc::fence_before();
          const bool raise = __syncthreads_or(!(over <= kTopWeight));
          tc::fence_after();
          return raise;
        };
        if constexpr (NR == 16) {  // (64 units of 64 blocks: 19.9 us so, 20.2 as below; 32 rows 24.3 and 23.9)
          if (weigh(std::false_type{})) weigh(std::true_type{});
        } else {
#pragma unroll 1
          for (bool pass = false; weigh(pass) && !pass; pass = true) {
          }
        }
        if ((warp == 3 || warp == 5) && tc::elect()) {
          const int b = warp == 5;
          {
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 16 tokens each
              tc::mma_f16_ta(tm + kTcO + b * NR, tm + kTcV + b * (kBlock / 2) + 8 * k, tc::sw128_desc_mn(sa + kTcP + b * 8192 + 2048 * k, 16384), idO, k > 0);
          }
          tc::commit(&bar_o);
        }
        __syncwarp();
        issue(c + 2, st);  // all have read the stage
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] += y[r];
        if (a.mass && j < n) {  // a warp's tokens are half a block
          const float sum = sum_rows<R>(y, lane);
          const size_t entry = (size_t)u * a.blocks + (a.sel ? list[j].z : b0 + j);
          if (lane < R && r0 + lane < a.rows)
            a.half[(entry * 2 + (quarter & 1)) * a.mass_rows + r0 + lane] = make_float2(top[r0 + lane], sum);
        }
        flying = true;
        st ^= 1;
      }
      if (late) break;
    }
    if (flying) add_products();
    late = __syncthreads_or(late || stuck);  // also: the operands' places are free
    if (late && tid == 0) atomicOr(a.err, kErrTimeout);

    // the partial: the thread's dim of its rows
    float* part = reinterpret_cast<float*>(sm);
    const int dim = 16 * (at & 7) + (at >> 3);
#pragma unroll
    for (int r = 0; r < R; ++r) part[(r0 + r) * kQaRowStride + dim] = o[r];
    const float sum = sum_rows<R>(l, lane);
    if (lane < R) sums[quarter][r0 + lane] = sum;
    __syncthreads();
    if (tid < NR) {
      wr[0][tid] = top[tid];
      wl[0][tid] = late ? __int_as_float(0x7fc00000) : (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]);
    }
    __syncthreads();
    finish_segment<1, NR>(a, share, seg, part, wr, wl, poison, merged, final, ph_raw & kLargeBit);
    ph_raw &= ~kLargeBit;
    if (share.todo > 0) {
      fence_proxy_async_smem();
      __syncthreads();
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(tm, kTcCols);
}

template <int NR>
static cudaError_t set_up_tc() {
  cudaError_t e = cudaFuncSetAttribute(byte_attend_tc_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(byte_attend_tc_kernel<NR>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(byte_attend_tc_kernel<NR>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  return e;
}

// Two CTAs share an SM by registers, shared memory and tensor-memory columns.  (The occupancy query counts one for any kernel
// that allocates tensor memory, whatever its shared memory.)
cudaError_t set_up_byte_attend_tc(int sms, int* wave) {
  *wave = 2 * sms;
  const cudaError_t e = set_up_tc<16>();
  return e == cudaSuccess ? set_up_tc<32>() : e;
}

cudaError_t launch_byte_attend_tc(const ByteArgs& a, int ctas, int cluster, cudaStream_t st) {
  return launch_ex(a.rows <= 16 ? byte_attend_tc_kernel<16> : byte_attend_tc_kernel<32>, dim3((unsigned)ctas), dim3(kTcThreads),
                   kTcSmem, st, true, cluster, a);
}

}  // namespace nosa
