// Rotary positions (nosa_rope_make, nosa_rope).
//
// A pair's angle at position p is p f.  Angles are counted in turns as 64-bit fractions: p times f / 2 pi in units of 2^-64
// turns wraps as the angle does, so the reduction is an integer product and exact at any position (float32 would lose
// 2^-4 of a radian a million tokens out, float64 is slow here).  The fraction's top 32 bits give sine and cosine.
//
// A CTA takes a tile of tokens and heads of one tensor: first the tile's sines and cosines, once for all its heads, into
// shared memory; then eight threads a row, 16 dims each, several rows in flight, the first of them loaded before the angles
// are computed.  A row is 256 bytes in and 256 out: bound by HBM.  8 sequences of 16,384 tokens with 16 + 2 heads (1.21 GB)
// take 182 us, 0.99 of measured HBM (CTAs of 256 threads: 198 before the frequencies came from shared memory, 190 with
// 128); one token of 32 sequences 2.7 us.  One head a token leaves a tile of 32 rows to 2,048 sines: 0.4 of HBM.  Rows
// through shared memory (98 dims in halves) 0.47, value by value (rows that begin anywhere) 0.28.
#include <algorithm>
#include <cmath>

#include "host.h"
#include "ptx.cuh"

namespace nosa {

constexpr int kRopeThreads = 128, kRopeRows = kRopeThreads / 8;  // rows side by side
constexpr int kRopeTokens = 32, kRopeHeads = 32, kRopeTile = 128;  // a tile: so many tokens and heads at most, rows about
constexpr int kRopePairs = kHeadDim / 2;
constexpr int kRopeFlight = 4;  // rows a thread has in flight

struct RopeView {
  const uint16_t* x;
  uint16_t* y;
  long long xs[3], ys[3];
  int heads, tokens, head_tiles;  // a tile's tokens; tiles of heads
  int vec, same;                  // rows that begin at whole 16-byte words; in place
};

struct RopeArgs {
  RopeView v[2];
  int tiles0, token_tiles0, token_tiles1;  // the first tensor's tiles; tiles of tokens of each
  int n, rot, interleaved, inverse;
  float factor;
  const int32_t* pos;
  const int32_t* count;
  int32_t* err;
  uint64_t turn[kRopePairs];
};

// Where a token's pair i is kept: in the order in which eight threads read four pairs each without bank conflicts.
__device__ __forceinline__ int pair_place(int i) { return (i & 4 ? 32 : 0) + (i >> 3) * 4 + (i & 3); }

__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = a;
  a = fmaf(x, c, -(b * s));
  b = fmaf(b, c, x * s);
}
__device__ __forceinline__ float lo_float(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_float(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// kStaged: rows of whole words go through shared memory, for pairs half the rotated dims apart that do not lie in a thread's
// words (the rotated dims are no multiple of 16).
template <bool kStaged>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float cosine[kRopeTokens][kRopePairs], sine[kRopeTokens][kRopePairs];
  __shared__ __align__(16) uint16_t staged[kStaged ? kRopeRows : 1][kHeadDim + 8];
  __shared__ uint64_t turn[kRopePairs];  // (a parameter that every lane reads at its own place is read lane by lane)
  pdl_wait();
  pdl_launch_dependents();
  const bool second = (int)blockIdx.x >= a.tiles0;
  const RopeView& v = a.v[second];
  int i = blockIdx.x - (second ? a.tiles0 : 0);
  const int hd = i % v.head_tiles;
  i /= v.head_tiles;
  const int token_tiles = second ? a.token_tiles1 : a.token_tiles0;
  const int t0 = i % token_tiles * v.tokens, b = i / token_tiles;
  const int c0 = a.count ? a.count[b] : a.n, count = min(max(c0, 0), a.n);
  if (blockIdx.x < a.tiles0 && hd == 0 && t0 == 0 && threadIdx.x == 0 && c0 != count && a.err) atomicOr(a.err, kErrBounds);
  const int tokens = min(v.tokens, count - t0);
  if (tokens <= 0) return;
  const int h0 = hd * kRopeHeads, heads = min(kRopeHeads, v.heads - h0), pairs = a.rot / 2;
  const long long p0 = (a.pos ? (long long)a.pos[b] : 0) + t0;
  const int rows = tokens * heads, part = threadIdx.x & 7;
  const uint16_t* xb = v.x + b * v.xs[0] + h0 * v.xs[1] + t0 * v.xs[2];
  uint16_t* yb = v.y + b * v.ys[0] + h0 * v.ys[1] + t0 * v.ys[2];
  // whole words: a thread's 16 dims, eight pairs (some of them, where the rotated dims end among interleaved ones) or what is
  // copied, of rows r0, r0 + kRopeRows, ...
  const bool turns = 16 * part < a.rot, idle = !v.vec || (!turns && v.same && !kStaged);
  const bool apart = turns && !a.interleaved && !kStaged;
  const int d0 = apart ? 8 * part : 16 * part, d1 = apart ? d0 + pairs : d0 + 8, mine = min(max(pairs - 8 * part, 0), 8);
  int r0 = threadIdx.x >> 3;
  uint4 x[kRopeFlight][2];
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < kRopeFlight; ++k) {
      const int r = r0 + k * kRopeRows;
      if (r >= rows) break;
      const uint16_t* p = xb + r % heads * v.xs[1] + r / heads * v.xs[2];
      x[k][0] = *reinterpret_cast<const uint4*>(p + d0);
      x[k][1] = *reinterpret_cast<const uint4*>(p + d1);
    }
  };
  if (!idle) load();  // while the angles are computed
  if (threadIdx.x < kRopePairs) turn[threadIdx.x] = a.turn[threadIdx.x];
  __syncthreads();
  for (int k = threadIdx.x; k < tokens * kRopePairs; k += kRopeThreads) {
    const int t = k / kRopePairs, p = k % kRopePairs;
    if (p >= pairs) continue;
    const uint64_t turns64 = (uint64_t)(p0 + t) * turn[p];
    float s, c;
    sincospif((float)(int32_t)(uint32_t)(turns64 >> 32) * 0x1p-31f, &s, &c);
    if (a.inverse) s = -s;
    const int at = pair_place(p);
    cosine[t][at] = c * a.factor;
    sine[t][at] = s * a.factor;
  }
  __syncthreads();

  if (kStaged && v.vec) {  // (a row's eight threads are in one warp; a thread rotates up to eight pairs, 8 part ..)
    uint16_t* row = staged[kStaged ? threadIdx.x >> 3 : 0];
    for (; r0 - (int)(threadIdx.x >> 3) < rows; r0 += kRopeRows * kRopeFlight, load()) {
#pragma unroll
      for (int k = 0; k < kRopeFlight; ++k) {
        const int r = r0 + k * kRopeRows, t = r / heads;
        const bool in = r < rows;
        uint32_t w[4] = {}, z[4] = {};  // the first values of the pairs, and the second ones
        if (in) {
          *reinterpret_cast<uint4*>(row + d0) = x[k][0];
          *reinterpret_cast<uint4*>(row + d1) = x[k][1];
        }
        __syncwarp();
        if (in && mine > 0) {
          const uint4 u = *reinterpret_cast<const uint4*>(row + 8 * part);
          const uint32_t first[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // two pairs
            const int at = (e & 2 ? 32 : 0) + 4 * part + 2 * (e & 1);
            const float2 c = *reinterpret_cast<const float2*>(&cosine[t][at]), s = *reinterpret_cast<const float2*>(&sine[t][at]);
            float f0 = lo_float(first[e]), f1 = bf16_to_float(row[pairs + 8 * part + 2 * e]);
            float g0 = hi_float(first[e]), g1 = bf16_to_float(row[pairs + 8 * part + 2 * e + 1]);
            rotate(f0, f1, c.x, s.x);
            rotate(g0, g1, c.y, s.y);
            w[e] = pack_bf16x2(f0, g0);
            z[e] = pack_bf16x2(f1, g1);
          }
        }
        __syncwarp();
        if (in) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < mine) {
              row[8 * part + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
              row[pairs + 8 * part + e] = (uint16_t)(z[e >> 1] >> (16 * (e & 1)));
            }
        }
        __syncwarp();
        if (in) {
          uint16_t* p = yb + r % heads * v.ys[1] + t * v.ys[2];
          *reinterpret_cast<uint4*>(p + d0) = *reinterpret_cast<const uint4*>(row + d0);
          *reinterpret_cast<uint4*>(p + d1) = *reinterpret_cast<const uint4*>(row + d1);
        }
        __syncwarp();
      }
    }
    return;
  }
  if (!kStaged && v.vec) {
    if (idle) return;
    for (; r0 < rows; r0 += kRopeRows * kRopeFlight, load()) {
#pragma unroll
      for (int k = 0; k < kRopeFlight; ++k) {
        const int r = r0 + k * kRopeRows;
        if (r >= rows) break;
        if (turns) {
          const int t = r / heads;
          uint32_t w[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // four pairs each
            const float4 c4 = *reinterpret_cast<const float4*>(&cosine[t][32 * q + 4 * part]);
            const float4 s4 = *reinterpret_cast<const float4*>(&sine[t][32 * q + 4 * part]);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
            if (a.interleaved) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float f0 = lo_float(w[4 * q + e]), f1 = hi_float(w[4 * q + e]);
                rotate(f0, f1, c[e], s[e]);
                if (4 * q + e < mine) w[4 * q + e] = pack_bf16x2(f0, f1);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // two pairs: words 2 q + e of both halves
                const uint32_t u0 = w[2 * q + e], u1 = w[4 + 2 * q + e];
                float f0 = lo_float(u0), f1 = lo_float(u1), g0 = hi_float(u0), g1 = hi_float(u1);
                rotate(f0, f1, c[2 * e], s[2 * e]);
                rotate(g0, g1, c[2 * e + 1], s[2 * e + 1]);
                w[2 * q + e] = pack_bf16x2(f0, g0);
                w[4 + 2 * q + e] = pack_bf16x2(f1, g1);
              }
            }
          }
          x[k][0] = make_uint4(w[0], w[1], w[2], w[3]);
          x[k][1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        uint16_t* p = yb + r % heads * v.ys[1] + r / heads * v.ys[2];
        *reinterpret_cast<uint4*>(p + d0) = x[k][0];
        *reinterpret_cast<uint4*>(p + d1) = x[k][1];
      }
    }
    return;
  }
  for (int r = threadIdx.x >> 3; r < rows; r += kRopeRows) {  // value by value
    const int t = r / heads;
    const uint16_t* x = xb + r % heads * v.xs[1] + t * v.xs[2];
    uint16_t* y = yb + r % heads * v.ys[1] + t * v.ys[2];
    for (int p = part; p < pairs; p += 8) {
      const int i0 = a.interleaved ? 2 * p : p, i1 = a.interleaved ? 2 * p + 1 : p + pairs, at = pair_place(p);
      float f0 = bf16_to_float(x[i0]), f1 = bf16_to_float(x[i1]);
      rotate(f0, f1, cosine[t][at], sine[t][at]);
      const uint32_t w = pack_bf16x2(f0, f1);
      y[i0] = (uint16_t)w;
      y[i1] = (uint16_t)(w >> 16);
    }
    if (!v.same)
      for (int d = a.rot + part; d < kHeadDim; d += 8) y[d] = x[d];
  }
}

}  // namespace nosa

using namespace nosa;

extern "C" nosa_status nosa_rope_make(const nosa_rope_config* cfg, nosa_rope_table* out) {
  if (!cfg || !out || cfg->struct_size != sizeof(nosa_rope_config)) return NOSA_ERR_INVALID_ARG;
  const nosa_rope_config& c = *cfg;
  auto real = [](double x, double least) { return x >= least && std::isfinite(x); };
  if (c.rot_dims < 2 || c.rot_dims > kHeadDim || c.rot_dims % 2 || c.interleaved < 0 || c.interleaved > 1 ||
      c.scaling < NOSA_ROPE_PLAIN || c.scaling > NOSA_ROPE_PARTS || !real(c.base, 1.0) || !real(c.attention_factor, 0.0) ||
      !std::isfinite((float)c.attention_factor))
    return NOSA_ERR_INVALID_ARG;
  if (c.scaling != NOSA_ROPE_PLAIN && !real(c.factor, 1.0)) return NOSA_ERR_INVALID_ARG;
  if (c.scaling == NOSA_ROPE_PARTS &&
      (!real(c.low, 0.0) || !real(c.high, 0.0) || !(c.high > c.low) || !real(c.original, 0.0) || !(c.original > 0)))
    return NOSA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  const int r = c.rot_dims;
  double base = c.base;
  if (c.scaling == NOSA_ROPE_BASE && r > 2) base *= std::pow(c.factor, (double)r / (r - 2));
  if (!std::isfinite(base)) return NOSA_ERR_INVALID_ARG;
  nosa_rope_table t = {};
  t.struct_size = sizeof(nosa_rope_table);
  t.rot_dims = r;
  t.interleaved = c.interleaved;
  t.attention_factor = c.attention_factor > 0 ? (float)c.attention_factor : 1.f;
  for (int i = 0; i < r / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (c.scaling == NOSA_ROPE_LINEAR) f /= c.factor;
    if (c.scaling == NOSA_ROPE_PARTS) {
      const double g = std::min(std::max((c.original * f / two_pi - c.low) / (c.high - c.low), 0.0), 1.0);
      f *= g + (1 - g) / c.factor;
    }
    t.turn[i] = (uint64_t)std::llround(std::ldexp(f / two_pi, 63)) << 1;  // f <= 1: below a sixth of a turn
  }
  *out = t;
  return NOSA_OK;
}

extern "C" nosa_status nosa_rope(const nosa_rope_table* table, const nosa_rope_view* views, int n_views, int batch,
                                 int n_tokens, const int32_t* pos, const int32_t* count, int inverse, int32_t* err_out,
                                 void* stream) {
  if (!table || !views || n_views < 1 || n_views > 2 || batch < 1 || n_tokens < 1 || n_tokens > (1 << 30))
    return NOSA_ERR_INVALID_ARG;
  if (table->struct_size != sizeof(nosa_rope_table) || table->rot_dims < 2 || table->rot_dims > kHeadDim ||
      table->rot_dims % 2)
    return NOSA_ERR_INVALID_ARG;
  auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (off(pos, 4) || off(count, 4) || off(err_out, 4)) return NOSA_ERR_INVALID_ARG;
  RopeArgs a{};
  a.n = n_tokens;
  a.rot = table->rot_dims;
  a.interleaved = table->interleaved;
  a.inverse = inverse != 0;
  a.factor = table->attention_factor;
  a.pos = pos;
  a.count = count;
  a.err = err_out;
  std::copy(table->turn, table->turn + kRopePairs, a.turn);
  long long tiles = 0;
  for (int i = 0; i < n_views; ++i) {
    const nosa_rope_view& w = views[i];
    RopeView& v = a.v[i];
    if (!w.x || !w.y || w.heads < 1 || w.heads > (1 << 20) || off(w.x, 2) || off(w.y, 2)) return NOSA_ERR_INVALID_ARG;
    const long long extent[3] = {batch, w.heads, n_tokens};
    bool same = w.x == w.y, whole = !off(w.x, 16) && !off(w.y, 16);
    for (int d = 0; d < 3; ++d) {
      if (extent[d] > 1) {
        if (w.x_stride[d] < 0 || w.y_stride[d] < kHeadDim) return NOSA_ERR_INVALID_ARG;
        if (w.x_stride[d] >= (1ll << 40) || w.y_stride[d] >= (1ll << 40)) return NOSA_ERR_INVALID_ARG;
        if (w.x == w.y && w.x_stride[d] != w.y_stride[d]) return NOSA_ERR_INVALID_ARG;
        v.xs[d] = w.x_stride[d];
        v.ys[d] = w.y_stride[d];
        whole = whole && v.xs[d] % 8 == 0 && v.ys[d] % 8 == 0;
      }
    }
    v.x = w.x;
    v.y = w.y;
    v.heads = w.heads;
    v.vec = whole;
    v.same = same;
    const int heads = std::min(w.heads, kRopeHeads);
    v.head_tiles = (w.heads + kRopeHeads - 1) / kRopeHeads;
    v.tokens = std::min(kRopeTokens, std::max(1, kRopeTile / heads));
    const int token_tiles = (n_tokens + v.tokens - 1) / v.tokens;
    (i ? a.token_tiles1 : a.token_tiles0) = token_tiles;
    if ((long long)batch * token_tiles >= (1ll << 31)) return NOSA_ERR_INVALID_ARG;
    tiles += (long long)batch * token_tiles * v.head_tiles;
    if (tiles >= (1ll << 31)) return NOSA_ERR_INVALID_ARG;
    if (i == 0) a.tiles0 = (int)tiles;
  }
  const bool staged = !a.interleaved && a.rot % 16 != 0;
  const cudaError_t e = launch_ex(staged ? rope_kernel<true> : rope_kernel<false>, dim3((unsigned)tiles), dim3(kRopeThreads), 0,
                                  static_cast<cudaStream_t>(stream), true, 0, a);
  if (e == cudaSuccess) return NOSA_OK;
  (void)cudaGetLastError();
  return NOSA_ERR_CUDA;
}
