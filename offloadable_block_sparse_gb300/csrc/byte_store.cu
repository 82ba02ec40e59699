// Writing the 8-bit KV block store (nosa_byte_append) and reading it back (nosa_byte_read).
//
// A scale belongs to a whole block of 64 tokens, so a CTA takes a block: four warps its K tiles, four its V tiles, each
// lane in the store's own layout (byte_core.cuh).  The lanes hold the new values in registers while the block's
// largest magnitude goes through shared memory.  A token and unit is 512 bytes of bf16 and 256 of the store.
#include <algorithm>

#include "byte_core.cuh"
#include "host.h"

namespace nosa {

constexpr int kByteWarps = 8;  // four tiles of K, four of V

// The exponent of the smallest power of two s with x <= 448 s, for the bf16 magnitude `top` > 0, within the scales' range:
// 448 = 1.75 x 2^8, so it is x's exponent less 8, or one more where x's mantissa is above 1.75.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u);
  return min(max(e, kLeastScale), kMostScale);
}
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Two bf16 values times inv as e4m3 codes.
__device__ __forceinline__ uint32_t two_codes(uint32_t x, float inv) {
  const float lo = __uint_as_float(x << 16) * inv, hi = __uint_as_float(x & 0xffff0000u) * inv;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  uint32_t c = r;
  if ((x & 0x7fffu) >= 0x7f80u) c = (c & 0xff00u) | 0x7fu;  // the conversion saturates infinities
  if ((x & 0x7fff0000u) >= 0x7f800000u) c = (c & 0x00ffu) | 0x7f00u;
  return c;
}

// Four codes c as e4m3(c ratio), ratio a power of two in f16x2.  The product is exact unless it is below 2^-10, where
// it becomes 0 either way.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, __half2 ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = codes_to_half2(i ? w >> 16 : w);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h), ratio);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&y)));
    out |= (uint32_t)r << (16 * i);
  }
  return out;
}

// The magnitude of the largest finite of the values in a register of two bf16, among which may be others.
__device__ __forceinline__ uint32_t finite_max(uint32_t top, uint32_t x) {
  const uint32_t lo = x & 0x7fffu, hi = (x >> 16) & 0x7fffu;
  top = lo < 0x7f80u ? max(top, lo) : top;
  return hi < 0x7f80u ? max(top, hi) : top;
}

__global__ void __launch_bounds__(kByteWarps * 32)
    byte_append_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, uint8_t* __restrict__ store, int n,
                       int max_blocks, const int32_t* __restrict__ pos, const int32_t* __restrict__ count,
                       const int32_t* __restrict__ slot_blk, int blocks, int32_t* err) {
  __shared__ uint32_t tops[kByteWarps];
  __shared__ int found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u = blockIdx.x / blocks, bi = blockIdx.x % blocks;
  pdl_wait();
  pdl_launch_dependents();
  const long long p0 = pos ? pos[u] : 0, cap = (long long)max_blocks * kBlock;
  const int c0 = count ? count[u] : n, c = min(max(c0, 0), n);
  if (bi == 0 && threadIdx.x == 0 && err && (c0 != c || (c > 0 && (p0 < 0 || (!slot_blk && p0 + c > cap)))))
    atomicOr(err, kErrBounds);
  const long long block = (p0 >> 6) + bi;  // an arithmetic shift: negative positions round down
  const int rel = (int)(block * kBlock - p0);  // the block's first token among the new ones, -63 at least
  if (c == 0 || rel >= c || block < 0) return;
  long long row = block;
  if (slot_blk) {
    if (threadIdx.x == 0) found = max_blocks;
    __syncthreads();
    for (int r = threadIdx.x; r < max_blocks; r += kByteWarps * 32)
      if (slot_blk[(size_t)u * max_blocks + r] == block) atomicMin(&found, r);
    __syncthreads();
    row = found;
    if (row == max_blocks && threadIdx.x == 0 && err) atomicOr(err, kErrBounds);
  }
  if (row >= max_blocks) return;
  uint8_t* dst = store + ((size_t)u * max_blocks + row) * kByteBlockBytes;
  const bool is_v = warp >= 4, begun = rel < 0;
  const int tile = warp & 3, first = rel + tile * kByteTileTokens;  // the tile's first token among the new ones
  auto is_new = [&](int j) { return (unsigned)(first + j) < (unsigned)c; };  // the tile's token j

  // the lane's new values, in its own order, and the block's earlier codes where they may be wanted
  uint4 x[8], old[4];
  const uint16_t* src = (is_v ? v : k) + (size_t)u * n * kHeadDim;
  bool any = false, all = true;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // K: tokens g, g + 8, halves of 16 dims; V: the four tokens
    const int j = is_v ? 2 * t + (i & 1) + 8 * (i >> 1) : g + 8 * (i >> 1);
    const bool in = is_new(j);
    any |= in;
    all &= in;
    const uint16_t* p = src + (size_t)(in ? first + j : 0) * kHeadDim + (is_v ? 16 * g : 32 * t + 16 * (i & 1));
    x[2 * i] = in ? ld_stream_v4(p) : zero;
    x[2 * i + 1] = in ? ld_stream_v4(p + 8) : zero;
  }
  uint8_t* words = dst + tile * kByteTile + (is_v ? kByteV : 0) + 16 * lane;
  const bool read = begun || (any && !all);
#pragma unroll
  for (int i = 0; i < 4; ++i) old[i] = read ? *reinterpret_cast<const uint4*>(words + 512 * i) : zero;
  float had = 0.f;  // the block's scale: what is not a scale (a store that was never written) counts as none
  if (begun) {
    const float s = *reinterpret_cast<const float*>(dst + kByteScales + (is_v ? 4 : 0));
    if (s >= power_of_2(kLeastScale) && s <= power_of_2(kMostScale) && (__float_as_uint(s) & 0x7fffffu) == 0) had = s;
  }

  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = finite_max(top, w[e]);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();  // also: every thread has the old scale
  top = max(max(tops[warp & 4], tops[(warp & 4) + 1]), max(tops[(warp & 4) + 2], tops[(warp & 4) + 3]));
  const float need = top ? power_of_2(scale_exponent(top)) : 0.f, scale = fmaxf(had, need);
  const float inv = scale > 0.f ? power_of_2(127 - (int)(__float_as_uint(scale) >> 23)) : 1.f;
  if (tile == 0 && lane == 0) *reinterpret_cast<float*>(dst + kByteScales + (is_v ? 4 : 0)) = scale;
  const bool grown = had > 0.f && scale > had;
  if (!any && !grown) return;
  const __half2 ratio = __float2half2_rn(grown ? fmaxf(had * inv, 0x1p-24f) : 1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4], keep[4];  // bytes of w that are not new
    if (!is_v) {  // chunk i: token g + 8 (i / 2), dims 32 t + 16 (i % 2) ..
      const uint4 a = x[2 * i], b = x[2 * i + 1];
      w[0] = two_codes(a.x, inv) | two_codes(a.y, inv) << 16;
      w[1] = two_codes(a.z, inv) | two_codes(a.w, inv) << 16;
      w[2] = two_codes(b.x, inv) | two_codes(b.y, inv) << 16;
      w[3] = two_codes(b.z, inv) | two_codes(b.w, inv) << 16;
#pragma unroll
      for (int e = 0; e < 4; ++e) keep[e] = is_new(g + 8 * (i >> 1)) ? 0u : 0xffffffffu;
    } else {  // chunk i: dims 16 g + 4 i .. + 3; word 2 jj + half: dims 2 jj, 2 jj + 1 of them, tokens 2t + 8 half, + 1
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int jj = e >> 1, half = e & 1, at = 2 * i + jj;  // of a token's 8 registers of two dims
        const uint4 a = x[4 * half + (at >> 2)], b = x[4 * half + 2 + (at >> 2)];
        const uint32_t xa = (at & 3) == 0 ? a.x : (at & 3) == 1 ? a.y : (at & 3) == 2 ? a.z : a.w;
        const uint32_t xb = (at & 3) == 0 ? b.x : (at & 3) == 1 ? b.y : (at & 3) == 2 ? b.z : b.w;
        w[e] = __byte_perm(two_codes(xa, inv), two_codes(xb, inv), 0x5140);
        keep[e] = (is_new(2 * t + 8 * half) ? 0u : 0x00ff00ffu) | (is_new(2 * t + 8 * half + 1) ? 0u : 0xff00ff00u);
      }
    }
    const uint32_t o[4] = {old[i].x, old[i].y, old[i].z, old[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (w[e] & ~keep[e]) | ((grown ? rescaled(o[e], ratio) : o[e]) & keep[e]);
    if (grown || is_v || keep[0] == 0) *reinterpret_cast<uint4*>(words + 512 * i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Two codes times the scale as bf16x2, exactly.
__device__ __forceinline__ uint32_t two_values(uint32_t two, float scale) {
  const uint32_t h = codes_to_half2(two);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x * scale, f.y * scale);
}

// A CTA takes a listed block, four warps its K tiles, four its V tiles.
__global__ void __launch_bounds__(kByteWarps * 32)
    byte_read_kernel(const uint8_t* __restrict__ store, int max_blocks, const int32_t* __restrict__ blocks,
                     const int32_t* __restrict__ slots, int n_blocks, const int32_t* __restrict__ lens,
                     uint16_t* __restrict__ kv, int32_t* err) {
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, tile = warp & 3;
  const bool is_v = warp >= 4;
  const int u = blockIdx.x / n_blocks, j = blockIdx.x % n_blocks;
  const int b = blocks ? blocks[blockIdx.x] : j, row = b >= 0 && slots ? slots[blockIdx.x] : b;
  const bool held = b >= 0 && row >= 0 && row < max_blocks;
  if (b >= 0 && !held && err && threadIdx.x == 0) atomicOr(err, kErrBounds);
  const long long left =
      !held ? 0 : lens ? (long long)lens[u] - ((long long)b * kBlock + tile * kByteTileTokens) : kByteTileTokens;
  const int rows = (int)min(max(left, 0ll), (long long)kByteTileTokens);  // rows of the tile below the length
  uint16_t* out = kv + ((size_t)blockIdx.x * 2 + is_v) * kBlockElems + tile * kByteTileTokens * kHeadDim;
  const uint8_t* src = store + ((size_t)u * max_blocks + (held ? row : 0)) * kByteBlockBytes;
  const uint8_t* words = src + tile * kByteTile + (is_v ? kByteV : 0) + 16 * lane;
  const float scale = rows > 0 ? *reinterpret_cast<const float*>(src + kByteScales + (is_v ? 4 : 0)) : 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = is_v ? 2 * t < rows : g + 8 * (i >> 1) < rows;
    c[i] = in ? ld_stream_v4(words + 512 * i) : zero;
  }
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t* p = out + (g + 8 * (i >> 1)) * kHeadDim + 32 * t + 16 * (i & 1);
      __stcs(reinterpret_cast<uint4*>(p), make_uint4(two_values(c[i].x, scale), two_values(c[i].x >> 16, scale),
                                                     two_values(c[i].y, scale), two_values(c[i].y >> 16, scale)));
      __stcs(reinterpret_cast<uint4*>(p + 8), make_uint4(two_values(c[i].z, scale), two_values(c[i].z >> 16, scale),
                                                         two_values(c[i].w, scale), two_values(c[i].w >> 16, scale)));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // token 2t + 8 (i / 2) + i % 2
    const int half = i >> 1, par = i & 1, token = 2 * t + 8 * half + par;
    uint32_t o[8];
#pragma unroll
    for (int at = 0; at < 8; ++at) {  // two dims each
      const uint4 w = c[at >> 1];
      const uint32_t x = at & 1 ? (half ? w.w : w.z) : (half ? w.y : w.x);
      o[at] = token < rows ? two_values(__byte_perm(x, 0, par ? 0x4431 : 0x4420), scale) : 0u;
    }
    uint16_t* p = out + token * kHeadDim + 16 * g;
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(o[0], o[1], o[2], o[3]));
    __stcs(reinterpret_cast<uint4*>(p + 8), make_uint4(o[4], o[5], o[6], o[7]));
  }
}

}  // namespace nosa

using namespace nosa;

static bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

static nosa_status launched(cudaError_t e) {
  if (e == cudaSuccess) return NOSA_OK;
  (void)cudaGetLastError();
  return NOSA_ERR_CUDA;
}

extern "C" nosa_status nosa_byte_append(const uint16_t* k, const uint16_t* v, uint8_t* store, int units, int n_tokens,
                                        int max_blocks, const int32_t* pos, const int32_t* count,
                                        const int32_t* slot_blk, int32_t* err_out, void* stream) {
  if (!k || !v || !store || units < 1 || n_tokens < 1 || n_tokens > (1 << 30) || max_blocks < 1) return NOSA_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(store, 16) || misaligned(pos, 4) || misaligned(count, 4) ||
      misaligned(slot_blk, 4) || misaligned(err_out, 4))
    return NOSA_ERR_INVALID_ARG;
  // blocks that n tokens touch at most, from any starting position
  const long long blocks = ((long long)n_tokens + 2 * kBlock - 2) / kBlock;
  if (units * blocks >= (1ll << 31) || (long long)units * max_blocks >= (1ll << 31)) return NOSA_ERR_INVALID_ARG;
  return launched(launch_ex(byte_append_kernel, dim3((unsigned)(units * blocks)), dim3(kByteWarps * 32), 0,
                            static_cast<cudaStream_t>(stream), true, 0, k, v, store, n_tokens, max_blocks, pos, count,
                            slot_blk, (int)blocks, err_out));
}

extern "C" nosa_status nosa_byte_read(const uint8_t* store, int units, int max_blocks, const int32_t* blocks,
                                      const int32_t* slots, int n_blocks, const int32_t* lens, uint16_t* kv,
                                      int32_t* err_out, void* stream) {
  if (!store || !kv || units < 1 || max_blocks < 1 || n_blocks < 1) return NOSA_ERR_INVALID_ARG;
  if (!blocks && (slots || n_blocks > max_blocks)) return NOSA_ERR_INVALID_ARG;
  if (misaligned(store, 16) || misaligned(kv, 16) || misaligned(blocks, 4) || misaligned(slots, 4) ||
      misaligned(lens, 4) || misaligned(err_out, 4))
    return NOSA_ERR_INVALID_ARG;
  if ((long long)units * n_blocks >= (1ll << 31) || (long long)units * max_blocks >= (1ll << 31))
    return NOSA_ERR_INVALID_ARG;
  return launched(launch_ex(byte_read_kernel, dim3((unsigned)(units * n_blocks)), dim3(kByteWarps * 32), 0,
                            static_cast<cudaStream_t>(stream), true, 0, store, max_blocks, blocks, slots, n_blocks,
                            lens, kv, err_out));
}
