// Writing the 8-bit KV block store (nosa_byte_append) and reading it back (nosa_byte_read).
//
// A scale belongs to a whole block of 64 tokens, so a CTA takes a block: four warps its K, four its V.  The new values
// wait in registers while the block's largest magnitude goes through shared memory.  A token and unit is 512 bytes of bf16
// and 256 of the store: bound by HBM.  16,384 tokens of 16 units take 30.8 us (30.1 of HBM; 48.6 with loads of 16 bytes,
// which fetch a lane's sector twice, and the largest magnitude value by value), 64 ragged chunks of up to 2,047 tokens at odd
// positions 10.3 (9.4).  One token of 256 units takes 2.4 us, 6.4 where the lanes had its tile's layout.  Reading 262,144
// tokens 31.0 us.
#include <algorithm>

#include "byte_core.cuh"
#include "host.h"

namespace nosa {

constexpr int kByteWarps = 8;   // four of K, four of V
constexpr int kFewTokens = 8;   // calls of so few tokens spread each over a warp

// The exponent of the smallest power of two s with x <= 448 s, for the bf16 magnitude `top` > 0, within the scales' range:
// 448 = 1.75 x 2^8, so it is x's exponent less 8, or one more where x's mantissa is above 1.75.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u);
  return min(max(e, kLeastScale), kMostScale);
}
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// The scale that a block has, for which `s` stands in it: what is not a scale (a store that was never written) counts as none.
__device__ __forceinline__ float held_scale(float s) {
  return s >= power_of_2(kLeastScale) && s <= power_of_2(kMostScale) && (__float_as_uint(s) & 0x7fffffu) == 0 ? s : 0.f;
}
// The scale for the finite magnitude `top` in a block that has the scale `had`, and 1 / it (1 for no scale).
__device__ __forceinline__ float new_scale(float had, uint32_t top) {
  return fmaxf(had, top ? power_of_2(scale_exponent(top)) : 0.f);
}
__device__ __forceinline__ float inverse_scale(float s) {
  return s > 0.f ? power_of_2(127 - (int)(__float_as_uint(s) >> 23)) : 1.f;
}

// Two bf16 values times inv as e4m3 codes; plain: both are finite (the conversion saturates infinities).
template <bool kPlain>
__device__ __forceinline__ uint32_t two_codes(uint32_t x, float inv) {
  uint32_t c = to_codes(__uint_as_float(x << 16) * inv, __uint_as_float(x & 0xffff0000u) * inv);
  if (!kPlain) {
    if ((x & 0x7fffu) >= 0x7f80u) c = (c & 0xff00u) | 0x7fu;
    if ((x & 0x7fff0000u) >= 0x7f800000u) c = (c & 0x00ffu) | 0x7f00u;
  }
  return c;
}

// Four codes c as e4m3(c ratio), ratio a power of two in f16x2.  The product is exact unless it is below 2^-10, where
// it becomes 0 either way.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, __half2 ratio) {
  uint32_t h[2], out = 0;
  codes_to_half2(w, h[0], h[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), ratio);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&y)));
    out |= (uint32_t)r << (16 * i);
  }
  return out;
}
// The factor of a block's codes whose scale grows from `had` to 1 / inv.
__device__ __forceinline__ __half2 growth(float had, float inv) { return __float2half2_rn(fmaxf(had * inv, 0x1p-24f)); }

// The larger magnitudes of two pairs of bf16 values, and that of the finite ones alone in a register of two.
__device__ __forceinline__ uint32_t max_magnitudes(uint32_t top, uint32_t x) { return __vmaxu2(top, x & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t finite_max(uint32_t top, uint32_t x) {
  const uint32_t lo = x & 0x7fffu, hi = (x >> 16) & 0x7fffu;
  top = lo < 0x7f80u ? max(top, lo) : top;
  return hi < 0x7f80u ? max(top, hi) : top;
}

// 32 bytes that are read once (wide: p is a multiple of 32 bytes, so that they are one load of a whole sector).
__device__ __forceinline__ void load_32(uint4& a, uint4& b, const void* p, bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = ld_stream_v4(p);
    b = ld_stream_v4(static_cast<const char*>(p) + 16);
  }
}
__device__ __forceinline__ void store_32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(static_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

struct AppendArgs {
  const uint16_t *k, *v;
  uint8_t* store;
  const int32_t *pos, *count, *slot_blk;
  int32_t* err;
  int n, max_blocks, blocks;  // blocks: that a unit's tokens touch at most
  int wide;                   // k and v are multiples of 32 bytes
};

// A CTA's block: its bytes (null: the CTA has nothing to write), and which of the unit's c new tokens are its first (rel < 0:
// the block has earlier ones).
struct AppendBlock {
  uint8_t* dst;
  int rel, c;
};
__device__ __forceinline__ AppendBlock append_block(const AppendArgs& a, int u, int bi, int* found) {
  const long long p0 = a.pos ? a.pos[u] : 0, cap = (long long)a.max_blocks * kBlock;
  const int c0 = a.count ? a.count[u] : a.n, c = min(max(c0, 0), a.n);
  if (bi == 0 && threadIdx.x == 0 && a.err && (c0 != c || (c > 0 && (p0 < 0 || (!a.slot_blk && p0 + c > cap)))))
    atomicOr(a.err, kErrBounds);
  const long long block = (p0 >> 6) + bi;  // an arithmetic shift: negative positions round down
  const int rel = (int)(block * kBlock - p0);  // -63 at least
  if (c == 0 || rel >= c || block < 0) return {nullptr, 0, 0};
  long long row = block;
  if (a.slot_blk) {
    if (threadIdx.x == 0) *found = a.max_blocks;
    __syncthreads();
    for (int r = threadIdx.x; r < a.max_blocks; r += kByteWarps * 32)
      if (a.slot_blk[(size_t)u * a.max_blocks + r] == block) atomicMin(found, r);
    __syncthreads();
    row = *found;
    if (row == a.max_blocks && threadIdx.x == 0 && a.err) atomicOr(a.err, kErrBounds);
  }
  if (row >= a.max_blocks) return {nullptr, 0, 0};
  return {a.store + ((size_t)u * a.max_blocks + row) * kByteBlockBytes, rel, c};
}

// The largest of what the four warps of K (or of V) have found.  Also a barrier.
__device__ __forceinline__ uint32_t block_top(uint32_t mine, uint32_t* tops) {
  const int warp = threadIdx.x >> 5, first = warp & 4;
  mine = __reduce_max_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0) tops[warp] = mine;
  __syncthreads();
  return max(max(tops[first], tops[first + 1]), max(tops[first + 2], tops[first + 3]));
}

// The lane's 16 words of a tile as they are to stand there: new codes in the bytes of new tokens (first: the tile's first
// token among the c new ones), the earlier ones elsewhere.
template <bool kPlain>
__device__ __forceinline__ void write_tile(uint8_t* words, const uint4 (&x)[8], const uint4 (&old)[4], bool is_v, int first, int c,
                                           bool grown, __half2 ratio, float inv, int lane) {
  const int g = lane >> 2, t = lane & 3;
  auto is_new = [&](int j) { return (unsigned)(first + j) < (unsigned)c; };  // the tile's token j
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4], keep[2];  // bytes of words e % 2 that are not new
    if (!is_v) {  // chunk i: token g + 8 (i / 2), dims 32 t + 16 (i % 2) ..
      const uint4 a = x[2 * i], b = x[2 * i + 1];
      w[0] = two_codes<kPlain>(a.x, inv) | two_codes<kPlain>(a.y, inv) << 16;
      w[1] = two_codes<kPlain>(a.z, inv) | two_codes<kPlain>(a.w, inv) << 16;
      w[2] = two_codes<kPlain>(b.x, inv) | two_codes<kPlain>(b.y, inv) << 16;
      w[3] = two_codes<kPlain>(b.z, inv) | two_codes<kPlain>(b.w, inv) << 16;
      keep[0] = keep[1] = is_new(g + 8 * (i >> 1)) ? 0u : 0xffffffffu;
    } else {  // chunk i: dims 16 g + 4 i .. + 3; word 2 jj + half: dims 2 jj, 2 jj + 1 of them, tokens 2t + 8 half, + 1
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int half = e & 1, at = 2 * i + (e >> 1);  // of a token's 8 registers of two dims
        const uint4 a = x[4 * half + (at >> 2)], b = x[4 * half + 2 + (at >> 2)];
        const uint32_t xa = (at & 3) == 0 ? a.x : (at & 3) == 1 ? a.y : (at & 3) == 2 ? a.z : a.w;
        const uint32_t xb = (at & 3) == 0 ? b.x : (at & 3) == 1 ? b.y : (at & 3) == 2 ? b.z : b.w;
        w[e] = __byte_perm(two_codes<kPlain>(xa, inv), two_codes<kPlain>(xb, inv), 0x5140);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half)
        keep[half] = (is_new(2 * t + 8 * half) ? 0u : 0x00ff00ffu) | (is_new(2 * t + 8 * half + 1) ? 0u : 0xff00ff00u);
    }
    if (keep[0] | keep[1]) {
      const uint32_t o[4] = {old[i].x, old[i].y, old[i].z, old[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = (w[e] & ~keep[e & 1]) | ((grown ? rescaled(o[e], ratio) : o[e]) & keep[e & 1]);
    }
    if (grown || (keep[0] & keep[1]) != 0xffffffffu)
      *reinterpret_cast<uint4*>(words + 512 * i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A warp takes a tile of K or V, each lane in the store's own layout (byte_core.cuh).
__global__ void __launch_bounds__(kByteWarps * 32) byte_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ uint32_t tops[kByteWarps];
  __shared__ int found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u = blockIdx.x / a.blocks, bi = blockIdx.x % a.blocks;
  pdl_wait();
  pdl_launch_dependents();
  const AppendBlock b = append_block(a, u, bi, &found);
  if (!b.dst) return;
  const bool is_v = warp >= 4, begun = b.rel < 0;
  const int tile = warp & 3, first = b.rel + tile * kByteTileTokens;

  // the lane's new values, in its own order, and the block's earlier codes where they may be wanted
  uint4 x[8], old[4];
  const uint16_t* src = (is_v ? a.v : a.k) + (size_t)u * a.n * kHeadDim;
  bool any = false, all = true;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // K: tokens g, g + 8, halves of 16 dims; V: the four tokens
    const int j = first + (is_v ? 2 * t + (i & 1) + 8 * (i >> 1) : g + 8 * (i >> 1));
    const bool in = (unsigned)j < (unsigned)b.c;
    any |= in;
    all &= in;
    x[2 * i] = x[2 * i + 1] = zero;
    if (in) load_32(x[2 * i], x[2 * i + 1], src + (size_t)j * kHeadDim + (is_v ? 16 * g : 32 * t + 16 * (i & 1)), a.wide);
  }
  uint8_t* words = b.dst + tile * kByteTile + (is_v ? kByteV : 0) + 16 * lane;
  const bool read = begun || (any && !all);
#pragma unroll
  for (int i = 0; i < 4; ++i) old[i] = read ? *reinterpret_cast<const uint4*>(words + 512 * i) : zero;
  float* held = reinterpret_cast<float*>(b.dst + kByteScales + (is_v ? 4 : 0));
  const float had = begun ? held_scale(*held) : 0.f;

  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    top = max_magnitudes(max_magnitudes(max_magnitudes(max_magnitudes(top, x[i].x), x[i].y), x[i].z), x[i].w);
  top = max(top & 0xffffu, top >> 16);
  const bool plain = __all_sync(0xffffffffu, top < 0x7f80u);
  if (!plain) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = finite_max(finite_max(finite_max(finite_max(top, x[i].x), x[i].y), x[i].z), x[i].w);
  }
  top = block_top(top, tops);  // also: every thread has the earlier scale
  const float scale = new_scale(had, top), inv = inverse_scale(scale);
  if (tile == 0 && lane == 0) *held = scale;
  const bool grown = had > 0.f && scale > had;
  if (!any && !grown) return;
  if (plain)
    write_tile<true>(words, x, old, is_v, first, b.c, grown, growth(had, inv), inv, lane);
  else
    write_tile<false>(words, x, old, is_v, first, b.c, grown, growth(had, inv), inv, lane);
}

// The same for calls of at most kFewTokens tokens, whose time is one warp's path through the code: a warp takes every
// fourth token of K or V, a lane four of its dims.
__global__ void __launch_bounds__(kByteWarps * 32) byte_append_few_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ uint32_t tops[kByteWarps];
  __shared__ int found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = blockIdx.x / a.blocks, bi = blockIdx.x % a.blocks;
  pdl_wait();
  pdl_launch_dependents();
  const AppendBlock b = append_block(a, u, bi, &found);
  if (!b.dst) return;
  const bool is_v = warp >= 4, begun = b.rel < 0;
  const int from = max(b.rel, 0), upto = min(b.c, b.rel + kBlock);  // the block's new tokens
  const uint16_t* src = (is_v ? a.v : a.k) + (size_t)u * a.n * kHeadDim + 4 * lane;
  uint2 x[kFewTokens / 4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kFewTokens / 4; ++i) {
    const int j = from + (warp & 3) + 4 * i;
    x[i] = j < upto ? *reinterpret_cast<const uint2*>(src + (size_t)j * kHeadDim) : make_uint2(0, 0);
    top = finite_max(finite_max(top, x[i].x), x[i].y);
  }
  float* held = reinterpret_cast<float*>(b.dst + kByteScales + (is_v ? 4 : 0));
  const float had = begun ? held_scale(*held) : 0.f;
  top = block_top(top, tops);  // also: every thread has the earlier scale
  const float scale = new_scale(had, top), inv = inverse_scale(scale);
  if ((warp & 3) == 0 && lane == 0) *held = scale;
  if (had > 0.f && scale > had) {  // a warp takes a tile; the new tokens' bytes are written after that
    uint4* words = reinterpret_cast<uint4*>(b.dst + (warp & 3) * kByteTile + (is_v ? kByteV : 0) + 16 * lane);
    const __half2 ratio = growth(had, inv);
    uint4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = words[32 * i];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      words[32 * i] = make_uint4(rescaled(o[i].x, ratio), rescaled(o[i].y, ratio), rescaled(o[i].z, ratio), rescaled(o[i].w, ratio));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kFewTokens / 4; ++i) {
    const int j = from + (warp & 3) + 4 * i;
    if (j >= upto) break;
    const uint32_t w = two_codes<false>(x[i].x, inv) | two_codes<false>(x[i].y, inv) << 16;
    const int token = (j - b.rel) % kByteTileTokens, d = 4 * lane;
    uint8_t* tile = b.dst + (j - b.rel) / kByteTileTokens * kByteTile;
    if (!is_v) {
      *reinterpret_cast<uint32_t*>(tile + 1024 * (token / 8) + 512 * (d % 32 / 16) + 16 * (4 * (token % 8) + d / 32) + d % 16) = w;
    } else {
      uint8_t* p = tile + kByteV + 512 * (d % 16 / 4) + 16 * (4 * (d / 16) + token % 8 / 2) + 4 * (token / 8) + token % 2;
      p[0] = (uint8_t)w;
      p[2] = (uint8_t)(w >> 8);
      p[8] = (uint8_t)(w >> 16);
      p[10] = (uint8_t)(w >> 24);
    }
  }
}

// Four codes times the scale as two bf16x2, exactly.
__device__ __forceinline__ void four_values(uint32_t four, float scale, uint32_t& a, uint32_t& b) {
  uint32_t lo, hi;
  codes_to_half2(four, lo, hi);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  a = pack_bf16x2(x.x * scale, x.y * scale);
  b = pack_bf16x2(y.x * scale, y.y * scale);
}

// A CTA takes a listed block, four warps its K tiles, four its V tiles.
__global__ void __launch_bounds__(kByteWarps * 32)
    byte_read_kernel(const uint8_t* __restrict__ store, int max_blocks, const int32_t* __restrict__ blocks,
                     const int32_t* __restrict__ slots, int n_blocks, const int32_t* __restrict__ lens,
                     uint16_t* __restrict__ kv, int32_t* err, bool wide) {
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
  uint32_t o[8];
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      four_values(c[i].x, scale, o[0], o[1]);
      four_values(c[i].y, scale, o[2], o[3]);
      four_values(c[i].z, scale, o[4], o[5]);
      four_values(c[i].w, scale, o[6], o[7]);
      store_32(out + (g + 8 * (i >> 1)) * kHeadDim + 32 * t + 16 * (i & 1), o, wide);
    }
    return;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {  // tokens 2t + 8 half, + 1
    uint32_t even[8], odd[8];
#pragma unroll
    for (int at = 0; at < 8; ++at) {  // two dims each
      const uint4 w = c[at >> 1];
      const uint32_t x = at & 1 ? (half ? w.w : w.z) : (half ? w.y : w.x);
      four_values(__byte_perm(x, 0, 0x3120), scale, even[at], odd[at]);
    }
    const int token = 2 * t + 8 * half;
#pragma unroll
    for (int at = 0; at < 8; ++at) {
      if (token >= rows) even[at] = 0;
      if (token + 1 >= rows) odd[at] = 0;
    }
    store_32(out + token * kHeadDim + 16 * g, even, wide);
    store_32(out + (token + 1) * kHeadDim + 16 * g, odd, wide);
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
  const AppendArgs a{k, v, store, pos, count, slot_blk, err_out, n_tokens, max_blocks, (int)blocks, !misaligned(k, 32) && !misaligned(v, 32)};
  return launched(launch_ex(n_tokens <= kFewTokens ? byte_append_few_kernel : byte_append_kernel,
                            dim3((unsigned)(units * blocks)), dim3(kByteWarps * 32), 0, static_cast<cudaStream_t>(stream), true,
                            0, a));
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
                            lens, kv, err_out, !misaligned(kv, 32)));
}
