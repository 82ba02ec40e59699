// Writing the 4-bit KV block store (nosa_quant_append) and reading it back (nosa_quant_read).
//
// Both move a tile of 16 tokens per warp through registers only: the lanes hold the tile in the
// store's own layout (quant_core.cuh), so each lane's codes leave (or arrive) as 16-byte words, and
// the bf16 side is touched in whole 32-byte sectors.  Both are bound by HBM: 512 bytes of bf16 and
// 160 of the store per token and unit.
#include "host.h"
#include "quant_core.cuh"

namespace nosa {

constexpr int kQuantWarps = 4;

// The range of a group spread over lanes that differ in the lane-index bits lo_bit .. hi_bit:
// packed (max x, max -x), so that one shuffle and one packed maximum serve both ends.  The maximum
// hands on NaN.
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Code of x in a group: clamp(rint((x - m) / s), 0, 15), exactly as the IEEE quotient rounds.  r is
// 1 / s rounded, so rint((x - m) r) is off by at most one, and only next to a border between two
// codes; the remainder e = (x - m) - n s is exact there (n s has at most 16 bits, and the two terms are
// within a factor of two of each other, or n = 0) and says which side x is on.  A division per value
// instead would cost more than the value's share of the memory time.
__device__ __forceinline__ uint32_t quant_code(float x, float m, float s, float r) {
  const float d = x - m;
  float n = rintf(d * r);
  const float e = 2.f * fmaf(-n, s, d);
  if (fabsf(e) >= s) {  // rare: a border
    if (fabsf(e) > s || (((int)n) & 1)) n += copysignf(1.f, e);
  }
  n = fminf(fmaxf(n, 0.f), 15.f);
  return s > 0.f ? (uint32_t)n : 0u;  // s = 0 or NaN: code 0
}

__global__ void __launch_bounds__(kQuantWarps * 32)
    quant_append_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, uint8_t* __restrict__ store,
                        int units, int n, int max_blocks, const int32_t* __restrict__ pos,
                        const int32_t* __restrict__ count, int tiles, int32_t* err) {
  pdl_wait();
  pdl_launch_dependents();
  const long long job = (long long)blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  const int u = (int)(job / tiles), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (u >= units) return;
  const long long p0 = pos ? pos[u] : 0, cap = (long long)max_blocks * kBlock;
  const int c0 = count ? count[u] : n, c = min(max(c0, 0), n);
  const long long tile = (p0 >> 4) + job % tiles;  // an arithmetic shift: negative positions round down
  if (job % tiles == 0 && lane == 0 && err && (c0 != c || (c > 0 && (p0 < 0 || p0 + c > cap)))) atomicOr(err, kErrBounds);
  const long long first = tile * kTileTokens;
  if (tile < 0 || first >= cap || first >= p0 + c) return;  // cap is a multiple of 16: a tile is in or out as a whole
  uint8_t* dst = store + (size_t)u * max_blocks * kQuantBlockBytes + (size_t)tile * kTileBytes;
  const size_t row0 = (size_t)u * n;
  // index of the tile's token i among the new ones, and whether it is one of them
  auto index = [&](int i) { return first + i - p0; };
  auto is_new = [&](int i) { return index(i) >= 0 && index(i) < c; };

  // loads of the whole tile, issued together
  uint4 kx[2][4];
  uint2 vx[2][2][4];  // [half][token of the pair][group]
  bool kin[2], vin[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    kin[h] = is_new(g + 8 * h);
    const uint16_t* src = k + (row0 + (kin[h] ? index(g + 8 * h) : 0)) * kHeadDim + 8 * t;
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) kx[h][gr] = kin[h] ? ld_stream_v4(src + 32 * gr) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int par = 0; par < 2; ++par) {
      vin[h][par] = is_new(8 * h + 2 * t + par);
      const uint16_t* vs = v + (row0 + (vin[h][par] ? index(8 * h + 2 * t + par) : 0)) * kHeadDim + 4 * g;
#pragma unroll
      for (int gr = 0; gr < 4; ++gr)
        vx[h][par][gr] = vin[h][par] ? __ldcs(reinterpret_cast<const uint2*>(vs + 32 * gr)) : make_uint2(0, 0);
    }
  }

  // K: token g + 8 h, dims 32 gr + 8 t + e in word gr
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4], sc[4], mn[4];
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      const uint32_t x[4] = {kx[h][gr].x, kx[h][gr].y, kx[h][gr].z, kx[h][gr].w};
      uint32_t hi = max2_nan(max2_nan(x[0], x[1]), max2_nan(x[2], x[3]));
      uint32_t lo = max2_nan(max2_nan(x[0] ^ 0x80008000u, x[1] ^ 0x80008000u),
                             max2_nan(x[2] ^ 0x80008000u, x[3] ^ 0x80008000u));
      // fold the two halves: (max x, max -x) in one register
      uint32_t both = max2_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
      both = max2_nan(both, __shfl_xor_sync(0xffffffffu, both, 1));
      both = max2_nan(both, __shfl_xor_sync(0xffffffffu, both, 2));
      const GroupScale q = group_scale(-bf16_to_float((uint16_t)(both >> 16)), bf16_to_float((uint16_t)both));
      sc[gr] = q.s;
      mn[gr] = q.m;
      const float s = half_bits_to_float(q.s), m = half_bits_to_float(q.m), r = __frcp_rn(s);
      w[gr] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[gr] |= quant_code(bf16_to_float((uint16_t)(x[e >> 1] >> (16 * (e & 1)))), m, s, r) << (4 * e);
    }
    if (kin[h]) {
      *reinterpret_cast<uint4*>(dst + 64 * (g + 8 * h) + 16 * t) = make_uint4(w[0], w[1], w[2], w[3]);
      if (t == 0)
        *reinterpret_cast<uint4*>(dst + kTileKs + 16 * (g + 8 * h)) =
            make_uint4(sc[0] | sc[1] << 16, sc[2] | sc[3] << 16, mn[0] | mn[1] << 16, mn[2] | mn[3] << 16);
    }
  }

  // V: tokens 8 h + 2 t + par, dims 32 gr + 4 g + e in word gr
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4] = {0, 0, 0, 0}, sc[4] = {0, 0, 0, 0}, mn[4] = {0, 0, 0, 0};
#pragma unroll
    for (int par = 0; par < 2; ++par)
#pragma unroll
      for (int gr = 0; gr < 4; ++gr) {
        const uint32_t x[2] = {vx[h][par][gr].x, vx[h][par][gr].y};
        const uint32_t hi = max2_nan(x[0], x[1]), lo = max2_nan(x[0] ^ 0x80008000u, x[1] ^ 0x80008000u);
        uint32_t both = max2_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) both = max2_nan(both, __shfl_xor_sync(0xffffffffu, both, o));
        const GroupScale q = group_scale(-bf16_to_float((uint16_t)(both >> 16)), bf16_to_float((uint16_t)both));
        const float s = half_bits_to_float(q.s), m = half_bits_to_float(q.m), r = __frcp_rn(s);
        sc[gr] |= q.s << (16 * par);
        mn[gr] |= q.m << (16 * par);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[gr] |= quant_code(bf16_to_float((uint16_t)(x[e >> 1] >> (16 * (e & 1)))), m, s, r) << (16 * par + 4 * e);
      }
    // lane (0, t) also writes the pair's scales, lane (1, t) its minima
    uint8_t* codes = dst + kTileV + 512 * h + 16 * lane;
    uint8_t* meta = dst + (g == 0 ? kTileVs : kTileVm) + 16 * (4 * h + t);
    const bool both_in = vin[h][0] && vin[h][1];
    if (both_in) {
      *reinterpret_cast<uint4*>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
      if (g == 0) *reinterpret_cast<uint4*>(meta) = make_uint4(sc[0], sc[1], sc[2], sc[3]);
      if (g == 1) *reinterpret_cast<uint4*>(meta) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
    } else if (vin[h][0] || vin[h][1]) {  // the pair's other token stays as it is
      const int par = vin[h][1];
#pragma unroll
      for (int gr = 0; gr < 4; ++gr) {
        *reinterpret_cast<uint16_t*>(codes + 4 * gr + 2 * par) = (uint16_t)(w[gr] >> (16 * par));
        if (g < 2) *reinterpret_cast<uint16_t*>(meta + 4 * gr + 2 * par) = (uint16_t)((g == 0 ? sc[gr] : mn[gr]) >> (16 * par));
      }
    }
  }
}

// Code e (of a 32-bit word's eight) as a float: the code in the low mantissa bits of 2^23.
__device__ __forceinline__ float code_float(uint32_t w, int e) {
  return __uint_as_float(((w >> (4 * e)) & 15u) | 0x4B000000u) - 8388608.f;
}

__global__ void __launch_bounds__(kQuantWarps * 32)
    quant_read_kernel(const uint8_t* __restrict__ store, int units, int max_blocks, const int32_t* __restrict__ blocks,
                      int n_blocks, const int32_t* __restrict__ lens, uint16_t* __restrict__ kv, int32_t* err) {
  pdl_wait();
  pdl_launch_dependents();
  // a CTA's four warps take the four tiles of one listed block
  const int tile = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u = blockIdx.x / n_blocks, j = blockIdx.x % n_blocks;
  const int b = blocks ? blocks[blockIdx.x] : j;
  if (b >= max_blocks && err && threadIdx.x == 0) atomicOr(err, kErrBounds);
  const bool held = b >= 0 && b < max_blocks;
  const long long left = !held ? 0 : lens ? (long long)lens[u] - ((long long)b * kBlock + tile * kTileTokens) : kTileTokens;
  const int rows = (int)min(max(left, 0ll), (long long)kTileTokens);  // rows of the tile below the length
  uint16_t* dk = kv + (size_t)blockIdx.x * 2 * kBlockElems + tile * kTileTokens * kHeadDim;
  uint16_t* dv = dk + kBlockElems;
  const uint8_t* src = store + ((size_t)u * max_blocks + (held ? b : 0)) * kQuantBlockBytes + tile * kTileBytes;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 kc[2], ks[2], vc[2], vs[2], vm[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool kin = g + 8 * h < rows, vin = 2 * t + 8 * h < rows;
    kc[h] = kin ? ld_stream_v4(src + 64 * (g + 8 * h) + 16 * t) : zero;
    ks[h] = kin ? ld_stream_v4(src + kTileKs + 16 * (g + 8 * h)) : zero;
    vc[h] = vin ? ld_stream_v4(src + kTileV + 512 * h + 16 * lane) : zero;
    vs[h] = vin ? ld_stream_v4(src + kTileVs + 16 * (4 * h + t)) : zero;
    vm[h] = vin ? ld_stream_v4(src + kTileVm + 16 * (4 * h + t)) : zero;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {kc[h].x, kc[h].y, kc[h].z, kc[h].w}, sm[4] = {ks[h].x, ks[h].y, ks[h].z, ks[h].w};
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      const float s = half_bits_to_float(sm[gr >> 1] >> (16 * (gr & 1)) & 0xffffu);
      const float m = half_bits_to_float(sm[2 + (gr >> 1)] >> (16 * (gr & 1)) & 0xffffu);
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack_bf16x2(fmaf(code_float(w[gr], 2 * e), s, m), fmaf(code_float(w[gr], 2 * e + 1), s, m));
      __stcs(reinterpret_cast<uint4*>(dk + (g + 8 * h) * kHeadDim + 32 * gr + 8 * t), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {vc[h].x, vc[h].y, vc[h].z, vc[h].w}, s4[4] = {vs[h].x, vs[h].y, vs[h].z, vs[h].w},
                   m4[4] = {vm[h].x, vm[h].y, vm[h].z, vm[h].w};
#pragma unroll
    for (int par = 0; par < 2; ++par) {
      const int row = 8 * h + 2 * t + par;
      const bool in = row < rows;
#pragma unroll
      for (int gr = 0; gr < 4; ++gr) {
        const float s = half_bits_to_float(s4[gr] >> (16 * par) & 0xffffu);
        const float m = half_bits_to_float(m4[gr] >> (16 * par) & 0xffffu);
        uint2 o;
        o.x = pack_bf16x2(fmaf(code_float(w[gr], 4 * par), s, m), fmaf(code_float(w[gr], 4 * par + 1), s, m));
        o.y = pack_bf16x2(fmaf(code_float(w[gr], 4 * par + 2), s, m), fmaf(code_float(w[gr], 4 * par + 3), s, m));
        __stcs(reinterpret_cast<uint2*>(dv + row * kHeadDim + 32 * gr + 4 * g), in ? o : make_uint2(0, 0));
      }
    }
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

extern "C" nosa_status nosa_quant_append(const uint16_t* k, const uint16_t* v, uint8_t* store, int units, int n_tokens,
                                         int max_blocks, const int32_t* pos, const int32_t* count, int32_t* err_out,
                                         void* stream) {
  if (!k || !v || !store || units < 1 || n_tokens < 1 || max_blocks < 1) return NOSA_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(store, 16) || misaligned(pos, 4) || misaligned(count, 4) ||
      misaligned(err_out, 4))
    return NOSA_ERR_INVALID_ARG;
  // tiles that n tokens touch at most, from any starting position
  const long long tiles = ((long long)n_tokens + 2 * kTileTokens - 2) / kTileTokens;
  const long long ctas = (units * tiles + kQuantWarps - 1) / kQuantWarps;
  if (ctas >= (1ll << 31) || (long long)units * max_blocks >= (1ll << 31)) return NOSA_ERR_INVALID_ARG;
  return launched(launch_ex(quant_append_kernel, dim3((unsigned)ctas), dim3(kQuantWarps * 32), 0,
                            static_cast<cudaStream_t>(stream), true, 0, k, v, store, units, n_tokens, max_blocks, pos,
                            count, (int)tiles, err_out));
}

extern "C" nosa_status nosa_quant_read(const uint8_t* store, int units, int max_blocks, const int32_t* blocks,
                                       int n_blocks, const int32_t* lens, uint16_t* kv, int32_t* err_out,
                                       void* stream) {
  if (!store || !kv || units < 1 || max_blocks < 1 || n_blocks < 1) return NOSA_ERR_INVALID_ARG;
  if (!blocks && n_blocks > max_blocks) return NOSA_ERR_INVALID_ARG;
  if (misaligned(store, 16) || misaligned(kv, 16) || misaligned(blocks, 4) || misaligned(lens, 4) ||
      misaligned(err_out, 4))
    return NOSA_ERR_INVALID_ARG;
  if ((long long)units * n_blocks >= (1ll << 31) || (long long)units * max_blocks >= (1ll << 31))
    return NOSA_ERR_INVALID_ARG;
  return launched(launch_ex(quant_read_kernel, dim3((unsigned)(units * n_blocks)), dim3(kQuantWarps * 32), 0,
                            static_cast<cudaStream_t>(stream), true, 0, store, units, max_blocks, blocks, n_blocks,
                            lens, kv, err_out));
}
