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

// A group's range is kept as one register of two bf16, (max x, max -x), so that one shuffle and one packed
// maximum serve both ends.  The maximum hands on NaN.
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t range_of(uint32_t hi, uint32_t lo) {  // the lane's maxima and minima, two each
  lo ^= 0x80008000u;
  return max2_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
}
// One step of a reduction that also deals its results out: of two values the lane keeps one and gives the other
// to its partner.
__device__ __forceinline__ uint32_t deal(uint32_t v0, uint32_t v1, bool keep1, int partner) {
  return max2_nan(keep1 ? v1 : v0, __shfl_xor_sync(0xffffffffu, keep1 ? v0 : v1, partner));
}
__device__ __forceinline__ GroupScale range_scale(uint32_t range) {
  return group_scale(-bf16_to_float((uint16_t)(range >> 16)), bf16_to_float((uint16_t)range));
}

// Code of x in a group: clamp(rint((x - m) / s), 0, 15), exactly as the IEEE quotient rounds.  r is
// 1 / s rounded, so rint((x - m) r) is off by at most one, and only next to a border between two
// codes; the remainder e = (x - m) - n s is exact there (n s has at most 16 bits, and the two terms are
// within a factor of two of each other, or n = 0) and says which side x is on.
__device__ __forceinline__ uint32_t exact_code(float x, float m, float s) {
  const float d = x - m;
  float n = rintf(d * __frcp_rn(s));
  const float e = 2.f * fmaf(-n, s, d);
  if (fabsf(e) > s || (fabsf(e) == s && (((int)n) & 1))) n += copysignf(1.f, e);
  n = fminf(fmaxf(n, 0.f), 15.f);
  return s > 0.f ? (uint32_t)n : 0u;  // s = 0 or NaN: code 0
}
__device__ __noinline__ uint32_t exact_codes(uint32_t x0, uint32_t x1, float s, float m) {
  uint32_t w = 0;
  for (int e = 0; e < 4; ++e)
    w |= exact_code(bf16_to_float((uint16_t)((e < 2 ? x0 : x1) >> (16 * (e & 1)))), m, s) << (4 * e);
  return w;
}

// Two float32 in one 64-bit register, the operands of the packed arithmetic.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) { return fmaxf(a, fmaxf(fabsf(b), fabsf(c))); }

// A group's scale as the code loop wants it.
struct CodeScale {
  float s, m;
  uint64_t r2, negm2;  // 1 / s (to 2^-23) and -m, twice
  bool plain;          // s a normal f16: no code can leave 0 .. 15 (s is within 2^-11 of the range's fifteenth)
};
__device__ __forceinline__ CodeScale code_scale(uint32_t s_bits, uint32_t m_bits) {
  CodeScale c;
  c.s = half_bits_to_float(s_bits);
  c.m = half_bits_to_float(m_bits);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(c.s));
  c.r2 = pair(r, r);
  c.negm2 = pair(-c.m, -c.m);
  c.plain = s_bits - 0x0400u < 0x7c00u - 0x0400u;
  return c;
}

// Codes of 2 N bf16 values, 4 bits each.  t = (x - m) r is within 2^-17 of the quotient, so its rounding is
// the quotient's unless t is that near to a border: then, and for an odd scale, the codes are taken exactly
// (a division per value instead would cost more than the value's share of the memory time).  Adding
// 1.5 x 2^23 rounds t to the integer that then stands in the sum's low bits.
template <int N>
__device__ __forceinline__ uint32_t codes(const uint32_t (&x)[N], const CodeScale& c) {
  const uint64_t magic = pair(12582912.f, 12582912.f), negmagic = pair(-12582912.f, -12582912.f), minus1 = pair(-1.f, -1.f);
  uint32_t w = 0xC0C00000u;  // what the constants' bits 0x4B400000 << 4 e add up to, negated
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t t = mul2(add2(pair(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u)), c.negm2), c.r2);
    const uint64_t u = add2(t, magic);
    float u0, u1, f0, f1;
    unpair(fma2(add2(u, negmagic), minus1, t), f0, f1);
    unpair(u, u0, u1);
    off = max3_abs(off, f0, f1);
    w += __float_as_uint(u0) << (8 * i);
    w += __float_as_uint(u1) << (8 * i + 4);
  }
  if (!c.plain || off > 0.5f - 0x1p-16f) {
    w = exact_codes(x[0], x[1], c.s, c.m);
    if constexpr (N == 4) w |= exact_codes(x[2], x[3], c.s, c.m) << 16;
  }
  return w;
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
  // index of the tile's token i among the new ones (-15 at least), and whether it is one of them
  const int rel = (int)(first - p0);
  auto index = [&](int i) { return rel + i; };
  auto is_new = [&](int i) { return (unsigned)(rel + i) < (unsigned)c; };

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

  // halves of the tile with a new token
  const bool any[2] = {rel < c && rel + 8 > 0, rel + 8 < c};

  // Ranges.  K: token g + 8 h, group gr, over the lanes t; dealt so that lane t ends up with group t.  V: token
  // 8 h + 2 t + par, group gr, over the lanes g; lane g ends up with half g / 4, group g % 4, both tokens.
  uint32_t kr[2], vr[2];
  {
    uint32_t v[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int gr = 0; gr < 4; ++gr) {
        const uint4& x = kx[h][gr];
        v[h][gr] = range_of(max2_nan(max2_nan(x.x, x.y), max2_nan(x.z, x.w)), min2_nan(min2_nan(x.x, x.y), min2_nan(x.z, x.w)));
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      kr[h] = deal(deal(v[h][0], v[h][2], t & 2, 2), deal(v[h][1], v[h][3], t & 2, 2), t & 1, 1);
  }
#pragma unroll
  for (int par = 0; par < 2; ++par) {
    uint32_t v[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int gr = 0; gr < 4; ++gr)
        v[h][gr] = range_of(max2_nan(vx[h][par][gr].x, vx[h][par][gr].y), min2_nan(vx[h][par][gr].x, vx[h][par][gr].y));
    uint32_t w[4];
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) w[gr] = deal(v[0][gr], v[1][gr], g & 4, 16);
    vr[par] = deal(deal(w[0], w[2], g & 2, 8), deal(w[1], w[3], g & 2, 8), g & 1, 4);
  }

  // K: dims 32 gr + 8 t + e of token g + 8 h in word gr
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!any[h]) continue;
    const GroupScale q = range_scale(kr[h]);
    uint32_t w[4], sm[4];
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      sm[gr] = __shfl_sync(0xffffffffu, q.s | q.m << 16, (lane & ~3) | gr);
      const CodeScale cs = code_scale(sm[gr] & 0xffffu, sm[gr] >> 16);
      const uint32_t x[4] = {kx[h][gr].x, kx[h][gr].y, kx[h][gr].z, kx[h][gr].w};
      w[gr] = codes<4>(x, cs);
    }
    if (kin[h]) {
      *reinterpret_cast<uint4*>(dst + 64 * (g + 8 * h) + 16 * t) = make_uint4(w[0], w[1], w[2], w[3]);
      if (t == 0)
        *reinterpret_cast<uint4*>(dst + kTileKs + 16 * (g + 8 * h)) =
            make_uint4(__byte_perm(sm[0], sm[1], 0x5410), __byte_perm(sm[2], sm[3], 0x5410),
                       __byte_perm(sm[0], sm[1], 0x7632), __byte_perm(sm[2], sm[3], 0x7632));
    }
  }

  // V: dims 32 gr + 4 g + e of token 8 h + 2 t + par in half `par` of word gr
  const GroupScale q0 = range_scale(vr[0]), q1 = range_scale(vr[1]);
  const uint32_t sp = q0.s | q1.s << 16, mp = q0.m | q1.m << 16;  // of half g / 4, group g % 4
  {
    uint8_t* meta = dst + kTileVs + 16 * (4 * (g >> 2) + t) + 4 * (g & 3);
    const bool in0 = g & 4 ? vin[1][0] : vin[0][0], in1 = g & 4 ? vin[1][1] : vin[0][1];
    if (in0 && in1) {
      *reinterpret_cast<uint32_t*>(meta) = sp;
      *reinterpret_cast<uint32_t*>(meta + kTileVm - kTileVs) = mp;
    } else if (in0 || in1) {  // the pair's other token stays as it is
      *reinterpret_cast<uint16_t*>(meta + 2 * in1) = (uint16_t)(sp >> (16 * in1));
      *reinterpret_cast<uint16_t*>(meta + kTileVm - kTileVs + 2 * in1) = (uint16_t)(mp >> (16 * in1));
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!any[h]) continue;
    uint32_t w[4];
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      const uint32_t s2 = __shfl_sync(0xffffffffu, sp, 16 * h + 4 * gr + t), m2 = __shfl_sync(0xffffffffu, mp, 16 * h + 4 * gr + t);
      const uint32_t x0[2] = {vx[h][0][gr].x, vx[h][0][gr].y}, x1[2] = {vx[h][1][gr].x, vx[h][1][gr].y};
      w[gr] = codes<2>(x0, code_scale(s2 & 0xffffu, m2 & 0xffffu)) | codes<2>(x1, code_scale(s2 >> 16, m2 >> 16)) << 16;
    }
    uint8_t* codes = dst + kTileV + 512 * h + 16 * lane;
    if (vin[h][0] && vin[h][1]) {
      *reinterpret_cast<uint4*>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (vin[h][0] || vin[h][1]) {
      const int par = vin[h][1];
#pragma unroll
      for (int gr = 0; gr < 4; ++gr) *reinterpret_cast<uint16_t*>(codes + 4 * gr + 2 * par) = (uint16_t)(w[gr] >> (16 * par));
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
