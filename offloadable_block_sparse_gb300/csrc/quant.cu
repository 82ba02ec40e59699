// Writing the 4-bit KV block store (nosa_quant_append) and reading it back (nosa_quant_read).
//
// Both move tiles of 16 tokens through registers only: the lanes hold a tile in the store's own layout
// (quant_core.cuh), so each lane's codes leave (or arrive) as 16-byte words, and the bf16 side is touched
// in whole 32-byte sectors.  A token and unit is 512 bytes of bf16 and 160 of the store.
#include <algorithm>

#include "host.h"
#include "quant_core.cuh"

namespace nosa {

constexpr int kQuantWarps = 4;
constexpr int kAppendTiles = 4, kAppendCtas = 3000;  // tiles a CTA takes in turn, while that leaves so many CTAs

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

// Code of x in a group: clamp(rint((x - m) / s), 0, 15), for s > 0.
__device__ __forceinline__ uint32_t exact_code(float x, float m, float s) {
  return (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(x - m, s)), 0.f), 15.f);
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

// What a group's owner computes and the code loop wants: m and s as f16 bits, and -m, -s and 1 / s (to 2^-23).
struct GroupCode {
  GroupScale q;
  float negm, negs, r;
  // s is a normal f16: no code can leave 0 .. 15 (s is within 2^-11 of the range's fifteenth)
  __device__ __forceinline__ bool plain() const { return q.s - 0x0400u < 0x7c00u - 0x0400u; }
};
__device__ __forceinline__ GroupCode group_code(uint32_t range) {
  GroupCode c;
  c.q = range_scale(range);
  c.negm = -half_bits_to_float(c.q.m);
  c.negs = -half_bits_to_float(c.q.s);
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(c.r) : "f"(-c.negs));
  return c;
}
// The group of lane `owner`, each value twice.
struct CodeScale {
  uint64_t negm2, negs2, r2;
};
__device__ __forceinline__ CodeScale code_scale(const GroupCode& c, int owner) {
  const float m = __shfl_sync(0xffffffffu, c.negm, owner), s = __shfl_sync(0xffffffffu, c.negs, owner);
  const float r = __shfl_sync(0xffffffffu, c.r, owner);
  return {pair(m, m), pair(s, s), pair(r, r)};
}

// Codes of eight bf16 values, 4 bits each, without a division: t = d r for d = x - m, then one Newton step on the
// remainder, t + (d - t s) r.  The remainder is exact (s has 11 bits, and the terms cancel), so a quotient that lies on
// a border between two codes, k + 1/2, comes out as just that and goes to the even code; ties are frequent with
// bf16 values (one in a thousand).  A quotient off the border is at least a unit of d's last place away from it in d,
// which t resolves unless d fills all of float32's bits (x below 2^-15 of m).  Adding 1.5 x 2^23 rounds t to the
// integer that then stands in the sum's low bits.
// plain = false (some group of the warp has a subnormal s, zero or a NaN): by division, and zeros for the latter two.
__device__ __forceinline__ uint32_t codes(const uint32_t (&x)[4], const CodeScale& c, bool plain) {
  const uint64_t magic = pair(12582912.f, 12582912.f);
  uint32_t w = 0xC0C00000u;  // what the constants' bits 0x4B400000 << 4 e add up to, negated
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t d = add2(pair(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u)), c.negm2);
    const uint64_t t = mul2(d, c.r2);
    float u0, u1;
    unpair(add2(fma2(fma2(t, c.negs2, d), c.r2, t), magic), u0, u1);
    w += __float_as_uint(u0) << (8 * i);
    w += __float_as_uint(u1) << (8 * i + 4);
  }
  if (!plain) {
    float negs, negm, unused;
    unpair(c.negs2, negs, unused);
    unpair(c.negm2, negm, unused);
    w = 0;
    if (negs < 0.f) w = exact_codes(x[0], x[1], -negs, -negm) | exact_codes(x[2], x[3], -negs, -negm) << 16;
  }
  return w;
}

// A CTA takes `per` tiles in turn, a warp half a tile (8 tokens) of K or V: short enough for a single token, whose time
// is one warp's path through the code, and small enough in registers for many warps.  One token of 256 units takes
// 2.2 us; 16,384 tokens of 16 units 32.7 us (176 MB, 0.80 of measured HBM; 38.6 with one tile a CTA, 28.6 without the
// codes): 1,400 instructions a tile keep two thirds of the issue slots busy.
__global__ void __launch_bounds__(kQuantWarps * 32)
    quant_append_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, uint8_t* __restrict__ store,
                        int n, int max_blocks, const int32_t* __restrict__ pos, const int32_t* __restrict__ count,
                        int tiles, int per, int32_t* err) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ctas = (tiles + per - 1) / per, u = blockIdx.x / ctas, i0 = blockIdx.x % ctas * per;
  pdl_wait();
  pdl_launch_dependents();
  const long long p0 = pos ? pos[u] : 0, cap = (long long)max_blocks * kBlock;
  const int c0 = count ? count[u] : n, c = min(max(c0, 0), n);
  if (i0 == 0 && threadIdx.x == 0 && err && (c0 != c || (c > 0 && (p0 < 0 || p0 + c > cap)))) atomicOr(err, kErrBounds);
  const int half = 8 * (warp >> 1);
  const bool is_v = warp & 1;
  long long tile = (p0 >> 4) + i0;                     // an arithmetic shift: negative positions round down
  int rel = (int)(tile * kTileTokens - p0) + half;     // the half's first token among the new ones, -15 at least
  uint8_t* dst = store + ((size_t)u * max_blocks * 4 + tile) * kTileBytes;  // (not used outside the store)
  for (int done = 0; done < per && rel < c; ++done, ++tile, rel += kTileTokens, dst += kTileBytes) {
    // cap is a multiple of 16: a tile is in or out as a whole
    if (tile < 0 || tile * kTileTokens >= cap || rel + 8 <= 0) continue;
    auto is_new = [&](int j) { return (unsigned)(rel + j) < (unsigned)c; };  // the half's token j
    auto row = [&](int j) { return ((size_t)u * n + (is_new(j) ? rel + j : 0)) * kHeadDim; };

    // the lane's part: dims 32 gr + 8 t + e of token g in word gr, which is K's own layout
    const bool in = is_new(g);
    const uint16_t* src = (is_v ? v : k) + row(g) + 8 * t;
    uint4 x[4];
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) x[gr] = in ? ld_stream_v4(src + 32 * gr) : make_uint4(0, 0, 0, 0);
    // ranges over the lanes t, dealt so that lane t ends up with group t
    uint32_t r[4], w[4];
#pragma unroll
    for (int gr = 0; gr < 4; ++gr)
      r[gr] = range_of(max2_nan(max2_nan(x[gr].x, x[gr].y), max2_nan(x[gr].z, x[gr].w)),
                       min2_nan(min2_nan(x[gr].x, x[gr].y), min2_nan(x[gr].z, x[gr].w)));
    const GroupCode q = group_code(deal(deal(r[0], r[2], t & 2, 2), deal(r[1], r[3], t & 2, 2), t & 1, 1));
    const bool plain = __all_sync(0xffffffffu, q.plain() || !in);
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      const uint32_t y[4] = {x[gr].x, x[gr].y, x[gr].z, x[gr].w};
      w[gr] = codes(y, code_scale(q, (lane & ~3) | gr), plain);
    }
    if (!is_v) {
      if (in) {
        *reinterpret_cast<uint4*>(dst + 64 * (half + g) + 16 * t) = make_uint4(w[0], w[1], w[2], w[3]);
        uint8_t* meta = dst + kTileKs + 16 * (half + g) + 2 * t;
        *reinterpret_cast<uint16_t*>(meta) = (uint16_t)q.q.s;
        *reinterpret_cast<uint16_t*>(meta + 8) = (uint16_t)q.q.m;
      }
      continue;
    }
    // V's words hold four dims of a token pair: the pair's lanes (g even and odd) swap halves of theirs, and the even one
    // keeps dims 8 t .. + 3 of both tokens, the odd one dims 8 t + 4 .. + 7
    const int odd = g & 1;
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      const uint32_t other = __shfl_xor_sync(0xffffffffu, w[gr], 4);
      w[gr] = odd ? __byte_perm(other, w[gr], 0x7632) : __byte_perm(w[gr], other, 0x5410);
    }
    uint8_t* out = dst + kTileV + 64 * half + 16 * (4 * (2 * t + odd) + (g >> 1));
    const bool in0 = is_new(g & ~1), in1 = is_new(g | 1);
    if (in0 && in1) {
      *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (in0 || in1) {  // the pair's other token stays as it is
#pragma unroll
      for (int gr = 0; gr < 4; ++gr) *reinterpret_cast<uint16_t*>(out + 4 * gr + 2 * in1) = (uint16_t)(w[gr] >> (16 * in1));
    }
    if (in) {
      uint8_t* meta = dst + kTileVs + 16 * ((half + g) >> 1) + 4 * t + 2 * odd;
      *reinterpret_cast<uint16_t*>(meta) = (uint16_t)q.q.s;
      *reinterpret_cast<uint16_t*>(meta + kTileVm - kTileVs) = (uint16_t)q.q.m;
    }
  }
}

// Code e (of a 32-bit word's eight) as a float: the code in the low mantissa bits of 2^23.
__device__ __forceinline__ float code_float(uint32_t w, int e) {
  return __uint_as_float(((w >> (4 * e)) & 15u) | 0x4B000000u) - 8388608.f;
}

// A CTA takes a listed block, a warp one of its tiles.  Bound by HBM: 81 blocks of each of 256 units (892 MB) in 133 us,
// 1.00 of measured HBM (with 12 bytes a thread spilled at the 64 registers that eight CTAs an SM leave).
__global__ void __launch_bounds__(kQuantWarps * 32, 8)
    quant_read_kernel(const uint8_t* __restrict__ store, int max_blocks, const int32_t* __restrict__ blocks,
                      int n_blocks, const int32_t* __restrict__ lens, uint16_t* __restrict__ kv, int32_t* err) {
  pdl_wait();
  pdl_launch_dependents();
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
  // Up to kAppendTiles tiles a CTA, which saves the others' set-up, as long as every SM keeps a few CTAs' worth.
  const int per = (int)std::min<long long>(kAppendTiles, std::max<long long>(1, units * tiles / kAppendCtas));
  const long long ctas = units * ((tiles + per - 1) / per);
  if (ctas >= (1ll << 31) || (long long)units * max_blocks >= (1ll << 31)) return NOSA_ERR_INVALID_ARG;
  return launched(launch_ex(quant_append_kernel, dim3((unsigned)ctas), dim3(kQuantWarps * 32), 0,
                            static_cast<cudaStream_t>(stream), true, 0, k, v, store, n_tokens, max_blocks, pos,
                            count, (int)tiles, per, err_out));
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
                            static_cast<cudaStream_t>(stream), true, 0, store, max_blocks, blocks, n_blocks,
                            lens, kv, err_out));
}
