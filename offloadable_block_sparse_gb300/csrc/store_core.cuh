// What the attention kernels over the quantised block stores share (quant_attend.cu, byte_attend.cu): the f16 MMA and
// its operands' packing, the waits for staged copies, the merging of partial results and how blocks are dealt to CTAs.
#pragma once

#include <cuda_fp16.h>

#include "nosa_internal.cuh"
#include "ptx.cuh"

namespace nosa {

constexpr int kQaSplitUnits = 2048;   // beyond, one CTA per unit
constexpr int kQaList = 256;          // listed blocks looked up at a time
constexpr int kQaMaxRows = 32;
constexpr int kMergeWarps = 8;
constexpr size_t kQaErrBytes = 256;   // the scratch starts with the device error word
constexpr int kQaRowStride = 132;     // floats per row of a warp's partial in shared memory (no bank conflicts)
constexpr float kNoRef = -3e38f;      // reference of a row that has seen no token

// How a call's CTAs share its units: one CTA each, equal pieces of all units' blocks, a cluster each.
enum { kWhole, kPieces, kCluster };

// D (16 x 8, f32) += A (16 x 16, row) . B (16 x 8, col), f16 inputs.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with D = A . B: a zero operand costs nothing, a zeroed accumulator four moves.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// SM cycles that a wait of this host thread's attention calls may take (nosa_debug_quant_wait; in quant_attend.cu).
extern thread_local long long g_wait_limit;
constexpr long long kProductsGiveUp = -2;  // of the 8-bit store's waits only those for products

// Waits for a staged half block.  Returns whether it came within `limit` cycles; waits on for those that did not, as long
// again as the longest limit, so that the copy has landed before the ring has another use or the CTA ends.
__device__ __forceinline__ bool stage_wait(uint64_t* bar, uint32_t phase, long long limit) {
  if (mbar_try_wait(bar, phase)) return limit >= 0;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, phase)) {
    if (clock64() - t0 > 2 * kWaitCycles) return false;
  }
  return clock64() - t0 <= limit;
}

// Adds a part (reference r, sum l, four dims o) to a running one.
__device__ __forceinline__ void merge_part(float& R, float& L, float4& O, float r, float l, const float4& o) {
  const float top = fmaxf(R, r), f = ex2(R - top), h = ex2(r - top);
  R = top;
  L = L * f + l * h;
  O.x = O.x * f + o.x * h;
  O.y = O.y * f + o.y * h;
  O.z = O.z * f + o.z * h;
  O.w = O.w * f + o.w * h;
}

// Four dims of an output row, o in units of `unit`: zeros where no token was seen.
__device__ __forceinline__ void store_out(uint16_t* out, const float4& o, float l, float unit = 1.f) {
  uint2 v = make_uint2(0, 0);
  if (l != 0.f) v = make_uint2(pack_bf16x2(o.x / l * unit, o.y / l * unit), pack_bf16x2(o.z / l * unit, o.w / l * unit));
  *reinterpret_cast<uint2*>(out) = v;
}

// The blocks that CTA i of n takes of `total`: [first(i), first(i + 1)), and the CTA that takes block b.
// (total is at most kQaSplitUnits x 16384, n one wave's CTAs: total i / n without a 64-bit division, some 500 cycles.)
__device__ __forceinline__ int cta_first(int total, int i, int n) {
  const uint32_t q = (uint32_t)total / (uint32_t)n, r = (uint32_t)total - q * n;
  return (int)(q * i + r * i / (uint32_t)n);
}
__device__ __forceinline__ int cta_of(int total, int b, int n) { return (int)(((long long)(b + 1) * n - 1) / total); }

}  // namespace nosa
