// The 4-bit KV block store's layout, shared by the kernels that write it (quant.cu) and the
// attention over it (quant_attend.cu); include/nosa.h (nosa_quant_append) states it byte by byte.
//
// The layout is the operand layout of mma.sync m16n8k16 over a tile of 16 tokens, so that the
// attention loads 16 bytes per lane and needs neither ldmatrix nor shuffles.  Lane (g, t) = (lane / 4,
// lane % 4) owns
//   K: of tokens g and g + 8, the 32-bit word of each group that holds dims 32 gr + 8 t .. + 7 (the A
//      rows are tokens; nibble e of a word is dim + e),
//   V: of the token pairs (2t, 2t + 1) and (2t + 8, 2t + 9), the word of each group that holds dims
//      32 gr + 4 g .. + 3 (the A rows are dims; the low half of a word is the even token's four
//      nibbles, the high half the odd token's).
// In both, `word & 0x000F000F` and its three shifted forms are pairs of codes along the operand's
// contraction index, and a single token's codes are whole bytes or halves of words, so that writing
// one token reads nothing back.
#pragma once

#include <cuda_fp16.h>

#include "nosa_internal.cuh"
#include "ptx.cuh"

namespace nosa {

constexpr int kTileTokens = 16;
constexpr int kTileBytes = 2560;
constexpr int kQuantBlockBytes = NOSA_QUANT_BLOCK_BYTES;
constexpr int kTileV = 1024, kTileKs = 2048, kTileVs = 2304, kTileVm = 2432;
static_assert(4 * kTileBytes == kQuantBlockBytes, "four tiles a block");

// A group's scale and minimum as f16 bits (NaN in both where either is not finite) from its float32
// extremes; the division is IEEE's, so that s is the correctly rounded quotient.
struct GroupScale {
  uint32_t s, m;  // f16 bits
};
__device__ __forceinline__ GroupScale group_scale(float lo, float hi) {
  const __half m = __float2half_rn(lo), s = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
  const bool fine = !__hisnan(m) && !__hisinf(m) && !__hisnan(s) && !__hisinf(s);
  return {fine ? (uint32_t)__half_as_ushort(s) : 0x7e00u, fine ? (uint32_t)__half_as_ushort(m) : 0x7e00u};
}

__device__ __forceinline__ float half_bits_to_float(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }

}  // namespace nosa
