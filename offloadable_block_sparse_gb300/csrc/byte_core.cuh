// The 8-bit KV block store's layout, shared by the kernels that write it (byte_store.cu) and the attention over it
// (byte_attend.cu); include/nosa.h (nosa_byte_append) states it byte by byte.
//
// As in the 4-bit store the layout is that of mma.sync operands over a tile of 16 tokens, so that a lane loads 16 bytes at
// a time, a warp 512 in a row.  Lane (g, t) = (lane / 4, lane % 4) owns
//   K: of tokens g and g + 8, dims 32 t .. + 31 (the A rows are tokens; a word is four places of the contraction index of
//      m16n8k32, which takes the codes as they are),
//   V: of tokens 2t, 2t + 1, 2t + 8 and 2t + 9, dims 16 g .. + 15 (the A rows are dims: a word holds two dims of a
//      token pair; two neighbouring bytes become an f16x2 in one conversion, a pair along m16n8k16's contraction index).
#pragma once

#include <cuda_fp16.h>

#include "nosa_internal.cuh"
#include "ptx.cuh"

namespace nosa {

constexpr int kByteTileTokens = 16, kByteTile = 4096, kByteV = 2048;
constexpr int kByteTiles = kBlock / kByteTileTokens;
constexpr int kByteScales = kByteTiles * kByteTile;  // s_K, s_V as float32
constexpr int kByteBlockBytes = NOSA_BYTE_BLOCK_BYTES;
static_assert(kByteScales + 128 == kByteBlockBytes, "four tiles and a line with the scales");
constexpr int kLeastScale = -118, kMostScale = 119;  // exponents of a scale

// Four e4m3 codes as two f16x2, exactly (NaN stays NaN).  (Naming the halves of the register saves a shift.)
__device__ __forceinline__ void codes_to_half2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
// Two floats as e4m3 codes, to nearest, ties to even; sizes above 448 become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace nosa
