// The 8-bit KV block store's layout, shared by the kernels that write it (byte_store.cu) and the attention over it
// (byte_attend.cu); include/nosa.h (nosa_byte_append) states it byte by byte.
//
// As in the 4-bit store the layout is the operand layout of mma.sync m16n8k16 over a tile of 16 tokens, so that a lane
// loads 16 bytes at a time, a warp 512 in a row.  Lane (g, t) = (lane / 4, lane % 4) owns
//   K: of tokens g and g + 8, dims 32 t .. + 31 (the A rows are tokens; a word's low two bytes and its high two are two
//      pairs along the operand's contraction index),
//   V: of tokens 2t, 2t + 1, 2t + 8 and 2t + 9, dims 16 g .. + 15 (the A rows are dims: a word holds two dims of a
//      token pair, so that a pair of tokens is a pair along the contraction index).
// Two neighbouring bytes become an f16x2 in one conversion.
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

// Two e4m3 codes as f16x2, exactly (NaN stays NaN).
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 c;\n cvt.u16.u32 c, %1;\n cvt.rn.f16x2.e4m3x2 %0, c;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return codes_to_half2(w); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return codes_to_half2(w >> 16); }

}  // namespace nosa
