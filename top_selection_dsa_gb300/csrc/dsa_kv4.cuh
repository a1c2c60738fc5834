// dsa_kv4.cuh -- the paged 4-bit key/value cache: its record layout and the
// conversions between packed E2M1 codes and fp16 pairs.
//
// One token of one key/value head is a record of D bytes: D/2 bytes of packed
// E2M1 key codes, then D/2 bytes of packed E2M1 value codes; next to it, in an
// array of its own, D/16 bytes of E8M0 scales (one per 32 consecutive elements):
// D/32 of the key, then D/32 of the value.  A scale is 2^(code - 127) for the
// codes 1 to 253 that an insert writes (and for 254), NaN for 255.  Code 0,
// which E8M0 gives 2^-127, is what an empty cache holds, and reads as zero:
// telling it from zero costs the 16-row attention 4 % (600 -> 624 us) for
// values below 2^-124.
//   records [num_blocks, Hkv, block_size, D], scales [num_blocks, Hkv,
//   block_size, D/16] -- a page's tokens of one head are contiguous.
// The codes of a record are ordered the way the attention kernel's matrix
// fragments take them, so that a lane's share is one shared-memory load and
// no code has to move between lanes (G = D/32 scale blocks):
//   key    8-element word w = 4 g + t  (elements 32 g + 8 t ..) at word t G + g
//          of the key half: lane quad member t holds its words of every block
//          side by side;
//   value  4-element unit u = 8 g + r (elements 32 g + 4 r ..) at unit r G + g
//          of the value half: the eight lane rows r likewise.
// In a byte the lower element is the low nibble.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_common.cuh"

namespace dsa {

constexpr int kMxBlock = 32;  // elements that share a scale

// Byte kByte of w (two E2M1 codes, low nibble first) -> two fp16 values.
template <int kByte>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (kByte == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (kByte == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (kByte == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Two fp32 values -> two E2M1 codes (round to nearest, ties to even,
// saturating); lo lands in the low nibble.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

}  // namespace dsa
