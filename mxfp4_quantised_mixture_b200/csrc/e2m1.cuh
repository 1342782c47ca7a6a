// E2M1 encoding of fp32 values by sm_100's conversion, shared by the
// deterministic quantisers.
#pragma once

#include <stdint.h>

namespace moe {

// E2M1 codes of 8 fp32 values (element 0 in the low nibble of the result):
// round to nearest, ties to even, saturating at 6, sign kept
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&f)[8]) {
  uint32_t out;
  asm("{\n"
      ".reg .b8 c0, c1, c2, c3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n"
      "mov.b32 %0, {c0, c1, c2, c3};\n"
      "}"
      : "=r"(out)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return out;
}

// Scale byte of a block whose largest bf16 magnitude pattern is m:
// floor(log2 amax) - 2 + 127, at least 0 (<= 252 for finite input).
__device__ __forceinline__ int scale_byte(uint32_t m) { return max(static_cast<int>(m >> 7) - 2, 0); }

// 2^(127 - sb) (sb <= 253 keeps it finite)
__device__ __forceinline__ float inverse_scale(int sb) {
  return __uint_as_float(static_cast<uint32_t>(254 - min(sb, 253)) << 23);
}

}  // namespace moe
