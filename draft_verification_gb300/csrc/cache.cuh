// The paged cache's codes and exponents (spec_cache.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace sv {

constexpr int kLowExp = -100, kHighExp = 100;

// 2^e, e in [-126, 127]
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two float32 values to e4m3, to nearest, the first in the low byte; beyond
// 448 they become 448 or -448, NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  unsigned short d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Two e4m3 codes as float32 (exact: e4m3 is a subset of float16).
__device__ __forceinline__ float2 unpack_e4m3(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(two)));
  float2 r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

}  // namespace sv
