// Heads of 16- and 32-bit elements, rotated pair by pair: what the rotation
// and the appending to the cache share.
//
// A head's D elements are handled in units of 2 V elements, two vectors of V:
// unit u < rot / (2 V) holds pairs u V .. u V + V - 1 (their a's and b's in
// one vector each for halves, interleaved over both for neighbouring pairs),
// a unit behind them 2 V elements that are not rotated.  V is 8 (bfloat16,
// 16-byte loads), 4 or 1, the largest that divides the sizes, strides and
// addresses.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace sv {

// V consecutive elements as float32.
template <int V>
__device__ __forceinline__ void load_elems(const bf16_t* p, float* x) {
  if constexpr (V == 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(r[i]), x[2 * i + 1] = bf16_hi(r[i]);
  } else if constexpr (V == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
  }
}
template <int V>
__device__ __forceinline__ void load_elems(const float* p, float* x) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 w = *reinterpret_cast<const float4*>(p + i);
      x[i] = w.x, x[i + 1] = w.y, x[i + 2] = w.z, x[i + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = p[i];
  }
}

// two float32 values rounded to bfloat16, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <int V>
__device__ __forceinline__ void store_elems(bf16_t* p, const float* x) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                              pack_bf16(x[6], x[7]));
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = static_cast<bf16_t>(pack_bf16(x[i], 0.f));
  }
}
template <int V>
__device__ __forceinline__ void store_elems(float* p, const float* x) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = x[i];
  }
}

// Where a unit's two vectors start in a head.
struct UnitPlace {
  int a, b;      // elements
  bool rotated;
};
template <int V>
__device__ __forceinline__ UnitPlace unit_place(int u, int rot, bool pairs) {
  if (u * 2 * V >= rot || pairs) return {u * 2 * V, u * 2 * V + V, u * 2 * V < rot};
  return {u * V, rot / 2 + u * V, true};
}

// The unit's V pairs rotated in place; a rounding per operation.
template <int V>
__device__ __forceinline__ void rotate_unit(float* a, float* b, const float* cs, const float* sn, bool pairs) {
  const auto turn = [](float& x, float& y, float c, float s) {
    const float nx = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = nx;
  };
  if (V == 1 || !pairs) {
#pragma unroll
    for (int i = 0; i < V; ++i) turn(a[i], b[i], cs[i], sn[i]);
  } else {
    // pair i of the unit: elements 2 i and 2 i + 1 of the two vectors
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      turn(a[2 * i], a[2 * i + 1], cs[i], sn[i]);
      turn(b[2 * i], b[2 * i + 1], cs[V / 2 + i], sn[V / 2 + i]);
    }
  }
}

// The largest V of a call: the sizes in elements, the strides (zero strides
// of axes of one entry do not matter), the addresses.
inline int vector_width(int elem, int D, int rot, const long long* ld, int B, int n, int H, const void* p) {
  for (int v = elem == 2 ? 8 : 4; v > 1; v /= 2) {
    if (v == 2) break;
    if (D % (2 * v) || rot % (2 * v) || (reinterpret_cast<uintptr_t>(p) % (static_cast<uintptr_t>(v) * elem))) continue;
    if ((B > 1 && ld[0] % v) || (n > 1 && ld[1] % v) || (H > 1 && ld[2] % v)) continue;
    return v;
  }
  return 1;
}

}  // namespace sv
