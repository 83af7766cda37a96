// Quantisation to 4-bit weights with group scales (the rule and the layout are
// in spec_logits.h).
//
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "spec_logits.h"

namespace sv {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A warp takes 256 columns of four rows at a time, 8 consecutive columns per
// lane and row, so a group is 4, 8 or 16 neighbouring lanes: its extremes come
// from two to four shuffles, every weight is read once and a lane's 8 codes are
// one 32-bit store.  What is computed once per group (a division, a reciprocal)
// is computed by a lane for one of its four rows and handed round.  The scales
// of one group lie a vocabulary apart for one row, so a CTA of 8 warps covers 32
// rows and hands their scales through shared memory: 32 neighbouring values per
// store.
//
// The codes are rint(w / s) with an IEEE division, without dividing:
//   bfloat16 weights  w and s have 8 significant bits, so w / s is half way
//     between two integers exactly or differs from every such point by 1/1020
//     or more.  One fma puts w (1 / s) on a grid of 2^-11 (adding 6144, whose
//     float32 neighbours are that far apart): an exact half lands on itself,
//     anything else stays on its side, and rounding the grid point to even is
//     rounding the quotient.
//   float32 weights   w (1 / s) is within 3e-6 of the quotient, so its rounding
//     is the quotient's unless it lies within 1e-4 of half way: those few
//     weights are divided.
// Groups whose scale is below 2^-120 (or 0, or not finite) are divided.
constexpr int kQuantThreads = 256;
constexpr int kQuantRows = 32;             // rows per CTA, 4 per warp
constexpr int kQuantCols = 256;            // columns per CTA
constexpr int kQuantGroups = kQuantCols / 32;

struct QuantParams {
  int V, d, group;
  long long ld, codes_ld, scales_ld, zeros_ld;
  const void* weights;
  unsigned char* codes;
  unsigned short* scales;
  unsigned char* zeros;
};

__device__ __forceinline__ unsigned short to_bf16(float x) {
  unsigned short r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* p, float (&w)[8]) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (kVec) {
      const uint4 v = ld_stream16(p);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[2 * j] = bf16_lo(u[j]);
        w[2 * j + 1] = bf16_hi(u[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = load_elem(p + j);
    }
  } else {
    if constexpr (kVec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 v = ld_stream16(p + 4 * h);
        w[4 * h] = __uint_as_float(v.x);
        w[4 * h + 1] = __uint_as_float(v.y);
        w[4 * h + 2] = __uint_as_float(v.z);
        w[4 * h + 3] = __uint_as_float(v.w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = load_elem(p + j);
    }
  }
}

constexpr float kGrid = 6144.f;            // float32 neighbours 2^-11 apart
constexpr float kWhole = 12582912.f;       // 1.5 * 2^23: neighbours 1 apart
constexpr float kTiny = 7.5231638e-37f;    // 2^-120

template <typename T, bool kVec, bool kZeros>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantParams P) {
  __shared__ unsigned short s_scale[kQuantGroups][kQuantRows];
  __shared__ unsigned char s_zero[kQuantGroups][kQuantRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = static_cast<int>(blockIdx.x) * kQuantRows;
  const int k0 = static_cast<int>(blockIdx.y) * kQuantCols;
  const int k = k0 + lane * 8;
  constexpr int kPer = kQuantRows / (kQuantThreads / 32);
  static_assert(kPer == 4, "a group has at least 4 lanes: one for each row");
  float w[kPer][8];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = v0 + warp * kPer + i;
    if (v < P.V && k < P.d) {
      load8<T, kVec>(static_cast<const T*>(P.weights) + static_cast<long long>(v) * P.ld + k, w[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 0.f;
    }
  }
  const int lanes = P.group >> 3;  // lanes of a group
  // extremes of this lane's group in each row, 0 included; NaN-propagating
  // (lo holds max(0, -min))
  float hi = 0.f, lo = 0.f;  // of row lane % 4
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float h = 0.f, l = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h = fmax_nan(h, kZeros ? w[i][j] : fabsf(w[i][j]));
      if constexpr (kZeros) l = fmax_nan(l, -w[i][j]);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      h = fmax_nan(h, __shfl_xor_sync(0xffffffffu, h, o));
      if constexpr (kZeros) l = fmax_nan(l, __shfl_xor_sync(0xffffffffu, l, o));
    }
    if ((lane & 3) == i) {
      hi = h;
      lo = l;
    }
  }
  // row lane % 4: the scale, its reciprocal and the zero point
  unsigned short sb = to_bf16(kZeros ? __fdiv_rn(__fadd_rn(hi, lo), 15.f) : __fdiv_rn(hi, 7.f));
  float s = __uint_as_float(static_cast<uint32_t>(sb) << 16);
  if (!(s < kInf)) {  // a NaN or an infinity in the group, or an overflow of s
    sb = 0x7fc0;
    s = 0.f;
  }
  const float r = s >= kTiny ? __frcp_rn(s) : 0.f;
  float z = 8.f;
  if constexpr (kZeros) z = s > 0.f ? fminf(rintf(__fdiv_rn(lo, s)), 15.f) : 0.f;
  if ((lane & (lanes - 1)) < kPer) {
    s_scale[lane / lanes][warp * kPer + (lane & 3)] = sb;
    if constexpr (kZeros) s_zero[lane / lanes][warp * kPer + (lane & 3)] = static_cast<unsigned char>(z);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = v0 + warp * kPer + i;
    const int from = (lane & ~3) | i;
    const float ri = __shfl_sync(0xffffffffu, r, from);
    const float zi = kZeros ? __shfl_sync(0xffffffffu, z, from) : 8.f;
    const float si = __shfl_sync(0xffffffffu, s, from);
    float c[8];
    if (ri > 0.f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(T) == 2) {
          const float t = __fadd_rn(__fmaf_rn(w[i][j], ri, kGrid), kWhole - kGrid);
          c[j] = __fadd_rn(t, zi - kWhole);
        } else {
          const float q = __fmul_rn(w[i][j], ri);
          float t = __fadd_rn(__fadd_rn(q, kWhole), -kWhole);
          if (fabsf(__fadd_rn(q, -t)) > 0.4999f) t = rintf(__fdiv_rn(w[i][j], si));
          c[j] = __fadd_rn(t, zi);
        }
        // without zeros |w / s| < 7.5, and with them w / s rounds to -z or more
        if constexpr (kZeros) c[j] = fminf(c[j], 15.f);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = si > 0.f ? rintf(__fdiv_rn(w[i][j], si)) : 0.f;
        c[j] = fminf(fmaxf(__fadd_rn(q, zi), 0.f), 15.f);
      }
    }
    // four codes at a time, exact in float32, then as an integer
    const auto four = [](const float* x) {
      const float p = __fmaf_rn(__fmaf_rn(__fmaf_rn(x[3], 16.f, x[2]), 16.f, x[1]), 16.f, x[0]);
      return __float_as_uint(__fadd_rn(p, 8388608.f));  // 2^23: the low bits are the integer
    };
    if (v < P.V && k < P.d)
      *reinterpret_cast<uint32_t*>(P.codes + static_cast<long long>(v) * P.codes_ld + (k >> 1)) =
          __byte_perm(four(c), four(c + 4), 0x5410);
  }
  __syncthreads();
  const int groups = kQuantCols / P.group;
  for (int i = tid; i < groups * kQuantRows; i += kQuantThreads) {
    const int g = i / kQuantRows, q = i % kQuantRows;
    const int v = v0 + q;
    if (v < P.V && k0 + g * P.group < P.d) {
      const long long row = k0 / P.group + g;
      P.scales[row * P.scales_ld + v] = s_scale[g][q];
      if constexpr (kZeros) P.zeros[row * P.zeros_ld + v] = s_zero[g][q];
    }
  }
}

template <typename T>
cudaError_t launch_quantize(const QuantParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.V + kQuantRows - 1) / kQuantRows),
                  static_cast<unsigned>((p.d + kQuantCols - 1) / kQuantCols));
  const bool vec = aligned(p.weights, 16) && (p.ld * static_cast<long long>(sizeof(T))) % 16 == 0;
  if (vec) {
    if (p.zeros) quantize_kernel<T, true, true><<<grid, kQuantThreads, 0, s>>>(p);
    else quantize_kernel<T, true, false><<<grid, kQuantThreads, 0, s>>>(p);
  } else {
    if (p.zeros) quantize_kernel<T, false, true><<<grid, kQuantThreads, 0, s>>>(p);
    else quantize_kernel<T, false, false><<<grid, kQuantThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

bool good_shape(int V, int d, int group) {
  return V >= 1 && V <= 2097152 && (group == 32 || group == 64 || group == 128) && d >= 32 && d <= 65536 &&
         d % group == 0;
}

}  // namespace
}  // namespace sv

extern "C" spec_status spec_quantize_int4(const spec_quantize_int4_args* a, cudaStream_t stream) {
  using namespace sv;
  NvtxRange nvtx_range("spec_quantize_int4");
  if (a == nullptr) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (!good_shape(a->V, a->d, a->group)) return SPEC_EINVAL;
  if (!a->weights || !a->codes || !a->scales) return SPEC_EINVAL;
  if (a->ld < a->d || a->codes_ld < a->d / 2 || a->codes_ld % 16 || a->scales_ld < a->V) return SPEC_EINVAL;
  if (a->zeros && a->zeros_ld < a->V) return SPEC_EINVAL;
  if (!aligned(a->weights, a->dtype == SPEC_F32 ? 4 : 2) || !aligned(a->codes, 16) || !aligned(a->scales, 2))
    return SPEC_EALIGN;
  QuantParams p{};
  p.V = a->V;
  p.d = a->d;
  p.group = a->group;
  p.ld = a->ld;
  p.codes_ld = a->codes_ld;
  p.scales_ld = a->scales_ld;
  p.zeros_ld = a->zeros_ld;
  p.weights = a->weights;
  p.codes = static_cast<unsigned char*>(a->codes);
  p.scales = static_cast<unsigned short*>(a->scales);
  p.zeros = a->zeros;
  const cudaError_t e =
      a->dtype == SPEC_BF16 ? launch_quantize<bf16_t>(p, stream) : launch_quantize<float>(p, stream);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}
