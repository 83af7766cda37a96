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

// A warp takes 256 columns of one row at a time, 8 consecutive ones per lane,
// so a group is 4, 8 or 16 neighbouring lanes: its extremes come from three
// to four shuffles, every weight is read once and a lane's 8 codes are one
// 32-bit store.  The scales of one group lie a vocabulary apart for one row,
// so a CTA of 8 warps covers 32 rows and hands their scales through shared
// memory: 32 neighbouring values per store.
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

template <typename T, bool kVec, bool kZeros>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantParams P) {
  __shared__ unsigned short s_scale[kQuantGroups][kQuantRows];
  __shared__ unsigned char s_zero[kQuantGroups][kQuantRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = static_cast<int>(blockIdx.x) * kQuantRows;
  const int k0 = static_cast<int>(blockIdx.y) * kQuantCols;
  const int k = k0 + lane * 8;
  constexpr int kPer = kQuantRows / (kQuantThreads / 32);
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
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = warp * kPer + i;
    const int v = v0 + r;
    float lo = 0.f, hi = 0.f;  // extremes, 0 included; NaN-propagating
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hi = fmax_nan(hi, kZeros ? w[i][j] : fabsf(w[i][j]));
      if constexpr (kZeros) lo = fmax_nan(lo, -w[i][j]);  // lo holds max(0, -min)
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      hi = fmax_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      if constexpr (kZeros) lo = fmax_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    const float span = kZeros ? __fdiv_rn(__fadd_rn(hi, lo), 15.f) : __fdiv_rn(hi, 7.f);
    unsigned short sb = to_bf16(span);
    float s = __uint_as_float(static_cast<uint32_t>(sb) << 16);
    if (!(s < kInf)) {  // a NaN or an infinity in the group, or an overflow of s
      sb = 0x7fc0;
      s = 0.f;
    }
    float z = 0.f;
    if constexpr (kZeros) {
      if (s > 0.f) z = fminf(rintf(__fdiv_rn(lo, s)), 15.f);
    }
    const float low = kZeros ? 0.f : -8.f, high = kZeros ? 15.f : 7.f;
    uint32_t packed = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float q = s > 0.f ? rintf(__fdiv_rn(w[i][j], s)) : 0.f;
      q = fminf(fmaxf(__fadd_rn(q, z), low), high);
      packed |= static_cast<uint32_t>(static_cast<int>(q) + (kZeros ? 0 : 8)) << (4 * j);
    }
    if (v < P.V && k < P.d)
      *reinterpret_cast<uint32_t*>(P.codes + static_cast<long long>(v) * P.codes_ld + (k >> 1)) = packed;
    if ((lane & (lanes - 1)) == 0) {
      s_scale[lane / lanes][r] = sb;
      if constexpr (kZeros) s_zero[lane / lanes][r] = static_cast<unsigned char>(z);
    }
  }
  __syncthreads();
  const int groups = kQuantCols / P.group;
  for (int i = tid; i < groups * kQuantRows; i += kQuantThreads) {
    const int g = i / kQuantRows, r = i % kQuantRows;
    const int v = v0 + r;
    if (v < P.V && k0 + g * P.group < P.d) {
      const long long row = k0 / P.group + g;
      P.scales[row * P.scales_ld + v] = s_scale[g][r];
      if constexpr (kZeros) P.zeros[row * P.zeros_ld + v] = s_zero[g][r];
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
