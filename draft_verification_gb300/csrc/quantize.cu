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
//
// What bounds it: instruction issue, with HBM (2.5 bytes per bfloat16 weight)
// not far behind.  128256 x 4096 bfloat16 weights in groups of 128 (1.32 GB, 195
// us at the measured 6.8 TB/s): 244 us, 5.4 TB/s, the schedulers issuing in 76 %
// of all cycles.  With a division per weight it took 623 us; with the group's
// size known only at run time 273 us, with the extremes found in float32 320.
// 50257 x 1024 in groups of 64 with zero points (131 MB, 19 us): 31 us, issuing in
// 77 %, HBM at 44 % of its peak: both extremes are found, and every code is clamped
// (128256 x 4096 with zero points 276 us).  float32 weights are half as much work
// per byte: 128256 x 2048 in groups of 128 (1.19 GB, 175 us) 205 us.
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

// 8 consecutive weights as they are in memory, their extremes, and one of them.
template <typename T, bool kVec>
struct Eight;

template <bool kVec>
struct Eight<bf16_t, kVec> {
  uint32_t u[4];
  __device__ __forceinline__ void load(const bf16_t* p) {
    if constexpr (kVec) {
      const uint4 v = ld_stream16(p);
      u[0] = v.x;
      u[1] = v.y;
      u[2] = v.z;
      u[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = __ldg(reinterpret_cast<const unsigned short*>(p) + 2 * j) |
               static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p) + 2 * j + 1)) << 16;
    }
  }
  __device__ __forceinline__ void clear() { u[0] = u[1] = u[2] = u[3] = 0u; }
  __device__ __forceinline__ float get(int j) const { return (j & 1) ? bf16_hi(u[j >> 1]) : bf16_lo(u[j >> 1]); }
};

template <bool kVec>
struct Eight<float, kVec> {
  float w[8];
  __device__ __forceinline__ void load(const float* p) {
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
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.f;
  }
  __device__ __forceinline__ float get(int j) const { return w[j]; }
};

// Extremes of the groups (kLanes lanes) of four rows, 0 included and
// NaN-propagating; this lane keeps those of row lane % 4.  hi: max w (max |w|
// without zeros); lo: max(0, -min w).
template <bool kZeros, int kLanes, bool kVec>
__device__ __forceinline__ void extremes(const Eight<float, kVec> (&x)[4], float& hi, float& lo) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float h = 0.f, l = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h = fmax_nan(h, kZeros ? x[i].w[j] : fabsf(x[i].w[j]));
      if constexpr (kZeros) l = fmax_nan(l, -x[i].w[j]);
    }
#pragma unroll
    for (int o = kLanes >> 1; o > 0; o >>= 1) {
      h = fmax_nan(h, __shfl_xor_sync(0xffffffffu, h, o));
      if constexpr (kZeros) l = fmax_nan(l, __shfl_xor_sync(0xffffffffu, l, o));
    }
    if ((lane & 3) == i) {
      hi = h;
      lo = l;
    }
  }
}
// bfloat16: two values to a register all the way (the extremes of bfloat16
// values are bfloat16), two rows or both extremes of one row per shuffle.
template <bool kZeros, int kLanes, bool kVec>
__device__ __forceinline__ void extremes(const Eight<bf16_t, kVec> (&x)[4], float& hi, float& lo) {
  const int lane = threadIdx.x & 31;
  const auto both = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {  // the maximum of eight, in both halves
    const uint32_t m = bmax2_nan(bmax2_nan(a, b), bmax2_nan(c, d));
    return bmax2_nan(m, __byte_perm(m, m, 0x1032));
  };
  constexpr int kRegs = kZeros ? 4 : 2;
  uint32_t m[kRegs];
  if constexpr (kZeros) {
    const uint32_t sign = 0x80008000u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t(&u)[4] = x[i].u;
      m[i] = __byte_perm(both(u[0], u[1], u[2], u[3]), both(u[0] ^ sign, u[1] ^ sign, u[2] ^ sign, u[3] ^ sign), 0x5410);
    }
  } else {
    const uint32_t magnitude = 0x7fff7fffu;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t(&u)[4] = x[i].u;
      const uint32_t(&v)[4] = x[i + 1].u;
      m[i / 2] = __byte_perm(both(u[0] & magnitude, u[1] & magnitude, u[2] & magnitude, u[3] & magnitude),
                             both(v[0] & magnitude, v[1] & magnitude, v[2] & magnitude, v[3] & magnitude), 0x5410);
    }
  }
#pragma unroll
  for (int o = kLanes >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kRegs; ++i) m[i] = bmax2_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
  if constexpr (kZeros) {
    const uint32_t mine = (lane & 2) ? ((lane & 1) ? m[3] : m[2]) : ((lane & 1) ? m[1] : m[0]);
    hi = fmax_nan(0.f, bf16_lo(mine));
    lo = fmax_nan(0.f, bf16_hi(mine));
  } else {
    const uint32_t mine = (lane & 2) ? m[1] : m[0];
    hi = (lane & 1) ? bf16_hi(mine) : bf16_lo(mine);
    lo = 0.f;
  }
}

constexpr float kGrid = 6144.f;            // float32 neighbours 2^-11 apart
constexpr float kWhole = 12582912.f;       // 1.5 * 2^23: neighbours 1 apart
constexpr float kTiny = 7.5231638e-37f;    // 2^-120

template <typename T, int kGroup, bool kVec, bool kZeros>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantParams P) {
  __shared__ unsigned short s_scale[kQuantGroups][kQuantRows];
  __shared__ unsigned char s_zero[kQuantGroups][kQuantRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = static_cast<int>(blockIdx.x) * kQuantRows;
  const int k0 = static_cast<int>(blockIdx.y) * kQuantCols;
  const int k = k0 + lane * 8;
  constexpr int kLanes = kGroup / 8;  // of a group
  constexpr int kPer = kQuantRows / (kQuantThreads / 32);
  static_assert(kPer == 4, "a group has at least 4 lanes: one for each row");
  Eight<T, kVec> x[kPer];
  const int row0 = v0 + warp * kPer;
  const int rows = k < P.d ? P.V - row0 : 0;  // this lane's (4 or more: all of the warp's)
  const T* src = static_cast<const T*>(P.weights) + static_cast<long long>(row0) * P.ld + k;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i < rows) x[i].load(src + i * P.ld);
    else x[i].clear();
  }
  float hi = 0.f, lo = 0.f;        // the group's in row lane % 4
  extremes<kZeros, kLanes>(x, hi, lo);
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
  if ((lane & (kLanes - 1)) < kPer) {
    s_scale[lane / kLanes][warp * kPer + (lane & 3)] = sb;
    if constexpr (kZeros) s_zero[lane / kLanes][warp * kPer + (lane & 3)] = static_cast<unsigned char>(z);
  }
  unsigned char* dst = P.codes + static_cast<long long>(row0) * P.codes_ld + (k >> 1);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int from = (lane & ~3) | i;
    const float ri = __shfl_sync(0xffffffffu, r, from);
    const float zi = kZeros ? __shfl_sync(0xffffffffu, z, from) : 8.f;
    const float si = __shfl_sync(0xffffffffu, s, from);
    float c[8];
    if (ri > 0.f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(T) == 2) {
          const float t = __fadd_rn(__fmaf_rn(x[i].get(j), ri, kGrid), kWhole - kGrid);
          c[j] = __fadd_rn(t, zi - kWhole);
        } else {
          const float q = __fmul_rn(x[i].get(j), ri);
          float t = __fadd_rn(__fadd_rn(q, kWhole), -kWhole);
          if (fabsf(__fadd_rn(q, -t)) > 0.4999f) t = rintf(__fdiv_rn(x[i].get(j), si));
          c[j] = __fadd_rn(t, zi);
        }
        // without zeros |w / s| < 7.5, and with them w / s rounds to -z or more
        if constexpr (kZeros) c[j] = fminf(c[j], 15.f);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = si > 0.f ? rintf(__fdiv_rn(x[i].get(j), si)) : 0.f;
        c[j] = fminf(fmaxf(__fadd_rn(q, zi), 0.f), 15.f);
      }
    }
    // four codes at a time, exact in float32, then as an integer
    const auto four = [](const float* x) {
      const float p = __fmaf_rn(__fmaf_rn(__fmaf_rn(x[3], 16.f, x[2]), 16.f, x[1]), 16.f, x[0]);
      return __float_as_uint(__fadd_rn(p, 8388608.f));  // 2^23: the low bits are the integer
    };
    if (i < rows) *reinterpret_cast<uint32_t*>(dst + i * P.codes_ld) = __byte_perm(four(c), four(c + 4), 0x5410);
  }
  __syncthreads();
  constexpr int groups = kQuantCols / kGroup;
  for (int i = tid; i < groups * kQuantRows; i += kQuantThreads) {
    const int g = i / kQuantRows, q = i % kQuantRows;
    const int v = v0 + q;
    if (v < P.V && k0 + g * kGroup < P.d) {
      const long long row = k0 / kGroup + g;
      P.scales[row * P.scales_ld + v] = s_scale[g][q];
      if constexpr (kZeros) P.zeros[row * P.zeros_ld + v] = s_zero[g][q];
    }
  }
}

template <typename T, int kGroup>
cudaError_t launch_quantize(const QuantParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.V + kQuantRows - 1) / kQuantRows),
                  static_cast<unsigned>((p.d + kQuantCols - 1) / kQuantCols));
  const bool vec = aligned(p.weights, 16) && (p.ld * static_cast<long long>(sizeof(T))) % 16 == 0;
  if (vec) {
    if (p.zeros) quantize_kernel<T, kGroup, true, true><<<grid, kQuantThreads, 0, s>>>(p);
    else quantize_kernel<T, kGroup, true, false><<<grid, kQuantThreads, 0, s>>>(p);
  } else {
    if (p.zeros) quantize_kernel<T, kGroup, false, true><<<grid, kQuantThreads, 0, s>>>(p);
    else quantize_kernel<T, kGroup, false, false><<<grid, kQuantThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_quantize(const QuantParams& p, cudaStream_t s) {
  switch (p.group) {
    case 32: return launch_quantize<T, 32>(p, s);
    case 64: return launch_quantize<T, 64>(p, s);
    default: return launch_quantize<T, 128>(p, s);
  }
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
