// Attention of drafted rows over the paged 8-bit cache (spec_attend_cache).
//
// One CTA per query row and head, a pass over its tokens in tiles of 128 with
// the running maximum and sum of the softmax.
#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "common.cuh"
#include "internal.h"
#include "spec_cache.h"

namespace sv {
namespace {

constexpr int kTile = 128;
constexpr float kNan = __builtin_nanf("");

struct AttendParams {
  int n, Hq, H, D, page, pages, table_pages;
  float c;  // scale * log2(e)
  long long q_ld[3], out_ld[3];
  const bf16_t* q;
  bf16_t* out;
  const int* prefix;
  const int* count;
  const int* parent;
  const int* block_table;
  const unsigned char* k_codes;
  const unsigned char* v_codes;
  const signed char* k_exps;
  const signed char* v_exps;
  int* seq_error;
  int* error_word;
};

__device__ void report(const AttendParams& P, int b, int bits) {
  if (P.seq_error) atomicOr(P.seq_error + b, bits);
  if (P.error_word) atomicOr(P.error_word, bits);
}

__global__ void __launch_bounds__(kTile) attend_kernel(const AttendParams P) {
  __shared__ float q_s[256], w_s[kTile], red_s[kTile / 32];
  __shared__ const unsigned char* v_s[kTile];
  __shared__ uint32_t own_s[32];  // the row's own nodes: ancestors and itself
  const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int hk = h / (P.Hq / P.H);
  const int prefix = P.prefix ? P.prefix[b] : 0, count = P.count ? P.count[b] : P.n;
  bf16_t* out = P.out + b * P.out_ld[0] + i * P.out_ld[1] + h * P.out_ld[2];
  const bool bad = prefix < 0 || count < 0 || count > P.n ||
                   static_cast<long long>(prefix) + count > static_cast<long long>(P.table_pages) * P.page;
  if (bad && tid == 0 && h == 0 && i == 0) report(P, b, SPEC_ERR_CACHE);
  if (bad || i >= count) {
    for (int d = tid; d < P.D; d += kTile) out[d] = 0;
    return;
  }
  for (int d = tid; d < P.D; d += kTile)
    q_s[d] = load_elem(P.q + b * P.q_ld[0] + i * P.q_ld[1] + h * P.q_ld[2] + d);
  if (tid < 32) own_s[tid] = P.parent ? 0u : (tid < i / 32 ? 0xffffffffu : tid == i / 32 ? (2u << (i % 32)) - 1u : 0u);
  __syncthreads();
  if (P.parent && tid == 0) {
    own_s[0] |= 1u;
    for (int j = i; j > 0;) {
      own_s[j / 32] |= 1u << (j % 32);
      const int p = P.parent[static_cast<long long>(b) * P.n + j];
      if (p < 0 || p >= j) report(P, b, SPEC_ERR_PARENT);
      j = p < 0 || p >= j ? 0 : p;
    }
  }
  __syncthreads();
  const auto all_max = [&](float v) {
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((tid & 31) == 0) red_s[tid >> 5] = v;
    __syncthreads();
    return fmaxf(fmaxf(red_s[0], red_s[1]), fmaxf(red_s[2], red_s[3]));
  };
  float m = -kInf, l = 0.f, o0 = 0.f, o1 = 0.f;
  const int keys = prefix + count;
  for (int t0 = 0; t0 < keys; t0 += kTile) {
    const int t = t0 + tid, j = t - prefix;
    const bool seen = t < keys && (j < 0 || (own_s[j / 32] >> (j % 32) & 1u));
    float x = -kInf;
    v_s[tid] = nullptr;
    float ve = 0.f;
    if (seen) {
      const int page = P.block_table[static_cast<long long>(b) * P.table_pages + t / P.page];
      if (page < 0 || page >= P.pages) {
        report(P, b, SPEC_ERR_CACHE);
        x = kNan;
      } else {
        const long long slab = static_cast<long long>(page) * P.H + hk;
        const long long at = (slab * P.page + t % P.page) * P.D;
        const unsigned char* k = P.k_codes + at;
        float s = 0.f;
        for (int d = 0; d < P.D; d += 2) {
          const float2 two = unpack_e4m3(*reinterpret_cast<const unsigned short*>(k + d));
          s = __fmaf_rn(two.x, q_s[d], s);
          s = __fmaf_rn(two.y, q_s[d + 1], s);
        }
        x = s * exp2i(P.k_exps[slab]) * P.c;
        v_s[tid] = P.v_codes + at;
        ve = exp2i(P.v_exps[slab]);
      }
    }
    const float top = all_max(x);
    const float mn = fmaxf(m, top), shift = mn == -kInf ? 0.f : mn;
    const float old = m == -kInf ? 0.f : ex2(m - shift);
    const float w = seen ? ex2(x - shift) : 0.f;
    l = l * old + w;
    w_s[tid] = w * ve;
    if (seen && w != w) w_s[tid] = kNan;
    __syncthreads();
    o0 *= old, o1 *= old;
    for (int k = 0; k < kTile; ++k) {
      if (v_s[k] == nullptr) continue;
      if (tid < P.D) o0 = __fmaf_rn(w_s[k], unpack_e4m3(v_s[k][tid]).x, o0);
      if (tid + kTile < P.D) o1 = __fmaf_rn(w_s[k], unpack_e4m3(v_s[k][tid + kTile]).x, o1);
    }
    __syncthreads();
    m = mn;
  }
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  __syncthreads();
  if ((tid & 31) == 0) red_s[tid >> 5] = l;
  __syncthreads();
  l = (red_s[0] + red_s[1]) + (red_s[2] + red_s[3]);
  const auto store = [&](int d, float v) {
    const float y = v / l;
    unsigned short bits;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(y));
    out[d] = bits;
  };
  if (tid < P.D) store(tid, o0);
  if (tid + kTile < P.D) store(tid + kTile, o1);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool good_shape(int B, int n, int Hq, int H, int D) {
  return B >= 1 && B <= 65535 && n >= 1 && n <= 1024 && H >= 1 && Hq >= H && Hq <= 1024 && Hq % H == 0 && D >= 16 &&
         D <= 256 && D % 16 == 0;
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_attend_workspace_size(int B, int n, int Hq, int H, int D) {
  return sv::good_shape(B, n, Hq, H, D) ? 256 : 0;
}

extern "C" spec_status spec_attend_cache(const spec_attend_args* a, cudaStream_t stream) {
  using namespace sv;
  NvtxRange nvtx_range("spec_attend_cache");
  if (a == nullptr) return SPEC_EINVAL;
  if (!good_shape(a->B, a->n, a->Hq, a->H, a->D)) return SPEC_EINVAL;
  if (a->page != 16 && a->page != 32 && a->page != 64 && a->page != 128) return SPEC_EINVAL;
  if (a->pages < 1 || static_cast<long long>(a->pages) * a->H * a->page > 0x7fffffffLL || a->table_pages < 1 ||
      static_cast<long long>(a->table_pages) * a->page > (1 << 30))
    return SPEC_EINVAL;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return SPEC_EINVAL;
  if (!a->q || !a->out || !a->block_table || !a->k_codes || !a->v_codes || !a->k_exps || !a->v_exps) return SPEC_EINVAL;
  for (int i = 0; i < 3; ++i)
    if (a->q_ld[i] % 8) return SPEC_EALIGN;
  if (!aligned(a->q, 16) || !aligned(a->out, 2) || !aligned(a->k_codes, 16) || !aligned(a->v_codes, 16))
    return SPEC_EALIGN;
  if (!a->workspace || a->workspace_bytes < spec_attend_workspace_size(a->B, a->n, a->Hq, a->H, a->D) ||
      !aligned(a->workspace, 256))
    return SPEC_EWORKSPACE;
  AttendParams p{};
  p.n = a->n;
  p.Hq = a->Hq;
  p.H = a->H;
  p.D = a->D;
  p.page = a->page;
  p.pages = a->pages;
  p.table_pages = a->table_pages;
  p.c = a->scale * 1.44269504088896340736f;
  for (int i = 0; i < 3; ++i) p.q_ld[i] = a->q_ld[i], p.out_ld[i] = a->out_ld[i];
  p.q = static_cast<const bf16_t*>(a->q);
  p.out = static_cast<bf16_t*>(a->out);
  p.prefix = a->prefix_len;
  p.count = a->count;
  p.parent = a->parent;
  p.block_table = a->block_table;
  p.k_codes = static_cast<const unsigned char*>(a->k_codes);
  p.v_codes = static_cast<const unsigned char*>(a->v_codes);
  p.k_exps = a->k_exps;
  p.v_exps = a->v_exps;
  p.seq_error = a->seq_error;
  p.error_word = a->error_word;
  attend_kernel<<<dim3(a->Hq, a->n, a->B), kTile, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}
