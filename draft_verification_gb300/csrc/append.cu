// Appending keys and values to the paged 8-bit cache (spec_append_cache).
//
// One CTA per page that gets rows, head and sequence: it alone reads and
// writes that page of that head.  It needs its rows' largest magnitude before
// it can round the first of them, so they stay in registers in between: a
// thread keeps up to kHold units (what it takes for pages of 64 tokens and 128
// elements: 1 of fp32 or bf16 for a chain's few rows, 2 for full pages of
// bf16, 4 for those of fp32), loaded before the block table's answer is
// there.  Larger pages, and rows that start anywhere, are read twice.
//
// It moves 2 x (element + code) bytes per row, head and element.  4 x 8191 rows
// of 8 heads of 128, bf16: 48 us, 4.2 TB/s, 0.63 of a copy's rate.  What bounds
// that: instructions (70 % of the issue slots, DRAM 44 % busy) and three waits
// of a CTA one behind another (its lengths; the page's name beside its rows; an
// older page's exponents beside the rotation's rows, which every head reads
// again, from L2).  When they were tried: a test of the range per element
// instead of per vector 53 us, three CTAs per SM instead of four 50, rows read
// twice 62, room for four units in every page 70 (fewer CTAs per SM).  Pages of
// more units than two per thread run at one CTA of 512 threads per SM: the same
// rows in pages of 128 72 us, in fp32 111 us (0.46).  A drafted chain (64 x 6
// rows) takes 5.4 us in a graph, one row 2.6; a call from the host costs more.
#include <algorithm>
#include <cstdint>

#include "cache.cuh"
#include "heads.cuh"
#include "internal.h"
#include "spec_cache.h"

namespace sv {
namespace {


struct AppendParams {
  int n, H, D, page, pages, table_pages, rot, units, table_rows, path_ld;
  bool pairs;
  long long k_ld[3], v_ld[3];
  const void* k;
  const void* v;
  const float* table;
  const int* positions;
  const int* prefix;
  const int* count;
  const int* path_nodes;
  const int* path_len;
  const int* block_table;
  unsigned char* k_codes;
  unsigned char* v_codes;
  signed char* k_exps;
  signed char* v_exps;
  int* seq_error;
  int* error_word;
};

// The larger magnitude, with some sign; NaN if one is.
__device__ __forceinline__ float larger(float a, float b) {
  float m;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// V float32 values times `scale` to codes; what e4m3 does not reach becomes NaN
// (and `bad`).  One test for all of them: it is instructions that a long call
// waits for.
template <int V>
__device__ __forceinline__ void store_codes(unsigned char* p, const float* x, float scale, bool& bad) {
  float y[V], m = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    y[i] = x[i] * scale;
    m = larger(m, y[i]);
  }
  if (!(fabsf(m) <= 448.f)) {
    bad = true;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!(fabsf(y[i]) <= 448.f)) y[i] = __uint_as_float(0x7fc00000u);
  }
  if constexpr (V == 8) {
    *reinterpret_cast<uint2*>(p) =
        make_uint2(pack_e4m3(y[0], y[1]) | pack_e4m3(y[2], y[3]) << 16, pack_e4m3(y[4], y[5]) | pack_e4m3(y[6], y[7]) << 16);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(p) = pack_e4m3(y[0], y[1]) | pack_e4m3(y[2], y[3]) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = static_cast<unsigned char>(pack_e4m3(y[i], 0.f));
  }
}

// The page's earlier codes, scaled by 2^-shift, shift >= 1.
template <int TH>
__device__ void scale_codes(unsigned char* p, int bytes, int shift) {
  const float f = shift > 126 ? 0.f : exp2i(-shift);
  for (int o = threadIdx.x * 16; o < bytes; o += TH * 16) {
    uint4 w = *reinterpret_cast<uint4*>(p + o);
    uint32_t* r = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 lo = unpack_e4m3(r[i] & 0xffffu), hi = unpack_e4m3(r[i] >> 16);
      r[i] = pack_e4m3(lo.x * f, lo.y * f) | pack_e4m3(hi.x * f, hi.y * f) << 16;
    }
    *reinterpret_cast<uint4*>(p + o) = w;
  }
}

// The least e with m <= 2^(e + 7), in range.
__device__ __forceinline__ int exponent_of(float m) {
  const uint32_t bits = __float_as_uint(m);
  if (bits < (1u << 23)) return kLowExp;  // (0, or below 2^-126)
  const int e = static_cast<int>(bits >> 23) - 127 + ((bits & 0x7fffffu) != 0 ? 1 : 0) - 7;
  return min(kHighExp, max(kLowExp, e));
}

// TH threads; kHold: units of a page's rows that a thread keeps in registers
// between the two passes, 0: none (they are read twice)
template <typename T, int V, int TH, int kHold>
__global__ void __launch_bounds__(TH, kHold == 2 ? 4 : kHold == 1 ? 3 : 1) append_kernel(const AppendParams P) {
  __shared__ float most_s[2][TH / 32];
  __shared__ int skip_s;
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const int prefix = P.prefix ? P.prefix[b] : 0;
  const int* path = P.path_nodes ? P.path_nodes + static_cast<long long>(b) * P.path_ld : nullptr;
  const bool reports = blockIdx.x == 0 && h == 0;  // one CTA per sequence reports what concerns all of it
  int rows, bits = 0;
  if (path) {
    const int depth = P.path_len[b];
    if (path[0] == -1) return;  // the verification's data-error marking
    if (tid == 0) skip_s = 0;
    __syncthreads();
    if (depth < 0 || depth >= P.path_ld) bits |= SPEC_ERR_CACHE;
    rows = bits ? 0 : depth + 1;
    bool bad = false;
    for (int i = tid; i < rows; i += TH) bad |= path[i] < 0 || path[i] >= P.n;
    if (bad) atomicOr(&skip_s, SPEC_ERR_PARENT);
    __syncthreads();
    bits |= skip_s;
  } else {
    rows = P.count ? P.count[b] : P.n;
    if (rows < 0 || rows > P.n) bits |= SPEC_ERR_CACHE;
  }
  if (prefix < 0 || static_cast<long long>(prefix) + rows > static_cast<long long>(P.table_pages) * P.page)
    bits |= SPEC_ERR_CACHE;
  if (bits) {
    if (reports && tid == 0) {
      if (P.seq_error) atomicOr(P.seq_error + b, bits);
      if (P.error_word) atomicOr(P.error_word, bits);
    }
    return;
  }
  const int entry = prefix / P.page + blockIdx.x;
  const int start = entry * P.page;  // first token of the page
  const int i0 = max(0, start - prefix), i1 = min(rows, start + P.page - prefix);
  if (i0 >= i1) return;
  const int page = P.block_table[static_cast<long long>(b) * P.table_pages + entry];
  const T* k = static_cast<const T*>(P.k) + b * P.k_ld[0] + h * P.k_ld[2];
  const T* v = static_cast<const T*>(P.v) + b * P.v_ld[0] + h * P.v_ld[2];
  const int work = (i1 - i0) * P.units;

  // the largest finite magnitudes
  float mk = 0.f, mv = 0.f;
  const auto most = [](float m, const float* x) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float a = fabsf(x[e]);
      if (a < kInf) m = fmaxf(m, a);
    }
    return m;
  };
  // a thread's units, TH apart, without a division for each
  const int step_i = TH / P.units, step_u = TH % P.units;
  const auto next = [&](int& i, int& u) {
    i += step_i;
    u += step_u;
    if (u >= P.units) u -= P.units, ++i;
  };
  uint4 raw[kHold ? kHold : 1][4];
  {
    int i = i0 + tid / P.units, u = tid % P.units;
    if constexpr (kHold > 0) {
#pragma unroll
      for (int j = 0; j < kHold; ++j, next(i, u)) {
        if (tid + j * TH >= work) break;
        const long long r = path ? path[i] : i;
        const UnitPlace w = unit_place<V>(u, P.rot, P.pairs);
        raw[j][0] = __ldcs(reinterpret_cast<const uint4*>(k + r * P.k_ld[1] + w.a));
        raw[j][1] = __ldcs(reinterpret_cast<const uint4*>(k + r * P.k_ld[1] + w.b));
        raw[j][2] = __ldcs(reinterpret_cast<const uint4*>(v + r * P.v_ld[1] + 2 * u * V));
        raw[j][3] = __ldcs(reinterpret_cast<const uint4*>(v + r * P.v_ld[1] + (2 * u + 1) * V));
      }
      // (all magnitudes first; infinities and NaN are set aside only where there are some)
      if constexpr (sizeof(T) == 2) {
        uint32_t m[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < kHold; ++j) {
          if (tid + j * TH >= work) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4& w = raw[j][e];
            const uint32_t s = 0x7fff7fffu;
            m[e >> 1] = __vmaxu2(m[e >> 1], __vmaxu2(__vmaxu2(w.x & s, w.y & s), __vmaxu2(w.z & s, w.w & s)));
          }
        }
        mk = __uint_as_float(max(m[0] & 0xffffu, m[0] >> 16) << 16);
        mv = __uint_as_float(max(m[1] & 0xffffu, m[1] >> 16) << 16);
      } else {
#pragma unroll
        for (int j = 0; j < kHold; ++j) {
          if (tid + j * TH >= work) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4& w = raw[j][e];
            float& m = e < 2 ? mk : mv;
            m = larger(larger(larger(m, __uint_as_float(w.x)), __uint_as_float(w.y)),
                       larger(__uint_as_float(w.z), __uint_as_float(w.w)));
          }
        }
        mk = fabsf(mk);
        mv = fabsf(mv);
      }
      if (!(mk < kInf) || !(mv < kInf)) {
        mk = mv = 0.f;
#pragma unroll
        for (int j = 0; j < kHold; ++j) {
          if (tid + j * TH >= work) break;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float x[V];
            load_elems<V>(reinterpret_cast<const T*>(&raw[j][half]), x);
            mk = most(mk, x);
            load_elems<V>(reinterpret_cast<const T*>(&raw[j][2 + half]), x);
            mv = most(mv, x);
          }
        }
      }
    } else {
      for (int o = tid; o < work; o += TH, next(i, u)) {
        const long long r = path ? path[i] : i;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[V];
          load_elems<V>(k + r * P.k_ld[1] + (2 * u + half) * V, x);
          mk = most(mk, x);
          load_elems<V>(v + r * P.v_ld[1] + (2 * u + half) * V, x);
          mv = most(mv, x);
        }
      }
    }
  }
  if (page < 0 || page >= P.pages) {
    if (h == 0 && tid == 0) {
      if (P.seq_error) atomicOr(P.seq_error + b, SPEC_ERR_CACHE);
      if (P.error_word) atomicOr(P.error_word, SPEC_ERR_CACHE);
    }
    return;
  }
  const long long slab = static_cast<long long>(page) * P.H + h;
  unsigned char* kc = P.k_codes + slab * P.page * P.D;
  unsigned char* vc = P.v_codes + slab * P.page * P.D;
  // (what is needed behind the barrier is on its way before it)
  const bool older = start < prefix;
  const int ok = older ? P.k_exps[slab] : kLowExp, ov = older ? P.v_exps[slab] : kLowExp;
  const auto turn = [&](int i, int u, long long r, float* cs, float* sn) {
    const int t = P.positions ? P.positions[static_cast<long long>(b) * P.n + r] : prefix + i;
    if (t >= 0 && t < P.table_rows) {
      const float* src = P.table + static_cast<long long>(t) * P.rot + u * V;
      load_elems<V>(src, cs);
      load_elems<V>(src + P.rot / 2, sn);
      return true;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) cs[e] = sn[e] = __uint_as_float(0x7fc00000u);
    return false;
  };
  float turn_c[V], turn_s[V];
  bool turn_inside = false;
  if constexpr (kHold == 1) {
    const int i = i0 + tid / P.units, u = tid % P.units;
    if (tid < work && unit_place<V>(u, P.rot, P.pairs).rotated)
      turn_inside = turn(i, u, path ? path[i] : i, turn_c, turn_s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
    mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
  }
  if ((tid & 31) == 0) most_s[0][tid >> 5] = mk, most_s[1][tid >> 5] = mv;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < TH / 32; ++w) mk = fmaxf(mk, most_s[0][w]), mv = fmaxf(mv, most_s[1][w]);
  int ek = exponent_of(mk), ev = exponent_of(mv);
  if (older) {
    ek = max(ek, ok);
    ev = max(ev, ov);
    const int bytes = (prefix - start) * P.D;
    if (ek > ok) scale_codes<TH>(kc, bytes, ek - ok);
    if (ev > ov) scale_codes<TH>(vc, bytes, ev - ov);
  }
  __syncthreads();
  if (tid == 0) {
    P.k_exps[slab] = static_cast<signed char>(ek);
    P.v_exps[slab] = static_cast<signed char>(ev);
  }

  // the codes
  const float fk = exp2i(-ek), fv = exp2i(-ev);
  bool bad = false, outside = false;
  const auto put = [&](int i, int u, long long r, const UnitPlace& w, float* a, float* c, const float* x, const float* y) {
    const long long at = static_cast<long long>(prefix + i - start) * P.D;
    if (w.rotated) {
      bool inside;
      float cs[V], sn[V];
      if constexpr (kHold == 1) {
        inside = turn_inside;
#pragma unroll
        for (int e = 0; e < V; ++e) cs[e] = turn_c[e], sn[e] = turn_s[e];
      } else {
        inside = turn(i, u, r, cs, sn);
      }
      outside |= !inside;
      rotate_unit<V>(a, c, cs, sn, P.pairs);
      bool hit = false;
      store_codes<V>(kc + at + w.a, a, fk, hit);
      store_codes<V>(kc + at + w.b, c, fk, hit);
      bad |= hit && inside;
    } else {
      store_codes<V>(kc + at + w.a, a, fk, bad);
      store_codes<V>(kc + at + w.b, c, fk, bad);
    }
    store_codes<V>(vc + at + 2 * u * V, x, fv, bad);
    store_codes<V>(vc + at + (2 * u + 1) * V, y, fv, bad);
  };
  int i = i0 + tid / P.units, u = tid % P.units;
  if constexpr (kHold > 0) {
#pragma unroll
    for (int j = 0; j < kHold; ++j, next(i, u)) {
      if (tid + j * TH >= work) break;
      float a[V], c[V], x[V], y[V];
      load_elems<V>(reinterpret_cast<const T*>(&raw[j][0]), a);
      load_elems<V>(reinterpret_cast<const T*>(&raw[j][1]), c);
      load_elems<V>(reinterpret_cast<const T*>(&raw[j][2]), x);
      load_elems<V>(reinterpret_cast<const T*>(&raw[j][3]), y);
      put(i, u, path ? path[i] : i, unit_place<V>(u, P.rot, P.pairs), a, c, x, y);
    }
  } else {
    for (int o = tid; o < work; o += TH, next(i, u)) {
      const long long r = path ? path[i] : i;
      const UnitPlace w = unit_place<V>(u, P.rot, P.pairs);
      float a[V], c[V], x[V], y[V];
      load_elems<V>(k + r * P.k_ld[1] + w.a, a);
      load_elems<V>(k + r * P.k_ld[1] + w.b, c);
      load_elems<V>(v + r * P.v_ld[1] + 2 * u * V, x);
      load_elems<V>(v + r * P.v_ld[1] + (2 * u + 1) * V, y);
      put(i, u, r, w, a, c, x, y);
    }
  }
  if (bad || outside) {
    const int err = (bad ? SPEC_ERR_NONFINITE : 0) | (outside ? SPEC_ERR_POSITION : 0);
    if (P.seq_error) atomicOr(P.seq_error + b, err);
    if (P.error_word) atomicOr(P.error_word, err);
  }
}

template <typename T, int V>
void launch_width(const AppendParams& p, dim3 grid, cudaStream_t s) {
  if constexpr (V * sizeof(T) == 16) {
    const int most = std::min(p.page, p.path_nodes ? p.path_ld : p.n) * p.units;  // a page's units, at most
    if (most <= 256) {
      append_kernel<T, V, 256, 1><<<grid, 256, 0, s>>>(p);
      return;
    }
    if (most <= 512) {
      append_kernel<T, V, 256, 2><<<grid, 256, 0, s>>>(p);
      return;
    }
    if (most <= 2048) {
      append_kernel<T, V, 512, 4><<<grid, 512, 0, s>>>(p);
      return;
    }
  }
  append_kernel<T, V, 256, 0><<<grid, 256, 0, s>>>(p);
}

template <typename T>
void launch_append(const AppendParams& p, int v, dim3 grid, cudaStream_t s) {
  if (v == 8) {
    if constexpr (sizeof(T) == 2) launch_width<T, 8>(p, grid, s);
  } else if (v == 4) {
    launch_width<T, 4>(p, grid, s);
  } else {
    launch_width<T, 1>(p, grid, s);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace sv

extern "C" spec_status spec_append_cache(const spec_append_args* a, cudaStream_t stream) {
  using namespace sv;
  NvtxRange nvtx_range("spec_append_cache");
  if (a == nullptr) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (a->B < 1 || a->B > 65535 || a->n < 1 || a->n > (1 << 20) || a->H < 1 || a->H > 1024 || a->D < 16 || a->D > 256 ||
      a->D % 16)
    return SPEC_EINVAL;
  if (a->page != 16 && a->page != 32 && a->page != 64 && a->page != 128) return SPEC_EINVAL;
  if (a->pages < 1 || static_cast<long long>(a->pages) * a->H * a->page > 0x7fffffffLL || a->table_pages < 1 ||
      static_cast<long long>(a->table_pages) * a->page > (1 << 30))
    return SPEC_EINVAL;
  if (a->rot < 0 || a->rot > a->D || a->rot % 2 || (a->rot && a->table_rows < 1)) return SPEC_EINVAL;
  if (!a->k || !a->v || !a->block_table || !a->k_codes || !a->v_codes || !a->k_exps || !a->v_exps ||
      (a->rot && !a->table))
    return SPEC_EINVAL;
  if ((a->path_nodes != nullptr) != (a->path_len != nullptr) || (a->path_nodes && a->count)) return SPEC_EINVAL;
  if (a->path_nodes && (a->max_depth < 0 || a->max_depth > 65534)) return SPEC_EINVAL;
  const int elem = a->dtype == SPEC_F32 ? 4 : 2;
  if (!aligned(a->k, elem) || !aligned(a->v, elem) || (a->rot && !aligned(a->table, 16)) || !aligned(a->k_codes, 16) ||
      !aligned(a->v_codes, 16))
    return SPEC_EALIGN;
  const int v = std::min(vector_width(elem, a->D, a->rot, a->k_ld, a->B, a->n, a->H, a->k),
                         vector_width(elem, a->D, a->rot, a->v_ld, a->B, a->n, a->H, a->v));
  AppendParams p{};
  p.n = a->n;
  p.H = a->H;
  p.D = a->D;
  p.page = a->page;
  p.pages = a->pages;
  p.table_pages = a->table_pages;
  p.rot = a->rot;
  p.units = a->D / (2 * v);
  p.table_rows = a->table_rows;
  p.path_ld = a->max_depth + 1;
  p.pairs = a->pairs != 0;
  for (int i = 0; i < 3; ++i) p.k_ld[i] = a->k_ld[i], p.v_ld[i] = a->v_ld[i];
  p.k = a->k;
  p.v = a->v;
  p.table = a->table;
  p.positions = a->positions;
  p.prefix = a->prefix_len;
  p.count = a->count;
  p.path_nodes = a->path_nodes;
  p.path_len = a->path_len;
  p.block_table = a->block_table;
  p.k_codes = static_cast<unsigned char*>(a->k_codes);
  p.v_codes = static_cast<unsigned char*>(a->v_codes);
  p.k_exps = a->k_exps;
  p.v_exps = a->v_exps;
  p.seq_error = a->seq_error;
  p.error_word = a->error_word;
  // the pages that so many rows can touch, wherever they start
  const int rows = a->path_nodes ? p.path_ld : a->n;
  const dim3 grid(static_cast<unsigned>((rows + a->page - 2) / a->page + 1), static_cast<unsigned>(a->H),
                  static_cast<unsigned>(a->B));
  if (a->dtype == SPEC_F32) launch_append<float>(p, v, grid, stream);
  else launch_append<bf16_t>(p, v, grid, stream);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}
