// Rotary positions (spec_rotation_table, spec_rotate_heads).
//
// spec_rotate_heads is bound by memory: it reads and writes every element
// once.  A thread takes one unit (heads.cuh) of kHeads heads of one row, so
// the row's cosines and sines are loaded once for them, and has two loads per
// head in flight.  2 x 4095 rows of 20 heads of 96, fp32: 23 us, 5.55 TB/s, 0.83
// of a copy's rate.  One row takes 2.5 us in a graph; a call from the host costs
// more (6 us).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "heads.cuh"
#include "internal.h"
#include "spec_cache.h"

namespace sv {
namespace {

constexpr int kRotateThreads = 128;
constexpr int kHeads = 4;

__global__ void __launch_bounds__(256)
    table_kernel(int rows, int half, const double* freq, double magnitude, float* table) {
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= static_cast<long long>(rows) * half) return;
  const long long t = at / half;
  const int i = static_cast<int>(at % half);
  double s, c;
  sincos(static_cast<double>(t) * freq[i], &s, &c);
  float* row = table + t * (2 * half);
  row[i] = static_cast<float>(c * magnitude);
  row[half + i] = static_cast<float>(s * magnitude);
}

struct RotateParams {
  unsigned n, units;
  int H, D, rot, groups, table_rows;  // groups of kHeads heads
  long long rows;                               // B * n
  bool pairs, transpose;
  long long x_ld[3], out_ld[3];
  const void* x;
  void* out;
  const float* table;
  const int* positions;
  const int* prefix;
  int* seq_error;
  int* error_word;
};

template <typename T, int V>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(const RotateParams P) {
  const long long at = static_cast<long long>(blockIdx.x) * kRotateThreads + threadIdx.x;
  const long long per_row = static_cast<long long>(P.units) * P.groups;
  // (divisions of 64 bits would take as long as the rest)
  const bool few = P.rows * per_row <= 0xffffffffLL;
  const long long row = few ? static_cast<unsigned>(at) / static_cast<unsigned>(per_row) : at / per_row;
  if (row >= P.rows) return;
  const unsigned rest = static_cast<unsigned>(at - row * per_row);
  const int u = static_cast<int>(rest % P.units), h0 = static_cast<int>(rest / P.units) * kHeads;
  const int b = few ? static_cast<int>(static_cast<unsigned>(row) / P.n) : static_cast<int>(row / P.n);
  const int i = static_cast<int>(row - static_cast<long long>(b) * P.n);
  const UnitPlace w = unit_place<V>(u, P.rot, P.pairs);
  float cs[V], sn[V];
  if (w.rotated) {
    const long long t = P.positions ? static_cast<long long>(P.positions[row])
                                    : static_cast<long long>(P.prefix ? P.prefix[b] : 0) + i;
    if (t >= 0 && t < P.table_rows) {
      const float* src = P.table + t * P.rot + u * V;
      load_elems<V>(src, cs);
      load_elems<V>(src + P.rot / 2, sn);
#pragma unroll
      for (int e = 0; e < V; ++e) sn[e] = P.transpose ? -sn[e] : sn[e];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) cs[e] = sn[e] = __uint_as_float(0x7fc00000u);
      if (u == 0 && h0 == 0) {
        if (P.seq_error) atomicOr(P.seq_error + b, SPEC_ERR_POSITION);
        if (P.error_word) atomicOr(P.error_word, SPEC_ERR_POSITION);
      }
    }
  }
  const T* x = static_cast<const T*>(P.x) + b * P.x_ld[0] + i * P.x_ld[1] + h0 * P.x_ld[2];
  T* y = static_cast<T*>(P.out) + b * P.out_ld[0] + i * P.out_ld[1] + h0 * P.out_ld[2];
  float a[kHeads][V], c[kHeads][V];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    if (h0 + k < P.H) {
      load_elems<V>(x + k * P.x_ld[2] + w.a, a[k]);
      load_elems<V>(x + k * P.x_ld[2] + w.b, c[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    if (h0 + k < P.H) {
      if (w.rotated) rotate_unit<V>(a[k], c[k], cs, sn, P.pairs);
      store_elems<V>(y + k * P.out_ld[2] + w.a, a[k]);
      store_elems<V>(y + k * P.out_ld[2] + w.b, c[k]);
    }
  }
}

template <typename T>
void launch_rotate(const RotateParams& p, int v, unsigned blocks, cudaStream_t s) {
  if (v == 8) {
    if constexpr (sizeof(T) == 2) rotate_kernel<T, 8><<<blocks, kRotateThreads, 0, s>>>(p);
  } else if (v == 4) {
    rotate_kernel<T, 4><<<blocks, kRotateThreads, 0, s>>>(p);
  } else {
    rotate_kernel<T, 1><<<blocks, kRotateThreads, 0, s>>>(p);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace sv

extern "C" spec_status spec_rotation_table(int rows, int rot, const double* freq, double magnitude, float* table,
                                           cudaStream_t stream) {
  using namespace sv;
  NvtxRange nvtx_range("spec_rotation_table");
  if (rows < 1 || rows > (1 << 30) || rot < 2 || rot > 1024 || rot % 2 || !freq || !table || !std::isfinite(magnitude))
    return SPEC_EINVAL;
  if (!aligned(freq, 8) || !aligned(table, 4)) return SPEC_EALIGN;
  const long long blocks = (static_cast<long long>(rows) * (rot / 2) + 255) / 256;
  if (blocks > 0x7fffffffLL) return SPEC_EINVAL;
  table_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(rows, rot / 2, freq, magnitude, table);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

extern "C" spec_status spec_rotate_heads(const spec_rotate_args* a, cudaStream_t stream) {
  using namespace sv;
  NvtxRange nvtx_range("spec_rotate_heads");
  if (a == nullptr) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (a->B < 1 || a->B > 65535 || a->n < 1 || a->n > (1 << 20) || a->H < 1 || a->H > 1024 || a->D < 2 || a->D > 1024 || a->D % 2 ||
      a->rot < 2 || a->rot > a->D || a->rot % 2 || a->table_rows < 1)
    return SPEC_EINVAL;
  if (!a->x || !a->out || !a->table) return SPEC_EINVAL;
  const bool same_ld = a->x_ld[0] == a->out_ld[0] && a->x_ld[1] == a->out_ld[1] && a->x_ld[2] == a->out_ld[2];
  if (a->x == a->out && !same_ld) return SPEC_EINVAL;
  const int elem = a->dtype == SPEC_F32 ? 4 : 2;
  if (!aligned(a->x, elem) || !aligned(a->out, elem) || !aligned(a->table, 16)) return SPEC_EALIGN;
  const int v = std::min(vector_width(elem, a->D, a->rot, a->x_ld, a->B, a->n, a->H, a->x),
                   vector_width(elem, a->D, a->rot, a->out_ld, a->B, a->n, a->H, a->out));
  RotateParams p{};
  p.n = a->n;
  p.H = a->H;
  p.D = a->D;
  p.rot = a->rot;
  p.pairs = a->pairs != 0;
  p.transpose = a->transpose != 0;
  p.table_rows = a->table_rows;
  p.rows = static_cast<long long>(a->B) * a->n;
  for (int i = 0; i < 3; ++i) p.x_ld[i] = a->x_ld[i], p.out_ld[i] = a->out_ld[i];
  p.x = a->x;
  p.out = a->out;
  p.table = a->table;
  p.positions = a->positions;
  p.prefix = a->prefix_len;
  p.seq_error = a->seq_error;
  p.error_word = a->error_word;
  p.units = a->D / (2 * v);
  p.groups = (a->H + kHeads - 1) / kHeads;
  const long long blocks = (p.rows * p.units * p.groups + kRotateThreads - 1) / kRotateThreads;
  if (blocks > 0x7fffffffLL) return SPEC_EINVAL;
  if (a->dtype == SPEC_F32) launch_rotate<float>(p, v, static_cast<unsigned>(blocks), stream);
  else launch_rotate<bf16_t>(p, v, static_cast<unsigned>(blocks), stream);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}
