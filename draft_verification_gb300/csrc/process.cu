// Per-request processing of logits: penalties for repeated tokens, biases and
// grammar masks, each row with the tokens before its own position (chain or
// tree).  The arithmetic and the argument meanings are in spec_logits.h.
//
// process_kernel: a CTA owns one slab of the vocabulary of one sequence.  It
// first streams that slab of the sequence's rows: a masked copy, which needs
// nothing but the mask bits (a vector whose bits are all 0 is not read; in
// place without masks nothing is streamed at all).  Then it rewrites the few
// tokens that something applies to, read again from the input (through L2)
// with all lanes busy: handled inside the stream, a token in a hundred would
// put nearly every warp on the slow path.
//
// What applies is a table of the slab in shared memory - per token a 32-bit
// word (low 31 bits: occurrences that count, bit 31: occurs in the prompt) and
// the sum of its bias entries - built by reading the whole history once while
// the first rows are in flight, and two lists of tokens: those that only the
// history and the biases touch, which are the same for every row, so that all
// (token, row) pairs are rewritten in any order; and those that are drafted,
// whose counts depend on the row.  For the latter the rows go in order, and one
// thread takes the table from row to row (leaving one path and entering the
// next, up to their last common node) where a drafted token of the slab is
// concerned (rows marked beforehand, all in parallel).
//
// The stream goes in 16-byte vectors aligned in memory: a row that starts at
// element m of its vector has tokens [k e - m, k e - m + e) in vector k, so the
// table starts e - 1 tokens before the slab and mask bits are taken by funnel
// shifts.  Vectors that stick out of the row, and rows whose output starts at
// another offset than the input, are written element by element.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "spec_logits.h"

namespace sv {
namespace {

constexpr int kProcThreads = 256;
constexpr int kMaxRows = 1024;       // rows per sequence
constexpr unsigned kInPrompt = 1u << 31;
constexpr int kFill = 152 * 5;       // CTAs that fill the GPU (shared memory: 5 per SM with long slabs)

struct ProcessParams {
  int B, n, V;
  long long ld, out_ld;
  const void* logits;
  void* out;
  const int* tokens;
  const int* parent;
  int tokens_ld, history_ld;
  const int* history;
  const int* history_len;
  const int* prompt_len;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int* bias_tokens;
  const float* bias_values;
  const int* bias_len;
  int bias_ld, mask_rows;
  const unsigned* mask;
  long long mask_ld;
  const int* mask_index;
  int* seq_error;
  int* error_word;
  int rows_per_cta;
};

// 16 bytes of logits.  Not the read-only path: the output may be the input.
__device__ __forceinline__ uint4 ld_row16(const void* p) {
  if (kDebugChecks && misaligned16(p)) return make_uint4(0x7fc00000u, 0x7fc00000u, 0x7fc00000u, 0x7fc00000u);
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

template <typename T>
struct Lanes;  // the elements of a 16-byte vector

template <>
struct Lanes<bf16_t> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ uint32_t bits(const uint32_t (&w)[4], int j) {
    return (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
  }
  static __device__ __forceinline__ void set_bits(uint32_t (&w)[4], int j, uint32_t b) {
    w[j >> 1] = (j & 1) ? (w[j >> 1] & 0xffffu) | (b << 16) : (w[j >> 1] & 0xffff0000u) | b;
  }
  static __device__ __forceinline__ uint32_t round(float x) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
    return r;
  }
  static __device__ __forceinline__ float widen(uint32_t b) { return __uint_as_float(b << 16); }
  static constexpr uint32_t kNegInf = 0xff80u;
  static constexpr uint32_t kNegInf4 = 0xff80ff80u;
};

template <>
struct Lanes<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ uint32_t bits(const uint32_t (&w)[4], int j) { return w[j]; }
  static __device__ __forceinline__ void set_bits(uint32_t (&w)[4], int j, uint32_t b) { w[j] = b; }
  static __device__ __forceinline__ uint32_t round(float x) { return __float_as_uint(x); }
  static __device__ __forceinline__ float widen(uint32_t b) { return __uint_as_float(b); }
  static constexpr uint32_t kNegInf = 0xff800000u;
  static constexpr uint32_t kNegInf4 = 0xff800000u;
};

template <typename T>
__device__ __forceinline__ uint32_t load_bits(const T* p) {
  if constexpr (sizeof(T) == 2) {
    return *reinterpret_cast<const volatile unsigned short*>(p);
  } else {
    return *reinterpret_cast<const volatile unsigned*>(p);
  }
}
template <typename T>
__device__ __forceinline__ void store_bits(T* p, uint32_t b) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(b);
  } else {
    *reinterpret_cast<unsigned*>(p) = b;
  }
}

// table entries: the slab and the e - 1 tokens before it
__host__ __device__ constexpr int table_tokens(int elems, int vecs) { return kProcThreads * vecs * elems + elems - 1; }
__host__ __device__ constexpr int bitmap_words(int elems, int vecs) { return (table_tokens(elems, vecs) + 31) / 32; }

template <typename T, int kVecs>
__global__ void __launch_bounds__(kProcThreads) process_kernel(const ProcessParams P) {
  using L = Lanes<T>;
  constexpr int E = L::kN;
  constexpr uint32_t kFull = (1u << E) - 1u;
  constexpr int kSlab = kProcThreads * kVecs * E;
  constexpr int kTable = table_tokens(E, kVecs);
  constexpr int kWords = bitmap_words(E, kVecs);

  extern __shared__ unsigned proc_dyn[];
  unsigned* count = proc_dyn;                         // [kTable]
  unsigned* drafted = count + kTable;                 // [kWords] tokens that some row's path may hold
  unsigned* listed = drafted + kWords;                // [kWords] tokens in either list
  unsigned* change = listed + kWords;                 // [kMaxRows / 32] rows before which the table changes
  int* s_tok = reinterpret_cast<int*>(change + kMaxRows / 32);  // [n]
  int* s_par = s_tok + P.n;                           // [n]
  int* s_mask = s_par + P.n;                          // [n]
  float* bias = reinterpret_cast<float*>(s_mask + P.n);  // [kTable], with biases
  // the lists grow towards each other: fixed tokens from the front, drafted ones from the back
  unsigned short* list = reinterpret_cast<unsigned short*>(bias + (P.bias_tokens ? kTable : 0));  // [kTable]
  __shared__ int s_err, s_fixed, s_drafted;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.z;
  const int r0 = blockIdx.y * P.rows_per_cta;
  const int r1 = min(P.n, r0 + P.rows_per_cta);
  const int v0 = blockIdx.x * (kProcThreads * kVecs);  // first vector of the slab
  const int lo = v0 * E - (E - 1);                     // first token of the table
  const bool checks = blockIdx.x == 0 && blockIdx.y == 0;
  const bool tree = P.parent != nullptr;
  const bool biased = P.bias_tokens != nullptr;
  const bool stream = P.mask != nullptr || P.logits != P.out;

  const auto mask_row = [&](int i) {
    if (!P.mask) return -1;
    const long long row = static_cast<long long>(b) * P.n + i;
    const long long mr = P.mask_index ? static_cast<long long>(__ldg(P.mask_index + row)) : row;
    return mr < P.mask_rows ? static_cast<int>(mr) : -1;
  };
  const auto lead_of = [&](int i) {  // element of its first vector at which row i starts
    return static_cast<int>(((static_cast<long long>(b) * P.n + i) * P.ld) % E);
  };
  // the mask bits of row i's vectors (mrow < 0: not masked; 0 for vectors outside the row)
  const auto load_mask = [&](int i, int mrow, uint32_t (&ok)[kVecs]) {
    const int m = lead_of(i);
    const unsigned* mk = mrow >= 0 ? P.mask + static_cast<long long>(mrow) * P.mask_ld : nullptr;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int t0 = (v0 + j * kProcThreads + tid) * E - m;
      ok[j] = t0 < P.V ? kFull : 0u;
      if (mk && t0 < P.V) {
        if (t0 < 0) {
          ok[j] = (__ldg(mk) << -t0) & kFull;
        } else {
          const int q = t0 >> 5, s = t0 & 31;
          const unsigned a = __ldg(mk + q);
          const unsigned c = (s + E > 32 && (q + 1) * 32 < P.V) ? __ldg(mk + q + 1) : 0u;
          ok[j] = __funnelshift_r(a, c, s) & kFull;
        }
      }
    }
  };
  // row i's vectors that have an allowed token
  const auto load_row = [&](int i, const uint32_t (&ok)[kVecs], uint32_t (&w)[kVecs][4]) {
    const T* src = static_cast<const T*>(P.logits) + (static_cast<long long>(b) * P.n + i) * P.ld;
    const int m = lead_of(i);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int t0 = (v0 + j * kProcThreads + tid) * E - m;
      if (!ok[j]) continue;
      if (t0 >= 0 && t0 + E <= P.V) {
        const uint4 x = ld_row16(src + t0);
        w[j][0] = x.x;
        w[j][1] = x.y;
        w[j][2] = x.z;
        w[j][3] = x.w;
      } else {
        w[j][0] = w[j][1] = w[j][2] = w[j][3] = 0u;
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (t0 + k >= 0 && t0 + k < P.V) L::set_bits(w[j], k, load_bits(src + t0 + k));
      }
    }
  };
  const auto store_row = [&](int i, const uint32_t (&ok)[kVecs], uint32_t (&w)[kVecs][4]) {
    const long long row = static_cast<long long>(b) * P.n + i;
    T* dst = static_cast<T*>(P.out) + row * P.out_ld;
    const int m = lead_of(i);
    const bool same = static_cast<int>((row * P.out_ld) % E) == m;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int t0 = (v0 + j * kProcThreads + tid) * E - m;
      if (t0 >= P.V) continue;
      if (!ok[j]) {
        w[j][0] = w[j][1] = w[j][2] = w[j][3] = L::kNegInf4;
      } else if (ok[j] != kFull) {
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (!((ok[j] >> k) & 1u)) L::set_bits(w[j], k, L::kNegInf);
      }
      if (same && t0 >= 0 && t0 + E <= P.V) {
        if (!(kDebugChecks && misaligned16(dst + t0)))
          *reinterpret_cast<uint4*>(dst + t0) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (t0 + k >= 0 && t0 + k < P.V) store_bits(dst + t0 + k, L::bits(w[j], k));
      }
    }
  };

  // The first row's vectors are in flight while the table is built, the
  // second row's mask bits as well: the stream always reads the vectors of one
  // row and the mask bits of the next ahead.
  uint32_t cur[kVecs][4], nxt[kVecs][4], ok0[kVecs], ok1[kVecs], ok2[kVecs];
  if (stream) {
    load_mask(r0, mask_row(r0), ok0);
    if (r0 + 1 < r1) load_mask(r0 + 1, mask_row(r0 + 1), ok1);
    load_row(r0, ok0, cur);
  }

  for (int i = tid; i < kTable; i += kProcThreads) count[i] = 0u;
  for (int i = tid; i < kWords; i += kProcThreads) drafted[i] = listed[i] = 0u;
  for (int i = tid; i < kMaxRows / 32; i += kProcThreads) change[i] = 0u;
  if (biased)
    for (int i = tid; i < kTable; i += kProcThreads) bias[i] = 0.f;
  if (tid == 0) s_err = s_fixed = s_drafted = 0;
  __syncthreads();

  int err = 0;
  const auto in_slab = [&](int t) { return t >= 0 && static_cast<unsigned>(t - lo) < static_cast<unsigned>(kTable); };

  // the drafted tokens, the tree and the mask rows
  for (int i = tid; i < P.n; i += kProcThreads) {
    int t = -1, p = 0;
    if (P.tokens && i < P.tokens_ld) t = __ldg(P.tokens + static_cast<long long>(b) * P.tokens_ld + i);
    const bool used = tree ? i > 0 : (P.tokens && i < P.n - 1);
    if (used && (t < 0 || t >= P.V)) {
      err |= SPEC_ERR_TOKEN;
      t = -1;
    }
    if (tree && i > 0) {
      p = __ldg(P.parent + static_cast<long long>(b) * P.n + i);
      if (p < 0 || p >= i) {
        err |= SPEC_ERR_PARENT;
        p = 0;
      }
    }
    if (!used) t = -1;
    s_tok[i] = t;
    s_par[i] = p;
    s_mask[i] = mask_row(i);
    if (in_slab(t)) {
      const int at = t - lo;
      if (!((atomicOr(&drafted[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1u))
        list[kTable - 1 - atomicAdd(&s_drafted, 1)] = static_cast<unsigned short>(at);
    }
    if (P.mask && P.mask_index) {
      const int mi = __ldg(P.mask_index + static_cast<long long>(b) * P.n + i);
      if (mi < -1 || mi >= P.mask_rows) err |= SPEC_ERR_MASK;
    }
  }
  __syncthreads();

  // a token that the history or a bias touches: into the list of fixed tokens unless it is drafted
  const auto touch = [&](unsigned at) {
    const unsigned bit = 1u << (at & 31);
    if (!((drafted[at >> 5] | listed[at >> 5]) & bit) && !(atomicOr(&listed[at >> 5], bit) & bit))
      list[atomicAdd(&s_fixed, 1)] = static_cast<unsigned short>(at);
  };
  // the history
  if (P.history) {
    int len = P.history_len ? __ldg(P.history_len + b) : P.history_ld;
    if (len < 0 || len > P.history_ld) {
      err |= SPEC_ERR_TOKEN;
      len = len < 0 ? 0 : P.history_ld;
    }
    const int prompt = P.prompt_len ? __ldg(P.prompt_len + b) : 0;
    const int* h = P.history + static_cast<long long>(b) * P.history_ld;
    const auto take = [&](int t, int at) {
      if (at >= len) return;
      if (t < 0 || t >= P.V) {
        err |= SPEC_ERR_TOKEN;
        return;
      }
      const unsigned o = static_cast<unsigned>(t - lo);
      if (o < static_cast<unsigned>(kTable)) {
        if (at < prompt) atomicOr(&count[o], kInPrompt);
        else atomicAdd(&count[o], 1u);
        touch(o);
      }
    };
    // a thread's loads go out together: 8192 tokens per round where rows allow 16-byte loads
    constexpr int kU = 8;
    if (P.history_ld % 4 == 0 && !misaligned16(P.history)) {
      for (int base = 4 * tid; base < len; base += 4 * kProcThreads * kU) {
        int4 t[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int at = base + 4 * k * kProcThreads;
          if (at < len) t[k] = __ldg(reinterpret_cast<const int4*>(h + at));
        }
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int at = base + 4 * k * kProcThreads;
          if (at >= len) break;
          take(t[k].x, at);
          take(t[k].y, at + 1);
          take(t[k].z, at + 2);
          take(t[k].w, at + 3);
        }
      }
    } else {
      for (int base = tid; base < len; base += kProcThreads * kU) {
        int t[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int at = base + k * kProcThreads;
          if (at < len) t[k] = __ldg(h + at);
        }
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int at = base + k * kProcThreads;
          if (at >= len) break;
          take(t[k], at);
        }
      }
    }
  }

  // the biases, one warp, in their order (entries of one token add up as listed)
  if (biased && warp == 0) {
    int len = P.bias_len ? __ldg(P.bias_len + b) : P.bias_ld;
    if (len < 0 || len > P.bias_ld) {
      err |= SPEC_ERR_TOKEN;
      len = len < 0 ? 0 : P.bias_ld;
    }
    constexpr int kAhead = 4;  // 32 entries a step, the loads of four steps at once
    int ts[kAhead];
    float xs[kAhead];
    for (int base = 0; base < len; base += 32) {
      const int step = base / 32 % kAhead;
      if (step == 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int at = base + 32 * k + lane;
          const long long src = static_cast<long long>(b) * P.bias_ld + at;
          ts[k] = at < len ? __ldg(P.bias_tokens + src) : -1;
          xs[k] = at < len ? __ldg(P.bias_values + src) : 0.f;
        }
      }
      int t = ts[0];
      float x = xs[0];
#pragma unroll
      for (int k = 1; k < kAhead; ++k) {
        t = step == k ? ts[k] : t;
        x = step == k ? xs[k] : x;
      }
      if (base + lane < len && (t < 0 || t >= P.V)) {
        err |= SPEC_ERR_TOKEN;
        t = -1;
      }
      const unsigned o = static_cast<unsigned>(t - lo);
      const bool mine = t >= 0 && o < static_cast<unsigned>(kTable);
      const unsigned peers = __match_any_sync(0xffffffffu, mine ? static_cast<int>(o) : -1 - lane);
      const bool alone = !mine || (peers & (peers - 1)) == 0;
      if (__all_sync(0xffffffffu, alone)) {
        if (mine) bias[o] += x;
      } else {
        for (int l = 0; l < 32; ++l) {
          if (l == lane && mine) bias[o] += x;
          __syncwarp();
        }
      }
      if (mine) touch(o);
      __syncwarp();
    }
  }
  if (checks && err) atomicOr(&s_err, err);

  // the stream
  if (stream) {
    for (int i = r0; i < r1; ++i) {
      if (i + 1 < r1) load_row(i + 1, ok1, nxt);
      if (i + 2 < r1) load_mask(i + 2, s_mask[i + 2], ok2);
      store_row(i, ok0, cur);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) cur[j][k] = nxt[j][k];
        ok0[j] = ok1[j];
        ok1[j] = ok2[j];
      }
    }
  }
  __syncthreads();
  if (checks && tid == 0) {
    if (P.seq_error) P.seq_error[b] = s_err;
    if (s_err && P.error_word) atomicOr(P.error_word, s_err);
  }

  const float rep = P.repetition ? __ldg(P.repetition + b) : 1.f;
  const float inv = __frcp_rn(rep);
  const float freq = P.frequency ? __ldg(P.frequency + b) : 0.f;
  const float pres = P.presence ? __ldg(P.presence + b) : 0.f;
  // Whether this CTA writes table entry `at` in row i: rows that start within
  // a vector shift the slab's tokens, and the mask must allow the token.
  const auto writes = [&](int i, int at) {
    const int v = lo + at;
    const int t = v + lead_of(i) - v0 * E;
    if (v < 0 || v >= P.V || t < 0 || t >= kSlab) return false;
    const int mrow = s_mask[i];
    return mrow < 0 || ((__ldg(P.mask + static_cast<long long>(mrow) * P.mask_ld + (v >> 5)) >> (v & 31)) & 1u);
  };
  const auto value = [&](int i, int at) {
    return static_cast<const T*>(P.logits) + (static_cast<long long>(b) * P.n + i) * P.ld + (lo + at);
  };
  const auto rewrite = [&](int i, int at, uint32_t bits) {
    const unsigned c = count[at];
    float x = L::widen(bits);
    if (c) x = __fmul_rn(x, x > 0.f ? inv : rep);
    const unsigned made = c & ~kInPrompt;
    if (made) x = __fsub_rn(x, __fmaf_rn(freq, static_cast<float>(made), pres));
    const float plus = biased ? bias[at] : 0.f;
    if (plus != 0.f) x = __fadd_rn(x, plus);
    if (c || plus != 0.f)
      store_bits(static_cast<T*>(P.out) + (static_cast<long long>(b) * P.n + i) * P.out_ld + (lo + at), L::round(x));
  };

  // tokens that are the same for every row: all (token, row) pairs, four in flight per thread
  const int fixed = s_fixed;
  const int pairs = fixed * (r1 - r0);
  constexpr int kU = 4;
  for (int base = tid; base < pairs; base += kProcThreads * kU) {
    int row[kU], at[kU];
    uint32_t x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int p = base + u * kProcThreads;
      at[u] = -1;
      if (p < pairs) {
        const int i = p / fixed;
        row[u] = r0 + i;
        at[u] = list[p - i * fixed];
        if (!writes(row[u], at[u])) at[u] = -1;
      }
      if (at[u] >= 0) x[u] = load_bits(value(row[u], at[u]));
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (at[u] >= 0) rewrite(row[u], at[u], x[u]);
  }

  // drafted tokens: row by row
  const int moving = s_drafted;
  if (moving == 0) return;
  if (!tree) {
    for (int j = tid; j < r0; j += kProcThreads)
      if (in_slab(s_tok[j])) atomicAdd(&count[s_tok[j] - lo], 1u);
    for (int i = r0 + 1 + tid; i < r1; i += kProcThreads)
      if (in_slab(s_tok[i - 1])) atomicOr(&change[i >> 5], 1u << (i & 31));
  } else {
    if (tid == 0)
      for (int a = r0; a > 0; a = s_par[a])
        if (in_slab(s_tok[a])) count[s_tok[a] - lo] += 1u;
    for (int i = r0 + 1 + tid; i < r1; i += kProcThreads) {
      int x = i - 1, y = i;
      bool any = false;
      while (x != y && !any) {
        any = in_slab(s_tok[x > y ? x : y]);
        if (x > y) x = s_par[x];
        else y = s_par[y];
      }
      if (any) atomicOr(&change[i >> 5], 1u << (i & 31));
    }
  }
  __syncthreads();
  for (int i = r0; i < r1; ++i) {
    if (i > r0 && (change[i >> 5] >> (i & 31)) & 1u) {
      __syncthreads();  // everyone is done with the previous row's counts
      if (tid == 0) {
        const auto add = [&](int t, unsigned d) {
          if (in_slab(t)) count[t - lo] += d;
        };
        if (!tree) {
          add(s_tok[i - 1], 1u);
        } else {
          int x = i - 1, y = i;  // leave x's path, enter y's, up to their last common node
          while (x != y) {
            if (x > y) {
              add(s_tok[x], ~0u);
              x = s_par[x];
            } else {
              add(s_tok[y], 1u);
              y = s_par[y];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int e = tid; e < moving; e += kProcThreads) {
      const int at = list[kTable - 1 - e];
      if (writes(i, at)) rewrite(i, at, load_bits(value(i, at)));
    }
  }
}

template <typename T, int kVecs>
size_t process_smem(const ProcessParams& p) {
  constexpr int E = Lanes<T>::kN;
  constexpr size_t table = table_tokens(E, kVecs);
  size_t words = table + 2 * bitmap_words(E, kVecs) + kMaxRows / 32 + 3 * static_cast<size_t>(p.n);
  if (p.bias_tokens) words += table;
  return words * 4 + (table + 1) / 2 * 4;
}

int slabs_of(const ProcessParams& p, int elems, int vecs) {
  // vectors of the longest row: a row may start anywhere in its first vector
  const int lead = p.ld % elems ? elems - 1 : 0;
  const int nvec = (p.V + lead + elems - 1) / elems;
  return (nvec + kProcThreads * vecs - 1) / (kProcThreads * vecs);
}

template <typename T, int kVecs>
cudaError_t launch_process(ProcessParams p, cudaStream_t s) {
  const size_t dyn = process_smem<T, kVecs>(p);
  cudaError_t e = cudaFuncSetAttribute(process_kernel<T, kVecs>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(dyn));
  if (e != cudaSuccess) return e;
  const int slabs = slabs_of(p, Lanes<T>::kN, kVecs);
  // few sequences and slabs: a sequence's rows are split as well (each part
  // reads the history again)
  const long long have = static_cast<long long>(slabs) * p.B;
  const long long parts = (kFill + have - 1) / have;
  const int chunks = static_cast<int>(parts < p.n ? parts : p.n);
  p.rows_per_cta = (p.n + chunks - 1) / chunks;
  const dim3 grid(static_cast<unsigned>(slabs), static_cast<unsigned>((p.n + p.rows_per_cta - 1) / p.rows_per_cta),
                  static_cast<unsigned>(p.B));
  process_kernel<T, kVecs><<<grid, kProcThreads, dyn, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch_process(const ProcessParams& p, cudaStream_t s) {
  // long slabs read the history fewer times; short ones fill the GPU
  if (static_cast<long long>(slabs_of(p, Lanes<T>::kN, 2)) * p.B * p.n >= kFill) return launch_process<T, 2>(p, s);
  return launch_process<T, 1>(p, s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace sv

extern "C" spec_status spec_process_logits(const spec_process_args* a, cudaStream_t stream) {
  using namespace sv;
  NvtxRange nvtx_range("spec_process_logits");
  if (a == nullptr) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (a->B < 1 || a->B > kMaxSeq || a->n < 1 || a->n > kMaxRows || a->V < 1 || a->V > 2097152) return SPEC_EINVAL;
  if (a->ld < a->V || a->out_ld < a->V || !a->logits || !a->out) return SPEC_EINVAL;
  if (a->logits == a->out && a->ld != a->out_ld) return SPEC_EINVAL;
  if (a->parent && !a->tokens) return SPEC_EINVAL;
  if (a->tokens && a->tokens_ld < (a->parent ? a->n : a->n - 1)) return SPEC_EINVAL;
  if (a->history && a->history_ld < 0) return SPEC_EINVAL;
  if (a->bias_tokens && (!a->bias_values || a->bias_ld < 0)) return SPEC_EINVAL;
  if (a->mask && (a->mask_rows < 1 || a->mask_ld < (a->V + 31) / 32)) return SPEC_EINVAL;
  if (a->mask && !a->mask_index && a->mask_rows < static_cast<long long>(a->B) * a->n) return SPEC_EINVAL;
  if (!aligned16(a->logits) || !aligned16(a->out)) return SPEC_EALIGN;
  ProcessParams p{};
  p.B = a->B;
  p.n = a->n;
  p.V = a->V;
  p.ld = a->ld;
  p.out_ld = a->out_ld;
  p.logits = a->logits;
  p.out = a->out;
  p.tokens = a->tokens;
  p.parent = a->parent;
  p.tokens_ld = a->tokens_ld;
  p.history = a->history_ld > 0 ? a->history : nullptr;
  p.history_ld = a->history_ld;
  p.history_len = a->history_len;
  p.prompt_len = a->prompt_len;
  p.repetition = a->repetition;
  p.frequency = a->frequency;
  p.presence = a->presence;
  p.bias_tokens = a->bias_ld > 0 ? a->bias_tokens : nullptr;
  p.bias_values = a->bias_values;
  p.bias_len = a->bias_len;
  p.bias_ld = a->bias_ld;
  p.mask = a->mask;
  p.mask_rows = a->mask_rows;
  p.mask_ld = a->mask_ld;
  p.mask_index = a->mask_index;
  p.seq_error = a->seq_error;
  p.error_word = a->error_word;
  const cudaError_t e =
      a->dtype == SPEC_BF16 ? dispatch_process<bf16_t>(p, stream) : dispatch_process<float>(p, stream);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}
