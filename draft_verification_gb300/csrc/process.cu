// Per-request processing of logits: penalties for repeated tokens, biases and
// grammar masks, each row with the tokens before its own position (chain or
// tree).  The arithmetic and the argument meanings are in spec_logits.h.
//
// A CTA owns one slab of the vocabulary of one sequence.  Row by row its part
// goes through shared memory: 16-byte vectors are read (those whose mask bits
// are all 0 are not), masked elements become -inf, the few tokens that anything
// else applies to are rewritten in shared memory with all lanes busy, and the
// vectors are written.  Rewritten in the registers of the stream, a token in a
// hundred would put nearly every warp on the slow path; rewritten in global
// memory afterwards, two-byte accesses a sector apart run at 25 to 50 per
// nanosecond on the whole GPU, which was slower than the stream itself.
//
// What applies to a token is an entry: a 32-bit word (low bits: occurrences
// that count; bit 31: occurs in the prompt; bit 30: drafted, its occurrences on
// the way to a row are counted for each row; bit 29: has a bias) and the sum of
// its bias entries.
//  - Most calls build a slab's entries in the same kernel, as a table of the
//    slab in shared memory, from the whole history, which is read while the
//    first row's vectors are in flight.
//  - Where that would have every SM read histories again and again (long ones of
//    many sequences over a large vocabulary), collect_kernel gathers each
//    sequence's distinct tokens once and writes their entries in ascending
//    order to the workspace; the slabs' CTAs (launched dependent: their first
//    vectors are in flight meanwhile) read a few hundred entries each.
// run_process has the rule and what it measured.
//
// What bounds it: HBM, which has to read every vector with an allowed token and
// write every element; where tokens are few, what precedes a CTA's first row.
//  - 128 sequences of 9 rows of 128256 bfloat16 logits with grammar masks and
//    histories of up to 8192 tokens: 109 us, of which collecting takes 15 and the
//    rows 97.  All bytes are 613 MB, 90.5 us at the measured 6.8 TB/s; the masks
//    leave a third of the vectors to read, 411 MB, and the kernel reads no others.
//    That gains little (without masks 118 us), because writing is the slower half:
//    a fill of the output alone takes 76 us, 3.9 TB/s, a copy of a third of it and
//    a fill of the rest 87.
//  - 16 trees of 64 nodes over 50257 tokens, whose rows start anywhere (212 MB, 31
//    us; 141 MB as the masks leave it; a fill of the output 29): 53 us, without
//    masks 59, over 50264 tokens 46.  DRAM is at 22 %, 45 % of the warps are
//    active: latency between the barriers.
//  - One row: 7 us, the launch.  One sequence of 9 rows with 131,072 tokens: 112 us,
//    the history.
//  - float32: the same 109 us for half as many sequences.  In place with masks the
//    same; without masks 97 us for the first.

// Vectors are aligned in memory: a row that starts at element m of its vector
// has tokens [k e - m, k e - m + e) in vector k, so a row's part is the slab
// shifted by m (entries of the slab before may belong to it), and mask bits are
// taken by funnel shifts.  Vectors that stick out of the row, and rows whose
// output starts at another offset than the input, are read or written element
// by element.
//
// In place and without masks only the touched elements are read and written.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "spec_logits.h"
#include "tma_host.h"

namespace sv {
namespace {

constexpr int kMaxRows = 1024;       // rows per sequence
// entries of a history or a bias list: with the rows' tokens their occurrences
// stay below a word's flags, and the loops' positions below 2^31
constexpr int kMaxList = 1 << 28;
// bits of a token's word; the low ones count its occurrences
constexpr unsigned kInPrompt = 1u << 31, kDrafted = 1u << 30, kBiased = 1u << 29;
constexpr unsigned kMade = kBiased - 1u;
static_assert(static_cast<unsigned>(kMaxList) + kMaxRows <= kMade, "the occurrences fit their bits");

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
  int window;          // collecting: entries gathered at a time
  int slab_tokens;     // collecting: tokens of a slab
  int slabs;
  int capacity;        // entries of a sequence in the workspace
  int* offsets;        // workspace [B][slabs + 1]: where each slab's entries start
  int* entry_token;    // workspace [B][capacity]
  unsigned* entry_count;
  float* entry_bias;
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
  // Elements whose bit of ok is 0 become -inf.  Four bits are spread to the
  // sign bits of four bytes by a product (their partial products do not meet),
  // and a byte permutation makes a mask of each sign: 11 operations for eight
  // elements, where a test and a selection of each took three times as many.
  static __device__ __forceinline__ void only(uint32_t (&w)[4], uint32_t ok) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t signs = ((ok >> 4 * h) & 15u) * 0x10204080u;
      uint32_t a, b;
      asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(a) : "r"(signs));
      asm("prmt.b32 %0, %1, 0, 0xbbaa;" : "=r"(b) : "r"(signs));
      w[2 * h] = (w[2 * h] & a) | (kNegInf4 & ~a);
      w[2 * h + 1] = (w[2 * h + 1] & b) | (kNegInf4 & ~b);
    }
  }
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
  static __device__ __forceinline__ void only(uint32_t (&w)[4], uint32_t ok) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = (ok >> k) & 1u ? w[k] : kNegInf;
  }
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

// What a sequence's arguments say, clamped to what they may.
struct Lengths {
  int history, prompt, bias;
};
__device__ __forceinline__ Lengths lengths_of(const ProcessParams& P, int b, int& err) {
  Lengths n{0, 0, 0};
  const auto within = [&](int len, int most) {
    if (len < 0 || len > most) err |= SPEC_ERR_TOKEN;
    return min(max(len, 0), most);
  };
  n.history = within(P.history_len ? __ldg(P.history_len + b) : P.history_ld, P.history_ld);
  if (P.prompt_len) n.prompt = __ldg(P.prompt_len + b);
  n.bias = within(P.bias_len ? __ldg(P.bias_len + b) : P.bias_ld, P.bias_ld);
  return n;
}

// The drafted token of row i (-1: none) and its parent.
__device__ __forceinline__ void draft_of(const ProcessParams& P, int b, int i, int& token, int& parent, int& err) {
  const bool tree = P.parent != nullptr;
  token = -1;
  parent = 0;
  if (tree ? i > 0 : (P.tokens && i < P.n - 1)) {
    token = __ldg(P.tokens + static_cast<long long>(b) * P.tokens_ld + i);
    if (token < 0 || token >= P.V) {
      err |= SPEC_ERR_TOKEN;
      token = -1;
    }
  }
  if (tree && i > 0) {
    parent = __ldg(P.parent + static_cast<long long>(b) * P.n + i);
    if (parent < 0 || parent >= i) {
      err |= SPEC_ERR_PARENT;
      parent = 0;
    }
  }
  if (P.mask && P.mask_index) {
    const int mi = __ldg(P.mask_index + static_cast<long long>(b) * P.n + i);
    if (mi < -1 || mi >= P.mask_rows) err |= SPEC_ERR_MASK;
  }
}

// take(token, place) for the history's tokens within [first, first + count),
// four at a time where rows allow 16-byte loads, the next four loading
// meanwhile.  Most tokens are of other slabs: four are sifted by a subtraction
// and a comparison each, and only the rest take a branch.  bad: also look for
// tokens outside the vocabulary.
template <int kThreads, typename F>
__device__ __forceinline__ void for_history(const ProcessParams& P, int b, int len, int first, int count, bool* bad,
                                            F&& take) {
  const int* h = P.history + static_cast<long long>(b) * P.history_ld;
  const bool wide = P.history_ld % 4 == 0 && !misaligned16(P.history);
  const int width = wide ? 4 : 1;
  const auto load = [&](int at) {
    int4 t = make_int4(0, 0, 0, 0);
    if (at < len) {
      if (wide) t = __ldg(reinterpret_cast<const int4*>(h + at));
      else t.x = __ldg(h + at);
    }
    return t;
  };
  const auto within = [](const int4& t, int from, int n) {
    const auto in = [&](int v) { return static_cast<unsigned>(v - from) < static_cast<unsigned>(n); };
    return (in(t.x) ? 1u : 0u) | (in(t.y) ? 2u : 0u) | (in(t.z) ? 4u : 0u) | (in(t.w) ? 8u : 0u);
  };
  int4 next = load(width * static_cast<int>(threadIdx.x));
  for (int at = width * static_cast<int>(threadIdx.x); at < len; at += width * kThreads) {
    const int4 t = next;
    next = load(at + width * kThreads);
    const unsigned there = (1u << min(width, len - at)) - 1u;
    if (bad && (there & ~within(t, 0, P.V))) *bad = true;
    for (unsigned todo = there & within(t, first, count); todo; todo &= todo - 1) {
      const int k = __ffs(todo) - 1;
      take(k < 2 ? (k == 0 ? t.x : t.y) : (k == 2 ? t.z : t.w), at + k);
    }
  }
}

// The biases.  enter(token) gives a token's place (negative: not of this
// table); words and bias are the tables' words and sums.  Entries of different
// tokens go in at once; where a token has several, one warp adds all of them up
// in their order, so that the sum is always the same.  Ends synchronised.
template <int kThreads, typename Enter>
__device__ __forceinline__ void add_biases(const ProcessParams& P, int b, int len, unsigned* words, float* bias,
                                           int* again, int& err, Enter&& enter) {
  if (len == 0) {
    __syncthreads();
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31;
  const long long src = static_cast<long long>(b) * P.bias_ld;
  if (tid == 0) *again = 0;
  __syncthreads();
  int first_at = -1;  // entry tid's place and value (most lists are no longer than the CTA)
  float first_x = 0.f;
  for (int e = tid; e < len; e += kThreads) {
    const int t = __ldg(P.bias_tokens + src + e);
    if (e == tid) first_x = __ldg(P.bias_values + src + e);
    if (t < 0 || t >= P.V) {
      err |= SPEC_ERR_TOKEN;
      continue;
    }
    const int at = enter(t);
    if (at < 0) continue;
    if (e == tid) first_at = at;
    if (atomicOr(&words[at], kBiased) & kBiased) *again = 1;
  }
  __syncthreads();
  if (!*again) {
    if (first_at >= 0) bias[first_at] = first_x;
    for (int e = tid + kThreads; e < len; e += kThreads) {
      const int t = __ldg(P.bias_tokens + src + e);
      const int at = t >= 0 && t < P.V ? enter(t) : -1;
      if (at >= 0) bias[at] = __ldg(P.bias_values + src + e);
    }
  } else if (tid < 32) {
    int t_next = lane < len ? __ldg(P.bias_tokens + src + lane) : -1;
    float x_next = lane < len ? __ldg(P.bias_values + src + lane) : 0.f;
    for (int base = 0; base < len; base += 32) {
      const int t = t_next;
      const float x = x_next;
      const int ahead = base + 32 + lane;
      t_next = ahead < len ? __ldg(P.bias_tokens + src + ahead) : -1;
      x_next = ahead < len ? __ldg(P.bias_values + src + ahead) : 0.f;
      const int at = t >= 0 && t < P.V ? enter(t) : -1;
      if (!__any_sync(0xffffffffu, at >= 0)) continue;
      // the lanes whose entries are one token's all add them up, lowest lane first
      const unsigned peers = __match_any_sync(0xffffffffu, at);
      float sum = at >= 0 ? bias[at] : 0.f;
      for (unsigned todo = at >= 0 ? peers : 0u; __any_sync(0xffffffffu, todo != 0u); todo &= todo - 1) {
        const float y = __shfl_sync(0xffffffffu, x, todo ? __ffs(todo) - 1 : 0);
        if (todo) sum = __fadd_rn(sum, y);
      }
      __syncwarp();
      if (at >= 0) bias[at] = sum;  // (the same value from each of them)
      __syncwarp();
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// collecting
// ---------------------------------------------------------------------------
// One CTA per sequence: a bitmap of the vocabulary marks the tokens, the bits
// before each word are counted, and a token's rank among the marked ones is its
// place.  No probing and no appending, so that every thread's work is a few
// instructions per token, and the entries come out sorted: a slab's start is
// the count at its first word.  (A hash table with appended entries took 25 to
// 45 us for 4000 to 8000 tokens, most of it in a warp's longest probe.)  Larger
// vocabularies go range by range, more than kWindow tokens window by window.
// (Calls with 128 histories of 8192 tokens: 177 us with 256 threads, 163 with
// 512, 160 with 1024.)
constexpr int kCollectThreads = 1024;
constexpr int kRangeWords = 8192;    // 262,144 tokens
constexpr int kWindow = 8192;

__global__ void __launch_bounds__(kCollectThreads) collect_kernel(const ProcessParams P) {
  extern __shared__ unsigned collect_dyn[];
  pdl_launch_dependents();
  const int words = min((P.V + 31) / 32, kRangeWords);
  unsigned* marked = collect_dyn;                             // [words] bitmap of the range
  unsigned* before = marked + words;                          // [words] marked tokens before the word
  unsigned* count = before + words;                           // [P.window] of the window's tokens
  float* bias = reinterpret_cast<float*>(count + P.window);   // [P.window]
  int* token = reinterpret_cast<int*>(bias + P.window);       // [P.window]
  __shared__ unsigned s_warp[kCollectThreads / 32];
  __shared__ int s_err, s_again;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x;
  int err = 0;
  const Lengths len = lengths_of(P, b, err);
  if (tid == 0) s_err = 0;
  const long long out = static_cast<long long>(b) * P.capacity;
  int* offsets = P.offsets + static_cast<long long>(b) * (P.slabs + 1);
  int base = 0;  // entries of the ranges before
  for (int first = 0; first < P.V; first += words * 32) {
    const int count_in = min(words * 32, P.V - first);  // the range's tokens
    // the word of a token in this range, or a negative number
    const auto word_of = [&](int t) {
      const int w = (t - first) >> 5;
      return t >= first && w < words ? w : -1;
    };
    const auto mark = [&](int t) {
      const int w = word_of(t);
      const unsigned bit = 1u << (t & 31);
      if (w >= 0 && !(*const_cast<volatile unsigned*>(marked + w) & bit)) atomicOr(&marked[w], bit);
    };
    for (int i = tid; i < words; i += kCollectThreads) marked[i] = 0u;
    __syncthreads();
    for (int i = tid; i < P.n; i += kCollectThreads) {
      int t, p;
      draft_of(P, b, i, t, p, err);
      if (t >= 0) mark(t);
    }
    bool bad = false;
    for_history<kCollectThreads>(P, b, len.history, first, count_in, first == 0 ? &bad : nullptr,
                                 [&](int t, int) { mark(t); });
    if (bad) err |= SPEC_ERR_TOKEN;
    for (int e = tid; e < len.bias; e += kCollectThreads) {
      const int t = __ldg(P.bias_tokens + static_cast<long long>(b) * P.bias_ld + e);
      if (t < 0 || t >= P.V) err |= SPEC_ERR_TOKEN;
      else mark(t);
    }
    if (first == 0 && err) atomicOr(&s_err, err);
    __syncthreads();
    if (first == 0 && tid == 0) {
      if (P.seq_error) P.seq_error[b] = s_err;
      if (s_err && P.error_word) atomicOr(P.error_word, s_err);
    }

    // marked tokens before each word: a thread's words, the warp's, the CTA's
    const int per = (words + kCollectThreads - 1) / kCollectThreads;
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
    unsigned own = 0;
    for (int i = w0; i < w1; ++i) own += __popc(marked[i]);
    unsigned sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    static_assert(kCollectThreads == 32 * 32, "a lane per warp");
    const unsigned total = __reduce_add_sync(0xffffffffu, s_warp[lane]);
    unsigned run = sum - own + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
    for (int i = w0; i < w1; ++i) {
      before[i] = run;
      // where the slab that begins here starts (slab_tokens is a power of two)
      const int t0 = first + i * 32;
      if (t0 < P.V && (t0 & (P.slab_tokens - 1)) == 0) offsets[t0 / P.slab_tokens] = base + static_cast<int>(run);
      run += __popc(marked[i]);
    }

    for (int window = 0; window < static_cast<int>(total); window += P.window) {
      // a token's place in the window; whoever comes to a place leaves the token there
      const auto enter = [&](int t) {
        const int w = word_of(t);
        if (w < 0) return -1;
        const int at = static_cast<int>(before[w] + __popc(marked[w] & ((1u << (t & 31)) - 1u))) - window;
        if (at < 0 || at >= P.window) return -1;
        token[at] = t;
        return at;
      };
      for (int i = tid; i < P.window; i += kCollectThreads) {
        count[i] = 0u;
        bias[i] = 0.f;
      }
      __syncthreads();
      for (int i = tid; i < P.n; i += kCollectThreads) {
        int t, p;
        draft_of(P, b, i, t, p, err);
        const int at = t >= 0 ? enter(t) : -1;
        if (at >= 0) atomicOr(&count[at], kDrafted);
      }
      for_history<kCollectThreads>(P, b, len.history, first, count_in, nullptr, [&](int t, int i) {
        const int at = enter(t);
        if (at < 0) return;
        if (i < len.prompt) atomicOr(&count[at], kInPrompt);
        else atomicAdd(&count[at], 1u);
      });
      add_biases<kCollectThreads>(P, b, len.bias, count, bias, &s_again, err, enter);
      const int n = min(P.window, static_cast<int>(total) - window);
      for (int i = tid; i < n; i += kCollectThreads) {
        P.entry_token[out + base + window + i] = token[i];
        P.entry_count[out + base + window + i] = count[i];
        P.entry_bias[out + base + window + i] = bias[i];
      }
      __syncthreads();
    }
    base += static_cast<int>(total);
    __syncthreads();
  }
  // slabs past the vocabulary's last token, and the end
  for (int s = (P.V - 1) / P.slab_tokens + 1 + tid; s <= P.slabs; s += kCollectThreads) offsets[s] = base;
}

// ---------------------------------------------------------------------------
// the rows
// ---------------------------------------------------------------------------
// kThreads threads with kVecs vectors each: the slab.  kListed: the entries
// come from the workspace.
template <typename T, int kThreads, int kVecs, bool kListed>
struct Slab {
  static constexpr int kE = Lanes<T>::kN;
  static constexpr int kTokens = kThreads * kVecs * kE;
  static constexpr int kTable = kTokens + kE - 1;        // and the e - 1 tokens before it
  static constexpr int kWords = (kTable + 31) / 32;      // a bitmap of the table
  static constexpr int kTileBytes = kTokens * static_cast<int>(sizeof(T));  // a row's part; there are two
  static constexpr int kCache = 1024;                    // listed entries kept in shared memory
  static_assert(!kListed || kTable <= 0x3fff, "an entry's place and two flags in 16 bits");
  static size_t smem(const ProcessParams& p) {
    const size_t rows = 2 * kTileBytes + 12 * static_cast<size_t>(p.n);
    if (kListed) return rows + 6 * static_cast<size_t>(kCache);
    return rows + 4 * (static_cast<size_t>(kTable) * (p.bias_tokens ? 2 : 1) + 2 * kWords) +
           2 * static_cast<size_t>(kTable);
  }
};

// Threads an SM holds: as many as leave the kernel its registers (56; with listed
// entries 40 and 4 to 64 bytes spilled).  Without the list, 128 sequences
// of 9 rows of 128256 tokens: 1024 threads 108 us, 1152 103, 1280 107; 16 trees of
// 64 rows of 50257: 51, 52, 68.
__host__ __device__ constexpr int resident_threads(bool listed) { return listed ? 1536 : 1152; }

template <typename T, int kThreads, int kVecs, bool kListed, bool kAligned>
__global__ void __launch_bounds__(kThreads, resident_threads(kListed) / kThreads) process_kernel(const ProcessParams P) {
  using L = Lanes<T>;
  using S = Slab<T, kThreads, kVecs, kListed>;
  constexpr int E = S::kE;
  constexpr uint32_t kFull = (1u << E) - 1u;

  extern __shared__ __align__(16) unsigned char proc_dyn[];
  T* tile = reinterpret_cast<T*>(proc_dyn);                              // [2][kTokens] rows' parts
  int* s_tok = reinterpret_cast<int*>(proc_dyn + 2 * S::kTileBytes);     // [n]
  int* s_par = s_tok + P.n;                                              // [n]
  int* s_mask = s_par + P.n;                                             // [n]
  // listed: the first kCache entries, as they apply to every row: what is added
  // (a penalty's negative or a bias), and the place in the table with two flags
  // (bit 14: repetition; bit 15: the entry is read again, because it is drafted,
  // so that the row matters, or has both a penalty and a bias)
  float* c_add = reinterpret_cast<float*>(s_mask + P.n);
  unsigned short* c_place = reinterpret_cast<unsigned short*>(c_add + S::kCache);
  // else: the table, two bitmaps and the list of touched tokens
  unsigned* count = reinterpret_cast<unsigned*>(s_mask + P.n);           // [kTable]
  unsigned* listed = count + S::kTable;                                  // [kWords]
  float* bias = reinterpret_cast<float*>(listed + S::kWords);            // [kTable], with biases
  unsigned short* list = reinterpret_cast<unsigned short*>(bias + (P.bias_tokens ? S::kTable : 0));  // [kTable]
  __shared__ int s_err, s_used, s_again;

  const int tid = threadIdx.x;
  const int b = blockIdx.x;
  const int r0 = blockIdx.y * P.rows_per_cta;
  const int r1 = min(P.n, r0 + P.rows_per_cta);
  const int v0 = blockIdx.z * (kThreads * kVecs);  // first vector of the slab
  const int lo = v0 * E - (E - 1);                 // first token of the table
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
    if constexpr (kAligned) return 0;
    return static_cast<int>(((static_cast<long long>(b) * P.n + i) * P.ld) % E);
  };
  // the mask bits of row i's vectors (mrow < 0: not masked; 0 for vectors outside the row)
  const auto load_mask = [&](int i, int mrow, uint32_t (&ok)[kVecs]) {
    const int m = lead_of(i);
    const unsigned* mk = mrow >= 0 ? P.mask + static_cast<long long>(mrow) * P.mask_ld : nullptr;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int t0 = (v0 + j * kThreads + tid) * E - m;
      ok[j] = t0 < P.V ? kFull : 0u;
      if (mk && t0 < P.V) {
        if constexpr (kAligned) {  // (a vector's bits lie in one word)
          ok[j] = (__ldg(mk + (t0 >> 5)) >> (t0 & 31)) & kFull;
        } else if (t0 < 0) {
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
      const int t0 = (v0 + j * kThreads + tid) * E - m;
      if (!ok[j]) continue;
      if ((kAligned || t0 >= 0) && t0 + E <= P.V) {
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

  // The stream reads the vectors of one row and the mask bits of the next
  // ahead; the first ones are in flight while the entries are fetched or built.
  uint32_t w[kVecs][4], ok0[kVecs], ok1[kVecs];
  if (stream) {
    load_mask(r0, mask_row(r0), ok0);
    if (r0 + 1 < r1) load_mask(r0 + 1, mask_row(r0 + 1), ok1);
    load_row(r0, ok0, w);
  }

  int err = 0;
  if constexpr (!kListed) {
    for (int i = tid; i < S::kTable + S::kWords; i += kThreads) count[i] = 0u;  // and the bitmap
    if (biased)
      for (int i = tid; i < S::kTable; i += kThreads) bias[i] = 0.f;
    if (tid == 0) s_err = s_used = 0;
    __syncthreads();
  }
  // a token of the slab that something applies to: into the list
  const auto touch = [&](unsigned at) {
    const unsigned bit = 1u << (at & 31);
    if (!(listed[at >> 5] & bit) && !(atomicOr(&listed[at >> 5], bit) & bit))
      list[atomicAdd(&s_used, 1)] = static_cast<unsigned short>(at);
  };
  const auto place_of = [&](int t) {
    const unsigned at = static_cast<unsigned>(t - lo);
    return t >= 0 && at < static_cast<unsigned>(S::kTable) ? static_cast<int>(at) : -1;
  };
  for (int i = tid; i < P.n; i += kThreads) {
    int t, p;
    draft_of(P, b, i, t, p, err);
    s_tok[i] = t;
    s_par[i] = p;
    s_mask[i] = mask_row(i);
    if constexpr (!kListed) {
      const int at = place_of(t);
      if (at >= 0) {
        atomicOr(&count[at], kDrafted);
        touch(at);
      }
    }
  }
  const float rep = P.repetition ? __ldg(P.repetition + b) : 1.f;
  const float inv = __frcp_rn(rep);
  const float freq = P.frequency ? __ldg(P.frequency + b) : 0.f;
  const float pres = P.presence ? __ldg(P.presence + b) : 0.f;
  // the penalty of a word's occurrences (one rounding for both terms)
  const auto penalty = [&](unsigned c) {
    const unsigned made = c & kMade;
    return made ? __fmaf_rn(freq, static_cast<float>(made), pres) : 0.f;
  };
  int e0 = 0, tokens;  // listed: the entries' first, in the workspace
  if constexpr (kListed) {
    pdl_wait();
    const int* offsets = P.offsets + static_cast<long long>(b) * (P.slabs + 1);
    const int slab = blockIdx.z;
    e0 = __ldcg(offsets + slab);
    tokens = __ldcg(offsets + slab + 1) - e0;
    if (!kAligned && P.ld % E && slab > 0) {
      // rows that start within a vector take up to e - 1 tokens of the slab before:
      // some of its last entries.  (With all of them, 128 sequences of 9 rows of
      // 128255 tokens, 8192 in the history: 138 us, so 133; of 50257 85 and 77.)
      const int at = e0 - 1 - (tid & 31);
      const bool ours = (tid & 31) < E - 1 && at >= __ldcg(offsets + slab - 1) &&
                        __ldcg(P.entry_token + static_cast<long long>(b) * P.capacity + at) >= lo;
      const int back = __popc(__ballot_sync(0xffffffffu, ours));
      e0 -= back;
      tokens += back;
    }
    const long long src = static_cast<long long>(b) * P.capacity + e0;
    for (int e = tid; e < min(tokens, S::kCache); e += kThreads) {
      const int at = __ldcg(P.entry_token + src + e) - lo;
      const unsigned c = __ldcg(P.entry_count + src + e);
      const float minus = penalty(c), plus = __ldcg(P.entry_bias + src + e);
      // (a penalty and a bias are two additions: such entries are read again)
      const bool both = minus != 0.f && plus != 0.f;
      c_add[e] = minus != 0.f ? -minus : plus;
      c_place[e] = static_cast<unsigned short>(at | (c & (kInPrompt | kMade) ? 0x4000 : 0) |
                                               (c & kDrafted || both ? 0x8000 : 0));
    }
    __syncthreads();
  } else {
    const Lengths len = lengths_of(P, b, err);
    const bool checks = blockIdx.z == 0 && blockIdx.y == 0;
    const int t0 = max(lo, 0);
    bool bad = false;
    for_history<kThreads>(P, b, len.history, t0, min(lo + S::kTable, P.V) - t0, checks ? &bad : nullptr,
                          [&](int t, int at) {
                            const int o = t - lo;
                            if (at < len.prompt) atomicOr(&count[o], kInPrompt);
                            else atomicAdd(&count[o], 1u);
                            touch(o);
                          });
    if (bad) err |= SPEC_ERR_TOKEN;
    add_biases<kThreads>(P, b, len.bias, count, bias, &s_again, err, [&](int t) {
      const int at = place_of(t);
      if (at >= 0) touch(at);
      return at;
    });
    if (checks && err) atomicOr(&s_err, err);
    __syncthreads();
    if (checks && tid == 0) {
      if (P.seq_error) P.seq_error[b] = s_err;
      if (s_err && P.error_word) atomicOr(P.error_word, s_err);
    }
    tokens = s_used;
  }

  // Rewrites entry e's element of row i, which starts at element m of its first
  // vector; `part` is the row's part of the slab.  (A masked element is -inf by
  // now and stays.)
  const auto rewrite = [&](int i, int e, T* part, int m) {
    int at;
    float first = 0.f, plus = 0.f;  // what is added: the penalty's negative, then the bias
    bool seen, again = true;
    if constexpr (kListed) {
      if (e < S::kCache) {
        at = c_place[e];
        first = c_add[e];
        seen = at & 0x4000;
        again = at & 0x8000;
        at &= 0x3fff;
      } else {
        at = __ldcg(P.entry_token + static_cast<long long>(b) * P.capacity + e0 + e) - lo;
      }
    } else {
      at = list[e];
    }
    // rows that start within a vector shift the slab: the neighbours' tokens are not ours
    const int place = at - (E - 1) + m;
    if (place < 0 || place >= S::kTokens) return;
    if (again) {
      unsigned c;
      if constexpr (kListed) {
        const long long src = static_cast<long long>(b) * P.capacity + e0 + e;
        c = __ldcg(P.entry_count + src);
        plus = __ldcg(P.entry_bias + src);
      } else {
        c = count[at];
        plus = biased ? bias[at] : 0.f;
      }
      // Its occurrences on the way to the row.  (This grows with the square of a
      // chain's rows: one of 1024 rows of 32000 logits takes 0.41 ms, 16 take 5.9,
      // where their bytes take 0.31; a tree of 1024 nodes, with short paths, 59 us.)
      if (c & kDrafted) {
        const int t = lo + at;
        if (tree) {
          for (int a = i; a > 0; a = s_par[a]) c += s_tok[a] == t;
        } else {
          for (int a = 0; a < i; ++a) c += s_tok[a] == t;
        }
      }
      seen = c & (kInPrompt | kMade);
      first = -penalty(c);
    }
    if (!seen && first == 0.f && plus == 0.f) return;
    const uint32_t x = load_bits(part + place);
    if (x == L::kNegInf) return;
    float y = L::widen(x);
    if (seen) y = __fmul_rn(y, y > 0.f ? inv : rep);
    if (first != 0.f) y = __fadd_rn(y, first);
    if (plus != 0.f) y = __fadd_rn(y, plus);
    store_bits(part + place, L::round(y));
  };

  if (!stream) {
    // in place: consecutive threads take the tokens of one row
    const long long pairs = static_cast<long long>(tokens) * (r1 - r0);
    for (long long p = tid; p < pairs; p += kThreads) {
      const int i = r0 + static_cast<int>(p / tokens), e = static_cast<int>(p % tokens), m = lead_of(i);
      rewrite(i, e,
              static_cast<T*>(P.out) + (static_cast<long long>(b) * P.n + i) * P.out_ld +
                  (static_cast<long long>(v0) * E - m),
              m);
    }
    return;
  }

  // Row i's vectors, masked, into its tile; then the loads of row i + 1 go out.
  const auto fill = [&](int i) {
    uint4* to = reinterpret_cast<uint4*>(tile + ((i - r0) & 1) * S::kTokens);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (!ok0[j]) {
        w[j][0] = w[j][1] = w[j][2] = w[j][3] = L::kNegInf4;
      } else if (ok0[j] != kFull) {
        L::only(w[j], ok0[j]);
      }
      to[j * kThreads + tid] = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
      ok0[j] = ok1[j];
    }
    if (i + 1 < r1) load_row(i + 1, ok0, w);
    if (i + 2 < r1) load_mask(i + 2, s_mask[i + 2], ok1);
  };
  // While row i is rewritten in one tile, row i + 1 fills the other: one
  // barrier per row.  (A thread fills a tile again after it has written out its
  // own vectors of it, which nobody else touches in between.)
  fill(r0);
  __syncthreads();
  for (int i = r0; i < r1; ++i) {
    const long long row = static_cast<long long>(b) * P.n + i;
    const int m = lead_of(i);
    T* part = tile + ((i - r0) & 1) * S::kTokens;
    for (int e = tid; e < tokens; e += kThreads) rewrite(i, e, part, m);
    if (i + 1 < r1) fill(i + 1);
    if (tokens > 0) __syncthreads();
    T* dst = static_cast<T*>(P.out) + row * P.out_ld;
    const bool same = kAligned || static_cast<int>((row * P.out_ld) % E) == m;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int t0 = (v0 + j * kThreads + tid) * E - m;
      if (t0 >= P.V) continue;
      const uint4 x = reinterpret_cast<const uint4*>(part)[j * kThreads + tid];
      if (same && (kAligned || t0 >= 0) && t0 + E <= P.V) {
        if (!(kDebugChecks && misaligned16(dst + t0))) *reinterpret_cast<uint4*>(dst + t0) = x;
      } else {
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (t0 + k >= 0 && t0 + k < P.V) store_bits(dst + t0 + k, L::bits(y, k));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// A kernel's dynamic shared memory limit, raised where a call needs more.
template <typename K>
cudaError_t raise_smem(K kernel, size_t bytes, std::map<int, size_t>& done) {
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev] >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done[dev] = bytes;
  return e;
}

template <typename T, int kThreads, int kVecs>
int slabs_of(int V, long long ld) {
  constexpr int E = Lanes<T>::kN;
  // vectors of the longest row: a row may start anywhere in its first vector
  const int lead = ld % E ? E - 1 : 0;
  const int nvec = (V + lead + E - 1) / E;
  return (nvec + kThreads * kVecs - 1) / (kThreads * kVecs);
}

// Rows that a CTA takes: few sequences and slabs have a sequence's rows split
// as well, into as many CTAs as the registers have room for.  (With biases the
// tables' shared memory has room for fewer: 3 of 256 threads instead of 4, 7 of
// 128 instead of 9, and the rest run in a second round.  Split by that as well:
// 32 sequences of 9 rows of 32000, 2048 tokens and 300 biases, 22.5 to 20.1 us
// where tokens are uniform, 19.7 to 25.0 where frequent ones share a slab; one
// sequence of 1024 rows of 700 67 to 94, 16 of 1024 rows of 32000 5.8 ms to 8.9.)
template <typename T, int kThreads, int kVecs, bool kListed>
int rows_of(const ProcessParams& p, int nsm) {
  const long long have = static_cast<long long>(slabs_of<T, kThreads, kVecs>(p.V, p.ld)) * p.B;
  const long long fill = static_cast<long long>(resident_threads(kListed) / kThreads) * nsm;
  const long long parts = std::min<long long>(p.n, std::max<long long>(1, fill / have));
  return static_cast<int>((p.n + parts - 1) / parts);
}

template <typename T, int kThreads, int kVecs, bool kListed, bool kAligned>
cudaError_t launch_rows(ProcessParams p, int nsm, cudaStream_t s) {
  using S = Slab<T, kThreads, kVecs, kListed>;
  static std::map<int, size_t> done;
  const size_t dyn = S::smem(p);
  const auto kernel = process_kernel<T, kThreads, kVecs, kListed, kAligned>;
  cudaError_t e = raise_smem(kernel, dyn, done);
  if (e != cudaSuccess) return e;
  const int slabs = slabs_of<T, kThreads, kVecs>(p.V, p.ld);
  p.rows_per_cta = rows_of<T, kThreads, kVecs, kListed>(p, nsm);
  cudaLaunchConfig_t cfg = {};
  // sequences first: a slab that takes long (the first, with the frequent tokens
  // of a vocabulary) does so for every sequence, and what takes long starts early
  cfg.gridDim = dim3(static_cast<unsigned>(p.B), static_cast<unsigned>((p.n + p.rows_per_cta - 1) / p.rows_per_cta),
                     static_cast<unsigned>(slabs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = dyn;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = kListed ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Rows that all start and end up on a vector boundary need no shifts of their
// mask bits and no choice of how to store.  Measured (128 sequences of 9 rows of
// 128256 bfloat16 logits, masks, histories of 8192 tokens): 109 us, by the
// kernel for any alignment 129; without masks 118 and 124.
template <typename T, int kThreads, int kVecs, bool kListed>
cudaError_t launch_process(const ProcessParams& p, int nsm, cudaStream_t s) {
  constexpr int E = Lanes<T>::kN;
  if (p.ld % E == 0 && p.out_ld % E == 0) return launch_rows<T, kThreads, kVecs, kListed, true>(p, nsm, s);
  return launch_rows<T, kThreads, kVecs, kListed, false>(p, nsm, s);
}

// The entries' places in the workspace.
struct ProcessLayout {
  int capacity;
  size_t token, count, bias, total;
};
ProcessLayout process_layout(long long B, int n, int V, int history, int biases) {
  ProcessLayout l{};
  const long long most = static_cast<long long>(n) + history + biases;
  l.capacity = static_cast<int>(std::min<long long>(most, V));
  const size_t part = align256(static_cast<size_t>(B) * l.capacity * 4);
  l.token = align256(static_cast<size_t>(B) * (V / 1024 + 4) * 4);  // slabs of 1024 tokens or more, and the end
  l.count = l.token + part;
  l.bias = l.count + part;
  l.total = l.bias + part;
  return l;
}

cudaError_t launch_collect(ProcessParams p, cudaStream_t s) {
  static std::map<int, size_t> done;
  p.window = std::min(kWindow, (p.capacity + 31) / 32 * 32);
  const size_t dyn =
      8 * static_cast<size_t>(std::min((p.V + 31) / 32, kRangeWords)) + 12 * static_cast<size_t>(p.window);
  const cudaError_t e = raise_smem(collect_kernel, dyn, done);
  if (e != cudaSuccess) return e;
  collect_kernel<<<p.B, kCollectThreads, dyn, s>>>(p);
  return cudaGetLastError();
}

// CTAs of the one-kernel form
template <typename T, int kThreads, int kVecs>
long long ctas_of(const ProcessParams& p, int nsm) {
  const int rows = rows_of<T, kThreads, kVecs, false>(p, nsm);
  return static_cast<long long>(slabs_of<T, kThreads, kVecs>(p.V, p.ld)) * p.B * ((p.n + rows - 1) / rows);
}

template <typename T>
cudaError_t run_process(ProcessParams p, int nsm, cudaStream_t s) {
  // (Here the host knows the buffers' widths, not the lists' lengths.)
  const int reads = p.history_ld + p.bias_ld;
  // The form for one kernel: CTAs of 128 threads stream better (more of them
  // overlap their phases), those of 256 get through a history sooner and read it
  // half as often: worth it where reading comes to 400 tokens per row or more.
  // Measured (bfloat16, 9 rows; 128 and 256 threads): V = 32000, 32 sequences of
  // 200 tokens, 40 per row, 9.4 and 10.2 us; 2000, 400, 12.0 and 11.5; 8000,
  // 1600, 24.9 and 20.1; V = 128256, 128 sequences of 500, 56 per row, 110 and 112.
  const bool wide = reads > 400LL * rows_of<T, 128, 2, false>(p, nsm);
  // One kernel or two.  With one, every CTA of a sequence (a slab and some of the
  // rows) goes through the whole history.  With two, one CTA per sequence goes
  // through it alone, once per range to mark its tokens and once per window of
  // them; the second launch and the entries' way through the workspace cost 5 to
  // 8 us.  So two are worth it where there is much to read (16M tokens by all
  // slabs) and an SM reads 1.3 times as much or more with one.
  // Measured (bfloat16, tokens uniform and mostly frequent ones; one kernel, two):
  //   much to read or not, 9 rows, V = 128256: 128 sequences of 500 tokens (4M)
  //     110 and 113 us; of 2000 (16M) 111 and 110; of 8192 (66M) 138 and 118, 132
  //     and 116; 64 of 8192 (33M) 77 and 71; 32 of 8192 (16M) 43 and 47
  //   an SM's reading with one over that with two, from 16M on: 1 row, V = 128256,
  //     128 sequences of 32768 (4.5) 151 and 81, 134 and 65; 9 rows, V = 32000, 128
  //     of 131072 (1.35) 330 and 324, 290 and 278; of 32768 (1.35) 128 and 137, 106
  //     and 118; V = 128256, 32 of 32768 (1.1) 82 and 101, 81 and 117; 64 of 131072
  //     (0.8) 413 and 557, 340 and 374; 16 of 32768 (0.6) 49 and 84, 76 and 113; 4
  //     of 131072 (0.15) 91 and 421, 147 and 292.
  p.slabs = slabs_of<T, 128, 2>(p.V, p.ld);
  const bool much = static_cast<long long>(p.slabs) * p.B * reads > (1LL << 24);
  const long long ctas = wide ? ctas_of<T, 256, 2>(p, nsm) : ctas_of<T, 128, 2>(p, nsm);
  const int ranges = (p.V + 32 * kRangeWords - 1) / (32 * kRangeWords);
  const long long passes = 2 * ranges - 1 + (p.capacity + kWindow - 1) / kWindow;
  const int rounds = (p.B + nsm - 1) / nsm;  // of collecting CTAs, taken as one per SM
  if (!much || 10 * ctas < 13 * passes * rounds * nsm) {
    if (wide) return launch_process<T, 256, 2, false>(p, nsm, s);
    return launch_process<T, 128, 2, false>(p, nsm, s);
  }
  using Listed = Slab<T, 128, 2, true>;
  static_assert((Listed::kTokens & (Listed::kTokens - 1)) == 0 && Listed::kTokens >= 1024,
                "collecting tests for a slab's start with a mask; the workspace's offsets");
  p.slab_tokens = Listed::kTokens;
  const cudaError_t e = launch_collect(p, s);
  return e == cudaSuccess ? launch_process<T, 128, 2, true>(p, nsm, s) : e;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace sv

extern "C" size_t spec_process_workspace_size(int B, int n, int V, int history_ld, int bias_ld) {
  if (B < 1 || B > sv::kMaxSeq || n < 1 || n > sv::kMaxRows || V < 1 || V > 2097152 || history_ld < 0 || bias_ld < 0 ||
      history_ld > sv::kMaxList || bias_ld > sv::kMaxList)
    return 0;
  return sv::process_layout(B, n, V, history_ld, bias_ld).total;
}

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
  if (a->history && (a->history_ld < 0 || a->history_ld > kMaxList)) return SPEC_EINVAL;
  if (a->bias_tokens && (!a->bias_values || a->bias_ld < 0 || a->bias_ld > kMaxList)) return SPEC_EINVAL;
  if (a->mask && (a->mask_rows < 1 || a->mask_ld < (a->V + 31) / 32)) return SPEC_EINVAL;
  if (a->mask && !a->mask_index && a->mask_rows < static_cast<long long>(a->B) * a->n) return SPEC_EINVAL;
  if (!aligned16(a->logits) || !aligned16(a->out)) return SPEC_EALIGN;
  const int history = a->history ? a->history_ld : 0, biases = a->bias_tokens ? a->bias_ld : 0;
  const ProcessLayout layout = process_layout(a->B, a->n, a->V, history, biases);
  if (!a->workspace || a->workspace_bytes < layout.total || (reinterpret_cast<uintptr_t>(a->workspace) & 255u))
    return SPEC_EWORKSPACE;
  const int nsm = sm_count();
  if (nsm < 1) return SPEC_ECUDA;
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
  // (a list of width 0 may have no address, but has lengths; without a list they are not read)
  p.history = history > 0 ? a->history : nullptr;
  p.history_ld = history;
  p.history_len = a->history || a->history_ld == 0 ? a->history_len : nullptr;
  p.prompt_len = a->history ? a->prompt_len : nullptr;
  p.repetition = a->repetition;
  p.frequency = a->frequency;
  p.presence = a->presence;
  p.bias_tokens = biases > 0 ? a->bias_tokens : nullptr;
  p.bias_values = a->bias_values;
  p.bias_len = a->bias_tokens || a->bias_ld == 0 ? a->bias_len : nullptr;
  p.bias_ld = biases;
  p.mask = a->mask;
  p.mask_rows = a->mask_rows;
  p.mask_ld = a->mask_ld;
  p.mask_index = a->mask_index;
  p.seq_error = a->seq_error;
  p.error_word = a->error_word;
  char* ws = static_cast<char*>(a->workspace);
  p.capacity = layout.capacity;
  p.offsets = reinterpret_cast<int*>(ws);
  p.entry_token = reinterpret_cast<int*>(ws + layout.token);
  p.entry_count = reinterpret_cast<unsigned*>(ws + layout.count);
  p.entry_bias = reinterpret_cast<float*>(ws + layout.bias);
  const cudaError_t e =
      a->dtype == SPEC_BF16 ? run_process<bf16_t>(p, nsm, stream) : run_process<float>(p, nsm, stream);
  return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}
