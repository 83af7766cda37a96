// Attention of drafted rows over the paged 8-bit cache (spec_attend_cache).
//
// The rows of one sequence that read one head of the cache, n rows of Hq / H
// query heads each, are cut into blocks of R (16, 32 or 64).  For a tile of
// 128 tokens a block needs
//    S^T [128 tokens x R] = K [128 x D] Q^T,   O^T [D x R] = V^T [D x 128] P^T,
// P = 2^(scores - maximum): tokens, then elements, are the 128 rows of a
// tensor-core product and the block's rows its N columns, so that few rows
// cost few columns.  The codes are e4m3 and go to the tensor cores as they
// lie in memory (tcgen05.mma kind::f8f6f4), K with D and V with the tokens as
// the inner products' axis; nothing is unpacked.  The other operands keep
// their precision as sums of two e4m3 numbers x = hi + lo, lo = e4m3(x - hi),
// two products into the same accumulators:
//    a query relative to its largest element (bfloat16's 8 significant bits
//       are the two's, so it is exact down to 2^-18 of that element);
//    a weight relative to the largest of its tile and row, hence from 256
//       down to 2^-9 / 2: rows whose first tokens have nearly all the weight
//       keep the others' precision.
// A page's exponents are 2's powers and uniform over a token: one factor per
// thread for K; V's exponent is added to the score before the maximum, so that
// P carries it (y = x + ve), and the sum of the weights takes it back.
//
// One persistent CTA per SM takes an equal run of the tiles of all blocks,
// in the order sequence, head, block; a block that two CTAs share is left in
// parts in the workspace and joined by a second kernel (in order, so that the
// sums do not depend on the timing).  Warps: 0 copies pages (TMA, 128-byte
// swizzle) into rings of K and V tiles; 1 issues the products; 2 and 3 bring
// in queries, tree masks and clear what lies behind the last token; 4-7 and
// 8-11 turn the scores of every other tile into weights; 12-15 add the tiles'
// outputs up in registers.
//
// Bound by the bytes of the cache for a few rows.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>

#include "cache.cuh"
#include "internal.h"
#include "spec_cache.h"
#include "tc.cuh"
#include "tma_host.h"

namespace sv {
namespace {

constexpr int kTile = 128;      // tokens per tile
constexpr int kPanel = 16384;   // bytes of 128 tokens x 128 elements
constexpr int kMaxRows = 1024;  // n
constexpr int kMaxCtas = 160;
constexpr int kAttendThreads = 512;
constexpr int kScaleRing = 16, kPatchRing = 8;

// R: a block's rows; NP: panels of 128 elements of a head.
template <int R, int NP>
struct Shape {
  static constexpr int kStages = NP == 1 ? (R == 64 ? 4 : 5) : 2;
  static constexpr int kSlot = NP * kPanel;
  static constexpr int kQHalf = NP * R * 128;  // hi or lo of a block's queries
  static constexpr int kPHalf = kTile * R;     // hi or lo of a tile's weights
  static constexpr int kMaskBytes = 2 * kMaxRows * 8;
  static constexpr int kSmem = 1024 + 2 * kStages * kSlot + 4 * kQHalf + 4 * kPHalf + kMaskBytes + kMaxRows * 2;
  static constexpr uint32_t kTmemCols = (2 + 2 * NP) * R <= 128 ? 128 : 256;
  static_assert((2 + 2 * NP) * R <= 256 && kStages + 3 <= kScaleRing && kStages < kPatchRing, "rings");
};

struct AttendParams {
  int B, n, Hq, H, G, D, page, pages, table_pages, blocks;
  float c;  // scale * log2(e)
  long long q_ld[3], out_ld[3];
  const bf16_t* q;
  bf16_t* out;
  const int* prefix;
  const int* count;
  const int* parent;
  const int* block_table;
  const signed char* k_exps;
  const signed char* v_exps;
  int* seq_error;
  int* error_word;
  int4* shared;      // [ctas]: sequence, head, block and CTAs of the block that CTA begins and shares; 0 CTAs: none
  float* parts;      // [ctas][2][R][Dp + 4]: a part's sums, then log2 of their unit, its sum of weights and log2 of theirs
  unsigned more_bytes;
};

__device__ __forceinline__ void report(const AttendParams& P, int b, int bits) {
  if (P.seq_error) atomicOr(P.seq_error + b, bits);
  if (P.error_word) atomicOr(P.error_word, bits);
}

// ---------------------------------------------------------------------------
// the tiles of a call, in order
// ---------------------------------------------------------------------------

// A sequence's lengths; a sequence with a data error has none.
struct Lengths {
  int prefix, count;
  bool bad;
};
__device__ __forceinline__ Lengths lengths_of(const AttendParams& P, int b) {
  Lengths s;
  s.prefix = P.prefix ? __ldg(P.prefix + b) : 0;
  s.count = P.count ? __ldg(P.count + b) : P.n;
  s.bad = s.prefix < 0 || s.count < 0 || s.count > P.n ||
          static_cast<long long>(s.prefix) + s.count > static_cast<long long>(P.table_pages) * P.page;
  if (s.bad) s.prefix = s.count = 0;
  return s;
}
// The tokens that a block's rows can see: none if it has no rows.
template <int R>
__device__ __forceinline__ int keys_of(const AttendParams& P, const Lengths& s, int block) {
  if (block * R / P.G >= s.count) return 0;
  if (P.parent) return s.prefix + s.count;
  return s.prefix + min(s.count, ((block + 1) * R + P.G - 1) / P.G);
}
__device__ __forceinline__ int tiles_of(int keys) { return max(1, (keys + kTile - 1) / kTile); }

// One after another, the pieces of blocks that a CTA works on.
template <int R>
struct Walk {
  int b, h, block;
  Lengths s;
  int keys, tiles;  // the block's
  int t0, t1;       // the piece's tiles
  long long left;   // of the CTA, after this piece

  __device__ void start(const AttendParams& P, int seq, long long offset, long long units) {
    b = seq;
    left = units;
    if (units == 0) return;
    s = lengths_of(P, b);
    long long per = 0;
    for (int i = 0; i < P.blocks; ++i) per += tiles_of(keys_of<R>(P, s, i));
    h = static_cast<int>(offset / per);
    int rest = static_cast<int>(offset % per);
    for (block = 0;; ++block) {
      keys = keys_of<R>(P, s, block);
      tiles = tiles_of(keys);
      if (rest < tiles) break;
      rest -= tiles;
    }
    t0 = t1 = rest;  // (an empty piece before the first)
  }
  __device__ bool next(const AttendParams& P) {
    if (left == 0) return false;
    if (t1 == tiles) {
      if (++block == P.blocks) {
        block = 0;
        if (++h == P.H) {
          h = 0;
          s = lengths_of(P, ++b);
        }
      }
      keys = keys_of<R>(P, s, block);
      tiles = tiles_of(keys);
      t1 = 0;
    }
    t0 = t1;
    t1 = static_cast<int>(min(static_cast<long long>(tiles), t0 + left));
    left -= t1 - t0;
    return true;
  }
  __device__ __forceinline__ int row0() const { return block * R; }
  // From this tile on, rows differ in what they see, or see nothing at the end.
  __device__ __forceinline__ int first_special() const {
    return s.count > 1 ? s.prefix / kTile : keys % kTile ? keys / kTile : 0x7fffffff;
  }
};

// ---------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------

// Whole warps wait together (see int4_product.cu); a wait that gives up, here
// or elsewhere in the CTA, ends the role.
__device__ __forceinline__ bool at_wait(uint64_t* bar, unsigned parity, volatile int* fault) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  for (int i = 0; i < kMaxPolls; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *fault)) return false;
  }
  *fault = 1;
  return false;
}

__device__ __forceinline__ bool one_lane() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// Shared-memory matrix descriptor: the 8-row (K-major) or 8-step (MN-major)
// groups `stride` bytes apart, the swizzle of `row` bytes (tc.cuh has the bits).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t stride, int row) {
  const uint64_t swizzle = row == 128 ? 2 : row == 64 ? 4 : row == 32 ? 6 : 0;
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>(stride >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | swizzle << 61;
}
// byte offset `o` of a tile whose rows have `row` bytes, after the swizzle
__device__ __forceinline__ uint32_t swizzled(uint32_t o, int row) {
  return o ^ ((o >> 3) & (row == 128 ? 0x70u : row == 64 ? 0x30u : row == 32 ? 0x10u : 0u));
}

// e4m3 operands (format 0), float32 accumulators; majors: 0 K, 1 MN.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_major, int b_major) {
  return (1u << 4) | (static_cast<uint32_t>(a_major) << 15) | (static_cast<uint32_t>(b_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A B, M x N x 32.
__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_columns(uint32_t at, float* v) {
  if constexpr (N == 16) {
    tmem_ld16(at, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 32) tmem_ld32(at + i, v + i);
  }
}

// largest value of a warp (a NaN is passed over)
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// The warp's sums of N columns (N 16 or 32): lane i gets column i % N's.
template <int N>
__device__ __forceinline__ float column_sums(float* v, int lane) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float give = up ? v[j] : v[j + o], keep = up ? v[j + o] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float s = v[0];
  if (N == 16) s += __shfl_xor_sync(0xffffffffu, s, 16);
  return s;
}

// Two values as hi + lo, two e4m3 codes each.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  uint32_t h, back, rest;
  unsigned short c, d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(c));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(rest));
  hi = c;
  lo = d;
}

// The warps of a role meet at `bar` (one arrival each; a bounded wait).
__device__ __forceinline__ bool meet(uint64_t* bar, unsigned parity, bool leader, volatile int* fault) {
  __syncwarp();
  if (leader) mbar_arrive(bar);
  return at_wait(bar, parity, fault);
}

struct PageScale {
  float ck, ve;  // 2^key exponent (NaN: not a page), value exponent
  int far;       // the tile's value exponents lie far apart
  int pad;
};

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int R, int NP>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const AttendParams P) {
  using S = Shape<R, NP>;
  extern __shared__ __align__(1024) unsigned char at_dyn[];
  __shared__ uint64_t kfull[S::kStages], kempty[S::kStages], vfull[S::kStages], vempty[S::kStages];
  // sfull: a tile's scores are there; sempty: read; pfull: its weights are in
  // shared memory; pempty: read by the products; ofull / oempty: its outputs;
  // mfull / mempty: its maxima and sums of weights
  __shared__ uint64_t sfull[2], sempty[2], pfull[2], pempty[2], ofull[2], oempty[2], mfull[2], mempty[2];
  __shared__ uint64_t qfull[2], qempty[2], landed[kPatchRing], patched[kPatchRing], drain;
  // meetings within a role
  __shared__ uint64_t most_met[2], ref_met[2], mix_met[2], row_met[2], parent_met[2];
  __shared__ uint32_t tmem_s;
  __shared__ int fault_s, k_issued_s, v_issued_s, start_b;
  __shared__ long long start_off, warp_sums[kAttendThreads / 32];
  __shared__ PageScale scale_s[kScaleRing][8];
  __shared__ __align__(16) float most_s[2][4][R], ref_s[2][R], top_s[2][R], sum_s[2][4][R], cq_s[2][R];
  __shared__ __align__(16) float2 mix_s[2][R];
  __shared__ float row_s[R];
  __shared__ unsigned char token_s[2][R], nan_s[kPatchRing][kTile];

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool leader = one_lane();
  unsigned char* kring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(at_dyn) + 1023) &
                                                          ~static_cast<uintptr_t>(1023));
  unsigned char* vring = kring + S::kStages * S::kSlot;
  unsigned char* qbuf = vring + S::kStages * S::kSlot;
  unsigned char* pbuf = qbuf + 4 * S::kQHalf;
  unsigned long long* mask_s = reinterpret_cast<unsigned long long*>(pbuf + 4 * S::kPHalf);
  unsigned short* parent_s = reinterpret_cast<unsigned short*>(mask_s + 2 * kMaxRows);
  volatile int* fault = &fault_s;

  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 2);
      mbar_init(&sempty[s], 4);
      mbar_init(&pfull[s], 4);
      mbar_init(&pempty[s], 1);
      mbar_init(&ofull[s], 1);
      mbar_init(&oempty[s], 4);
      mbar_init(&mfull[s], 4);
      mbar_init(&mempty[s], 4);
      mbar_init(&most_met[s], 4);
      mbar_init(&ref_met[s], 4);
      mbar_init(&mix_met[s], 4);
      mbar_init(&row_met[s], 4);
      mbar_init(&parent_met[s], 2);
      mbar_init(&qfull[s], 2);
      mbar_init(&qempty[s], 4);
    }
    for (int s = 0; s < kPatchRing; ++s) {
      mbar_init(&landed[s], 1);
      mbar_init(&patched[s], 2);
    }
    mbar_init(&drain, 1);
    fault_s = k_issued_s = v_issued_s = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_s, S::kTmemCols);
    tmem_relinquish();
  }
  // the CTA's run of tiles
  long long total, mine = 0, before;
  const int per = (P.B + kAttendThreads - 1) / kAttendThreads;
  const int b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
  const auto tiles_of_seq = [&](int b) {
    const Lengths s = lengths_of(P, b);
    long long t = 0;
    for (int i = 0; i < P.blocks; ++i) t += tiles_of(keys_of<R>(P, s, i));
    return t * P.H;
  };
  for (int b = b0; b < b1; ++b) mine += tiles_of_seq(b);
  before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) warp_sums[warp] = before;
  before -= mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  total = 0;
  for (int w = 0; w < kAttendThreads / 32; ++w) {
    if (w == warp) before += total;
    total += warp_sums[w];
  }
  const long long ctas = min(static_cast<long long>(gridDim.x), total);
  const int cta = blockIdx.x;
  const long long u0 = cta < ctas ? total * cta / ctas : total, u1 = cta < ctas ? total * (cta + 1) / ctas : total;
  if (u0 < u1 && u0 >= before && u0 < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const long long t = tiles_of_seq(b);
      if (u0 < at + t) {
        start_b = b;
        start_off = u0 - at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  const uint32_t tmem_sc = tmem_s, tmem_o = tmem_s + 2 * R;
  Walk<R> w;
  w.start(P, u0 < u1 ? start_b : 0, u0 < u1 ? start_off : 0, u1 - u0);

  if (warp == 0) {
    // ---------------- pages ----------------
    const int pp = kTile / P.page, slot_in = lane % pp, batch = 32 / pp;
    int it = 0;
    bool ok = true;
    while (ok && w.next(P)) {
      if (w.keys == 0) continue;
      const int* table = P.block_table + static_cast<long long>(w.b) * P.table_pages;
      // the pages of `batch` tiles, a lane each
      const auto page_of = [&](int tb) {
        const int tile = tb + lane / pp, at = tile * pp + slot_in;
        return tile < w.t1 && at * P.page < w.keys ? __ldg(table + at) : 0;
      };
      int ahead = page_of(w.t0);
      for (int tb = w.t0; ok && tb < w.t1; tb += batch) {
        int page = ahead;
        const int mine_t = tb + lane / pp;
        const bool has = mine_t < w.t1 && (mine_t * pp + slot_in) * P.page < w.keys;
        const bool bad = has && (page < 0 || page >= P.pages);
        if (bad) report(P, w.b, SPEC_ERR_CACHE);
        if (!has || bad) page = 0;
        const long long slab = static_cast<long long>(page) * P.H + w.h;
        int ke = 0, ve = 0;
        if (has && !bad) {
          ke = __ldg(P.k_exps + slab);
          ve = __ldg(P.v_exps + slab);
        }
        ahead = page_of(tb + batch);
        int lo = has ? ve : 127, hi = has ? ve : -127;
        for (int o = 1; o < pp; o <<= 1) {
          lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        const unsigned groups = __ballot_sync(0xffffffffu, has);
        for (int i = 0; i < batch && tb + i < w.t1; ++i, ++it) {
          const int s = it % S::kStages;
          const unsigned parity = (static_cast<unsigned>(it / S::kStages) & 1u) ^ 1u;
          const bool here = has && lane / pp == i;
          const unsigned bytes =
              static_cast<unsigned>(__popc(groups >> (i * pp) & ((1u << pp) - 1u))) * static_cast<unsigned>(P.page) * 128u * NP +
              P.more_bytes;
          ok = at_wait(&kempty[s], parity, fault);
          if (!ok) break;
          if (lane / pp == i) {
            PageScale x;
            x.ck = bad ? __uint_as_float(0x7fc00000u) : exp2i(ke);
            x.ve = static_cast<float>(ve);
            x.far = hi - lo > 100;
            scale_s[it % kScaleRing][slot_in] = x;
          }
          __syncwarp();
          if (leader) mbar_expect_tx(&kfull[s], bytes);
          __syncwarp();
          if (here) {
#pragma unroll
            for (int p = 0; p < NP; ++p)
              tma_load_2d(kring + s * S::kSlot + p * kPanel + slot_in * P.page * 128, &tm_k, p * 128,
                          static_cast<int>(slab * P.page), &kfull[s]);
          }
          __syncwarp();
          if (leader) k_issued_s = it + 1;
          ok = at_wait(&vempty[s], parity, fault);
          if (!ok) break;
          if (leader) mbar_expect_tx(&vfull[s], bytes);
          __syncwarp();
          if (here) {
#pragma unroll
            for (int p = 0; p < NP; ++p)
              tma_load_2d(vring + s * S::kSlot + p * kPanel + slot_in * P.page * 128, &tm_v, p * 128,
                          static_cast<int>(slab * P.page), &vfull[s]);
          }
          __syncwarp();
          if (leader) v_issued_s = it + 1;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- products ----------------
    constexpr uint32_t idesc_s = idesc_e4m3(kTile, R, 0, 0), idesc_o = idesc_e4m3(128, R, 1, 1);
    const int steps = (P.D + 31) / 32;
    int it = 0, qn = 0, patches = 0;
    int last_patch = -1;  // the tile before's place among the patched ones
    bool ok = true;
    // the outputs of tile j
    const auto outputs = [&](int j, int patch) {
      const int s = j % S::kStages, d = j & 1;
      const unsigned half = static_cast<unsigned>(j >> 1) & 1u;
      if (!at_wait(&vfull[s], static_cast<unsigned>(j / S::kStages) & 1u, fault)) return false;
      if (patch >= 0 && !at_wait(&patched[patch % kPatchRing], static_cast<unsigned>(patch / kPatchRing) & 1u, fault))
        return false;
      if (!at_wait(&pfull[d], half, fault) || !at_wait(&oempty[d], half ^ 1u, fault)) return false;
      tc_fence_after();
      if (leader) {
        const uint64_t b = operand(smem_addr(pbuf + 2 * d * S::kPHalf), 8 * R, R);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const uint64_t a = operand(smem_addr(vring + s * S::kSlot + p * kPanel), 1024, 128);
#pragma unroll
          for (int k = 0; k < 2 * kTile / 32; ++k)  // hi's 4 steps of 32 tokens, then lo's
            umma_e4m3(tmem_o + (d * NP + p) * R, a + static_cast<uint64_t>((k & 3) * (32 * 128 >> 4)),
                      b + static_cast<uint64_t>((k >> 2) * (S::kPHalf >> 4) + (k & 3) * (32 * R >> 4)), idesc_o, k != 0);
        }
        umma_commit(&ofull[d]);
        umma_commit(&vempty[s]);
        umma_commit(&pempty[d]);
      }
      __syncwarp();
      return true;
    };
    while (ok && w.next(P)) {
      if (w.keys == 0) continue;
      const int special = w.first_special(), qb = qn & 1;
      ok = at_wait(&qfull[qb], static_cast<unsigned>(qn >> 1) & 1u, fault);
      for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
        const int s = it % S::kStages, d = it & 1;
        ok = at_wait(&kfull[s], static_cast<unsigned>(it / S::kStages) & 1u, fault) &&
             at_wait(&sempty[d], (static_cast<unsigned>(it >> 1) & 1u) ^ 1u, fault);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint64_t a = operand(smem_addr(kring + s * S::kSlot), 1024, 128);
          const uint64_t b = operand(smem_addr(qbuf + 2 * qb * S::kQHalf), 1024, 128);
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < 4 * NP; ++k)
              if (k < steps)
                umma_e4m3(tmem_sc + d * R, a + static_cast<uint64_t>((k >> 2) * (kPanel >> 4) + (k & 3) * 2),
                          b + static_cast<uint64_t>(half * (S::kQHalf >> 4) + (k >> 2) * (R * 128 >> 4) + (k & 3) * 2),
                          idesc_s, half != 0 || k != 0);
          umma_commit(&sfull[d]);
          umma_commit(&kempty[s]);
          mbar_arrive(&sfull[d]);  // what the copies' and queries' warps wrote is visible behind it
        }
        __syncwarp();
        if (t >= special) {
          // (a warp that comes to a barrier's phase two phases early would pass: the
          // patching warps, which skip tiles, are told when their tile's V is there)
          ok = at_wait(&vfull[s], static_cast<unsigned>(it / S::kStages) & 1u, fault);
          if (!ok) break;
          if (leader) mbar_arrive(&landed[patches % kPatchRing]);
        }
        if (it > 0) ok = outputs(it - 1, last_patch);
        last_patch = t >= special ? patches++ : -1;
      }
      ++qn;
    }
    if (ok && it > 0) ok = outputs(it - 1, last_patch);
    // every product issued has completed before tensor memory is released
    if (leader) umma_commit(&drain);
    __syncwarp();
    mbar_wait(&drain, 0);
  } else if (warp < 4) {
    // ---------------- queries, masks, what no row sees ----------------
    const int me = tid - 64;
    constexpr int kLanes = 16 * NP;          // lanes of a row, 8 elements each
    constexpr int kAtOnce = 64 / kLanes;     // rows of the two warps at a time
    const auto prepare = [&](const Walk<R>& x, int n) {
      const int qb = n & 1;
      if (!at_wait(&qempty[qb], (static_cast<unsigned>(n >> 1) & 1u) ^ 1u, fault)) return false;
      unsigned char* dst = qbuf + 2 * qb * S::kQHalf;
      const int row0 = x.row0(), tok0 = row0 / P.G, d0 = lane % kLanes * 8;
      constexpr int kBatch = R / kAtOnce < 8 ? R / kAtOnce : 8;
#pragma unroll 1
      for (int r1 = 0; r1 < R; r1 += kBatch * kAtOnce) {
        uint4 raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = r1 + i * kAtOnce + me / kLanes, row = row0 + r, tok = row / P.G, g = row % P.G;
          raw[i] = make_uint4(0, 0, 0, 0);
          if (tok < x.s.count && d0 < P.D)
            raw[i] = *reinterpret_cast<const uint4*>(P.q + x.b * P.q_ld[0] + tok * P.q_ld[1] +
                                                     (x.h * P.G + g) * P.q_ld[2] + d0);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = r1 + i * kAtOnce + me / kLanes;
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          float v[8], most = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = e & 1 ? bf16_hi(u[e / 2]) : bf16_lo(u[e / 2]);
            if (fabsf(v[e]) < kInf) most = fmaxf(most, fabsf(v[e]));
            else v[e] = __uint_as_float(0x7fc00000u);
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          // the least exponent with most <= 448 2^eq
          const uint32_t bits = __float_as_uint(most);
          int eq = static_cast<int>(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
          eq = max(eq, -100);
          const float f = exp2i(-eq);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = v[2 * e] * f, c = v[2 * e + 1] * f;
            hi[e] = pack_e4m3(a, c);
            const float2 back = unpack_e4m3(hi[e]);
            lo[e] = pack_e4m3(a - back.x, c - back.y);
          }
          const uint32_t at = (d0 >> 7) * R * 128 + swizzled(r * 128 + (d0 & 127), 128);
          *reinterpret_cast<uint2*>(dst + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2*>(dst + S::kQHalf + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          if (d0 == 0) {
            cq_s[qb][r] = exp2i(eq) * P.c;
            token_s[qb][r] = static_cast<unsigned char>((row0 + r) / P.G - tok0);
          }
        }
      }
      if (P.parent) {
        // which of the block's rows' tokens see drafted token j
        unsigned long long* mask = mask_s + qb * kMaxRows;
        const int* parent = P.parent + static_cast<long long>(x.b) * P.n;
        bool bad = false;
        for (int j = me; j < x.s.count; j += 64) {
          int p = j ? __ldg(parent + j) : 0;
          if (j && (p < 0 || p >= j)) {
            bad = true;
            p = 0;
          }
          parent_s[j] = static_cast<unsigned short>(p);
          mask[j] = 0;
        }
        if (bad && x.h == 0) report(P, x.b, SPEC_ERR_PARENT);
        if (!meet(&parent_met[0], static_cast<unsigned>(n) & 1u, leader, fault)) return false;
        const int tok = tok0 + me;
        if (tok < x.s.count && tok * P.G < row0 + R) {
          const unsigned long long bit = 1ull << me;
          for (int j = tok;; j = parent_s[j]) {
            atomicOr(mask + j, bit);
            if (j == 0) break;
          }
        }
        if (!meet(&parent_met[1], static_cast<unsigned>(n) & 1u, leader, fault)) return false;
      }
      fence_proxy_async();
      __syncwarp();
      if (leader) mbar_arrive(&qfull[qb]);
      return true;
    };
    Walk<R> ahead = w;
    int qn = 0, it = 0, patches = 0;
    bool ok = true;
    const auto next_full = [&](Walk<R>& x) {
      while (x.next(P))
        if (x.keys) return true;
      return false;
    };
    bool more = next_full(ahead);
    if (more) ok = prepare(ahead, qn++);
    while (ok && next_full(w)) {
      if (more) more = next_full(ahead);
      if (more) ok = prepare(ahead, qn++);
      const int special = w.first_special();
      it += w.t1 - w.t0;
      for (int t = max(w.t0, special); ok && t < w.t1; ++t, ++patches) {
        const int j = it - (w.t1 - t), s = j % S::kStages;
        ok = at_wait(&landed[patches % kPatchRing], static_cast<unsigned>(patches / kPatchRing) & 1u, fault) &&
             at_wait(&vfull[s], static_cast<unsigned>(j / S::kStages) & 1u, fault);
        if (!ok) break;
        for (int row = me; row < kTile; row += 64) {
          const int pos = t * kTile + row;
          unsigned char* v = vring + s * S::kSlot + row * 128;
          bool clear = pos >= w.keys, nan = false;
          if (!clear && pos >= w.s.prefix) {
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
              for (int o = 0; o < 128; o += 16) {
                const uint4 x = *reinterpret_cast<const uint4*>(v + p * kPanel + o);
                const uint32_t m = 0x7f7f7f7fu, one = 0x01010101u;
                nan |= ((((x.x & m) + one) | ((x.y & m) + one) | ((x.z & m) + one) | ((x.w & m) + one)) & 0x80808080u) != 0;
              }
            clear = nan;
          }
          if (clear) {
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
              for (int o = 0; o < 128; o += 16) *reinterpret_cast<uint4*>(v + p * kPanel + o) = make_uint4(0, 0, 0, 0);
          }
          nan_s[patches % kPatchRing][row] = nan;
        }
        fence_proxy_async();
        __syncwarp();
        if (leader) mbar_arrive(&patched[patches % kPatchRing]);
      }
    }
  } else if (warp < 12) {
    // ---------------- weights ----------------
    const int grp = (warp - 4) >> 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    int it = 0, qn = 0, patches = 0;
    bool ok = true;
    while (ok && w.next(P)) {
      if (w.keys == 0) continue;
      const int special = w.first_special(), qb = qn & 1, tok0 = w.row0() / P.G;
      for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
        const int patch = t >= special ? patches++ : -1;
        if ((it & 1) != grp) continue;
        const unsigned half = static_cast<unsigned>(it >> 1) & 1u;
        ok = at_wait(&sfull[grp], half, fault);
        if (!ok) break;
        tc_fence_after();
        float y[R];
        tmem_columns<R>(tmem_sc + grp * R + lanes, y);
        tc_fence_before();
        __syncwarp();
        if (leader) mbar_arrive(&sempty[grp]);
        const PageScale ps = scale_s[it % kScaleRing][row / P.page];
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 c = *reinterpret_cast<const float4*>(&cq_s[qb][r]);
          y[r] = __fmaf_rn(y[r] * c.x, ps.ck, ps.ve);
          y[r + 1] = __fmaf_rn(y[r + 1] * c.y, ps.ck, ps.ve);
          y[r + 2] = __fmaf_rn(y[r + 2] * c.z, ps.ck, ps.ve);
          y[r + 3] = __fmaf_rn(y[r + 3] * c.w, ps.ck, ps.ve);
        }
        if (patch >= 0) {
          ok = at_wait(&patched[patch % kPatchRing], static_cast<unsigned>(patch / kPatchRing) & 1u, fault);
          if (!ok) break;
          const int pos = t * kTile + row, j = pos - w.s.prefix;
          unsigned long long seen = ~0ull;
          if (pos >= w.keys) seen = 0;
          else if (j >= 0 && P.parent) seen = mask_s[qb * kMaxRows + j];
          else if (j > tok0) seen = j - tok0 > 63 ? 0 : ~0ull << (j - tok0);
          const bool nan = nan_s[patch % kPatchRing][row];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (nan) y[r] = __uint_as_float(0x7fc00000u);
            if (!(seen >> token_s[qb][r] & 1ull)) y[r] = -kInf;
          }
        }
        // the columns' largest
        float keep[R / 32 + 1];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float m = warp_max(y[r]);
          if ((r & 31) == 0 || lane == (r & 31)) keep[r / 32] = m;
        }
        ok = at_wait(&mempty[grp], half ^ 1u, fault);
        if (!ok) break;
#pragma unroll
        for (int r = 0; r < R; r += 32)
          if (r + lane < R) most_s[grp][q][r + lane] = keep[r / 32];
        ok = meet(&most_met[grp], half, leader, fault);
        if (!ok) break;
        if (row < R) {
          const float m = fmaxf(fmaxf(most_s[grp][0][row], most_s[grp][1][row]),
                                fmaxf(most_s[grp][2][row], most_s[grp][3][row]));
          top_s[grp][row] = m - 8.f;
          ref_s[grp][row] = m == -kInf ? 0.f : m - 8.f;
        }
        ok = meet(&ref_met[grp], half, leader, fault);
        if (!ok) break;
        float e[R];
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 c = *reinterpret_cast<const float4*>(&ref_s[grp][r]);
          e[r] = ex2(y[r] - c.x);
          e[r + 1] = ex2(y[r + 1] - c.y);
          e[r + 2] = ex2(y[r + 2] - c.z);
          e[r + 3] = ex2(y[r + 3] - c.w);
        }
        ok = at_wait(&pempty[grp], half ^ 1u, fault);
        if (!ok) break;
        unsigned char* p = pbuf + 2 * grp * S::kPHalf;
#pragma unroll
        for (int r = 0; r < R; r += 16) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) split2(e[r + 2 * i], e[r + 2 * i + 1], hi[i], lo[i]);
          const uint32_t at = swizzled(row * R + r, R);
          *reinterpret_cast<uint4*>(p + at) =
              make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, hi[4] | hi[5] << 16, hi[6] | hi[7] << 16);
          *reinterpret_cast<uint4*>(p + S::kPHalf + at) =
              make_uint4(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16, lo[4] | lo[5] << 16, lo[6] | lo[7] << 16);
        }
        fence_proxy_async();
        __syncwarp();
        if (leader) mbar_arrive(&pfull[grp]);
        // the sums of the weights themselves: without the values' exponents
        if (!ps.far) {
          const float f = exp2i(-static_cast<int>(ps.ve));
#pragma unroll
          for (int r = 0; r < R; ++r) e[r] *= f;
        } else {
          // (2^(y - reference) may underflow where a page's values are tiny against another's)
#pragma unroll
          for (int r = 0; r < R; ++r) e[r] = ex2((y[r] - ref_s[grp][r]) - ps.ve);
        }
        constexpr int kSum = R < 32 ? R : 32;
#pragma unroll
        for (int r = 0; r < R; r += kSum) {
          const float s = column_sums<kSum>(e + r, lane);
          if (lane < kSum) sum_s[grp][q][r + lane] = s;
        }
        __syncwarp();
        if (leader) mbar_arrive(&mfull[grp]);
      }
      ++qn;
    }
  } else {
    // ---------------- outputs ----------------
    const int q = warp & 3, d = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    int it = 0, qn = 0;
    unsigned whole = 0;
    bool ok = true;
    while (ok && w.next(P)) {
      if (w.keys == 0) {
        if (w.s.bad || w.s.count < P.n) {
          // rows of nothing
          for (int r = 0; r < R && w.row0() + r < P.n * P.G; ++r) {
            bf16_t* out = P.out + w.b * P.out_ld[0] + (w.row0() + r) / P.G * P.out_ld[1] +
                          (w.h * P.G + (w.row0() + r) % P.G) * P.out_ld[2];
            for (int e = d; e < P.D; e += 128) out[e] = 0;
          }
        }
        if (w.s.bad && w.h == 0 && w.block == 0 && d == 0) report(P, w.b, SPEC_ERR_CACHE);
        continue;
      }
      float acc[NP][R];
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[p][r] = 0.f;
      // row d's: log2 of the unit of acc, the sum of weights and log2 of its unit
      float unit = -kInf, sum = 0.f, sum_unit = -kInf;
      for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
        const int k = it & 1;
        const unsigned half = static_cast<unsigned>(it >> 1) & 1u;
        ok = at_wait(&mfull[k], half, fault);
        if (!ok) break;
        if (d < R) {
          const float top = top_s[k][d];
          const float s = (sum_s[k][0][d] + sum_s[k][1][d]) + (sum_s[k][2][d] + sum_s[k][3][d]);
          const float next = fmaxf(unit, top), ref = next == -kInf ? 0.f : next;
          mix_s[k][d] = make_float2(unit == -kInf ? 0.f : ex2(unit - ref), top == -kInf ? 0.f : ex2(top - ref));
          unit = next;
          if (s != 0.f) {  // (a NaN too)
            // s = part 2^power; the sums' unit is the largest 2^(top + power) so far
            const int power = static_cast<int>(__float_as_uint(s) >> 23 & 255u) - 127;
            const float su = (top == -kInf ? 0.f : top) + static_cast<float>(power);
            const float sn = fmaxf(sum_unit, su);
            sum = (sum_unit == -kInf ? 0.f : sum * ex2(sum_unit - sn)) + s * exp2i(min(126, max(-126, -power))) * ex2(su - sn);
            sum_unit = sn;
          }
        }
        __syncwarp();
        if (leader) mbar_arrive(&mempty[k]);
        ok = meet(&mix_met[k], half, leader, fault) && at_wait(&ofull[k], half, fault);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          if (p * 128 + q * 32 >= P.D) break;
          float o[R];
          tmem_columns<R>(tmem_o + (k * NP + p) * R + lanes, o);
#pragma unroll
          for (int r = 0; r < R; r += 2) {
            const float4 m = *reinterpret_cast<const float4*>(&mix_s[k][r]);
            acc[p][r] = __fmaf_rn(o[r], m.y, acc[p][r] * m.x);
            acc[p][r + 1] = __fmaf_rn(o[r + 1], m.w, acc[p][r + 1] * m.z);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (leader) mbar_arrive(&oempty[k]);
      }
      if (!ok) break;
      if (leader) mbar_arrive(&qempty[qn & 1]);
      ++qn;
      if (w.t0 == 0 && w.t1 == w.tiles) {
        if (d < R) row_s[d] = sum == 0.f ? 0.f : ex2(unit - sum_unit) / sum;
        ok = meet(&row_met[0], whole & 1u, leader, fault);
        if (!ok) break;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int row = w.row0() + r, tok = row / P.G;
          if (tok >= P.n) break;
          bf16_t* out = P.out + w.b * P.out_ld[0] + tok * P.out_ld[1] + (w.h * P.G + row % P.G) * P.out_ld[2];
          const float f = row_s[r];
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            unsigned short bits;
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(tok < w.s.count ? acc[p][r] * f : 0.f));
            if (p * 128 + d < P.D) out[p * 128 + d] = bits;
          }
        }
        ok = meet(&row_met[1], whole++ & 1u, leader, fault);
      } else {
        constexpr int kLd = NP * 128 + 4;
        float* part = P.parts + (static_cast<long long>(2 * cta) + (w.t0 == 0 ? 1 : 0)) * R * kLd;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int p = 0; p < NP; ++p) __stcg(part + r * kLd + p * 128 + d, acc[p][r]);
        if (d < R) {
          float* end = part + d * kLd + NP * 128;
          __stcg(end, unit);
          __stcg(end + 1, sum);
          __stcg(end + 2, sum_unit);
        }
      }
    }
    // the block that this CTA begins and others end
    if (ok && d == 0 && cta < ctas) {
      int4 x = make_int4(0, 0, 0, 0);
      if (u1 > u0 && w.t0 == 0 && w.t1 < w.tiles) {
        const long long last = u1 + (w.tiles - w.t1) - 1;  // the block's last tile
        x = make_int4(w.b, w.h, w.block, static_cast<int>(((last + 1) * ctas - 1) / total) - cta + 1);
      }
      P.shared[cta] = x;
    }
  }

  __syncthreads();
  if (*fault && tid == 0) {
    // copies still in flight land before the CTA exits: wait (bounded) for
    // the last phase of every stage that was issued
    for (int k = max(0, k_issued_s - S::kStages); k < k_issued_s; ++k)
      mbar_wait(&kfull[k % S::kStages], static_cast<unsigned>(k / S::kStages) & 1u);
    for (int k = max(0, v_issued_s - S::kStages); k < v_issued_s; ++k)
      mbar_wait(&vfull[k % S::kStages], static_cast<unsigned>(k / S::kStages) & 1u);
    if (P.error_word) atomicOr(P.error_word, SPEC_ERR_INTERNAL);
    P.shared[cta] = make_int4(0, 0, 0, 0);
  }
  if (tid == 0 && cta >= ctas) P.shared[cta] = make_int4(0, 0, 0, 0);
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_s, S::kTmemCols);
  }
}

// The blocks that several CTAs share: CTA (x, y) joins rows 4 y .. 4 y + 3 of
// the one that attend CTA x begins, its parts in the order of the tokens.
template <int R, int NP>
__global__ void __launch_bounds__(128) join_kernel(const AttendParams P) {
  constexpr int kLd = NP * 128 + 4;
  pdl_wait();
  const int4 it = __ldcg(P.shared + blockIdx.x);
  if (it.w == 0) return;
  const int d = threadIdx.x;
  const Lengths s = lengths_of(P, it.x);
  for (int r = blockIdx.y * 4; r < blockIdx.y * 4 + 4; ++r) {
    const int row = it.z * R + r, tok = row / P.G;
    if (tok >= P.n) return;
    bf16_t* out = P.out + it.x * P.out_ld[0] + tok * P.out_ld[1] + (it.y * P.G + row % P.G) * P.out_ld[2];
    if (tok >= s.count) {
      for (int e = d; e < P.D; e += 128) out[e] = 0;
      continue;
    }
    const auto part = [&](int i) {
      return P.parts + (static_cast<long long>(2 * (blockIdx.x + i)) + (i == 0 ? 1 : 0)) * R * kLd + r * kLd;
    };
    float unit = -kInf, sum_unit = -kInf;
    for (int i = 0; i < it.w; ++i) {
      const float* e = part(i) + NP * 128;
      unit = fmaxf(unit, __ldcg(e));
      sum_unit = fmaxf(sum_unit, __ldcg(e + 2));
    }
    float acc[NP], sum = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) acc[p] = 0.f;
    for (int i = 0; i < it.w; ++i) {
      const float* e = part(i);
      const float u = __ldcg(e + NP * 128), su = __ldcg(e + NP * 128 + 2);
      const float f = u == -kInf ? 0.f : ex2(u - unit);
      if (su != -kInf) sum += __ldcg(e + NP * 128 + 1) * ex2(su - sum_unit);
#pragma unroll
      for (int p = 0; p < NP; ++p) acc[p] = __fmaf_rn(__ldcg(e + p * 128 + d), f, acc[p]);
    }
    const float f = sum == 0.f ? 0.f : ex2(unit - sum_unit) / sum;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      unsigned short bits;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(acc[p] * f));
      if (p * 128 + d < P.D) out[p * 128 + d] = bits;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool good_shape(int B, int n, int Hq, int H, int D) {
  return B >= 1 && B <= 65535 && n >= 1 && n <= kMaxRows && H >= 1 && Hq >= H && Hq <= 1024 && Hq % H == 0 &&
         D >= 16 && D <= 256 && D % 16 == 0;
}

int block_rows(int n, int G, int D) {
  const int rows = n * G;
  return rows <= 16 ? 16 : rows <= 32 || D > 128 ? 32 : 64;
}

size_t attend_workspace(int n, int Hq, int H, int D) {
  const int R = block_rows(n, Hq / H, D), ld = (D > 128 ? 256 : 128) + 4;
  return align256(kMaxCtas * sizeof(int4)) + static_cast<size_t>(2) * kMaxCtas * R * ld * sizeof(float);
}

// Codes as rows of D bytes: boxes of a page's tokens x 128 elements, 128-byte swizzle, zeros beyond D.
bool code_map(CUtensorMap* map, const void* base, long long rows, int D, int page) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(page)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel's dynamic shared memory limit, raised once per device.
template <int R, int NP>
cudaError_t raise_smem() {
  static std::mutex mu;
  static std::map<int, bool> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (done.count(dev)) return cudaSuccess;
  e = cudaFuncSetAttribute(attend_kernel<R, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<R, NP>::kSmem);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

// Test hook (spec_test_inject_cache_copy_timeout): nonzero makes every tile
// wait for 16 bytes that never come, so that the bounded waits of the roles
// behind it give up.  Zero in normal operation.
std::atomic<unsigned> g_more_bytes{0};

template <int R, int NP>
spec_status launch_attend(const spec_attend_args& a, AttendParams& p, cudaStream_t s) {
  const int nsm = sm_count();
  if (nsm < 1) return SPEC_ECUDA;
  const long long rows = static_cast<long long>(a.pages) * a.H * a.page;
  CUtensorMap tk, tv;
  if (!code_map(&tk, a.k_codes, rows, a.D, a.page) || !code_map(&tv, a.v_codes, rows, a.D, a.page)) return SPEC_ECUDA;
  if (raise_smem<R, NP>() != cudaSuccess) return SPEC_ECUDA;
  p.blocks = (a.n * p.G + R - 1) / R;
  p.more_bytes = g_more_bytes.load();
  const int ctas = std::min(nsm, kMaxCtas);
  attend_kernel<R, NP><<<ctas, kAttendThreads, Shape<R, NP>::kSmem, s>>>(tk, tv, p);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>((std::min(R, a.n * p.G) + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<R, NP>, static_cast<const AttendParams>(p)) == cudaSuccess ? SPEC_OK
                                                                                                       : SPEC_ECUDA;
}

}  // namespace
}  // namespace sv

extern "C" spec_status spec_test_inject_cache_copy_timeout(int enable) {
  sv::g_more_bytes = enable ? 16u : 0u;
  return SPEC_OK;
}

extern "C" size_t spec_attend_workspace_size(int B, int n, int Hq, int H, int D) {
  return sv::good_shape(B, n, Hq, H, D) ? sv::attend_workspace(n, Hq, H, D) : 0;
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
  if (!a->workspace || a->workspace_bytes < attend_workspace(a->n, a->Hq, a->H, a->D) || !aligned(a->workspace, 256))
    return SPEC_EWORKSPACE;
  AttendParams p{};
  p.B = a->B;
  p.n = a->n;
  p.Hq = a->Hq;
  p.H = a->H;
  p.G = a->Hq / a->H;
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
  p.k_exps = a->k_exps;
  p.v_exps = a->v_exps;
  p.seq_error = a->seq_error;
  p.error_word = a->error_word;
  p.shared = static_cast<int4*>(a->workspace);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + align256(kMaxCtas * sizeof(int4)));
  const int R = block_rows(a->n, p.G, a->D);
  if (a->D > 128) return R == 16 ? launch_attend<16, 2>(*a, p, stream) : launch_attend<32, 2>(*a, p, stream);
  switch (R) {
    case 16: return launch_attend<16, 1>(*a, p, stream);
    case 32: return launch_attend<32, 1>(*a, p, stream);
    default: return launch_attend<64, 1>(*a, p, stream);
  }
}
