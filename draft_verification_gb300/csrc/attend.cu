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
constexpr int kScaleRing = 16, kPatchRing = 8, kPieceRing = 4;
constexpr int kScores = 4;  // places of tiles' scores: those are two tiles ahead of the outputs, every group meets all phases of its places
constexpr int kFar = 30;  // value exponents of a tile that lie further apart than this

// R: a block's rows; NP: panels of 128 elements of a head.
template <int R, int NP>
struct Shape {
  // the softmax warpgroups: kGroups, each with kW of the block's rows, of every
  // tile or of every other one
  static constexpr int kW = R == 16 ? 8 : 16, kColumns = R / kW, kTurns = kColumns == 2 ? 2 : 1;
  static constexpr int kGroups = kColumns * kTurns;
  static constexpr int kThreads = 128 * (2 + kGroups);
  static constexpr int kStages = NP == 1 ? (R > 32 ? 4 : 5) : 2;
  static constexpr int kPRow = R == 48 ? 64 : R;  // bytes of a token's weights
  static constexpr int kSlot = NP * kPanel;
  static constexpr int kQHalf = NP * R * 128;  // hi or lo of a block's queries
  static constexpr int kPHalf = kTile * kPRow;  // hi or lo of a tile's weights
  static constexpr int kMaskBytes = 2 * kMaxRows * 8;
  static constexpr int kSmem = 1024 + 2 * kStages * kSlot + 4 * kQHalf + 4 * kPHalf + kMaskBytes + kMaxRows * 2;
  static constexpr int kCols = (kScores + 2 * NP) * R;
  static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512 && kStages + 3 <= kScaleRing && kStages < kPatchRing, "rings");
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
// the tiles of a call, in order: sequence, head, block, tile
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

// A piece of a block: what one CTA does of it.
struct Piece {
  int b, h, block, prefix;  // b < 0: no more
  int count, keys, t0, t1;  // keys: the tokens that the block's rows can see; t0, t1: the piece's tiles
  int part, pad[3];         // part: -1 all of the block, 1 its first tiles, 0 others
};
// From this tile on, rows differ in what they see, or see nothing at the end.
__device__ __forceinline__ int first_special(const Piece& w) {
  return w.count > 1 ? w.prefix / kTile : w.keys % kTile ? w.keys / kTile : 0x7fffffff;
}

// ---------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------

// Whole warps wait together (see int4_product.cu); a wait that gives up, here
// or elsewhere in the CTA, ends the role.
__device__ __forceinline__ bool at_wait(uint64_t* bar, unsigned parity, volatile int* fault) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
#pragma unroll 1
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

// The four warps of a warpgroup meet, and go on only if all of them can (so
// that they leave a role together when a wait gave up).
__device__ __forceinline__ bool meet(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(id)
      : "memory");
  return all != 0;
}

// Shared-memory matrix descriptor (tc.cuh has the bits) in two words: the
// address; the 8-row (K-major) or 8-step (MN-major) groups `stride` bytes
// apart and the swizzle of `row` bytes.
__device__ __forceinline__ uint32_t operand_low(uint32_t addr, uint32_t stride) {
  return ((addr >> 4) & 0x3FFFu) | (stride >> 4) << 16;
}
__host__ __device__ constexpr uint32_t operand_high(uint32_t stride, int row) {
  return (stride >> 4) | 1u << 14 | (row == 128 ? 2u : row == 64 ? 4u : row == 32 ? 6u : 0u) << 29;
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
// D[tmem] (+)= A B, M x N x 32, by the lane that `issues`.  The whole warp runs
// it: in a branch of one lane the operands would leave the uniform registers
// that the instruction takes, at some 50 cycles per product.
template <bool kAccumulate>
__device__ __forceinline__ void umma_e4m3(uint32_t issues, uint32_t d, uint32_t a, uint32_t a_high, uint32_t b,
                                          uint32_t b_high, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 da, db;\n mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n"
      " setp.ne.b32 p, %6, 0;\n setp.ne.b32 q, %7, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n}" ::"r"(d),
      "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(idesc), "n"(kAccumulate ? 1 : 0), "r"(issues)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t issues, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_addr(bar)),
      "r"(issues)
      : "memory");
}

// 8 consecutive float32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// N columns, a multiple of 8
template <int N>
__device__ __forceinline__ void tmem_columns(uint32_t at, float* v) {
  if constexpr (N >= 32) {
    tmem_ld32(at, v);
    if constexpr (N > 32) tmem_columns<N - 32>(at + 32, v + 32);
  } else if constexpr (N >= 16) {
    tmem_ld16(at, v);
    if constexpr (N > 16) tmem_columns<N - 16>(at + 16, v + 16);
  } else {
    tmem_ld8(at, v);
  }
}

// largest value of a warp (a NaN is passed over)
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// The warp's sums of N columns (N a power of two): lane i gets column i % N's.
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
#pragma unroll
  for (int o = N; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
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

__device__ __forceinline__ float4 lds_f4(const float* p) { return *reinterpret_cast<const float4*>(p); }

struct PageScale {
  float ck, ve;   // 2^key exponent (NaN: not a page), value exponent
  float ve_low;   // the tile's least value exponent
  int far;        // the tile's value exponents lie far apart
};

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int R, int NP>
__global__ void __launch_bounds__(Shape<R, NP>::kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const AttendParams P) {
  using S = Shape<R, NP>;
  constexpr int kW = S::kW, kFirstOut = 4 + 4 * S::kGroups;
  extern __shared__ __align__(1024) unsigned char at_dyn[];
  // full / empty: a tile's codes; sfull: its scores are there; pfull / pempty:
  // its weights in shared memory (its scores are read); ofull / oempty: its outputs;
  // mfull / mempty: its maxima (top_s); efull / eempty: a piece's sums of
  // weights; qfull / qempty: its queries; rfull / rempty: its record;
  // landed: a patched tile's V is there; patched: it is patched
  struct Bars {
    uint64_t full[S::kStages], empty[S::kStages];
    uint64_t sfull[kScores], pfull[2], pempty[2], ofull[2], oempty[2], mfull[2], mempty[2], efull[2], eempty[2];
    uint64_t qfull[2], qempty[2], landed[kPatchRing], patched[kPatchRing], rfull[kPieceRing], rempty[kPieceRing], drain;
  };
  constexpr int kBars = sizeof(Bars) / 8;
  __shared__ Bars bar;
  __shared__ uint32_t tmem_s;
  __shared__ int fault_s, issued_s;
  __shared__ __align__(16) Piece piece_s[kPieceRing];
  __shared__ __align__(16) PageScale scale_s[kScaleRing][8];
  __shared__ __align__(16) float most_s[S::kGroups][2][4][kW], most_x_s[S::kGroups][4][kW];
  __shared__ __align__(16) float ref_s[4 * S::kGroups][3][kW], cq_s[2][R], top_s[2][R], sum_s[2][S::kTurns][4][R];
  __shared__ __align__(16) float2 mix_s[2][R];
  __shared__ float sum_unit_s[2][S::kTurns][R];
  __shared__ __align__(16) float row_s[R];
  __shared__ long long place_s[R];
  __shared__ unsigned char token_s[2][R];
  __shared__ unsigned nan_s[kPatchRing][kTile / 32];

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
  if (tid < kBars) {
    uint64_t* at = reinterpret_cast<uint64_t*>(&bar) + tid;
    unsigned count = 1;
    if (at >= bar.pfull && at < bar.pempty) count = 4 * S::kColumns;  // pfull
    if (at >= bar.oempty && at < bar.mfull) count = 4;            // oempty
    if (at >= bar.sfull && at < bar.pfull) count = 2;             // sfull
    if (at >= bar.mfull && at < bar.mempty) count = S::kColumns;  // mfull
    if (at >= bar.mempty && at < bar.efull) count = 4;            // mempty
    if (at >= bar.efull && at < bar.eempty) count = 4 * S::kGroups;  // efull
    if (at >= bar.eempty && at < bar.qfull) count = 4;            // eempty
    if (at >= bar.qempty && at < bar.landed) count = 4;           // qempty
    if (at >= bar.rempty && at < &bar.drain) count = 7 + 4 * S::kGroups;  // rempty
    mbar_init(at, count);
    mbar_fence_init();
  }
  if (tid == 0) fault_s = issued_s = 0;
  if (warp == 1) {
    tmem_alloc(&tmem_s, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_sc = tmem_s, tmem_o = tmem_s + kScores * R;

  // the next piece, for all roles but the one that makes them
  int pieces = 0;
  const auto next_piece = [&](Piece& w) {
    const int s = pieces % kPieceRing;
    if (!at_wait(&bar.rfull[s], static_cast<unsigned>(pieces / kPieceRing) & 1u, fault)) return false;
    w = piece_s[s];
    // (a shuffle makes a warp's value uniform to the compiler as well)
    w.b = __shfl_sync(0xffffffffu, w.b, 0);
    w.keys = __shfl_sync(0xffffffffu, w.keys, 0);
    w.prefix = __shfl_sync(0xffffffffu, w.prefix, 0);
    w.count = __shfl_sync(0xffffffffu, w.count, 0);
    w.t0 = __shfl_sync(0xffffffffu, w.t0, 0);
    w.t1 = __shfl_sync(0xffffffffu, w.t1, 0);
    if (leader) mbar_arrive(&bar.rempty[s]);
    ++pieces;
    return w.b >= 0;
  };

  if (warp == 0) {
    // ---------------- pages ----------------
    const int pp = kTile / P.page, slot_in = lane % pp, mine = lane / pp, batch = 32 / pp;
    const unsigned page_bytes = static_cast<unsigned>(P.page) * 128u;
    int it = 0;
    bool ok = true;
    Piece w;
    while (ok && next_piece(w)) {
      const int* table = P.block_table + static_cast<long long>(w.b) * P.table_pages;
      // the pages of `batch` tiles, a lane each
      const auto has_page = [&](int tb) { return tb + mine < w.t1 && ((tb + mine) * pp + slot_in) * P.page < w.keys; };
      int ahead = has_page(w.t0) ? __ldg(table + (w.t0 + mine) * pp + slot_in) : 0;
#pragma unroll 1
      for (int tb = w.t0; ok && tb < w.t1; tb += batch) {
        const bool has = has_page(tb);
        int page = ahead;
        const bool bad = has && (page < 0 || page >= P.pages);
        if (bad) report(P, w.b, SPEC_ERR_CACHE);
        if (!has || bad) page = 0;
        const long long slab = static_cast<long long>(page) * P.H + w.h;
        int ke = 0, ve = 0;
        if (has && !bad) {
          ke = __ldg(P.k_exps + slab);
          ve = __ldg(P.v_exps + slab);
        }
        if (has_page(tb + batch)) ahead = __ldg(table + (tb + batch + mine) * pp + slot_in);
        int lo = has ? ve : 127, hi = has ? ve : -127;
        for (int o = 1; o < pp; o <<= 1) {
          lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        PageScale x;
        x.ck = bad ? __uint_as_float(0x7fc00000u) : exp2i(ke);
        x.ve = static_cast<float>(ve);
        x.ve_low = static_cast<float>(lo);
        x.far = hi - lo > kFar;
        const unsigned groups = __ballot_sync(0xffffffffu, has);
        const int y = static_cast<int>(slab * P.page);
#pragma unroll 1
        for (int i = 0; i < batch && tb + i < w.t1; ++i, ++it) {
          const int s = it % S::kStages;
          const unsigned parity = (static_cast<unsigned>(it / S::kStages) & 1u) ^ 1u;
          const unsigned bytes = static_cast<unsigned>(__popc(groups >> (i * pp) & ((1u << pp) - 1u))) * page_bytes * 2 * NP +
                                 P.more_bytes;
          unsigned char* dst = kring + s * S::kSlot + slot_in * page_bytes;
          ok = at_wait(&bar.empty[s], parity, fault);
          if (!ok) break;
          if (mine == i) scale_s[it % kScaleRing][slot_in] = x;
          __syncwarp();
          if (leader) mbar_expect_tx(&bar.full[s], bytes);
          __syncwarp();
          if (mine == i && has) {
#pragma unroll
            for (int p = 0; p < NP; ++p) tma_load_2d(dst + p * kPanel, &tm_k, p * 128, y, &bar.full[s]);
#pragma unroll
            for (int p = 0; p < NP; ++p)
              tma_load_2d(dst + S::kStages * S::kSlot + p * kPanel, &tm_v, p * 128, y, &bar.full[s]);
          }
          __syncwarp();
          if (leader) issued_s = it + 1;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- products ----------------
    constexpr uint32_t idesc_s = idesc_e4m3(kTile, R, 0, 0), idesc_o = idesc_e4m3(128, R, 1, 1);
    const int steps = (P.D + 31) / 32;
    int it = 0, qn = 0, patches = 0;
    bool ok = true;
    const uint32_t issues = leader ? 1u : 0u;
    // the outputs of tile j
    const auto outputs = [&](int j, int patch) {
      const int s = j % S::kStages, d = j & 1;
      const unsigned half = static_cast<unsigned>(j >> 1) & 1u;
      if (patch >= 0 && !at_wait(&bar.patched[patch % kPatchRing], static_cast<unsigned>(patch / kPatchRing) & 1u, fault))
        return false;
      if (!at_wait(&bar.oempty[d], half ^ 1u, fault) || !at_wait(&bar.pfull[d], half, fault)) return false;
      tc_fence_after();
      const uint32_t b = operand_low(smem_addr(pbuf + 2 * d * S::kPHalf), 8 * S::kPRow);
      constexpr uint32_t a_high = operand_high(1024, 128), b_high = operand_high(8 * S::kPRow, S::kPRow);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const uint32_t a = operand_low(smem_addr(vring + s * S::kSlot + p * kPanel), 1024), o = tmem_o + (d * NP + p) * R;
        umma_e4m3<false>(issues, o, a, a_high, b, b_high, idesc_o);
#pragma unroll
        for (int k = 1; k < 2 * kTile / 32; ++k)  // hi's 4 steps of 32 tokens, then lo's
          umma_e4m3<true>(issues, o, a + (k & 3) * (32 * 128 >> 4), a_high,
                          b + (k >> 2) * (S::kPHalf >> 4) + (k & 3) * (32 * S::kPRow >> 4), b_high, idesc_o);
      }
      commit_if(issues, &bar.ofull[d]);
      commit_if(issues, &bar.empty[s]);
      commit_if(issues, &bar.pempty[d]);
      return true;
    };
    // one loop over the tiles, scores two tiles ahead of the outputs
    Piece w;
    bool more = next_piece(w);
    int t = more ? w.t0 : 0, special = more ? first_special(w) : 0;
    int sb = 0, patch0 = -1, patch1 = -1;  // place of the scores; the last two tiles' among the patched ones
    constexpr int kUnknown = 0x40000000;
    int end = kUnknown;  // the number of tiles, once it is known
    for (; it < end + 2; ++it) {
      int patch = -1;
      // (where a piece's queries, or the codes' place, wait for the outputs of the tile two before: those first)
      const bool outputs_first = more && (t == w.t0 || S::kStages == 2);
#pragma unroll 1
      for (int turn = 0; turn < 2 && ok; ++turn) {
        if ((turn == 0) == outputs_first) {
          if (it > 1) ok = outputs(it - 2, patch1);
        } else if (more) {
          const int s = it % S::kStages;
          if (t == w.t0) ok = at_wait(&bar.qfull[qn & 1], static_cast<unsigned>(qn >> 1) & 1u, fault);
          ok = ok && at_wait(&bar.full[s], static_cast<unsigned>(it / S::kStages) & 1u, fault);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = operand_low(smem_addr(kring + s * S::kSlot), 1024), d = tmem_sc + sb * R;
          const uint32_t b = operand_low(smem_addr(qbuf + 2 * (qn & 1) * S::kQHalf), 1024);
          constexpr uint32_t high = operand_high(1024, 128);
          umma_e4m3<false>(issues, d, a, high, b, high, idesc_s);
#pragma unroll
          for (int k = 1; k < 8 * NP; ++k) {  // hi's steps of 32 elements, then lo's
            const int step = k % (4 * NP);
            if (step < steps)
              umma_e4m3<true>(issues, d, a + (step >> 2) * (kPanel >> 4) + (step & 3) * 2, high,
                              b + k / (4 * NP) * (S::kQHalf >> 4) + (step >> 2) * (R * 128 >> 4) + (step & 3) * 2, high,
                              idesc_s);
          }
          commit_if(issues, &bar.sfull[sb]);
          if (leader) mbar_arrive(&bar.sfull[sb]);  // what the copies' and queries' warps wrote is visible behind it
          if (t >= special) {
            // (a warp that comes to a barrier's phase two phases early would pass: the
            // patching warp, which skips tiles, is told when its tile is there)
            patch = patches++;
            if (leader) mbar_arrive(&bar.landed[patch % kPatchRing]);
          }
          __syncwarp();
          sb = sb == kScores - 1 ? 0 : sb + 1;
        }
      }
      if (!ok) break;
      patch1 = patch0;
      patch0 = patch;
      if (more && ++t == w.t1) {
        ++qn;
        more = next_piece(w);
        if (more) {
          t = w.t0;
          special = first_special(w);
        } else {
          end = it + 1;
        }
      } else if (!more && end == kUnknown) {
        break;  // (no tiles at all)
      }
    }
    // every product issued has completed before tensor memory is released
    if (leader) umma_commit(&bar.drain);
    __syncwarp();
    mbar_wait(&bar.drain, 0);
  } else if (warp == 2) {
    // ---------------- pieces, queries, masks ----------------
    const auto lengths = [&](int b) { return lengths_of(P, b); };
    const auto tiles_of_seq = [&](const Lengths& s) {
      int n = 0;
#pragma unroll 1
      for (int i = 0; i < P.blocks; ++i) n += tiles_of(keys_of<R>(P, s, i));
      return n * P.H;
    };
    int total = 0;
#pragma unroll 1
    for (int b = lane; b < P.B; b += 32) total += tiles_of_seq(lengths(b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    // equal runs: `more` CTAs have one tile more than the others
    const int ctas = min(static_cast<int>(gridDim.x), total), cta = blockIdx.x;
    const int each = total / ctas, more = total - each * ctas;
    const auto first_tile = [&](int c) { return each * c + min(c, more); };
    const int u0 = first_tile(min(cta, ctas)), u1 = first_tile(min(cta + 1, ctas));
    int left = u1 - u0;
    // the sequence of tile u0, and the tile's place in it
    int b = 0, offset = 0;
    if (left > 0) {
      int before = 0;
#pragma unroll 1
      for (int b1 = 0;; b1 += 32) {
        const int n = b1 + lane < P.B ? tiles_of_seq(lengths(b1 + lane)) : 0;
        int up = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, up, o);
          if (lane >= o) up += x;
        }
        const unsigned over = __ballot_sync(0xffffffffu, before + up > u0);
        if (over) {
          const int l = __ffs(over) - 1;
          b = b1 + l;
          offset = u0 - before - __shfl_sync(0xffffffffu, up - n, l);
          break;
        }
        before += __shfl_sync(0xffffffffu, up, 31);
      }
    }
    Lengths s = lengths(b);
    int h = 0, block = 0, keys = 0, tiles = 0, t1 = 0;
    if (left > 0) {
      const int per = tiles_of_seq(s) / P.H;
      h = offset / per;
      offset -= h * per;
#pragma unroll 1
      for (;; ++block) {
        keys = keys_of<R>(P, s, block);
        tiles = tiles_of(keys);
        if (offset < tiles) break;
        offset -= tiles;
      }
      t1 = offset;
    }
    int4 shared = make_int4(0, 0, 0, 0);
    int qn = 0, made = 0;
    bool ok = true;
#pragma unroll 1
    while (ok) {
      const bool last = left == 0;
      const int t0 = t1;
      if (!last) {
        t1 = min(tiles, t0 + left);
        left -= t1 - t0;
      }
      if (!last && keys == 0) {
        // rows of nothing (a block of one tile that no other role hears of)
#pragma unroll 1
        for (int r = block * R; r < min(block * R + R, P.n * P.G); ++r) {
          const int tok = r / P.G;
          bf16_t* out = P.out + b * P.out_ld[0] + tok * P.out_ld[1] + (h * P.G + r - tok * P.G) * P.out_ld[2];
          for (int e = lane; e < P.D; e += 32) out[e] = 0;
        }
        if (s.bad && h == 0 && block == 0 && leader) report(P, b, SPEC_ERR_CACHE);
      } else {
        const int rs = made % kPieceRing;
        ok = at_wait(&bar.rempty[rs], (static_cast<unsigned>(made / kPieceRing) & 1u) ^ 1u, fault);
        if (!ok) break;
        if (leader) {
          Piece w;
          w.b = last ? -1 : b;
          w.h = h;
          w.block = block;
          w.prefix = s.prefix;
          w.count = s.count;
          w.keys = keys;
          w.t0 = t0;
          w.t1 = t1;
          w.part = t0 == 0 ? (t1 == tiles ? -1 : 1) : 0;
          w.pad[0] = w.pad[1] = w.pad[2] = 0;
          piece_s[rs] = w;
        }
        __syncwarp();
        if (leader) mbar_arrive(&bar.rfull[rs]);
        ++made;
        if (last) break;
      }
      if (t0 == 0 && t1 < tiles) {
        // the block's last tile is another CTA's
        const int u = u1 + (tiles - t1) - 1, few = each + 1;
        const int c = u < few * more ? u / few : more + (u - few * more) / each;
        shared = make_int4(b, h, block, c - cta + 1);
      }
      if (keys > 0) {
        // the block's rows: two e4m3 numbers for each element
        constexpr int kLanes = 16 * NP;       // lanes of a row, 8 elements each
        constexpr int kAtOnce = 32 / kLanes;  // rows at a time
        constexpr int kBatch = 8;
        const int qb = qn & 1, row0 = block * R, tok0 = row0 / P.G, d0 = lane % kLanes * 8;
        ok = at_wait(&bar.qempty[qb], (static_cast<unsigned>(qn >> 1) & 1u) ^ 1u, fault);
        if (!ok) break;
        unsigned char* dst = qbuf + 2 * qb * S::kQHalf;
        const bf16_t* q = P.q + b * P.q_ld[0] + static_cast<long long>(h) * P.G * P.q_ld[2] + d0;
#pragma unroll 1
        for (int r1 = 0; r1 < R; r1 += kBatch * kAtOnce) {
          uint4 raw[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int row = row0 + r1 + i * kAtOnce + lane / kLanes, tok = row / P.G, g = row - tok * P.G;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (tok < s.count && d0 < P.D && r1 + i * kAtOnce < R)
              raw[i] = *reinterpret_cast<const uint4*>(q + tok * P.q_ld[1] + g * P.q_ld[2]);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = r1 + i * kAtOnce + lane / kLanes;
            if (r1 + i * kAtOnce >= R) break;
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
            const int eq =
                max(static_cast<int>(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7), -100);
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
          const int* parent = P.parent + static_cast<long long>(b) * P.n;
          bool bad = false;
          for (int j = lane; j < s.count; j += 32) {
            int p = j ? __ldg(parent + j) : 0;
            if (j && (p < 0 || p >= j)) {
              bad = true;
              p = 0;
            }
            parent_s[j] = static_cast<unsigned short>(p);
            mask[j] = 0;
          }
          if (bad && h == 0) report(P, b, SPEC_ERR_PARENT);
          __syncwarp();
          for (int i = lane; i < R; i += 32) {
            const int tok = tok0 + i;
            if (tok >= s.count || tok * P.G >= row0 + R) break;
            const unsigned long long bit = 1ull << i;
            for (int j = tok;; j = parent_s[j]) {
              atomicOr(mask + j, bit);
              if (j == 0) break;
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (leader) mbar_arrive(&bar.qfull[qb]);
        ++qn;
      }
      if (t1 == tiles && left > 0) {
        if (++block == P.blocks) {
          block = 0;
          if (++h == P.H) {
            h = 0;
            s = lengths(++b);
          }
        }
        keys = keys_of<R>(P, s, block);
        tiles = tiles_of(keys);
        t1 = 0;
      }
    }
    if (leader) P.shared[cta] = ok ? shared : make_int4(0, 0, 0, 0);
  } else if (warp == 3) {
    // ---------------- what no row sees, and NaN values among the drafted tokens ----------------
    int it = 0, patches = 0;
    bool ok = true;
    Piece w;
    while (ok && next_piece(w)) {
      it += w.t1 - w.t0;
      for (int t = max(w.t0, first_special(w)); ok && t < w.t1; ++t, ++patches) {
        const int j = it - (w.t1 - t), s = j % S::kStages;
        ok = at_wait(&bar.landed[patches % kPatchRing], static_cast<unsigned>(patches / kPatchRing) & 1u, fault) &&
             at_wait(&bar.full[s], static_cast<unsigned>(j / S::kStages) & 1u, fault);
        if (!ok) break;
#pragma unroll 1
        for (int row = lane; row < kTile; row += 32) {
          const int pos = t * kTile + row;
          unsigned char* v = vring + s * S::kSlot + row * 128;
          bool clear = pos >= w.keys, nan = false;
          if (!clear && pos >= w.prefix) {
#pragma unroll 1
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
#pragma unroll 1
            for (int p = 0; p < NP; ++p)
#pragma unroll
              for (int o = 0; o < 128; o += 16) *reinterpret_cast<uint4*>(v + p * kPanel + o) = make_uint4(0, 0, 0, 0);
          }
          const unsigned all = __ballot_sync(0xffffffffu, nan);
          if (leader) nan_s[patches % kPatchRing][row >> 5] = all;
        }
        fence_proxy_async();
        __syncwarp();
        if (leader) mbar_arrive(&bar.patched[patches % kPatchRing]);
      }
    }
  } else if (warp < kFirstOut) {
    // ---------------- weights ----------------
    const int group = (warp - 4) >> 2, turn = group / S::kColumns, q = warp & 3, row = q * 32 + lane;
    const int col0 = group % S::kColumns * kW;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    const int page_row = row / P.page;
    const int col = lane % kW;  // lanes i and i + kW do the same for row col0 + i
    float(*refs)[kW] = ref_s[warp - 4];
    int it = 0, qn = 0, patches = 0;
    bool ok = true;  // (what a wait of this warp's gave; the warpgroup goes by what its warps agree on)
    Piece w;
    while (true) {
      const bool got = next_piece(w);
      if (!meet(1 + group, got)) break;
      const int special = first_special(w), qb = qn & 1, tok0 = w.block * R / P.G;
      float sum_unit = -kInf;  // log2 of the sums' unit, of row col0 + col
      float2 sum[kW / 2];
#pragma unroll
      for (int i = 0; i < kW / 2; ++i) sum[i] = make_float2(0.f, 0.f);
      bool go = true;
#pragma unroll 1
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int patch = t >= special ? patches++ : -1, k = it & 1;
        if (S::kTurns == 2 && k != turn) continue;
        const unsigned half = static_cast<unsigned>(it >> 1) & 1u;
        const int sb = it % kScores;
        ok = at_wait(&bar.sfull[sb], static_cast<unsigned>(it / kScores) & 1u, fault) && ok;
        tc_fence_after();
        float y[kW];
        tmem_columns<kW>(tmem_sc + sb * R + col0 + lanes, y);
        const PageScale ps = scale_s[it % kScaleRing][page_row];
        // y = score + value exponent
#pragma unroll
        for (int r = 0; r < kW; r += 4) {
          const float4 c = lds_f4(&cq_s[qb][col0 + r]);
          const float2 ck = make_float2(ps.ck, ps.ck), ve = make_float2(ps.ve, ps.ve);
          const float2 a = ffma2(fmul2(make_float2(y[r], y[r + 1]), make_float2(c.x, c.y)), ck, ve);
          const float2 b = ffma2(fmul2(make_float2(y[r + 2], y[r + 3]), make_float2(c.z, c.w)), ck, ve);
          y[r] = a.x, y[r + 1] = a.y, y[r + 2] = b.x, y[r + 3] = b.y;
        }
        if (patch >= 0) {
          ok = at_wait(&bar.patched[patch % kPatchRing], static_cast<unsigned>(patch / kPatchRing) & 1u, fault) && ok;
          const int pos = t * kTile + row, j = pos - w.prefix;
          unsigned long long seen = ~0ull;
          if (pos >= w.keys) seen = 0;
          else if (j >= 0 && P.parent) seen = mask_s[qb * kMaxRows + j];
          else if (j > tok0) seen = j - tok0 > 63 ? 0 : ~0ull << (j - tok0);
          const bool nan = nan_s[patch % kPatchRing][q] >> lane & 1u;
#pragma unroll
          for (int r = 0; r < kW; ++r) {
            if (nan) y[r] = __uint_as_float(0x7fc00000u);
            if (!(seen >> token_s[qb][col0 + r] & 1ull)) y[r] = -kInf;
          }
        }
        // the rows' largest
        const int slot = S::kTurns == 2 ? it >> 1 & 1 : k;
#pragma unroll
        for (int r = 0; r < kW; r += 4) {
          const float4 m = make_float4(warp_max(y[r]), warp_max(y[r + 1]), warp_max(y[r + 2]), warp_max(y[r + 3]));
          if (leader) *reinterpret_cast<float4*>(&most_s[group][slot][q][r]) = m;
        }
        if (ps.far) {
#pragma unroll
          for (int r = 0; r < kW; ++r) {
            const float m = warp_max(y[r] - ps.ve);
            if (leader) most_x_s[group][q][r] = m;
          }
        }
        go = meet(1 + group, ok);
        if (!go) break;
        // every warp for itself: a lane per row
        const float m = fmaxf(fmaxf(most_s[group][slot][0][col], most_s[group][slot][1][col]),
                              fmaxf(most_s[group][slot][2][col], most_s[group][slot][3][col]));
        const bool none = m == -kInf;
        refs[0][col] = none ? 0.f : m - 8.f;
        if (q == 0) {
          ok = at_wait(&bar.mempty[k], half ^ 1u, fault);
          top_s[k][col0 + col] = m - 8.f;
        }
        __syncwarp();
        if (q == 0 && leader) mbar_arrive(&bar.mfull[k]);
        // the sums' reference: the largest score without exponents, or a bound of it
        float most_x = m - ps.ve_low;
        if (ps.far) {
          // (2^(y - reference) may underflow where a page's values are tiny against another's)
          most_x = fmaxf(fmaxf(most_x_s[group][0][col], most_x_s[group][1][col]),
                         fmaxf(most_x_s[group][2][col], most_x_s[group][3][col]));
          const float next = fmaxf(sum_unit, most_x);
          refs[1][col] = sum_unit == -kInf ? 0.f : ex2(sum_unit - next);
          refs[2][col] = none ? 0.f : next;
          sum_unit = next;
          __syncwarp();
#pragma unroll
          for (int r = 0; r < kW; r += 2) {
            sum[r / 2].x = __fmaf_rn(sum[r / 2].x, refs[1][r], ex2((y[r] - ps.ve) - refs[2][r]));
            sum[r / 2].y = __fmaf_rn(sum[r / 2].y, refs[1][r + 1], ex2((y[r + 1] - ps.ve) - refs[2][r + 1]));
          }
          meet(1 + group, true);  // (there is one most_x_s)
        }
#pragma unroll
        for (int r = 0; r < kW; r += 4) {
          const float4 c = lds_f4(&refs[0][r]);
          y[r] = ex2(y[r] - c.x);
          y[r + 1] = ex2(y[r + 1] - c.y);
          y[r + 2] = ex2(y[r + 2] - c.z);
          y[r + 3] = ex2(y[r + 3] - c.w);
        }
        ok = at_wait(&bar.pempty[k], half ^ 1u, fault) && ok;
        unsigned char* p = pbuf + 2 * k * S::kPHalf;
#pragma unroll
        for (int r = 0; r < kW; r += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) split2(y[r + 2 * i], y[r + 2 * i + 1], hi[i], lo[i]);
          const uint32_t at = swizzled(row * S::kPRow + col0 + r, S::kPRow);
          *reinterpret_cast<uint2*>(p + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2*>(p + S::kPHalf + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (leader) mbar_arrive(&bar.pfull[k]);
        if (!ps.far) {
          // the sums of the weights themselves: without the values' exponents
          const float next = fmaxf(sum_unit, most_x);
          refs[1][col] = sum_unit == -kInf ? 0.f : ex2(sum_unit - next);
          refs[2][col] = none ? 0.f : ex2(most_x - next) * 0.00390625f;
          sum_unit = next;
          __syncwarp();
          const float f = exp2i(static_cast<int>(ps.ve_low - ps.ve));
#pragma unroll
          for (int r = 0; r < kW; r += 4) {
            const float4 a = lds_f4(&refs[1][r]), b = lds_f4(&refs[2][r]);
            sum[r / 2] = ffma2(sum[r / 2], make_float2(a.x, a.y),
                               fmul2(make_float2(y[r], y[r + 1]), fmul2(make_float2(b.x, b.y), make_float2(f, f))));
            sum[r / 2 + 1] = ffma2(sum[r / 2 + 1], make_float2(a.z, a.w),
                                   fmul2(make_float2(y[r + 2], y[r + 3]), fmul2(make_float2(b.z, b.w), make_float2(f, f))));
          }
        }
      }
      // the piece's sums and their units
      if (!go) break;
      ok = at_wait(&bar.eempty[qb], (static_cast<unsigned>(qn >> 1) & 1u) ^ 1u, fault) && ok;
      if (!meet(1 + group, ok)) break;
      float all[kW];
#pragma unroll
      for (int i = 0; i < kW / 2; ++i) all[2 * i] = sum[i].x, all[2 * i + 1] = sum[i].y;
      sum_s[qb][turn][q][col0 + col] = column_sums<kW>(all, lane);
      if (q == 0) sum_unit_s[qb][turn][col0 + col] = sum_unit;
      __syncwarp();
      if (leader) mbar_arrive(&bar.efull[qb]);
      ++qn;
    }
  } else {
    // ---------------- outputs ----------------
    const int q = warp & 3, d = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    int it = 0, qn = 0;
    bool ok = true;
    Piece w;
    while (true) {
      const bool got = next_piece(w);
      if (!meet(5, got)) break;
      const int row0 = w.block * R;
      const int qb = qn & 1;
      const unsigned piece_half = static_cast<unsigned>(qn >> 1) & 1u;
      float2 acc[NP][R / 2];
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; r < R / 2; ++r) acc[p][r] = make_float2(0.f, 0.f);
      float unit = -kInf;  // log2 of the outputs' unit, of row d
      bool go = true;
#pragma unroll 1
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int k = it & 1;
        const unsigned half = static_cast<unsigned>(it >> 1) & 1u;
        ok = at_wait(&bar.mfull[k], half, fault) && ok;
        if (d < R) {
          const float top = top_s[k][d], next = fmaxf(unit, top);
          mix_s[k][d] = make_float2(unit == -kInf ? 0.f : ex2(unit - next), top == -kInf ? 0.f : ex2(top - next));
          unit = next;
        }
        go = meet(5, ok);
        if (!go) break;
        if (leader) mbar_arrive(&bar.mempty[k]);
        ok = at_wait(&bar.ofull[k], half, fault);
        tc_fence_after();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          if (p * 128 + q * 32 >= P.D) break;
#pragma unroll
          for (int r = 0; r < R; r += 16) {
            float o[16];
            tmem_ld16(tmem_o + (k * NP + p) * R + r + lanes, o);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float4 m = *reinterpret_cast<const float4*>(&mix_s[k][r + e]);
              float2& x = acc[p][(r + e) / 2];
              x = ffma2(make_float2(o[e], o[e + 1]), make_float2(m.y, m.w), fmul2(x, make_float2(m.x, m.z)));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (leader) mbar_arrive(&bar.oempty[k]);
      }
      if (!go) break;
      ok = at_wait(&bar.efull[qb], piece_half, fault) && ok;
      if (!meet(5, ok)) break;
      constexpr int kLd = NP * 128 + 4;
      float* part = P.parts + (static_cast<long long>(2 * blockIdx.x) + max(w.part, 0)) * R * kLd;
      if (d < R) {
        float s = (sum_s[qb][0][0][d] + sum_s[qb][0][1][d]) + (sum_s[qb][0][2][d] + sum_s[qb][0][3][d]);
        float su = sum_unit_s[qb][0][d];
        if constexpr (S::kTurns == 2) {
          const float s2 = (sum_s[qb][1][0][d] + sum_s[qb][1][1][d]) + (sum_s[qb][1][2][d] + sum_s[qb][1][3][d]);
          const float su2 = sum_unit_s[qb][1][d], next = fmaxf(su, su2);
          s = (su == -kInf ? s : s * ex2(su - next)) + (su2 == -kInf ? s2 : s2 * ex2(su2 - next));
          su = next;
        }
        if (w.part < 0) {
          const int tok = (row0 + d) / P.G, g = row0 + d - tok * P.G;
          row_s[d] = s == 0.f ? 0.f : ex2(unit - su) / s;
          place_s[d] = tok >= P.n ? -1 : w.b * P.out_ld[0] + tok * P.out_ld[1] + (w.h * P.G + g) * P.out_ld[2];
          if (tok >= w.count) row_s[d] = 0.f;
        } else {
          float* e = part + d * kLd + NP * 128;
          __stcg(e, unit);
          __stcg(e + 1, s);
          __stcg(e + 2, su);
        }
      }
      meet(5, true);
      if (leader) {
        mbar_arrive(&bar.qempty[qb]);
        mbar_arrive(&bar.eempty[qb]);
      }
      ++qn;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const long long at = w.part < 0 ? place_s[r] : r * kLd;
        if (at < 0) break;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const float v = r & 1 ? acc[p][r / 2].y : acc[p][r / 2].x;
          if (w.part < 0) {
            unsigned short bits;
            const float f = row_s[r];
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(f == 0.f ? 0.f : v * f));
            if (p * 128 + d < P.D) P.out[at + p * 128 + d] = bits;
          } else {
            __stcg(part + at + p * 128 + d, v);
          }
        }
      }
      meet(5, true);
    }
  }

  __syncthreads();
  if (*fault && tid == 0) {
    // copies still in flight land before the CTA exits: wait (bounded) for
    // the last phase of every stage that was issued
    for (int k = max(0, issued_s - S::kStages); k < issued_s; ++k)
      mbar_wait(&bar.full[k % S::kStages], static_cast<unsigned>(k / S::kStages) & 1u);
    if (P.error_word) atomicOr(P.error_word, SPEC_ERR_INTERNAL);
    P.shared[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
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
  return rows <= 16 ? 16 : rows <= 32 || D > 128 ? 32 : rows <= 48 ? 48 : 64;
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
  p.blocks = (a.n * p.G + R - 1) / R;
  // tiles are counted in 31 bits
  const long long most = static_cast<long long>(a.table_pages) * a.page / kTile + 1;
  if (most * p.blocks * a.H * a.B > 0x7fffffffLL) return SPEC_EINVAL;
  const int nsm = sm_count();
  if (nsm < 1) return SPEC_ECUDA;
  const long long rows = static_cast<long long>(a.pages) * a.H * a.page;
  CUtensorMap tk, tv;
  if (!code_map(&tk, a.k_codes, rows, a.D, a.page) || !code_map(&tv, a.v_codes, rows, a.D, a.page)) return SPEC_ECUDA;
  if (raise_smem<R, NP>() != cudaSuccess) return SPEC_ECUDA;
  p.more_bytes = g_more_bytes.load();
  const int ctas = std::min(nsm, kMaxCtas);
  attend_kernel<R, NP><<<ctas, Shape<R, NP>::kThreads, Shape<R, NP>::kSmem, s>>>(tk, tv, p);
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
    case 48: return launch_attend<48, 1>(*a, p, stream);
    default: return launch_attend<64, 1>(*a, p, stream);
  }
}
