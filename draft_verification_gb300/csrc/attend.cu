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
#include <type_traits>

#include "cache.cuh"
#include "internal.h"
#include "spec_cache.h"
#include "tc.cuh"
#include "tma_host.h"

namespace sv {
namespace {

constexpr int kTile = 128;      // tokens per tile; two tiles make a step
constexpr int kPanel = 16384;   // bytes of 128 tokens x 128 elements
constexpr int kMaxRows = 1024;  // n
constexpr int kMaxCtas = 160;
constexpr int kThreads = 512;
constexpr int kMaskBytes = 10 * kMaxRows;  // of shared memory for a tree's masks, at most
constexpr int kScaleRing = 16, kPatchRing = 8, kPieceRing = 4;
constexpr int kFar = 9;    // value exponents of a step that lie further apart than this: 2^-9 is the least e4m3 code
constexpr int kAhead = 2;  // tiles that K is copied ahead of V, as its products are ahead

// R: a block's rows; NP: panels of 128 elements of a head.
template <int R, int NP>
struct Shape {
  // places of K tiles, and as many of V tiles (each with barriers of its own: a
  // warp has to meet all phases of a barrier that it waits on)
  static constexpr int kStages = NP == 2 ? 2 : R == 16 ? 5 : R == 32 ? 4 : 3;
  static constexpr int kSlot = NP * kPanel;
  static constexpr int kPRow = R == 48 ? 64 : R;  // bytes of a token's weights
  static constexpr int kPHalf = 2 * kTile * kPRow;  // hi or lo of a step's weights
  static constexpr int kQHalf = NP * R * 128;       // hi or lo of a block's queries
  static constexpr int kScores = R > 32 ? 2 : 4;    // places of steps' scores
  static constexpr int kOnes = 1024;                // a tile's factors of the sums of weights (one row of 128 bytes)
  static constexpr int kSmem = 1024 + 2 * kStages * kSlot + 4 * kQHalf + 4 * kPHalf + 4 * kOnes;
  static constexpr int kCols = (2 * kScores + 2 * NP + 2) * R;
  static constexpr uint32_t kTmemCols = kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512 && kStages + kAhead + 6 <= kScaleRing && 2 * kStages + kPatchRing <= 32, "rings");
  using Mask = typename std::conditional<(R > 32), unsigned long long, unsigned>::type;  // a bit per token of a block
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
__device__ __forceinline__ void umma_e4m3(uint32_t issues, uint32_t d, uint32_t a, uint32_t a_high, uint32_t b,
                                          uint32_t b_high, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 da, db;\n mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n"
      " setp.ne.b32 p, %6, 0;\n setp.ne.b32 q, %7, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n}" ::"r"(d),
      "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(idesc), "r"(accumulate), "r"(issues)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t issues, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_addr(bar)),
      "r"(issues)
      : "memory");
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
  float ck, ve;           // 2^key exponent (NaN: not a page), value exponent
  float ve_low, ve_high;  // the tile's least and largest value exponents
};

// Where a CTA's n-th tile of K (or of V) is among N places, and its parity there.
template <int N>
struct Place {
  int slot;
  unsigned parity;
  __device__ __forceinline__ explicit Place(unsigned number) : slot(number % N), parity(number / N & 1u) {}
};

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int R, int NP>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const AttendParams P) {
  using S = Shape<R, NP>;
  extern __shared__ __align__(1024) unsigned char at_dyn[];
  // kfull / kempty, vfull / vempty: a tile's K, V; sfull / sempty: a step's scores; pfull /
  // pempty: its weights in shared memory; ofull / oempty: its outputs; mfull /
  // mempty: its maxima (top_s); qfull / qempty: a piece's queries; rfull /
  // rempty: its record; landed: V of a tile that is patched before it is vfull;
  // patched: it is; drain: no product is under way
  struct Bars {
    uint64_t kfull[S::kStages], vfull[S::kStages], kempty[S::kStages], vempty[S::kStages];
    uint64_t sfull[S::kScores], sempty[S::kScores], pfull[2], pempty[2], ofull[2], oempty[2], mfull[2], mempty[2];
    uint64_t qfull[2], qempty[2], landed[kPatchRing], patched[kPatchRing], rfull[kPieceRing], rempty[kPieceRing], drain[2];
  };
  constexpr int kBars = sizeof(Bars) / 8;
  __shared__ Bars bar;
  __shared__ uint32_t tmem_s;
  __shared__ int fault_s;
  __shared__ unsigned issued_s, parity_s;  // barriers that copies count on (kfull, vfull, landed), the last one's parity
  __shared__ __align__(16) Piece piece_s[kPieceRing];
  __shared__ __align__(16) PageScale scale_s[kScaleRing][8];
  __shared__ int place_of_page_s[kScaleRing][8];  // rows of the pages' copies, -1: none
  __shared__ bool special_s[kScaleRing];          // tiles that are patched
  __shared__ __align__(16) float most_s[2][2][4][R], ref_s[8][R], cq_s[2][R], top_s[2][R], sum_s[R];
  __shared__ __align__(16) float2 mix_s[2][R], far_s[2][4][R];
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
  unsigned char* ones = pbuf + 4 * S::kPHalf;
  using Mask = typename S::Mask;
  Mask* mask_s = reinterpret_cast<Mask*>(ones + 4 * S::kOnes);  // [2][n], with parents
  unsigned short* parent_s = reinterpret_cast<unsigned short*>(mask_s + 2 * P.n);
  volatile int* fault = &fault_s;

  pdl_launch_dependents();
  if (tid < kBars) {
    uint64_t* at = reinterpret_cast<uint64_t*>(&bar) + tid;
    unsigned count = 1;
    if (at >= bar.sfull && at < bar.sempty) count = 2;   // sfull
    if (at >= bar.sempty && at < bar.pempty) count = 4;  // sempty, pfull
    if (at >= bar.oempty && at < bar.mfull) count = 4;   // oempty
    if (at >= bar.mempty && at < bar.qfull) count = 4;   // mempty
    if (at >= bar.qempty && at < bar.landed) count = 4;  // qempty
    if (at >= bar.rempty && at < bar.drain) count = 15;  // rempty
    mbar_init(at, count);
    mbar_fence_init();
  }
  if (tid == 0) fault_s = 0, issued_s = parity_s = 0u;
  // (rows of the sums' factors that are not the first: of no use, but of defined values)
  for (int i = tid; i < 4 * S::kOnes / 16; i += kThreads) reinterpret_cast<uint4*>(ones)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  if (warp == 1) {
    tmem_alloc(&tmem_s, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_sc = tmem_s, tmem_o = tmem_s + 2 * S::kScores * R, tmem_l = tmem_o + 2 * NP * R;

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
    // K or V of a tile to its place, counted on a barrier that is number `on` among kfull, vfull and landed
    const auto copy = [&](const CUtensorMap* map, int tile, unsigned char* to, uint64_t* empty, uint64_t* full, int on,
                          unsigned on_parity) {
      const Place<S::kStages> at(tile);
      const int y = lane < pp ? place_of_page_s[tile % kScaleRing][lane] : -1;
      const unsigned bytes =
          static_cast<unsigned>(__popc(__ballot_sync(0xffffffffu, y >= 0))) * page_bytes * NP + P.more_bytes;
      if (!at_wait(&empty[at.slot], at.parity ^ 1u, fault)) return false;
      if (leader) {
        mbar_expect_tx(full, bytes);
        issued_s |= 1u << on;
        parity_s = (parity_s & ~(1u << on)) | on_parity << on;
      }
      __syncwarp();
      if (y >= 0) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
          tma_load_2d(to + at.slot * S::kSlot + lane * page_bytes + p * kPanel, map, p * 128, y, full);
      }
      __syncwarp();
      return true;
    };
    int patches = 0;
    const auto copy_k = [&](int tile) {
      const Place<S::kStages> at(tile);
      return copy(&tm_k, tile, kring, bar.kempty, &bar.kfull[at.slot], at.slot, at.parity);
    };
    const auto copy_v = [&](int tile) {
      if (special_s[tile % kScaleRing]) {
        const Place<kPatchRing> at(patches++);
        return copy(&tm_v, tile, vring, bar.vempty, &bar.landed[at.slot], 2 * S::kStages + at.slot, at.parity);
      }
      const Place<S::kStages> at(tile);
      return copy(&tm_v, tile, vring, bar.vempty, &bar.vfull[at.slot], S::kStages + at.slot, at.parity);
    };
    Piece w;
    while (ok && next_piece(w)) {
      const int special = first_special(w);
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
        x.ve_high = static_cast<float>(hi);
        const int y = static_cast<int>(slab * P.page);
#pragma unroll 1
        for (int i = 0; i < batch && tb + i < w.t1; ++i, ++it) {
          if (mine == i) {
            scale_s[it % kScaleRing][slot_in] = x;
            place_of_page_s[it % kScaleRing][slot_in] = has ? y : -1;
          }
          if (leader) special_s[it % kScaleRing] = tb + i >= special;
          __syncwarp();
          ok = copy_k(it) && (tb + i - w.t0 < kAhead || copy_v(it - kAhead));
          if (!ok) break;
        }
      }
      // (V's last ones wait for no other piece, whose queries may wait for this one's end)
      const int n = w.t1 - w.t0;
#pragma unroll 1
      for (int j = max(0, n - kAhead); ok && j < n; ++j) ok = copy_v(it - n + j);
    }
  } else if (warp == 1) {
    // ---------------- scores ----------------
    constexpr uint32_t idesc = idesc_e4m3(kTile, R, 0, 0), high = operand_high(1024, 128);
    const int steps = (P.D + 31) / 32;
    const uint32_t issues = leader ? 1u : 0u;
    int it = 0, step = 0, qn = 0;
    bool ok = true;
    Piece w;
    while (ok && next_piece(w)) {
      const uint32_t q_hi = operand_low(smem_addr(qbuf + 2 * (qn & 1) * S::kQHalf), 1024);
      ok = at_wait(&bar.qfull[qn & 1], static_cast<unsigned>(qn >> 1) & 1u, fault);
      ++qn;
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
        // (a step's two tiles, the second one perhaps missing)
        const int sb = step % S::kScores, sub = (t - w.t0) & 1;
        const Place<S::kStages> at(it);
        if (sub == 0) ok = at_wait(&bar.sempty[sb], (static_cast<unsigned>(step / S::kScores) & 1u) ^ 1u, fault);
        ok = ok && at_wait(&bar.kfull[at.slot], at.parity, fault);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = operand_low(smem_addr(kring + at.slot * S::kSlot), 1024), d = tmem_sc + (2 * sb + sub) * R;
        umma_e4m3(issues, d, a, high, q_hi, high, idesc, 0u);
#pragma unroll
        for (int k = 1; k < 8 * NP; ++k) {  // hi's steps of 32 elements, then lo's
          const int e = k % (4 * NP);
          if (e < steps)
            umma_e4m3(issues, d, a + (e >> 2) * (kPanel >> 4) + (e & 3) * 2, high,
                            q_hi + k / (4 * NP) * (S::kQHalf >> 4) + (e >> 2) * (R * 128 >> 4) + (e & 3) * 2, high,
                      idesc, 1u);
        }
        commit_if(issues, &bar.kempty[at.slot]);
        if (sub == 1 || t + 1 == w.t1) {
          commit_if(issues, &bar.sfull[sb]);
          if (leader) mbar_arrive(&bar.sfull[sb]);  // what the copies' and queries' warps wrote is visible behind it
          ++step;
        }
        __syncwarp();
      }
    }
    // every product issued has completed before tensor memory is released
    commit_if(issues, &bar.drain[0]);
    mbar_wait(&bar.drain[0], 0);
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
          Mask* mask = mask_s + qb * P.n;
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
            const Mask bit = static_cast<Mask>(1) << i;
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
    // ---------------- outputs' products ----------------
    // (and, before them, V of what no row sees, and NaN values among the drafted tokens)
    constexpr uint32_t idesc = idesc_e4m3(128, R, 1, 1), idesc_l = idesc_e4m3(64, R, 0, 1);
    constexpr uint32_t a_high = operand_high(1024, 128), b_high = operand_high(8 * S::kPRow, S::kPRow);
    const uint32_t issues = leader ? 1u : 0u;
    int it = 0, step = 0, patches = 0;
    bool ok = true;
    Piece w;
    while (ok && next_piece(w)) {
      const int special = first_special(w);
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
        const int k = step & 1, sub = (t - w.t0) & 1;
        const unsigned half = static_cast<unsigned>(step >> 1) & 1u;
        if (sub == 0) {
          // (the weights of a step wait for its patches)
#pragma unroll 1
          for (int u = max(t, special); ok && u < min(t + 2, w.t1); ++u, ++patches) {
            ok = at_wait(&bar.landed[patches % kPatchRing], static_cast<unsigned>(patches / kPatchRing) & 1u, fault);
            if (!ok) break;
            const Place<S::kStages> at(it + u - t);
#pragma unroll 1
            for (int row = lane; row < kTile; row += 32) {
              const int pos = u * kTile + row;
              unsigned char* v = vring + at.slot * S::kSlot + row * 128;
              bool clear = pos >= w.keys, nan = false;
              if (!clear && pos >= w.prefix) {
#pragma unroll 1
                for (int p = 0; p < NP; ++p)
#pragma unroll
                  for (int o = 0; o < 128; o += 16) {
                    const uint4 x = *reinterpret_cast<const uint4*>(v + p * kPanel + o);
                    const uint32_t m = 0x7f7f7f7fu, one = 0x01010101u;
                    nan |=
                        ((((x.x & m) + one) | ((x.y & m) + one) | ((x.z & m) + one) | ((x.w & m) + one)) & 0x80808080u) != 0;
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
            if (leader) {
              mbar_arrive(&bar.patched[patches % kPatchRing]);
              mbar_arrive(&bar.vfull[at.slot]);
            }
          }
          ok = ok && at_wait(&bar.oempty[k], half ^ 1u, fault) && at_wait(&bar.pfull[k], half, fault);
        }
        const Place<S::kStages> at(it);
        ok = ok && at_wait(&bar.vfull[at.slot], at.parity, fault);
        if (!ok) break;
        tc_fence_after();
        const uint32_t b = operand_low(smem_addr(pbuf + 2 * k * S::kPHalf + sub * kTile * S::kPRow), 8 * S::kPRow);
        const uint32_t a0 = operand_low(smem_addr(vring + at.slot * S::kSlot), 1024);
        const uint32_t first = sub == 0 ? 0u : 1u;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const uint32_t a = a0 + p * (kPanel >> 4), o = tmem_o + (k * NP + p) * R;
#pragma unroll
          for (int i = 0; i < 2 * kTile / 32; ++i)  // hi's 4 steps of 32 tokens, then lo's
            umma_e4m3(issues, o, a + (i & 3) * (32 * 128 >> 4), a_high,
                      b + (i >> 2) * (S::kPHalf >> 4) + (i & 3) * (32 * S::kPRow >> 4), b_high, idesc,
                      i == 0 ? first : 1u);
        }
        // the sums of the weights: products with one row of factors (every 8 rows of
        // the operand are the same, a stride of 0), the first of the 64 results is used
        const uint32_t f = operand_low(smem_addr(ones + (2 * k + sub) * S::kOnes), 0);
#pragma unroll
        for (int i = 0; i < 2 * kTile / 32; ++i)
          umma_e4m3(issues, tmem_l + k * R, f + (i & 3) * 2, operand_high(0, 128),
                    b + (i >> 2) * (S::kPHalf >> 4) + (i & 3) * (32 * S::kPRow >> 4), b_high, idesc_l,
                    i == 0 ? first : 1u);
        commit_if(issues, &bar.vempty[at.slot]);
        if (sub == 1 || t + 1 == w.t1) {
          commit_if(issues, &bar.ofull[k]);
          commit_if(issues, &bar.pempty[k]);
          ++step;
        }
      }
    }
    commit_if(issues, &bar.drain[1]);
    mbar_wait(&bar.drain[1], 0);
  } else if (warp < 12) {
    // ---------------- weights ----------------
    // Every other step, all rows of the block; a thread has a token of each of
    // the step's tiles.  The scores are read twice, for the maxima and for the
    // weights, 16 rows at a time: the same few instructions again and again
    // (what these warps wait for most is instructions).
    const int turn = (warp - 4) >> 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    const int page_row = row / P.page;
    float* refs = ref_s[warp - 4];
    unsigned char* weights = pbuf + 2 * turn * S::kPHalf;
    unsigned char* factors = ones + 2 * turn * S::kOnes + row;
    int it = 0, step = 0, qn = 0, patches = 0;
    bool ok = true;  // (what a wait of this warp's gave; the warpgroup goes by what its warps agree on)
    Piece w;
    while (true) {
      const bool got = next_piece(w);
      if (!meet(1 + turn, got)) break;
      const int special = first_special(w), qb = qn & 1, tok0 = w.block * R / P.G;
      bool go = true;
#pragma unroll 1
      for (int t = w.t0; t < w.t1; t += 2, ++step) {
        const int tiles = min(2, w.t1 - t);
        const int at = it, patch = patches;
        it += tiles;
        patches += max(0, min(tiles, t + tiles - special));
        if ((step & 1) != turn) continue;
        const unsigned half = static_cast<unsigned>(step >> 1) & 1u;
        const int sb = step % S::kScores;
        ok = at_wait(&bar.sfull[sb], static_cast<unsigned>(step / S::kScores) & 1u, fault) && ok;
        tc_fence_after();
        const PageScale ps0 = scale_s[at % kScaleRing][page_row], ps1 = scale_s[(at + tiles - 1) % kScaleRing][page_row];
        // what the rows see of this thread's tokens
        Mask seen0 = ~static_cast<Mask>(0), seen1 = seen0;
        bool nan0 = false, nan1 = false;
        if (t + tiles > special) {
          const auto look = [&](int tile, int patch, Mask& seen, bool& nan) {
            if (tile < special) return;
            ok = at_wait(&bar.patched[patch % kPatchRing], static_cast<unsigned>(patch / kPatchRing) & 1u, fault) && ok;
            const int pos = tile * kTile + row, j = pos - w.prefix;
            if (pos >= w.keys) seen = 0;
            else if (j >= 0 && P.parent) seen = mask_s[qb * P.n + j];
            else if (j > tok0) seen = j - tok0 >= static_cast<int>(8 * sizeof(Mask)) ? 0 : ~static_cast<Mask>(0) << (j - tok0);
            nan = nan_s[patch % kPatchRing][q] >> lane & 1u;
          };
          look(t, patch, seen0, nan0);
          if (tiles == 2) look(t + 1, patch + (t >= special ? 1 : 0), seen1, nan1);
        }
        // 16 rows' scores, base 2, plus the value exponent
        const auto scores = [&](int sub, int c, float* y) {
          tmem_ld16(tmem_sc + (2 * sb + sub) * R + c + lanes, y);
          const float ck = sub ? ps1.ck : ps0.ck, ve = sub ? ps1.ve : ps0.ve;
          const float2 ck2 = make_float2(ck, ck), ve2 = make_float2(ve, ve);
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const float4 f = lds_f4(&cq_s[qb][c + r]);
            const float2 a = ffma2(fmul2(make_float2(y[r], y[r + 1]), make_float2(f.x, f.y)), ck2, ve2);
            const float2 b = ffma2(fmul2(make_float2(y[r + 2], y[r + 3]), make_float2(f.z, f.w)), ck2, ve2);
            y[r] = a.x, y[r + 1] = a.y, y[r + 2] = b.x, y[r + 3] = b.y;
          }
          if (t + sub >= special) {
            const Mask seen = sub ? seen1 : seen0;
            const bool nan = sub ? nan1 : nan0;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              if (nan) y[r] = __uint_as_float(0x7fc00000u);
              if (!(seen >> token_s[qb][c + r] & 1)) y[r] = -kInf;
            }
          }
        };
        // the rows' largest
        const int slot = step >> 1 & 1;
#pragma unroll 1
        for (int c = 0; c < R; c += 16) {
          float top[16];
          scores(0, c, top);
          if (tiles == 2) {
            float y[16];
            scores(1, c, y);
#pragma unroll
            for (int r = 0; r < 16; ++r) top[r] = fmaxf(top[r], y[r]);
          }
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const float4 m =
                make_float4(warp_max(top[r]), warp_max(top[r + 1]), warp_max(top[r + 2]), warp_max(top[r + 3]));
            if (leader) *reinterpret_cast<float4*>(&most_s[turn][slot][q][c + r]) = m;
          }
        }
        go = meet(1 + turn, ok);
        if (!go) break;
        // every warp for itself: a lane per row
        if (q == 0) ok = at_wait(&bar.mempty[turn], half ^ 1u, fault);
#pragma unroll
        for (int c = lane; c < R; c += 32) {
          const float m = fmaxf(fmaxf(most_s[turn][slot][0][c], most_s[turn][slot][1][c]),
                                fmaxf(most_s[turn][slot][2][c], most_s[turn][slot][3][c]));
          refs[c] = m == -kInf ? 0.f : m - 8.f;
          if (q == 0) top_s[turn][c] = m - 8.f;
        }
        ok = at_wait(&bar.pempty[turn], half ^ 1u, fault) && ok;
        const float low = fminf(ps0.ve_low, ps1.ve_low);
        if (fmaxf(ps0.ve_high, ps1.ve_high) - low > static_cast<float>(kFar)) {
          // The values' exponents lie too far apart for the factors: the sums of
          // the weights 2^x themselves, each warp's with its own largest as unit
#pragma unroll 1
          for (int c = 0; c < R; c += 16) {
            float x[16], x1[16];
            scores(0, c, x);
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] -= ps0.ve, x1[r] = -kInf;
            if (tiles == 2) {
              scores(1, c, x1);
#pragma unroll
              for (int r = 0; r < 16; ++r) x1[r] -= ps1.ve;
            }
            float unit = -kInf;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const float m = warp_max(fmaxf(x[r], x1[r])), ref = m == -kInf ? 0.f : m;
              x[r] = ex2(x[r] - ref) + ex2(x1[r] - ref);
              if ((lane & 15) == r) unit = m;
            }
            const float sum = column_sums<16>(x, lane);
            if (lane < 16) far_s[turn][q][c + lane] = make_float2(sum, unit);
          }
        } else {
          const auto code = [&](float ve) {  // of 2^(low - ve), in [2^-9, 1]
            const int e = static_cast<int>(low - ve);
            return static_cast<unsigned char>(e >= -6 ? (e + 7) << 3 : 1 << (e + 9));
          };
          factors[0] = code(ps0.ve);
          factors[S::kOnes] = code(ps1.ve);
        }
        __syncwarp();
        if (q == 0 && leader) mbar_arrive(&bar.mfull[turn]);
#pragma unroll 1
        for (int sub = 0; sub < tiles; ++sub) {
#pragma unroll 1
          for (int c = 0; c < R; c += 16) {
            float y[16];
            scores(sub, c, y);
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
              const float4 f = lds_f4(refs + c + r);
              const float2 a = fadd2(make_float2(y[r], y[r + 1]), make_float2(-f.x, -f.y));
              const float2 b = fadd2(make_float2(y[r + 2], y[r + 3]), make_float2(-f.z, -f.w));
              y[r] = ex2(a.x), y[r + 1] = ex2(a.y), y[r + 2] = ex2(b.x), y[r + 3] = ex2(b.y);
            }
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) split2(y[2 * i], y[2 * i + 1], hi[i], lo[i]);
            unsigned char* p = weights + swizzled((sub * kTile + row) * S::kPRow + c, S::kPRow);
            *reinterpret_cast<uint4*>(p) =
                make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, hi[4] | hi[5] << 16, hi[6] | hi[7] << 16);
            *reinterpret_cast<uint4*>(p + S::kPHalf) =
                make_uint4(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16, lo[4] | lo[5] << 16, lo[6] | lo[7] << 16);
          }
        }
        tc_fence_before();
        fence_proxy_async();
        __syncwarp();
        if (leader) {
          mbar_arrive(&bar.sempty[sb]);
          mbar_arrive(&bar.pfull[turn]);
        }
      }
      if (!go) break;
      ++qn;
    }
  } else {
    // ---------------- outputs ----------------
    const int q = warp & 3, d = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    int it = 0, step = 0, qn = 0;
    bool ok = true;
    Piece w;
    while (true) {
      const bool got = next_piece(w);
      if (!meet(3, got)) break;
      const int row0 = w.block * R, qb = qn & 1;
      float2 acc[NP][R / 2];
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; r < R / 2; ++r) acc[p][r] = make_float2(0.f, 0.f);
      float unit = -kInf;  // log2 of the outputs' unit, of row d
      // of rows `lane` and `lane` + 32 (warp 0): the sum of weights, log2 of its unit
      constexpr int kMine = (R + 31) / 32;
      float sum[kMine], sum_unit[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) sum[i] = 0.f, sum_unit[i] = -kInf;
      const auto add = [&](int i, float s, float u) {  // s 2^u more (of nothing, u is -infinity and s 0 or NaN)
        const float next = fmaxf(sum_unit[i], u);
        sum[i] = (sum_unit[i] == -kInf ? sum[i] : sum[i] * ex2(sum_unit[i] - next)) + (u == -kInf ? s : s * ex2(u - next));
        sum_unit[i] = next;
      };
      bool go = true;
#pragma unroll 1
      for (int t = w.t0; t < w.t1; t += 2, ++step) {
        const int k = step & 1, tiles = min(2, w.t1 - t);
        const unsigned half = static_cast<unsigned>(step >> 1) & 1u;
        ok = at_wait(&bar.mfull[k], half, fault) && ok;
        if (d < R) {
          const float top = top_s[k][d], next = fmaxf(unit, top);
          mix_s[k][d] = make_float2(unit == -kInf ? 0.f : ex2(unit - next), top == -kInf ? 0.f : ex2(top - next));
          unit = next;
        }
        go = meet(3, ok);
        if (!go) break;
        const PageScale ps0 = scale_s[it % kScaleRing][0], ps1 = scale_s[(it + tiles - 1) % kScaleRing][0];
        it += tiles;
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
        if (q == 0) {
          const float low = fminf(ps0.ve_low, ps1.ve_low);
          const bool far = fmaxf(ps0.ve_high, ps1.ve_high) - low > static_cast<float>(kFar);
          if (!far) {
#pragma unroll 1
            for (int r = 0; r < R; r += 16) {
              float s[16];
              tmem_ld16(tmem_l + k * R + r, s);
              if (lane == 0) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                  *reinterpret_cast<float4*>(&sum_s[r + e]) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
              }
            }
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const int r = min(lane + 32 * i, R - 1);
            if (!far) {
              add(i, sum_s[r], top_s[k][r] - low);
            } else {
              for (int v = 0; v < 4; ++v) add(i, far_s[k][v][r].x, far_s[k][v][r].y);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (leader) {
          mbar_arrive(&bar.oempty[k]);
          mbar_arrive(&bar.mempty[k]);
        }
      }
      if (!go) break;
      constexpr int kLd = NP * 128 + 4;
      float* part = P.parts + (static_cast<long long>(2 * blockIdx.x) + max(w.part, 0)) * R * kLd;
      if (d < R) row_s[d] = unit;
      if (!meet(3, ok)) break;
      if (leader) mbar_arrive(&bar.qempty[qb]);
      ++qn;
      if (q == 0) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int r = lane + 32 * i;
          if (r >= R) break;
          const float s = sum[i], u = row_s[r];
          if (w.part < 0) {
            const int tok = (row0 + r) / P.G, g = row0 + r - tok * P.G;
            place_s[r] = tok >= P.n ? -1 : w.b * P.out_ld[0] + tok * P.out_ld[1] + (w.h * P.G + g) * P.out_ld[2];
            row_s[r] = s == 0.f || tok >= w.count ? 0.f : ex2(u - sum_unit[i]) / s;
          } else {
            float* e = part + r * kLd + NP * 128;
            __stcg(e, u);
            __stcg(e + 1, s);
            __stcg(e + 2, sum_unit[i]);
          }
        }
      }
      meet(3, true);
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
      meet(3, true);
    }
  }

  __syncthreads();
  if (*fault && tid == 0) {
    // copies still in flight land before the CTA exits: wait (bounded) for
    // the last phase of every stage that was issued
    uint64_t* first = bar.kfull;  // (vfull behind it)
    for (int k = 0; k < 2 * S::kStages + kPatchRing; ++k)
      if (issued_s >> k & 1u)
        mbar_wait(k < 2 * S::kStages ? first + k : &bar.landed[k - 2 * S::kStages], parity_s >> k & 1u);
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
      const float mine = __ldcg(e + NP * 128 + 1);
      sum += su == -kInf ? mine : mine * ex2(su - sum_unit);
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
  // (of trees of more than 512 nodes the masks of 64 rows do not fit)
  return rows <= 16 ? 16 : rows <= 32 || D > 128 || n > 512 ? 32 : rows <= 48 ? 48 : 64;
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
  e = cudaFuncSetAttribute(attend_kernel<R, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<R, NP>::kSmem + kMaskBytes);
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
  const int smem = Shape<R, NP>::kSmem + (p.parent ? a.n * static_cast<int>(2 * sizeof(typename Shape<R, NP>::Mask) + 2) : 0);
  if (smem > Shape<R, NP>::kSmem + kMaskBytes) return SPEC_EINVAL;  // (block_rows sees to it)
  attend_kernel<R, NP><<<ctas, kThreads, smem, s>>>(tk, tv, p);
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
