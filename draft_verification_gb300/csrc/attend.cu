// Attention of drafted rows over the paged 8-bit cache (spec_attend_cache).
//
// The rows of one sequence that read one head of the cache, n rows of Hq / H
// query heads each, are cut into blocks of R (8 to 64).  For a tile of 128
// tokens a block needs
//    S^T [128 tokens x R] = K [128 x D] Q^T,   O^T [D x R] = V^T [D x 128] P^T,
// P = 2^(scores - maximum): tokens, then elements, are the 128 rows of a
// tensor-core product and the block's rows its N columns, so that few rows
// cost few columns.  The codes are e4m3 and go to the tensor cores as they
// lie in memory (tcgen05.mma kind::f8f6f4), K with D and V with the tokens as
// the inner products' axis; nothing is unpacked.  The other operands keep
// their precision as sums of two e4m3 numbers x = hi + lo, lo = e4m3(x - hi),
// side by side as rows of one product:
//    a query relative to its largest element (bfloat16's 8 significant bits
//       are the two's, so it is exact down to 2^-18 of that element);
//    a weight relative to the largest of its step (one or two tiles) and row,
//       hence from 256 down to 2^-9 / 2: rows whose first tokens have nearly
//       all the weight keep the others' precision.
// A page's exponents are 2's powers and uniform over a token: one factor per
// thread for K; V's exponent is added to the score before the maximum, so that
// P carries it (y = x + ve).  The sum of the weights is a third product, of P
// with one row of factors 2^(least ve - ve) that take it back; where a step's
// exponents lie far apart the weights' warps sum 2^x themselves.
//
// Persistent CTAs, two per SM up to 24 rows, take equal runs of the tiles of
// all blocks, in the order sequence, head, block; a block that CTAs share is
// left in parts in the workspace and joined by a second kernel (in order, so
// that the sums do not depend on the timing).  Warps: 0 copies pages (TMA,
// 128-byte swizzle) into rings of K and V tiles; 1 issues the scores' products;
// 2 finds the pieces of the CTA's run and makes their queries' codes and tree
// masks; 3 issues the outputs' products; 4-7 and 8-11 turn the scores of every
// other step into weights (and clear V behind the last token); 12-15 add the
// steps' outputs up in registers.  All waits are bounded, and the warps of a
// role leave it together.
//
// What bounds it: up to 32 rows the bytes (1.07 GB of cache, 8 heads of 128,
// 4 query heads each: 2 rows 167 us, 96 % of a copy's rate; 6 rows 176, 91 %;
// 8 rows 192, 84 %), above that the instructions of the weights' warps (12
// rows, blocks of 48: 241 us, 67 %; 16, blocks of 64: 285, 57 %): some 18 per
// score, at a third of the issue slots.  Beside its tiles (1.16 us each with 64
// rows) a block costs queries, masks, outputs and its share of the joining: 16
// trees of 64 nodes over 4096 tokens take 236 us, 127 of them for the 110 tiles
// of a CTA, the others for its 3.4 blocks.
// Short calls are latency: one piece takes about 14,000 cycles from launch to
// the end, a third of it until the lengths, the block table and the queries
// have come.
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

constexpr int kTile = 128;      // tokens per tile; one or two tiles make a step
constexpr int kPanel = 16384;   // bytes of 128 tokens x 128 elements
constexpr int kMaxRows = 1024;  // n
constexpr int kMaxCtas = 320;
constexpr int kThreads = 512;
constexpr int kMaskBytes = 10 * kMaxRows;  // of shared memory for a tree's masks, at most
constexpr int kScaleRing = 32, kPatchRing = 8, kPieceRing = 4;
// Value exponents of a step that lie further apart than this: its weights are
// summed apart.  Weights are held to 2^-18 of the step's largest, exponents
// included, so their sum without them to 2^(kFar - 18) of the largest per token.
constexpr int kFar = 3;

// R: a block's rows; NP: panels of 128 elements of a head.
template <int R, int NP>
struct Shape {
  // CTAs per SM: two, whose roles fill each other's waits, as long as registers
  // (64 a thread) and memories hold them.  Tiles of a step: two share a maximum, a
  // meeting and their hand-overs.  Measured both ways on the form that the kernel
  // had when this was chosen (its calls take 150 and 132 us now): 64 chains of 6
  // rows of 4 heads, 24 rows, two CTAs per SM 190 us, one 225; 36 rows, 2 x 131072
  // tokens, steps of two tiles 187 us, of one 192; 24 rows, one CTA per SM, steps
  // of two tiles 241 us, of one 225.
  static constexpr int kCtas = NP == 1 && R <= 24 ? 2 : 1;
  static constexpr int kSubs = NP == 1 && R >= 32 ? 2 : 1;
  // An operand from shared memory costs its bytes (a product of 128 x 32 with 32
  // rows some 60 cycles, with 64 hardly more), so K and V are taken once for hi
  // and lo: as rows of their own, whose results are added later.  Where tensor
  // memory is short (64 rows) the outputs' hi and lo are two products instead.
  static constexpr bool kStackedS = R <= 32;   // the scores' hi and lo
  static constexpr bool kStacked = R <= 48;    // the outputs'
  static constexpr bool kStackedL = R <= 32;   // the sums'
  // places of K tiles, and as many of V tiles (each with barriers of its own: a
  // warp has to meet all phases of a barrier that it waits on)
  static constexpr int kStages = NP == 2 || kCtas == 2 ? 2 : R > 32 ? 3 : 4;
  static constexpr int kSlot = NP * kPanel;
  // a token's weights: hi's rows, then lo's, in one row of bytes, or in two planes
  static constexpr int kPRow = !kStacked ? R : R == 48 ? 128 : R == 24 ? 64 : 2 * R;
  static constexpr int kPPlane = kTile * kPRow;
  static constexpr int kPTile = kPPlane * (kStacked ? 1 : 2);  // a tile's weights
  static constexpr int kQBytes = NP * 2 * R * 128;  // a block's queries: of each panel hi's rows, then lo's
  static constexpr int kScores = R <= 16 && NP == 1 ? 4 : 2;  // places of steps' scores
  static constexpr int kCut = R == 48 ? 24 : R < 32 ? R : 32;  // rows that the softmax warps take at a time
  static constexpr int kOnes = 1024;  // a tile's factors of the sums of weights (one row of 128 bytes)
  static constexpr int kSmem = 1024 + 2 * kStages * kSlot + 2 * kQBytes + 2 * kSubs * (kPTile + kOnes);
  static constexpr int kLBufs = R == 24 && kCtas == 2 ? 1 : 2;  // places of the sums
  // (a product of bytes whose rows lie along the other axis takes 16 of them at a time)
  static_assert(kStackedL ? 2 * R % 16 == 0 : R % 16 == 0, "the sums' products");
  static constexpr int kSCols = kStackedS ? 2 * R : R, kOCols = kStacked ? 2 * R : R, kLCols = kStackedL ? 2 * R : R;
  static constexpr int kCols = kScores * kSubs * kSCols + 2 * NP * kOCols + kLBufs * kLCols;
  static constexpr uint32_t kTmemCols = kCols <= 256 ? 256 : 512;
  static_assert(kCols * kCtas <= 512 && (kScores + 4) * kSubs + kStages + 1 <= kScaleRing && 2 * kStages + kPatchRing <= 32, "rings");
  using Mask = typename std::conditional<(R > 32), unsigned long long, unsigned>::type;  // a bit per row of a block
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
  float2* far;       // [ctas][4][4][64]: of a step whose value exponents lie far apart, each warp's sums and units
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

__device__ __forceinline__ bool mbar_test(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

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

// The warps of a role, kCount threads, meet, and go on only if all of them can
// (so that they leave the role together when a wait gave up).
template <int kCount>
__device__ __forceinline__ bool meet(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(id), "n"(kCount)
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
// A warp's common value, so that the compiler takes it for one.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
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

// Four values as hi + lo, four e4m3 codes each.
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t& hi, uint32_t& lo) {
  asm("{\n .reg .b32 x, y, u, v;\n .reg .b16 p, q, r, s;\n"
      " cvt.rn.f16x2.f32 x, %3, %2;\n cvt.rn.f16x2.f32 y, %5, %4;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 p, x;\n cvt.rn.satfinite.e4m3x2.f16x2 q, y;\n mov.b32 %0, {p, q};\n"
      " cvt.rn.f16x2.e4m3x2 u, p;\n cvt.rn.f16x2.e4m3x2 v, q;\n sub.f16x2 x, x, u;\n sub.f16x2 y, y, v;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 r, x;\n cvt.rn.satfinite.e4m3x2.f16x2 s, y;\n mov.b32 %1, {r, s};\n}"
      : "=r"(hi), "=r"(lo)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}

// 8 bytes of global memory to shared memory, or zeros; and the thread's wait for all of them.
__device__ __forceinline__ void copy8_async(void* to, const void* from, bool has) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(has ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Two float32 numbers in a register pair, each lane rounded as by itself (in
// 64 bits throughout: as two floats the pairs cost moves at every operation).
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float first_of(F2 x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float second_of(F2 x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ ulonglong2 lds_pairs(const void* p) { return *static_cast<const ulonglong2*>(p); }

// Both rounded to bfloat16, the first in the lower half.
__device__ __forceinline__ uint32_t pack_bf16(F2 x) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(second_of(x)), "f"(first_of(x)));
  return d;
}

// Consecutive float32 columns of this warp's 32 lanes, in pairs.
__device__ __forceinline__ void tmem_load8(uint32_t taddr, F2* v) {
  asm volatile(
      "{\n .reg .b32 a<8>;\n tcgen05.ld.sync.aligned.32x32b.x8.b32 {a0, a1, a2, a3, a4, a5, a6, a7}, [%4];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      " mov.b64 %0, {a0, a1};\n mov.b64 %1, {a2, a3};\n mov.b64 %2, {a4, a5};\n mov.b64 %3, {a6, a7};\n}"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t taddr, F2* v) {
  asm volatile(
      "{\n .reg .b32 a<16>;\n"
      " tcgen05.ld.sync.aligned.32x32b.x16.b32 {a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15}, "
      "[%8];\n tcgen05.wait::ld.sync.aligned;\n"
      " mov.b64 %0, {a0, a1};\n mov.b64 %1, {a2, a3};\n mov.b64 %2, {a4, a5};\n mov.b64 %3, {a6, a7};\n"
      " mov.b64 %4, {a8, a9};\n mov.b64 %5, {a10, a11};\n mov.b64 %6, {a12, a13};\n mov.b64 %7, {a14, a15};\n}"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]), "=l"(v[7])
      : "r"(taddr)
      : "memory");
}
// N columns, a multiple of 8
template <int N>
__device__ __forceinline__ void tmem_pairs(uint32_t taddr, F2* v) {
  if constexpr (N >= 16) {
    tmem_load16(taddr, v);
    if constexpr (N > 16) tmem_pairs<N - 16>(taddr + 16, v + 8);
  } else {
    tmem_load8(taddr, v);
  }
}

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
__global__ void __launch_bounds__(kThreads, Shape<R, NP>::kCtas)
    attend_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const AttendParams P) {
  using S = Shape<R, NP>;
  constexpr int kCut = S::kCut;
  extern __shared__ __align__(1024) unsigned char at_dyn[];
  // kfull / kempty, vfull / vempty: a tile's K, V; sfull / sempty: a step's scores; pfull /
  // pempty: its weights in shared memory; ofull / oempty: its outputs; mfull /
  // mempty: its maxima (top_s); qfull / qempty: a piece's queries; rfull /
  // rempty: its record; landed: V of a tile that is patched before it is
  // vfull; drain: no product is under way
  struct Bars {
    uint64_t kfull[S::kStages], vfull[S::kStages], kempty[S::kStages], vempty[S::kStages];
    uint64_t sfull[S::kScores], sempty[S::kScores], pfull[2], pempty[2], ofull[2], oempty[2], mfull[2], mempty[2];
    uint64_t qfull[2], qempty[2], landed[kPatchRing], rfull[kPieceRing], rempty[kPieceRing], drain[2];
  };
  constexpr int kBars = sizeof(Bars) / 8;
  __shared__ Bars bar;
  __shared__ uint32_t tmem_s;
  __shared__ int fault_s;
  __shared__ unsigned issued_s, parity_s;  // (see the copying warp)
  __shared__ __align__(16) Piece piece_s[kPieceRing];
  __shared__ __align__(16) PageScale scale_s[kScaleRing][8];
  __shared__ int copies_s[kScaleRing][9];  // rows of the pages' copies, -1: none; a copy's bytes, negative: patched
  __shared__ __align__(16) float most_s[2][2][4][kCut], ref_s[8][kCut], cq_s[2][R], top_s[2][R], sum_s[R];
  __shared__ __align__(16) float keep_s[2][R], take_s[2][R];
  __shared__ __align__(16) float row_s[R];
  __shared__ __align__(16) long long place_s[R];

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool leader = one_lane();
  unsigned char* kring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(at_dyn) + 1023) &
                                                          ~static_cast<uintptr_t>(1023));
  unsigned char* vring = kring + S::kStages * S::kSlot;
  unsigned char* qbuf = vring + S::kStages * S::kSlot;
  unsigned char* pbuf = qbuf + 2 * S::kQBytes;
  unsigned char* ones = pbuf + 2 * S::kSubs * S::kPTile;
  using Mask = typename S::Mask;
  Mask* mask_s = reinterpret_cast<Mask*>(ones + 2 * S::kSubs * S::kOnes);  // [2][n], with parents
  unsigned short* parent_s = reinterpret_cast<unsigned short*>(mask_s + 2 * P.n);
  volatile int* fault = &fault_s;
  float2* far_sums = P.far + blockIdx.x * 1024;

  pdl_launch_dependents();
  if (tid < kBars) {
    uint64_t* at = reinterpret_cast<uint64_t*>(&bar) + tid;
    unsigned count = 1;
    if (at >= bar.sfull && at < bar.sempty) count = 2;   // sfull
    if (at >= bar.ofull && at < bar.oempty) count = 2;   // ofull
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
  for (int i = tid; i < 2 * S::kSubs * S::kOnes / 16; i += kThreads) reinterpret_cast<uint4*>(ones)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  // the tiles of a sequence; those of this lane's, found while tensor memory is allocated
  const auto lengths = [&](int b) { return lengths_of(P, b); };
  const auto tiles_of_seq = [&](const Lengths& s) {
    int n = 0;
#pragma unroll 1
    for (int i = 0; i < P.blocks; ++i) n += tiles_of(keys_of<R>(P, s, i));
    return n * P.H;
  };
  const int own = warp == 2 && lane < P.B ? tiles_of_seq(lengths(lane)) : 0;
  if (warp == 1) {
    tmem_alloc(&tmem_s, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_sc = tmem_s, tmem_o = tmem_s + S::kScores * S::kSubs * S::kSCols, tmem_l = tmem_o + 2 * NP * S::kOCols;

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
    // (some 40 instructions per copy: more, and this warp would be what the others wait for)
    const int pp = kTile / P.page, slot_in = lane % pp, mine = lane / pp, batch = 32 / pp;
    const unsigned page_bytes = static_cast<unsigned>(P.page) * 128u;
    int it = 0;
    bool ok = true;
    unsigned issued = 0, parities = 0;  // barriers that copies count on (kfull, vfull, landed), the last one's parity
    const auto count_on = [&](uint64_t* full, int number, unsigned parity, unsigned bytes) {
      if (leader) mbar_expect_tx(full, bytes);
      issued |= 1u << number;
      parities = (parities & ~(1u << number)) | parity << number;
    };
    int kslot = 0, vslot = 0, vt = 0, patches = 0;  // the places of the next tiles, the next tile of V
    unsigned kparity = 0, vparity = 0;
    const auto v_free = [&] { return vt < it && __all_sync(0xffffffffu, mbar_test(&bar.vempty[vslot], vparity ^ 1u)); };
    const auto copy_v = [&] {
      const int x = copies_s[vt % kScaleRing][lane < 9 ? lane : 8];  // rows of the pages' copies, bytes and a flag
      const unsigned y = static_cast<unsigned>(__shfl_sync(0xffffffffu, x, 8));
      const unsigned bytes = y & 0x7fffffffu;
      uint64_t* full = &bar.vfull[vslot];
      if (y >> 31) {  // a tile that is patched
        full = &bar.landed[patches % kPatchRing];
        count_on(full, 2 * S::kStages + patches % kPatchRing, static_cast<unsigned>(patches / kPatchRing) & 1u, bytes);
        ++patches;
      } else {
        count_on(full, S::kStages + vslot, vparity, bytes);
      }
      if (lane < pp && x >= 0) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
          tma_load_2d(vring + vslot * S::kSlot + lane * page_bytes + p * kPanel, &tm_v, p * 128, x, full);
      }
      __syncwarp();
      ++vt;
      if (++vslot == S::kStages) vslot = 0, vparity ^= 1u;
    };
    // Waits for a barrier; V's copies go on meanwhile.
    const auto wait_for = [&](uint64_t* on, unsigned parity) {
#pragma unroll 1
      for (int polls = 0; polls < 8 * kMaxPolls; ++polls) {
        if (v_free()) copy_v();
        if (__all_sync(0xffffffffu, mbar_test(on, parity))) return true;
        if ((polls & 15) == 15 && __any_sync(0xffffffffu, *fault)) return false;
      }
      *fault = 1;
      return false;
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
        x.ve = static_cast<float>(has ? ve : lo);  // (behind the last page: one that is there)
        x.ve_low = static_cast<float>(lo);
        x.ve_high = static_cast<float>(hi);
        const int y = has ? static_cast<int>(slab * P.page) : -1;
        // the bytes of this lane's tile's K, or V, and whether it is patched
        const unsigned all = __ballot_sync(0xffffffffu, has);
        const unsigned bytes =
            static_cast<unsigned>(__popc(all >> (mine * pp) & ((1u << pp) - 1u))) * page_bytes * NP + P.more_bytes;
        const int flags = static_cast<int>(bytes | (tb + mine >= special ? 0x80000000u : 0u));
#pragma unroll 1
        for (int i = 0; i < batch && tb + i < w.t1; ++i) {
          if (mine == i) {
            const int at = it % kScaleRing;
            scale_s[at][slot_in] = x;
            copies_s[at][slot_in] = y;
            if (slot_in == 0) copies_s[at][8] = flags;
          }
          __syncwarp();
          const unsigned k_bytes = __shfl_sync(0xffffffffu, bytes, i * pp);
          ok = wait_for(&bar.kempty[kslot], kparity ^ 1u);
          if (!ok) break;
          count_on(&bar.kfull[kslot], kslot, kparity, k_bytes);
          if (mine == i && has) {
#pragma unroll
            for (int p = 0; p < NP; ++p)
              tma_load_2d(kring + kslot * S::kSlot + slot_in * page_bytes + p * kPanel, &tm_k, p * 128, y,
                          &bar.kfull[kslot]);
          }
          __syncwarp();
          ++it;
          if (++kslot == S::kStages) kslot = 0, kparity ^= 1u;
        }
      }
      // the next record, which may come only when this piece is done
      ok = ok && wait_for(&bar.rfull[pieces % kPieceRing], static_cast<unsigned>(pieces / kPieceRing) & 1u);
    }
    while (ok && vt < it) {
      ok = at_wait(&bar.vempty[vslot], vparity ^ 1u, fault);
      if (ok) copy_v();
    }
    if (leader) issued_s = issued, parity_s = parities;
  } else if (warp == 1) {
    // ---------------- scores ----------------
    constexpr uint32_t idesc = idesc_e4m3(kTile, S::kSCols, 0, 0), high = operand_high(1024, 128);
    const int steps = (P.D + 31) / 32;
    const uint32_t issues = leader ? 1u : 0u;
    int it = 0, step = 0, qn = 0;
    bool ok = true;
    Piece w;
    while (ok && next_piece(w)) {
      const uint32_t q = uniform(operand_low(smem_addr(qbuf + (qn & 1) * S::kQBytes), 1024));
      ok = at_wait(&bar.qfull[qn & 1], static_cast<unsigned>(qn >> 1) & 1u, fault);
      ++qn;
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
        // (a step's two tiles, the second one perhaps missing)
        const int sb = step % S::kScores, sub = S::kSubs == 2 ? (t - w.t0) & 1 : 0;
        const Place<S::kStages> at(it);
        if (sub == 0) ok = at_wait(&bar.sempty[sb], (static_cast<unsigned>(step / S::kScores) & 1u) ^ 1u, fault);
        ok = ok && at_wait(&bar.kfull[at.slot], at.parity, fault);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = uniform(operand_low(smem_addr(kring + at.slot * S::kSlot), 1024));
        const uint32_t d = uniform(tmem_sc + (S::kSubs * sb + sub) * S::kSCols);
        umma_e4m3(issues, d, a, high, q, high, idesc, 0u);
#pragma unroll
        for (int e = 1; e < 4 * NP; ++e)  // steps of 32 elements
          if (e < steps)
            umma_e4m3(issues, d, a + (e >> 2) * (kPanel >> 4) + (e & 3) * 2, high,
                      q + (e >> 2) * (2 * R * 128 >> 4) + (e & 3) * 2, high, idesc, 1u);
        if constexpr (!S::kStackedS) {
#pragma unroll
          for (int e = 0; e < 4 * NP; ++e)
            if (e < steps)
              umma_e4m3(issues, d, a + (e >> 2) * (kPanel >> 4) + (e & 3) * 2, high,
                        q + (R * 128 >> 4) + (e >> 2) * (2 * R * 128 >> 4) + (e & 3) * 2, high, idesc, 1u);
        }
        commit_if(issues, &bar.kempty[at.slot]);
        if (sub == S::kSubs - 1 || t + 1 == w.t1) {
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
    int total = own;
#pragma unroll 1
    for (int b = lane + 32; b < P.B; b += 32) total += tiles_of_seq(lengths(b));
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
        const int n = b1 == 0 ? own : b1 + lane < P.B ? tiles_of_seq(lengths(b1 + lane)) : 0;
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
        // The block's rows: two e4m3 numbers for each element.  A lane's 8 elements
        // of a row are copied to where their 16 codes will lie, all rows at once, and
        // are turned into codes there.  (One warp does it beside the other roles'
        // work: short loops, since it waits for instructions most of all.)
        constexpr int kLanes = 16 * NP;       // lanes of a row, 8 elements each
        constexpr int kAtOnce = 32 / kLanes;  // rows at a time
        const int qb = qn & 1, row0 = block * R, tok0 = row0 / P.G, d0 = lane % kLanes * 8, r0 = lane / kLanes;
        ok = at_wait(&bar.qempty[qb], (static_cast<unsigned>(qn >> 1) & 1u) ^ 1u, fault);
        if (!ok) break;
        unsigned char* dst = qbuf + qb * S::kQBytes + (d0 >> 7) * 2 * R * 128;
        const auto place = [&](int r) { return dst + swizzled(r * 128 + (d0 & 127), 128); };
        {
          const bf16_t* q = P.q + b * P.q_ld[0] + static_cast<long long>(h) * P.G * P.q_ld[2] + d0;
          int tok = (row0 + r0) / P.G, g = row0 + r0 - tok * P.G;
#pragma unroll 4
          for (int r1 = 0; r1 < R; r1 += kAtOnce) {
            const int r = r1 + r0;
            const bool has = tok < s.count && d0 < P.D;
            const bf16_t* from = has ? q + tok * P.q_ld[1] + g * P.q_ld[2] : P.q;
            unsigned char* to = place(r);
            copy8_async(to, from, has);
            copy8_async(to + R * 128, from + (has ? 4 : 0), has);
            for (g += kAtOnce; g >= P.G; g -= P.G) ++tok;
          }
        }
        copies_wait();
#pragma unroll 4
        for (int r1 = 0; r1 < R; r1 += kAtOnce) {
          const int r = r1 + r0;
          uint2* to = reinterpret_cast<uint2*>(place(r));
          const uint2 x = to[0], y = to[R * 16];
          const uint32_t sign = 0x7fff7fffu;
          uint32_t m = __vmaxu2(__vmaxu2(x.x & sign, x.y & sign), __vmaxu2(y.x & sign, y.y & sign));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
          m = max(m & 0xffffu, m >> 16);  // the row's largest magnitude
          const bool lost = m >= 0x7f80u;
          // the least exponent with magnitude <= 448 2^eq
          const int eq = lost ? 0 : max(static_cast<int>(m >> 7) - 127 - ((m & 0x7fu) <= 0x60u ? 8 : 7), -100);
          const float f = exp2i(-eq);
          uint2 hi, lo;
          split4(bf16_lo(x.x) * f, bf16_hi(x.x) * f, bf16_lo(x.y) * f, bf16_hi(x.y) * f, hi.x, lo.x);
          split4(bf16_lo(y.x) * f, bf16_hi(y.x) * f, bf16_lo(y.y) * f, bf16_hi(y.y) * f, hi.y, lo.y);
          to[0] = hi;
          to[R * 16] = lo;
          if (d0 == 0) cq_s[qb][r] = lost ? __uint_as_float(0x7fc00000u) : exp2i(eq) * P.c;
        }
        if (P.parent) {
          // which of the block's rows see drafted token j
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
          for (int tok = tok0 + lane; tok < s.count && tok * P.G < row0 + R; tok += 32) {
            const int from = max(tok * P.G - row0, 0), many = min((tok + 1) * P.G - row0, R) - from;
            const Mask bits = (~static_cast<Mask>(0) >> (8 * sizeof(Mask) - many)) << from;
            for (int j = tok;; j = parent_s[j]) {
              unsigned* m = reinterpret_cast<unsigned*>(mask + j);
              if (static_cast<unsigned>(bits)) atomicOr(m, static_cast<unsigned>(bits));
              if constexpr (sizeof(Mask) == 8)
                if (bits >> 32) atomicOr(m + 1, static_cast<unsigned>(bits >> 32));
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
    constexpr uint32_t idesc = idesc_e4m3(128, S::kOCols, 1, 1), idesc_l = idesc_e4m3(64, S::kLCols, 0, 1);
    constexpr uint32_t a_high = operand_high(1024, 128), b_high = operand_high(8 * S::kPRow, S::kPRow);
    const uint32_t issues = leader ? 1u : 0u;
    int it = 0, step = 0;
    bool ok = true;
    Piece w;
    while (ok && next_piece(w)) {
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
        const int k = step & 1, sub = S::kSubs == 2 ? (t - w.t0) & 1 : 0;
        const unsigned half = static_cast<unsigned>(step >> 1) & 1u;
        if (sub == 0)
          ok = at_wait(&bar.oempty[k], half ^ 1u, fault) && at_wait(&bar.pfull[k], half, fault);
        const Place<S::kStages> at(it);
        ok = ok && at_wait(&bar.vfull[at.slot], at.parity, fault);
        if (!ok) break;
        tc_fence_after();
        const uint32_t b = uniform(operand_low(smem_addr(pbuf + (S::kSubs * k + sub) * S::kPTile), 8 * S::kPRow));
        const uint32_t a0 = uniform(operand_low(smem_addr(vring + at.slot * S::kSlot), 1024));
        const uint32_t o0 = uniform(tmem_o + k * NP * S::kOCols), l = uniform(tmem_l + (S::kLBufs == 2 ? k : 0) * S::kLCols);
        const uint32_t first = sub == 0 ? 0u : 1u;
        constexpr int kB = 32 * S::kPRow >> 4, kPlane = S::kPPlane >> 4;  // 32 tokens, lo's plane
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const uint32_t a = a0 + p * (kPanel >> 4), o = o0 + p * S::kOCols;
#pragma unroll
          for (int i = 0; i < (S::kStacked ? 4 : 8); ++i)  // 4 steps of 32 tokens, hi's, then lo's
            umma_e4m3(issues, o, a + (i & 3) * (32 * 128 >> 4), a_high, b + (i >> 2) * kPlane + (i & 3) * kB, b_high, idesc,
                      i == 0 ? first : 1u);
        }
        if (S::kLBufs == 1 && sub == 0 && step > 0) {
          ok = at_wait(&bar.oempty[k ^ 1], static_cast<unsigned>((step - 1) >> 1) & 1u, fault);
          if (!ok) break;
        }
        // the sums of the weights: products with one row of factors (every 8 rows of
        // the operand are the same, a stride of 0), the first of the 64 results is used
        const uint32_t f = uniform(operand_low(smem_addr(ones + (S::kSubs * k + sub) * S::kOnes), 0));
        constexpr int kLo = S::kStacked ? R >> 4 : kPlane;  // from hi's weights to lo's
#pragma unroll
        for (int i = 0; i < (S::kStackedL ? 4 : 8); ++i)
          umma_e4m3(issues, l, f + (i & 3) * 2, operand_high(0, 128), b + (i >> 2) * kLo + (i & 3) * kB, b_high, idesc_l,
                    i == 0 ? first : 1u);
        commit_if(issues, &bar.vempty[at.slot]);
        if (sub == S::kSubs - 1 || t + 1 == w.t1) {
          commit_if(issues, &bar.ofull[k]);
          if (leader) mbar_arrive(&bar.ofull[k]);  // what the weights' warps wrote is visible behind it
          commit_if(issues, &bar.pempty[k]);
          ++step;
        }
      }
    }
    commit_if(issues, &bar.drain[1]);
    mbar_wait(&bar.drain[1], 0);
  } else if (warp < 12) {
    // ---------------- weights ----------------
    // Every other step, kCut of the block's rows at a time; a thread has a token
    // of each of the step's tiles and keeps its scores in registers.
    const int turn = (warp - 4) >> 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    const int page_row = row / P.page;
    const int col = lane < kCut ? lane : 0;  // the row that this lane sees to
    float* refs = ref_s[warp - 4];
    unsigned char* weights = pbuf + S::kSubs * turn * S::kPTile;
    int it = 0, step = 0, qn = 0, patches = 0;
    bool ok = true;  // (what a wait of this warp's gave; the warpgroup goes by what its warps agree on)
    Piece w;
    while (true) {
      const bool got = next_piece(w);
      if (!meet<128>(1 + turn, got)) break;
      const int special = first_special(w), qb = qn & 1;
      bool go = true;
#pragma unroll 1
      for (int t = w.t0; t < w.t1; t += S::kSubs, ++step) {
        const int tiles = S::kSubs == 2 ? min(2, w.t1 - t) : 1;
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
        using Mask = typename S::Mask;
        const bool special_step = t + tiles > special;
        Mask seen0 = ~static_cast<Mask>(0), seen1 = seen0;
        bool nan0 = false, nan1 = false;
        if (special_step) {
          // V of what no row sees is cleared, and NaN values of drafted tokens, which
          // are passed on by the scores (a drafted token that a row does not see must
          // not reach it).  Of the ring's phases this warp meets some: 8 patched tiles
          // earlier is at least 4 steps earlier, whose outputs are known to be done.
          const auto look = [&](int tile, int number, int patch, Mask& seen, bool& nan) {
            if (tile < special) return;
            const int pos = tile * kTile + row, j = pos - w.prefix;
            bool clear = pos >= w.keys;
            if (clear) seen = 0;
            else if (j >= 0 && P.parent) seen = mask_s[qb * P.n + j];
            else if (j * P.G > w.block * R) seen = j * P.G >= w.block * R + R ? 0 : seen << (j * P.G - w.block * R);
            ok = at_wait(&bar.landed[patch % kPatchRing], static_cast<unsigned>(patch / kPatchRing) & 1u, fault) && ok;
            const Place<S::kStages> v_at(number);
            unsigned char* v = vring + v_at.slot * S::kSlot + row * 128;
            if (!clear && j >= 0) {
#pragma unroll 1
              for (int p = 0; p < NP; ++p)
#pragma unroll 2
                for (int o = 0; o < 8; ++o) {
                  const uint4 x = *reinterpret_cast<const uint4*>(v + p * kPanel + ((o + lane) & 7) * 16);
                  const uint32_t m = 0x7f7f7f7fu, one = 0x01010101u;
                  nan |= ((((x.x & m) + one) | ((x.y & m) + one) | ((x.z & m) + one) | ((x.w & m) + one)) & 0x80808080u) != 0;
                }
              clear = nan;
            }
            if (clear) {
#pragma unroll 1
              for (int p = 0; p < NP; ++p)
#pragma unroll 2
                for (int o = 0; o < 8; ++o)
                  *reinterpret_cast<uint4*>(v + p * kPanel + ((o + lane) & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            // (the outputs' products wait for the weights too, hence for all four warps)
            if (q == 0 && leader) mbar_arrive(&bar.vfull[v_at.slot]);
          };
          look(t, at, patch, seen0, nan0);
          if (tiles == 2) look(t + 1, at + 1, patch + (t >= special ? 1 : 0), seen1, nan1);
        }
        const float low = fminf(ps0.ve_low, ps1.ve_low);
        const bool far = fmaxf(ps0.ve_high, ps1.ve_high) - low > static_cast<float>(kFar);
#pragma unroll 1
        for (int c = 0; c < R; c += kCut) {
          // scores, base 2, plus the value exponent, of rows c on
          F2 y0[kCut / 2], y1[kCut / 2];
          const auto scores = [&](int sub, const PageScale& ps, F2* y) {
            const uint32_t from = tmem_sc + (S::kSubs * sb + sub) * S::kSCols + c + lanes;
            const F2 ck = pair(ps.ck, ps.ck), ve = pair(ps.ve, ps.ve);
            tmem_pairs<kCut>(from, y);
#pragma unroll
            for (int i = 0; i < kCut / 2; i += 4) {  // hi's and lo's
              if constexpr (S::kStackedS) {
                F2 lo[4];
                tmem_load8(from + R + 2 * i, lo);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[i + j] = add2(y[i + j], lo[j]);
              }
              const ulonglong2 f = lds_pairs(&cq_s[qb][c + 2 * i]), g = lds_pairs(&cq_s[qb][c + 2 * i + 4]);
              y[i] = fma2(mul2(y[i], f.x), ck, ve);
              y[i + 1] = fma2(mul2(y[i + 1], f.y), ck, ve);
              y[i + 2] = fma2(mul2(y[i + 2], g.x), ck, ve);
              y[i + 3] = fma2(mul2(y[i + 3], g.y), ck, ve);
            }
          };
          scores(0, ps0, y0);
          if (tiles == 2) {
            scores(1, ps1, y1);
          } else {
#pragma unroll
            for (int i = 0; i < kCut / 2; ++i) y1[i] = pair(-kInf, -kInf);
          }
          if (special_step) {
            const auto cover = [&](F2* y, Mask rows, bool nan) {
              const unsigned seen = static_cast<unsigned>(rows >> c);
              const float none = -kInf, lost = __uint_as_float(0x7fc00000u);
              if (nan) {
#pragma unroll
                for (int i = 0; i < kCut / 2; ++i) y[i] = pair(lost, lost);
              }
#pragma unroll
              for (int i = 0; i < kCut / 2; ++i)
                y[i] = pair(seen & 1u << 2 * i ? first_of(y[i]) : none, seen & 2u << 2 * i ? second_of(y[i]) : none);
            };
            cover(y0, seen0, nan0);
            if (tiles == 2) cover(y1, seen1, nan1);
          }
          // the rows' largest (stored by all lanes: a branch costs the warp more)
          const int slot = S::kCut == R ? step >> 1 & 1 : c == 0 ? 0 : 1;
          const auto top = [&](int i) {
            return make_float2(warp_max(fmaxf(first_of(y0[i]), first_of(y1[i]))),
                               warp_max(fmaxf(second_of(y0[i]), second_of(y1[i]))));
          };
#pragma unroll
          for (int i = 0; i < kCut / 2; i += 2) {
            const float2 a = top(i), b = top(i + 1);
            *reinterpret_cast<float4*>(&most_s[turn][slot][q][2 * i]) = make_float4(a.x, a.y, b.x, b.y);
          }
          go = meet<128>(1 + turn, ok);
          if (!go) break;
          // every warp for itself: a lane per row
          const float m = fmaxf(fmaxf(most_s[turn][slot][0][col], most_s[turn][slot][1][col]),
                                fmaxf(most_s[turn][slot][2][col], most_s[turn][slot][3][col]));
          refs[col] = m == -kInf ? 0.f : 8.f - m;  // (negated)
          __syncwarp();
          if (q == 0) {
            if (c == 0) ok = at_wait(&bar.mempty[turn], half ^ 1u, fault);
            top_s[turn][c + col] = m - 8.f;
            __syncwarp();
            if (leader && c + kCut == R) mbar_arrive(&bar.mfull[turn]);
          }
          if (c == 0) {
            ok = at_wait(&bar.pempty[turn], half ^ 1u, fault) && ok;
            if (!far) {
              static_assert(kFar <= 6, "normal e4m3 numbers");
              const auto code = [&](float ve) {  // of 2^(low - ve), in [2^-kFar, 1]
                return static_cast<unsigned char>((static_cast<int>(low - ve) + 7) << 3);
              };
              ones[S::kSubs * turn * S::kOnes + row] = code(ps0.ve);
              if (S::kSubs == 2) ones[(S::kSubs * turn + 1) * S::kOnes + row] = code(ps1.ve);
            }
          }
          if (far) {
            // The values' exponents lie too far apart for the factors: the sums of
            // the weights 2^x themselves, each warp's with its own largest as unit.
            // (Behind the wait for pempty: the products of step - 2 are done, so
            // they were begun, behind oempty of step - 4, whose sums lay in this
            // place: they have been read.)
#pragma unroll
            for (int r = 0; r < kCut; ++r) {
              const float x0 = (r & 1 ? second_of(y0[r / 2]) : first_of(y0[r / 2])) - ps0.ve;
              const float x1 = (r & 1 ? second_of(y1[r / 2]) : first_of(y1[r / 2])) - ps1.ve;
              const float unit = warp_max(fmaxf(x0, x1)), ref = unit == -kInf ? 0.f : unit;
              float sum = ex2(x0 - ref) + ex2(x1 - ref);
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              if (lane == 0) __stcg(far_sums + (4 * (step & 3) + q) * 64 + c + r, make_float2(sum, unit));
            }
          }
          const auto store = [&](int sub, const F2* y) {
            uint32_t hi[kCut / 4], lo[kCut / 4];
#pragma unroll
            for (int i = 0; i < kCut / 2; i += 2) {
              const ulonglong2 f = lds_pairs(refs + 2 * i);
              const F2 a = add2(y[i], f.x), b = add2(y[i + 1], f.y);
              split4(ex2(first_of(a)), ex2(second_of(a)), ex2(first_of(b)), ex2(second_of(b)), hi[i / 2], lo[i / 2]);
            }
            const auto put = [&](int at, const uint32_t* x) {
              unsigned char* p = weights + sub * S::kPTile;
              if constexpr (kCut % 16 == 0) {
#pragma unroll
                for (int i = 0; i < kCut / 4; i += 4)
                  *reinterpret_cast<uint4*>(p + swizzled(at + 4 * i, S::kPRow)) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
              } else {
#pragma unroll
                for (int i = 0; i < kCut / 4; i += 2)
                  *reinterpret_cast<uint2*>(p + swizzled(at + 4 * i, S::kPRow)) = make_uint2(x[i], x[i + 1]);
              }
            };
            put(row * S::kPRow + c, hi);
            put(row * S::kPRow + c + (S::kStacked ? R : S::kPPlane), lo);
          };
          store(0, y0);
          if (tiles == 2) store(1, y1);
        }
        if (!go) break;
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
      if (!meet<128>(3, got)) break;
      const int row0 = w.block * R, qb = qn & 1;
      F2 acc[NP][R / 2];
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; r < R / 2; ++r) acc[p][r] = 0;
      float unit = -kInf;  // log2 of the outputs' unit, of row d
      // of rows `lane` and `lane` + 32 (warp 0): the sum of weights, log2 of its unit
      constexpr int kMine = (R + 31) / 32, kSome = R % 16 ? 8 : 16;
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
      for (int t = w.t0; t < w.t1; t += S::kSubs, ++step) {
        const int k = step & 1, tiles = S::kSubs == 2 ? min(2, w.t1 - t) : 1;
        const unsigned half = static_cast<unsigned>(step >> 1) & 1u;
        ok = at_wait(&bar.mfull[k], half, fault) && ok;
        if (d < R) {
          const float top = top_s[k][d], next = fmaxf(unit, top);
          keep_s[k][d] = unit == -kInf ? 0.f : ex2(unit - next);
          take_s[k][d] = top == -kInf ? 0.f : ex2(top - next);
          unit = next;
        }
        float tops[kMine];  // of warp 0's rows
#pragma unroll
        for (int i = 0; i < kMine; ++i) tops[i] = q == 0 ? top_s[k][min(lane + 32 * i, R - 1)] : 0.f;
        go = meet<128>(3, ok);
        if (!go) break;
        if (leader) mbar_arrive(&bar.mempty[k]);
        const PageScale ps0 = scale_s[it % kScaleRing][0], ps1 = scale_s[(it + tiles - 1) % kScaleRing][0];
        it += tiles;
        ok = at_wait(&bar.ofull[k], half, fault);
        tc_fence_after();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          if (p * 128 + q * 32 >= P.D) break;
#pragma unroll
          for (int r = 0; r < R; r += kSome) {
            F2 o[kSome / 2];
            tmem_pairs<kSome>(tmem_o + (k * NP + p) * S::kOCols + r + lanes, o);
            if constexpr (S::kStacked) {
              F2 lo[kSome / 2];
              tmem_pairs<kSome>(tmem_o + (k * NP + p) * S::kOCols + R + r + lanes, lo);
#pragma unroll
              for (int i = 0; i < kSome / 2; ++i) o[i] = add2(o[i], lo[i]);
            }
#pragma unroll
            for (int i = 0; i < kSome / 2; i += 2) {
              const ulonglong2 old = lds_pairs(&keep_s[k][r + 2 * i]), fresh = lds_pairs(&take_s[k][r + 2 * i]);
              acc[p][r / 2 + i] = fma2(o[i], fresh.x, mul2(acc[p][r / 2 + i], old.x));
              acc[p][r / 2 + i + 1] = fma2(o[i + 1], fresh.y, mul2(acc[p][r / 2 + i + 1], old.y));
            }
          }
        }
        if (q == 0) {
          const float low = fminf(ps0.ve_low, ps1.ve_low);
          const bool far = fmaxf(ps0.ve_high, ps1.ve_high) - low > static_cast<float>(kFar);
          if (!far) {
#pragma unroll 1
            for (int r = 0; r < R; r += kSome) {
              F2 s[kSome / 2];
              tmem_pairs<kSome>(tmem_l + (S::kLBufs == 2 ? k : 0) * S::kLCols + r, s);
              if constexpr (S::kStackedL) {
                F2 lo[kSome / 2];
                tmem_pairs<kSome>(tmem_l + (S::kLBufs == 2 ? k : 0) * S::kLCols + R + r, lo);
#pragma unroll
                for (int e = 0; e < kSome / 2; ++e) s[e] = add2(s[e], lo[e]);
              }
              if (lane == 0) {
#pragma unroll
                for (int e = 0; e < kSome / 2; e += 2)
                  *reinterpret_cast<ulonglong2*>(&sum_s[r + 2 * e]) = make_ulonglong2(s[e], s[e + 1]);
              }
            }
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const int r = min(lane + 32 * i, R - 1);
            if (!far) {
              add(i, sum_s[r], tops[i] - low);
            } else {
              for (int v = 0; v < 4; ++v) {
                const float2 x = __ldcg(far_sums + (4 * (step & 3) + v) * 64 + r);
                add(i, x.x, x.y);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (leader) mbar_arrive(&bar.oempty[k]);
      }
      if (!go) break;
      constexpr int kLd = NP * 128 + 4;
      float* part = P.parts + (static_cast<long long>(2 * blockIdx.x) + max(w.part, 0)) * R * kLd;
      if (d < R) row_s[d] = unit;
      if (!meet<128>(3, ok)) break;
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
            place_s[r] = w.b * P.out_ld[0] + tok * P.out_ld[1] + (w.h * P.G + g) * P.out_ld[2];
            row_s[r] = s == 0.f ? 0.f : ex2(u - sum_unit[i]) / s;
          } else {
            float* e = part + r * kLd + NP * 128;
            __stcg(e, u);
            __stcg(e + 1, s);
            __stcg(e + 2, sum_unit[i]);
          }
        }
      }
      meet<128>(3, true);
      if (w.part >= 0) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int r = 0; r < R; r += 2) {
            __stcg(part + r * kLd + p * 128 + d, first_of(acc[p][r / 2]));
            __stcg(part + (r + 1) * kLd + p * 128 + d, second_of(acc[p][r / 2]));
          }
      } else {
        const int live = w.count * P.G - row0, all = P.n * P.G - row0;  // rows with a result, rows
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          bf16_t* out = P.out + p * 128 + d;
          const bool has = p * 128 + d < P.D;
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            if (r >= live) break;
            const ulonglong2 f = lds_pairs(row_s + r);
            const longlong2 to0 = *reinterpret_cast<const longlong2*>(place_s + r);
            const longlong2 to1 = *reinterpret_cast<const longlong2*>(place_s + r + 2);
            const uint32_t x = pack_bf16(mul2(acc[p][r / 2], f.x)), y = pack_bf16(mul2(acc[p][r / 2 + 1], f.y));
            if (has) out[to0.x] = static_cast<bf16_t>(x);
            if (has && r + 1 < live) out[to0.y] = static_cast<bf16_t>(x >> 16);
            if (has && r + 2 < live) out[to1.x] = static_cast<bf16_t>(y);
            if (has && r + 3 < live) out[to1.y] = static_cast<bf16_t>(y >> 16);
          }
          if (has) {
#pragma unroll 1
            for (int r = max(live, 0); r < min(R, all); ++r) out[place_s[r]] = 0;
          }
        }
      }
      meet<128>(3, true);
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
  __shared__ float factor_s[4][kMaxCtas];
  pdl_wait();
  const int4 it = __ldcg(P.shared + blockIdx.x);
  if (it.w == 0) return;
  const int lane = threadIdx.x & 31, r = blockIdx.y * 4 + (threadIdx.x >> 5);
  float* factors = factor_s[threadIdx.x >> 5];
  const Lengths s = lengths_of(P, it.x);
  const int row = it.z * R + r, tok = row / P.G;
  if (tok >= P.n) return;
  bf16_t* out = P.out + it.x * P.out_ld[0] + tok * P.out_ld[1] + (it.y * P.G + row % P.G) * P.out_ld[2];
  const auto part = [&](int i) {
    return P.parts + (static_cast<long long>(2 * (blockIdx.x + i)) + (i == 0 ? 1 : 0)) * R * kLd + r * kLd;
  };
  // (the first 32 parts' sums are read once)
  const auto sums = [&](int i) { return __ldcg(reinterpret_cast<const float4*>(part(i) + NP * 128)); };
  const float4 own = lane < it.w ? sums(lane) : make_float4(-kInf, 0.f, -kInf, 0.f);
  float unit = own.x, sum_unit = own.z, sum = 0.f;
  for (int i = lane + 32; i < it.w; i += 32) {
    const float4 x = sums(i);
    unit = fmaxf(unit, x.x);
    sum_unit = fmaxf(sum_unit, x.z);
  }
  unit = warp_max(unit);
  sum_unit = warp_max(sum_unit);
  for (int i = lane; i < it.w; i += 32) {
    const float4 x = i == lane ? own : sums(i);
    factors[i] = x.x == -kInf ? 0.f : ex2(x.x - unit);
    sum += x.z == -kInf ? x.y : x.y * ex2(x.z - sum_unit);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncwarp();
  const float f = sum == 0.f || tok >= s.count ? 0.f : ex2(unit - sum_unit) / sum;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < it.w; ++i) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(part(i) + p * 128 + lane * 4));
      const float g = factors[i];
      acc = make_float4(__fmaf_rn(x.x, g, acc.x), __fmaf_rn(x.y, g, acc.y), __fmaf_rn(x.z, g, acc.z),
                        __fmaf_rn(x.w, g, acc.w));
    }
    const bool live = tok < s.count;  // (the parts of the other rows are of no meaning)
    const uint32_t lo = live ? pack_bf16(pair(acc.x * f, acc.y * f)) : 0u;
    const uint32_t hi = live ? pack_bf16(pair(acc.z * f, acc.w * f)) : 0u;
    const int e = p * 128 + lane * 4;  // (D is a multiple of 16)
    if (e < P.D) {
      out[e] = static_cast<bf16_t>(lo);
      out[e + 1] = static_cast<bf16_t>(lo >> 16);
      out[e + 2] = static_cast<bf16_t>(hi);
      out[e + 3] = static_cast<bf16_t>(hi >> 16);
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

// The rows of a block: those that need the least time per tile of 128 tokens,
// blocks times what a tile took with so many rows (ns per SM, 1.07 GB of cache,
// 4 query heads per head, 128 elements; the bytes alone take 740).  For 2 x 36
// rows two blocks of 48 so take 1130 each, two of 64 would take 1290.
int block_rows(int n, int G, int D) {
  const int rows = n * G;
  if (D > 128) return rows <= 16 ? 16 : 32;  // (registers and tensor memory hold no more)
  static constexpr int kRows[6] = {8, 16, 24, 32, 48, 64}, kTime[6] = {780, 820, 850, 910, 1130, 1290};
  int best = 0;
  long long least = 0;
  // (the masks of 64 bits of a tree of more than 512 nodes do not fit; chains of as
  // many rows have none, but the workspace is asked for without word of parents)
  for (int i = 0; i < (n > 512 ? 4 : 6); ++i) {
    const long long time = static_cast<long long>((rows + kRows[i] - 1) / kRows[i]) * kTime[i];
    if (i == 0 || time <= least) least = time, best = i;
    if (rows <= kRows[i]) break;
  }
  return kRows[best];
}

size_t attend_workspace(int n, int Hq, int H, int D) {
  const int R = block_rows(n, Hq / H, D), ld = (D > 128 ? 256 : 128) + 4;
  return align256(kMaxCtas * sizeof(int4)) + static_cast<size_t>(kMaxCtas) * 1024 * sizeof(float2) +
         static_cast<size_t>(2) * kMaxCtas * R * ld * sizeof(float);
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
  const int ctas = std::min(nsm * Shape<R, NP>::kCtas, kMaxCtas);
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
  p.far = reinterpret_cast<float2*>(static_cast<char*>(a->workspace) + align256(kMaxCtas * sizeof(int4)));
  p.parts = reinterpret_cast<float*>(p.far + kMaxCtas * 1024);
  const int R = block_rows(a->n, p.G, a->D);
  if (a->D > 128) return R == 16 ? launch_attend<16, 2>(*a, p, stream) : launch_attend<32, 2>(*a, p, stream);
  switch (R) {
    case 8: return launch_attend<8, 1>(*a, p, stream);
    case 16: return launch_attend<16, 1>(*a, p, stream);
    case 24: return launch_attend<24, 1>(*a, p, stream);
    case 32: return launch_attend<32, 1>(*a, p, stream);
    case 48: return launch_attend<48, 1>(*a, p, stream);
    default: return launch_attend<64, 1>(*a, p, stream);
  }
}
