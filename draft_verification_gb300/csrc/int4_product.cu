// Products of a few bfloat16 rows with a 4-bit matrix (layout and rule in
// spec_logits.h):
//   y(r, v) = sum_g s(g, v) * D_g(v, r),
//   D_g(v, r) = sum over k in group g of (q(v, k) - z(g, v)) x(r, k).
//
// q - z is an integer of at most 15 in magnitude, exact in bfloat16, so D_g is
// a tensor-core product of exact operands with a float32 accumulator, and the
// scale multiplies it in float32: no weight is rounded.  Folding the scale into
// the weights instead would round each of them to 8 bits.
//
// A tile is 128 vocabulary entries (M) by N rows (N = 16, 32, 64 or 128).  The
// weights are the A operand: they are unpacked in registers and stored to
// tensor memory, which tcgen05.mma reads A from, so they cross shared memory
// once, packed.  A unit of work is 256 columns of a tile.  Roles of a CTA:
//   warp 0          copies units of weights (128 entries x 128 bytes) into a
//                   ring with TMA, with the scales and zero points of the same
//                   columns;
//   warp 1          issues the MMAs (one thread);
//   warp 2          copies the rows' columns (N x 256) with TMA;
//   warp 3          settles the tiles shared with other CTAs;
//   unpacking       four warpgroups (two for 128 rows) in turns: thread t owns
//                   entry t of the tile, reads up to 128 of its columns (64
//                   bytes), turns them into q - z and stores them to tensor
//                   memory, a ring of two to four chunks;
//   epilogue        one warpgroup (two for 64 rows, four for 128, each with
//                   some of the rows): thread t owns entry t, reads each
//                   group's D_g and adds s D_g to its float32 sums.
//
// The work is a list of units, tile by tile, divided over the CTAs: by whole
// tiles or equal parts of tiles where that is even enough, else evenly
// (launch_product has the rule).  Where a tile is shared along the width each
// CTA leaves its partial sums in the workspace, and whichever arrives last at
// the tile's counter adds them in the order of the columns, so the result does
// not depend on who that is.
//
// What bounds it: for few rows HBM, which has to read half a byte per weight.
// With 128256 x 4096 weights in groups of 128 (271 MB, 40 us at the measured
// 6.8 TB/s) 1 row takes 66 us, 4.1 TB/s; 64 rows 79.  No role is alone at
// fault: a unit takes about 1150 cycles, of which the copying, MMA and epilogue
// warps are each busy for 600 or more, and the warp schedulers issue in 64 % of
// all cycles, most of it the unpacking.  Of 66 us (before tiles stayed whole)
// 60 were left without the unpacking's arithmetic, 62 without the epilogue's, 64
// without the weights' copies, 66 with one MMA of sixteen.  128 rows (134 GFLOP,
// 70.6 us at the measured bfloat16 rate) take 118 us: there the epilogue's reads
// of tensor memory, N values per entry and group, are the longest.  Small groups
// multiply those reads: with groups of 32, 16 rows take 82 us and 128 rows 239.
// More rows take a pass over the weights per 128: 129 rows 221 us, 256 231.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <map>
#include <mutex>
#include <type_traits>

#include "blocks.h"
#include "common.cuh"
#include "internal.h"
#include "spec_logits.h"
#include "tc.cuh"
#include "tma_host.h"

namespace sv {
namespace {

constexpr int kTileV = 128;                 // vocabulary entries per tile (MMA M)
constexpr int kStageK = 256;                // columns of a stage (a unit): 128 packed bytes per entry
constexpr int kStageBytes = kTileV * kStageK / 2;
// 128 scales (256 bytes) or zero points (128) that may start anywhere are copied
// as the 16-byte blocks they lie in
constexpr int kScalePitch = 272;
constexpr int kZeroPitch = 144;
constexpr int kTmemCols = 512;              // the chunks' weights, then the accumulators
constexpr int kMaxCtas = 152;               // persistent CTAs the workspace is sized for
constexpr size_t kCounterBytes = 1024;      // workspace: one counter per CTA, then the partial sums
static_assert(kMaxCtas * 4 <= kCounterBytes, "one counter per CTA");

struct I4Params {
  int R, V, d;
  int ntv, nk;              // tiles of the vocabulary, stages of the width
  int units;                // row blocks * ntv * nk
  int grain, grains;        // units that stay together: 1 or a tile's; and how many
  long long scales_ld, zeros_ld, out_ld;
  const unsigned short* scales;
  const unsigned char* zeros;
  void* out;
  int out_bf16;
  int ragged;               // scales or zero points begin or end within a 16-byte block
  unsigned stage_bytes;     // what a stage of weights waits for (kStageBytes; more: see the test hook)
  int* counters;
  float* partials;          // [2 * CTAs][N][128]
  int* error_word;
};

// N rows and groups of G columns.
template <int N, int G>
struct Shape {
  // Warpgroups.  The epilogue's work grows with the rows, the unpacking's does
  // not.  Measured (V = 128256, d = 4096; epilogue + unpacking): 128 rows, groups
  // of 128: 4 + 2 131 us, 2 + 4 147; 64 rows, groups of 64: 2 + 4 103 us, 2 + 3
  // 103, 4 + 3 114, 4 + 2 115; 32 rows: 1 + 4 84 us, 2 + 3 84.
  static constexpr int kEpiGroups = N == 128 ? 4 : N == 64 ? 2 : 1;
  static constexpr int kUnpackGroups = N == 128 ? 2 : 4;
  static constexpr int kThreads = 128 * (1 + kUnpackGroups + kEpiGroups);
  static constexpr int kCols = N / kEpiGroups;           // rows of x per epilogue thread
  // the epilogue computes its places in the rings from the unit's number, or
  // carries them along: at 80 registers carrying spills (128 rows, d = 4096,
  // groups of 128 and 32: 131 and 255 us, computed 122 and 247); with room for
  // them, computing costs more (64 rows, groups of 64 and 32: 133 and 252 us,
  // carried 103 and 144)
  static constexpr bool kCounted = N == 128;
  // a chunk (what is handed from unpacking to MMA to epilogue at once): the
  // whole unit, or as many columns as leave its accumulators 128
  // tensor-memory columns
  static constexpr int kChunkK = N * (kStageK / G) <= 128 ? kStageK : 128 * G / N;
  static constexpr int kChunks = kStageK / kChunkK;      // per unit
  static constexpr int kGroups = kChunkK / G;            // per chunk
  static constexpr int kDBuf = kGroups * N;              // columns of a chunk's accumulators
  // chunks in flight: their weights take kChunkK / 2 columns each
  static constexpr int kSlots = kChunkK < kStageK ? 4 : kDBuf <= 64 ? 3 : 2;
  static constexpr int kACols = kSlots * (kChunkK / 2);
  static constexpr int kDBufs = (kTmemCols - kACols) / kDBuf < kSlots ? (kTmemCols - kACols) / kDBuf : kSlots;
  static_assert(kDBufs >= 2, "products and epilogue overlap");
  // a piece: what one warpgroup unpacks at a time; the warpgroups take turns
  static constexpr int kPieceK = kChunkK < 128 ? kChunkK : 128;
  static constexpr int kPieces = kStageK / kPieceK;      // per unit
  // A warpgroup that comes to a chunk finished one at most kSlots before, whose
  // slot was free then: so the slot it waits for is one round behind at most,
  // and the round's parity says which.
  static_assert(kUnpackGroups * kPieceK <= kSlots * kChunkK, "no slot two rounds behind");
  static constexpr int kXBytes = N * kStageK * 2;        // the rows' columns of a unit: four 64-column blocks
  // the rows come from L2, the weights from HBM: the weights' ring is the deep one
  static constexpr int kXStages = N <= 32 ? 4 : N == 64 ? 3 : 2;
  static constexpr int kWStages = N <= 32 ? 8 : N == 64 ? 6 : 4;
  // registers per thread (warps 0-3, unpacking, epilogue): shares of what the
  // launch holds (128 rows in groups of 32 spill one)
  static constexpr int kRegsLaunch = 65536 / kThreads / 8 * 8;
  static constexpr int kRegsCopy = 40;
  static constexpr int kRegsUnpack = N == 64 ? 64 : 72;
  static constexpr int kRegsEpi = N == 128 ? 80 : N == 64 ? 104 : 152;
  static_assert(128 * (kRegsCopy + kUnpackGroups * kRegsUnpack + kEpiGroups * kRegsEpi) <= kThreads * kRegsLaunch,
                "no more registers than the launch holds");
  static_assert(kRegsCopy <= kRegsLaunch && kRegsUnpack <= kRegsLaunch && kRegsEpi >= kRegsLaunch,
                "the first two give registers back, the last takes them");
  // scales and zero points of a weight stage: one row of a tile per group
  static constexpr int kPer = kStageK / G;
  static constexpr int kSideBytes = kPer * (kScalePitch + kZeroPitch);
  static constexpr int kSmem = kXStages * kXBytes + kWStages * (kStageBytes + kSideBytes) + 1024;
  static_assert(kSmem <= 225 * 1024, "one CTA's shared memory");
};

// A place in a ring: slot and the parity of its current round.
template <int kSize>
struct Ring {
  int slot = 0;
  unsigned parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kSize) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// A whole warp's wait: gives up when the bound is reached or another role did,
// so that all of them leave.  The lanes vote on every poll, which keeps the
// warp together: a warp whose lanes part over a wait runs several times slower
// (it is put to sleep and woken lane set by lane set), and so does every role
// that depends on it.
__device__ __forceinline__ bool i4_wait(uint64_t* bar, unsigned parity, volatile int* fault) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  for (int i = 0; i < kMaxPolls; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *fault)) return false;
  }
  *fault = 1;
  return false;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, M = 128, N x 16, bfloat16 in, float32 out.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

// kN (16 or 32) consecutive float32 columns of this warp's 32 lanes.
template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
  static_assert(kN == 16 || kN == 32, "widths that have a load");
  if constexpr (kN == 16) tmem_ld16(taddr, v);
  else tmem_ld32(taddr, v);
}

// 32 columns of this warp's 32 lanes from 32 registers.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 8 codes (one word, columns ascending from the low nibble) -> 4 packed pairs
// of (q - z) / 64 in bfloat16.  The codes of one byte are neighbouring columns
// and go to the two halves of a register as they lie in the byte: a small
// integer in the low bits of a bfloat16 is a subnormal, and the first binade
// continues the subnormals, so the low nibble (bits 0-3) reads as q 2^-133 and
// the high one (bits 4-7) as q 2^-129.  One multiply-add by (2^127, 2^123)
// makes both q / 64 and subtracts z / 64, all exact.  (The unused bytes are
// sign copies of the low nibble's byte: zero.)  Two logic operations, four
// byte permutations and four multiply-adds for 8 weights: the byte and logic
// operations run at half the rate of the multiply-adds and bound the unpacking.
constexpr uint32_t kUnpackScale = 0x7d007f00u;  // (2^127, 2^123)
constexpr float kUnpackUnit = 64.f;
__device__ __forceinline__ uint32_t fma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Four bytes of a (0-3) and b (4-7); selector 8 + i: copies of byte i's sign.
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
// -z / 64 twice
__device__ __forceinline__ uint32_t minus_zero(uint32_t z) {
  return fma2_bf16(z * 0x10001u, 0xff00ff00u, 0x80008000u);  // z 2^-133 times -2^127
}
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t mz, uint32_t* out) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = w & 0xf0f0f0f0u;
  out[0] = fma2_bf16(pick(even, odd, 0x8480u), kUnpackScale, mz);
  out[1] = fma2_bf16(pick(even, odd, 0x9591u), kUnpackScale, mz);
  out[2] = fma2_bf16(pick(even, odd, 0xa6a2u), kUnpackScale, mz);
  out[3] = fma2_bf16(pick(even, odd, 0xb7b3u), kUnpackScale, mz);
}

// first unit of CTA c of `ctas`
__device__ __forceinline__ int first_unit(int c, int ctas, const I4Params& P) {
  return static_cast<int>(static_cast<long long>(c) * P.grains / ctas) * P.grain;
}

// Place in the CTA's list of units: stage k of tile vt of row block rb.  The
// CTA has units [u0, u1), but begins at `start`, the first unit of the tile
// that it shares with the next CTA, goes on at u0 with the tile that it shares
// with the one before, and ends with whole tiles: shared tiles are complete
// early, and nobody's last work is a sum that others must contribute to.
struct Place {
  int rb, vt, k;
  __device__ __forceinline__ void set(int u, const I4Params& P) {
    const int t = u / P.nk;
    k = u - t * P.nk;
    rb = t / P.ntv;
    vt = t - rb * P.ntv;
  }
};
struct Cursor {
  Place at, again;  // here; where [u0, ...) begins (kept: no division in the loops)
  int left;         // units to go before u0
  __device__ __forceinline__ Cursor(int start, int u0, int u1, const I4Params& P) : left(u1 - start) {
    at.set(start, P);
    again.set(u0, P);
  }
  __device__ __forceinline__ void next(const I4Params& P) {
    if (--left == 0) {
      at = again;
    } else if (++at.k == P.nk) {
      at.k = 0;
      if (++at.vt == P.ntv) {
        at.vt = 0;
        ++at.rb;
      }
    }
  }
};

// The same list as runs of units of one tile.
struct Runs {
  Place at;  // the run's first unit
  int run;   // its units
  int todo, u0;
  bool begun = false;
  __device__ __forceinline__ Runs(int start, int u0_, int u1, const I4Params& P) : run(0), todo(u1 - u0_), u0(u0_) {
    at.set(start, P);
    run = min(P.nk - at.k, u1 - start);
  }
  // on to the next run (at first: to the first); false at the end
  __device__ __forceinline__ bool next(const I4Params& P) {
    if (begun) {
      todo -= run;
      at.k += run;
      if (at.k < P.nk) {
        at.set(u0, P);  // the tail was left: on to the head
      } else {
        at.k = 0;
        if (++at.vt == P.ntv) {
          at.vt = 0;
          ++at.rb;
        }
      }
      run = min(P.nk - at.k, todo);
    }
    begun = true;
    return todo > 0;
  }
};

// The tile of a unit, its units' CTAs and its first unit.
struct SharedTile {
  int u0, first, last;
  __device__ __forceinline__ void find(int u, int ctas, const I4Params& P) {
    u0 = u / P.nk * P.nk;
    first = static_cast<int>(static_cast<long long>(u0) * ctas / P.units);
    while (first_unit(first + 1, ctas, P) <= u0) ++first;
    while (first_unit(first, ctas, P) > u0) --first;
    last = first;
    while (first_unit(last + 1, ctas, P) < u0 + P.nk) ++last;
  }
};

// The 16-byte blocks that `bytes` bytes at `src` lie in: their size, and a copy
// of them (the data is at the same place within its first block).  Only where
// none of them reaches out of the matrix.
__device__ __forceinline__ unsigned blocks_of(const void* src, int bytes) {
  const unsigned lead = static_cast<unsigned>(reinterpret_cast<uintptr_t>(src)) & 15u;
  return (lead + bytes + 15u) & ~15u;
}
__device__ __forceinline__ void load_blocks(void* dst, const void* src, int bytes, uint64_t* bar) {
  bulk_load(dst, reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(src) & ~static_cast<uintptr_t>(15)),
            blocks_of(src, bytes), bar);
}

// Announce more bytes of bulk copies on a barrier, without an arrival.
__device__ __forceinline__ void mbar_expect_more(uint64_t* bar, unsigned bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

// The same copies by a whole warp, where blocks may reach out of the matrices:
// a lane that `has` a row copies those of its blocks that do not, and the warp
// copies the bytes that are left.  [lo, hi): the bytes of the lane's matrix.
__device__ __forceinline__ void load_blocks_at_the_ends(bool has, uint32_t dst, const char* src, int bytes,
                                                        uint64_t lo, uint64_t hi, uint64_t* bar) {
  const uint64_t first = reinterpret_cast<uint64_t>(src) & ~static_cast<uint64_t>(15);
  const unsigned lead = static_cast<unsigned>(reinterpret_cast<uint64_t>(src)) & 15u;
  const Blocks b = blocks_within(reinterpret_cast<uint64_t>(src), static_cast<unsigned>(bytes), lo, hi);
  if (has && b.end > b.begin) {
    mbar_expect_more(bar, b.end - b.begin);
    bulk_load_at(dst + b.begin, reinterpret_cast<const void*>(first + b.begin), b.end - b.begin, bar);
  }
  unsigned todo = __ballot_sync(0xffffffffu, has && (b.begin > lead || b.end < lead + bytes));
  const unsigned range = lead | (lead + bytes) << 16, whole = b.begin | b.end << 16;
  for (; todo; todo &= todo - 1) {
    const int l = __ffs(todo) - 1;
    const unsigned r = __shfl_sync(0xffffffffu, range, l), w = __shfl_sync(0xffffffffu, whole, l);
    const uint64_t from = __shfl_sync(0xffffffffu, first, l);
    const uint32_t to = __shfl_sync(0xffffffffu, dst, l);
    for (unsigned i = (r & 0xffffu) + (threadIdx.x & 31u); i < r >> 16; i += 32)
      if (i < (w & 0xffffu) || i >= w >> 16)
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + i),
                     "r"(static_cast<unsigned>(*reinterpret_cast<const unsigned char*>(from + i)))
                     : "memory");
  }
  // (the next copies into these places are bulk copies)
  fence_proxy_async();
}

// One lane of the warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

template <int N, int G>
__global__ void __launch_bounds__(Shape<N, G>::kThreads, 1)
    int4_product_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                        const I4Params P) {
  using S = Shape<N, G>;
  extern __shared__ __align__(1024) unsigned char i4_dyn[];
  __shared__ uint64_t wfull[S::kWStages], wempty[S::kWStages], xfull[S::kXStages], xempty[S::kXStages];
  // ready: a chunk's weights are in tensor memory and its accumulators are
  // free; done: its products are complete (its weights' slot is free again)
  __shared__ uint64_t ready[S::kSlots], done[S::kSlots], drain;
  // left: the epilogue's partial sums of the CTA's i-th shared tile are in the
  // workspace; settled: it is known whether this CTA adds them all (won_s)
  __shared__ uint64_t left_s[2], settled[2];
  __shared__ uint32_t tmem_s;
  __shared__ int fault_s, won_s[2], w_issued_s, x_issued_s;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const bool leader = elect_one();  // one lane issues what a warp does once
  unsigned char* wring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(i4_dyn) + 1023) &
                                                          ~static_cast<uintptr_t>(1023));
  unsigned char* xring = wring + S::kWStages * kStageBytes;
  unsigned char* sring = xring + S::kXStages * S::kXBytes;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int u0 = first_unit(cta, ctas, P), u1 = first_unit(cta + 1, ctas, P);
  const int units = u1 - u0;
  int start = u1 - u1 % P.nk;
  if (start <= u0 || start == u1) start = u0;
  // shared tiles: start's, which the next CTA ends, and u0's, which another began
  const bool tail = u1 % P.nk != 0, head = u0 % P.nk != 0 && !(start == u0 && tail);
  volatile int* fault = &fault_s;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kWStages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], 4 * (S::kPieces + S::kEpiGroups));
    }
    for (int s = 0; s < S::kXStages; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(&ready[s], 4 * (S::kChunkK / S::kPieceK) + 4 * S::kEpiGroups);
      mbar_init(&done[s], 1);
    }
    mbar_init(&drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&left_s[i], 4 * S::kEpiGroups);
      mbar_init(&settled[i], 1);
    }
    fault_s = 0;
    w_issued_s = 0;
    x_issued_s = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_s, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_a = tmem_s, tmem_d = tmem_s + S::kACols;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsCopy));
    if (warp == 0) {
      // ---------------- weight stages ----------------
      // (what a warp does here per unit is on every unit's path: addresses are
      // carried along, and each lane announces its own bytes)
      if (leader) tma_prefetch_desc(&tm_w);
      Ring<S::kWStages> w;
      // lane i < kPer: the scales of group i of the stage; lane 16 + i: its zero points
      const int g = lane & 15;
      const bool zeros = lane >= 16;
      const bool serves = g < S::kPer && (!zeros || P.zeros);
      const long long step = S::kPer * (zeros ? P.zeros_ld : 2 * P.scales_ld);  // bytes from unit to unit
      unsigned char* side = sring + (zeros ? S::kPer * kScalePitch + g * kZeroPitch : g * kScalePitch);
      int issued = 0;
      bool ok = true;
      for (Runs runs(start, u0, u1, P); ok && runs.next(P);) {
        const int v0 = runs.at.vt * kTileV, len = min(kTileV, P.V - v0) * (zeros ? 1 : 2);
        int left = P.d / G - runs.at.k * S::kPer;  // groups from the unit's first on
        const long long first = static_cast<long long>(runs.at.k * S::kPer + g);
        const char* src = zeros ? reinterpret_cast<const char*>(P.zeros) + first * P.zeros_ld + v0
                                : reinterpret_cast<const char*>(P.scales + first * P.scales_ld + v0);
        int x = runs.at.k * (kStageK / 2);  // packed byte column
        const auto copy_run = [&](auto at_the_ends) {
          for (int n = runs.run; n > 0; --n, x += kStageK / 2, src += step, left -= S::kPer) {
            ok = i4_wait(&wempty[w.slot], w.parity ^ 1u, fault);
            if (!ok) break;
            const bool has = serves && g < left;
            if (decltype(at_the_ends)::value && blocks_may_stick_out(P.V, v0, x == 0, left <= S::kPer)) {
              const int last = P.d / G - 1;
              const uint64_t lo = reinterpret_cast<uint64_t>(zeros ? static_cast<const void*>(P.zeros) : P.scales);
              const uint64_t hi = lo + (zeros ? last * P.zeros_ld + P.V : 2 * (last * P.scales_ld + P.V));
              load_blocks_at_the_ends(has, smem_addr(side + w.slot * S::kSideBytes), src, len, lo, hi, &wfull[w.slot]);
            } else if (has) {
              mbar_expect_more(&wfull[w.slot], blocks_of(src, len));
              load_blocks(side + w.slot * S::kSideBytes, src, len, &wfull[w.slot]);
            }
            __syncwarp();  // the stage expects all its bytes before its one arrival
            if (leader) {
              mbar_expect_tx(&wfull[w.slot], P.stage_bytes);
              tma_load_2d(wring + w.slot * kStageBytes, &tm_w, x, v0, &wfull[w.slot]);
            }
            w.next();
            ++issued;
          }
        };
        if (P.ragged && blocks_may_stick_out(P.V, v0, true, true)) copy_run(std::true_type{});
        else copy_run(std::false_type{});
      }
      if (leader) w_issued_s = issued;
    } else if (warp == 1) {
      // ---------------- MMAs ----------------
      // The whole warp keeps the loop's values, so that they stay in uniform
      // registers, and one lane issues; everything that varies from MMA to MMA
      // is a constant: a lone thread's instruction latency is the limit here.
      constexpr uint32_t idesc = umma_idesc_bf16_f32(kTileV, N);
      Ring<S::kXStages> x;
      Ring<S::kSlots> a;
      int db = 0;
      bool ok = true;
      for (int it = 0; it < units; ++it) {
        ok = i4_wait(&xfull[x.slot], x.parity, fault);
        if (!ok) break;
        const uint64_t dx = umma_desc_sw128(smem_addr(xring + x.slot * S::kXBytes));
  #pragma unroll
        for (int i = 0; i < S::kChunks; ++i) {
          ok = i4_wait(&ready[a.slot], a.parity, fault);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = tmem_a + a.slot * (S::kChunkK / 2), dt = tmem_d + db * S::kDBuf;
          if (leader) {
  #pragma unroll
            for (int k = 0; k < S::kChunkK / 16; ++k) {
              // K step ks of the unit: 8 columns of A; of the rows' block
              // ks / 4, 32 bytes further per step
              const int ks = i * (S::kChunkK / 16) + k;
              umma_bf16_ta(dt + (k * 16 / G) * N, at + k * 8,
                           dx + static_cast<uint64_t>((ks >> 2) * (N * 128 >> 4) + (ks & 3) * 2), idesc,
                           k * 16 % G != 0);
            }
            umma_commit(&done[a.slot]);
            if (i + 1 == S::kChunks) umma_commit(&xempty[x.slot]);
          }
          a.next();
          if (++db == S::kDBufs) db = 0;
        }
        if (!ok) break;
        x.next();
      }
      // every MMA issued has completed before tensor memory is released
      if (leader) umma_commit(&drain);
      __syncwarp();
      mbar_wait(&drain, 0);
    } else if (warp == 2) {
      // ---------------- the rows' columns ----------------
      if (leader) tma_prefetch_desc(&tm_x);
      Ring<S::kXStages> x;
      int issued = 0;
      bool ok = true;
      for (Runs runs(start, u0, u1, P); ok && runs.next(P);) {
        for (int k = runs.at.k * kStageK, n = runs.run; n > 0; --n, k += kStageK) {
          ok = i4_wait(&xempty[x.slot], x.parity ^ 1u, fault);
          if (!ok) break;
          if (leader) {
            unsigned char* st = xring + x.slot * S::kXBytes;
            mbar_expect_tx(&xfull[x.slot], S::kXBytes);
#pragma unroll
            for (int i = 0; i < kStageK / 64; ++i)
              tma_load_2d(st + i * N * 128, &tm_x, k + i * 64, runs.at.rb * N, &xfull[x.slot]);
          }
          __syncwarp();
          x.next();
          ++issued;
        }
      }
      if (leader) x_issued_s = issued;
    } else if (warp == 3) {
      // ---------------- shared tiles ----------------
      // In the order in which the epilogue leaves them: the tile of unit
      // `start` where the CTA does not end it, then that of u0 where it does
      // not begin it.  One arrival per part; the last one's CTA adds them up.
      int n = 0;
      for (int i = 0; i < 2; ++i) {
        if (!(i == 0 ? tail : head)) continue;
        SharedTile t;
        t.find(i == 0 ? start : u0, ctas, P);
        if (!i4_wait(&left_s[n], 0u, fault)) break;
        if (leader) {
          // the counter wraps to zero with the last arrival: the workspace is as it was
          asm volatile("fence.acq_rel.gpu;" ::: "memory");
          const unsigned before =
              atomicInc(reinterpret_cast<unsigned*>(P.counters + t.first), static_cast<unsigned>(t.last - t.first));
          asm volatile("fence.acq_rel.gpu;" ::: "memory");
          won_s[n] = before == static_cast<unsigned>(t.last - t.first);
          mbar_arrive(&settled[n]);
        }
        __syncwarp();
        ++n;
      }
    }
  } else if (warp < 4 + 4 * S::kUnpackGroups) {
    // ---------------- unpacking ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsUnpack));
    constexpr int kVecs = S::kPieceK / 32;  // 16-byte vectors of an entry's piece, one zero point each
    const int grp = (warp - 4) >> 2, q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t key = static_cast<uint32_t>(row & 7);
    Cursor c(start, u0, u1, P);  // (with zero points) the piece's unit
    int c_it = 0;
    // low bits of addresses: where a row of zero points starts in its first block
    const uint32_t zeros_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(P.zeros));
    const uint32_t zeros_ld = static_cast<uint32_t>(P.zeros_ld);
    uint32_t minus[kVecs];  // -z / 64 twice, of the piece's 32-column vectors
#pragma unroll
    for (int i = 0; i < kVecs; ++i) minus[i] = minus_zero(8u);
    // pieces counted from the CTA's first; this warpgroup's are n % kUnpackGroups == grp
    for (int n = grp; n < units * S::kPieces; n += S::kUnpackGroups) {
      const int it = n / S::kPieces, i = n % S::kPieces;  // unit, and piece of the unit
      const int ws = it % S::kWStages;
      if (!i4_wait(&wfull[ws], static_cast<unsigned>(it / S::kWStages) & 1u, fault)) break;
      const unsigned char* src = wring + ws * kStageBytes + row * (kStageK / 2);
      uint4 code[kVecs];
#pragma unroll
      for (int e = 0; e < kVecs; ++e) code[e] = lds16(src + (((i * kVecs + e) ^ key) << 4));
      if (P.zeros) {
        for (; c_it < it; ++c_it) c.next(P);
        const unsigned char* z = sring + ws * S::kSideBytes + S::kPer * kScalePitch + row;
        const uint32_t lead = zeros_at + static_cast<uint32_t>(c.at.vt * kTileV);
#pragma unroll
        for (int e = 0; e < kVecs; ++e) {
          const int g = (i * S::kPieceK + e * 32) / G;  // of the unit
          minus[e] = minus_zero(
              z[g * kZeroPitch + ((lead + static_cast<uint32_t>(c.at.k * S::kPer + g) * zeros_ld) & 15u)]);
        }
      }
      __syncwarp();
      if (leader) mbar_arrive(&wempty[ws]);
      const unsigned chunk = static_cast<unsigned>(it * S::kChunks + i * S::kPieceK / S::kChunkK);
      const unsigned slot = chunk % S::kSlots;
      if (!i4_wait(&done[slot], ((chunk / S::kSlots) & 1u) ^ 1u, fault)) break;
      tc_fence_after();
      const uint32_t dst =
          tmem_a + slot * (S::kChunkK / 2) + static_cast<uint32_t>(i * S::kPieceK % S::kChunkK) / 2 + lanes;
      if constexpr (kVecs == 1) {
        uint32_t r[16];
        unpack8(code[0].x, minus[0], r);
        unpack8(code[0].y, minus[0], r + 4);
        unpack8(code[0].z, minus[0], r + 8);
        unpack8(code[0].w, minus[0], r + 12);
        tmem_st16(dst, r);
      } else {
#pragma unroll
        for (int h = 0; h < kVecs / 2; ++h) {
          uint32_t r[32];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 x = code[2 * h + e];
            const uint32_t z = minus[2 * h + e];
            unpack8(x.x, z, r + 16 * e);
            unpack8(x.y, z, r + 16 * e + 4);
            unpack8(x.z, z, r + 16 * e + 8);
            unpack8(x.w, z, r + 16 * e + 12);
          }
          tmem_st32(dst + 32 * h, r);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (leader) mbar_arrive(&ready[slot]);
    }
  } else {
    // ---------------- epilogue ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsEpi));
    const int grp = (warp - 4 - 4 * S::kUnpackGroups) >> 2, q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    const int col0 = grp * S::kCols;
    // this thread's sums of a tile, to their places in out
    const auto store = [&](const Place& at, const float2 (&acc)[S::kCols / 2]) {
      const int v = at.vt * kTileV + row;
      if (v >= P.V) return;
      const int r0 = at.rb * N + col0, rows = min(S::kCols, P.R - r0);
      const long long first = static_cast<long long>(r0) * P.out_ld + v;
      if (P.out_bf16) {
        unsigned short* y = static_cast<unsigned short*>(P.out) + first;
#pragma unroll
        for (int i = 0; i < S::kCols; ++i, y += P.out_ld) {
          if (i >= rows) break;
          unsigned short bits;
          asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(kUnpackUnit * ((i & 1) ? acc[i / 2].y : acc[i / 2].x)));
          *y = bits;
        }
      } else {
        float* y = static_cast<float*>(P.out) + first;
#pragma unroll
        for (int i = 0; i < S::kCols; ++i, y += P.out_ld) {
          if (i >= rows) break;
          *y = kUnpackUnit * ((i & 1) ? acc[i / 2].y : acc[i / 2].x);
        }
      }
    };
    float2 acc[S::kCols / 2];
#pragma unroll
    for (int i = 0; i < S::kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
    // the accumulators of the first chunks are free
    if (leader)
      for (int i = 0; i < S::kDBufs; ++i) mbar_arrive(&ready[i]);
    Ring<S::kWStages> w;
    Ring<S::kSlots> a;
    int db = 0;
    int shared = 0;  // shared tiles so far
    int unit0 = 0;   // the run's first unit, counted from the CTA's first
    bool ok = true;
    for (Runs runs(start, u0, u1, P); ok && runs.next(P); unit0 += runs.run) {
      const Place& c = runs.at;
      // low bits of addresses: where a row of scales starts in its first block
      const uint32_t step = static_cast<uint32_t>(P.scales_ld) * 2u;
      uint32_t lead = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(P.scales)) +
                      static_cast<uint32_t>(c.vt * kTileV) * 2u + static_cast<uint32_t>(c.k * S::kPer) * step;
      int width = P.d - c.k * kStageK;  // columns from the unit's first on
      for (int j = 0; j < runs.run; ++j, width -= kStageK) {
        const int it = unit0 + j;
        const int ws = S::kCounted ? it % S::kWStages : w.slot;
        ok = i4_wait(&wfull[ws], S::kCounted ? static_cast<unsigned>(it / S::kWStages) & 1u : w.parity, fault);
        if (!ok) break;
        uint32_t s_now[S::kPer];  // the scales of the unit's groups
        const unsigned char* sp = sring + ws * S::kSideBytes + row * 2;
#pragma unroll
        for (int i = 0; i < S::kPer; ++i, lead += step)
          s_now[i] = *reinterpret_cast<const unsigned short*>(sp + i * kScalePitch + (lead & 15u));
        __syncwarp();
        if (leader) mbar_arrive(&wempty[ws]);
        if (!S::kCounted) w.next();
#pragma unroll
        for (int i = 0; i < S::kChunks; ++i) {
          const unsigned chunk = static_cast<unsigned>(it * S::kChunks + i);
          const unsigned slot = S::kCounted ? chunk % S::kSlots : a.slot;
          ok = i4_wait(&done[slot], S::kCounted ? (chunk / S::kSlots) & 1u : a.parity, fault);
          if (!ok) break;
          tc_fence_after();
          // the chunk's accumulators, group by group, in loads of at most 32 columns
          constexpr int kAll = S::kGroups * S::kCols;
          constexpr int kLd = kAll < 32 ? kAll : 32;
          const uint32_t src = tmem_d + (S::kCounted ? chunk % S::kDBufs : db) * S::kDBuf + lanes;
#pragma unroll
          for (int n = 0; n < kAll; n += kLd) {
            float v[kLd];
            // (with two epilogue warpgroups a chunk of more than one group is read group by group)
            tmem_ld<kLd>(src + n / S::kCols * N + col0 + n % S::kCols, v);
#pragma unroll
            for (int e = 0; e < kLd; e += 2) {
              const int g = i * S::kGroups + (n + e) / S::kCols;
              // (a group beyond the width has no scale and is not added)
              if (g * G < width) {
                const float s = __uint_as_float(s_now[g] << 16);
                float2& sum = acc[(n + e) % S::kCols / 2];
                sum = ffma2(make_float2(s, s), make_float2(v[e], v[e + 1]), sum);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          // these accumulators are the ones of the chunk kDBufs further on
          if (leader) mbar_arrive(&ready[(slot + S::kDBufs) % S::kSlots]);
          if (!S::kCounted) a.next();
          if (!S::kCounted && ++db == S::kDBufs) db = 0;
        }
        if (!ok) break;
      }
      if (!ok) break;
      if (runs.run == P.nk) {
        store(c, acc);
      } else {
        // a shared tile: leave the sums in this CTA's slot
        float* mine = P.partials + (static_cast<long long>(2 * cta + (c.k == 0 ? 1 : 0)) * N + col0) * kTileV + row;
#pragma unroll
        for (int i = 0; i < S::kCols / 2; ++i) {
          __stcg(mine + (2 * i) * kTileV, acc[i].x);
          __stcg(mine + (2 * i + 1) * kTileV, acc[i].y);
        }
        __syncwarp();
        if (leader) mbar_arrive(&left_s[shared]);
        ++shared;
      }
#pragma unroll
      for (int i = 0; i < S::kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
    }
    // the shared tiles whose last part this CTA was: all parts, in the order of the columns
    for (int i = 0; i < shared && ok; ++i) {
      ok = i4_wait(&settled[i], 0u, fault);
      if (!ok || !won_s[i]) continue;
      SharedTile t;
      t.find(tail && i == 0 ? start : u0, ctas, P);
      Place c;
      c.set(t.u0, P);
      for (int o = t.first; o <= t.last; ++o) {
        const float* src =
            P.partials + (static_cast<long long>(2 * o + (o == t.first ? 1 : 0)) * N + col0) * kTileV + row;
#pragma unroll
        for (int n = 0; n < S::kCols / 2; ++n) {
          acc[n].x = __fadd_rn(acc[n].x, __ldcg(src + (2 * n) * kTileV));
          acc[n].y = __fadd_rn(acc[n].y, __ldcg(src + (2 * n + 1) * kTileV));
        }
      }
      store(c, acc);
#pragma unroll
      for (int n = 0; n < S::kCols / 2; ++n) acc[n] = make_float2(0.f, 0.f);
    }
  }

  __syncthreads();
  if (*fault && threadIdx.x == 0) {
    // copies still in flight land before the CTA exits: wait (bounded) for
    // the last phase of every stage that was issued
    for (int k = max(0, w_issued_s - S::kWStages); k < w_issued_s; ++k)
      mbar_wait(&wfull[k % S::kWStages], static_cast<unsigned>(k / S::kWStages) & 1u);
    for (int k = max(0, x_issued_s - S::kXStages); k < x_issued_s; ++k)
      mbar_wait(&xfull[k % S::kXStages], static_cast<unsigned>(k / S::kXStages) & 1u);
    if (P.error_word) atomicOr(P.error_word, SPEC_ERR_INTERNAL);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_s, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// MMA N: the rows of a block, rounded up to a width that has a kernel.  (The
// narrowest that fits: with 128256 x 4096 weights in groups of 128 the widths
// take 65, 71, 79 and 118 us whatever part of their rows is used.)
int rows_tile(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }

// the units of all row blocks
long long units_of(int R, int V, int d) {
  const int N = rows_tile(R);
  return static_cast<long long>((R + N - 1) / N) * ((V + kTileV - 1) / kTileV) * ((d + kStageK - 1) / kStageK);
}

bool good_shape(int R, int V, int d, int group) {
  return R >= 1 && R <= 65535 && V >= 1 && V <= 2097152 && (group == 32 || group == 64 || group == 128) && d >= 32 &&
         d <= 65536 && d % group == 0 && units_of(R, V, d) < 1LL << 30;
}

size_t product_workspace(int R) {
  return kCounterBytes + static_cast<size_t>(2) * kMaxCtas * rows_tile(R) * kTileV * sizeof(float);
}

// Packed weights [V, d / 2] bytes: boxes of 128 entries x 128 bytes, 128-byte swizzle, zeros outside.
bool weight_map(CUtensorMap* map, const void* base, int V, int d, long long ld) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d / 2), static_cast<cuuint64_t>(V)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {kStageK / 2, kTileV};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [R, d] bfloat16: boxes of N rows x 64 columns, 128-byte swizzle, zeros outside.
bool rows_map(CUtensorMap* map, const void* base, int R, int d, long long ld, int N) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(R)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(N)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel's dynamic shared memory limit, raised once per device.
template <int N, int G>
cudaError_t raise_smem() {
  static std::mutex mu;
  static std::map<int, bool> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (done.count(dev)) return cudaSuccess;
  e = cudaFuncSetAttribute(int4_product_kernel<N, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<N, G>::kSmem);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

// Test hook (spec_test_inject_product_copy_timeout): nonzero makes every stage
// of weights wait for 16 bytes that never come, so that the bounded waits of the
// roles behind it give up.  Zero in normal operation.
std::atomic<unsigned> g_more_bytes{0};

template <int N, int G>
spec_status launch_product(const spec_int4_product_args& a, cudaStream_t s) {
  I4Params P{};
  P.R = a.R;
  P.V = a.V;
  P.d = a.d;
  P.ntv = (a.V + kTileV - 1) / kTileV;
  P.nk = (a.d + kStageK - 1) / kStageK;
  P.units = static_cast<int>(units_of(a.R, a.V, a.d));
  P.scales_ld = a.scales_ld;
  P.zeros_ld = a.zeros_ld;
  P.out_ld = a.out_ld;
  P.scales = static_cast<const unsigned short*>(a.scales);
  P.zeros = a.zeros;
  P.out = a.out;
  P.out_bf16 = a.out_dtype == SPEC_BF16;
  P.counters = static_cast<int*>(a.workspace);
  P.partials = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kCounterBytes);
  P.error_word = a.error_word;
  P.stage_bytes = kStageBytes + g_more_bytes.load();
  // whether a matrix begins or ends within a 16-byte block (the kernel's test is
  // kept out of the common loop, where it cost 2 to 9 %: 33 rows 50257, 2048, 64
  // with zero points 28.7 us without it, 31.3 with it, 28.8 as it is)
  const uintptr_t scales = reinterpret_cast<uintptr_t>(a.scales), zeros = reinterpret_cast<uintptr_t>(a.zeros);
  const long long last = a.d / G - 1;
  P.ragged = ((scales | (scales + 2 * (last * a.scales_ld + a.V))) & 15u) != 0 ||
             (a.zeros && ((zeros | (zeros + last * a.zeros_ld + a.V)) & 15u) != 0);
  const int nsm = sm_count();
  if (nsm < 1) return SPEC_ECUDA;
  // A tile shared by CTAs that each have parts of two tiles costs them 4 to 8 us
  // at the end of the call, its join included.  So tiles stay whole, or are cut
  // into the same number of equal parts (of 4 units or more, which begin and end
  // with a tile), where the longest CTA has at most 8 units more than an even
  // division would give it.  Measured (by graph replays, which read 2 to 4 %
  // below single launches; V, d, group; evenly divided, and so):
  // 128 rows 128256, 4096, 128 124 and 114 us, 1 row 66 and 64; 33 rows 50257,
  // 2048, 64 31 and 27; 128 rows 1000, 8192, 64 33 and 23, 12800, 4096, 128
  // 27 and 22.  With 12 instead of 8 units: 16 rows 25000, 4096, 128 21 and 23,
  // 12800, 8192, 128 23 and 21.
  const int most = std::min(nsm, kMaxCtas), tiles = P.units / P.nk;
  const int even = (P.units + most - 1) / most;
  int ctas = std::min(most, P.units);
  P.grain = 1;
  if (tiles > most) {
    if ((tiles + most - 1) / most * P.nk <= even + 8) P.grain = P.nk;
  } else {
    const int parts = std::min(most / tiles, std::max(1, P.nk / 4));
    if ((P.nk + parts - 1) / parts <= even + 8) ctas = tiles * parts;
  }
  P.grains = P.units / P.grain;
  CUtensorMap tw, tx;
  if (!weight_map(&tw, a.codes, a.V, a.d, a.codes_ld) || !rows_map(&tx, a.x, a.R, a.d, a.x_ld, N)) return SPEC_ECUDA;
  if (raise_smem<N, G>() != cudaSuccess) return SPEC_ECUDA;
  int4_product_kernel<N, G><<<ctas, Shape<N, G>::kThreads, Shape<N, G>::kSmem, s>>>(tw, tx, P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ECUDA;
}

template <int N>
spec_status launch_product(const spec_int4_product_args& a, cudaStream_t s) {
  switch (a.group) {
    case 32: return launch_product<N, 32>(a, s);
    case 64: return launch_product<N, 64>(a, s);
    default: return launch_product<N, 128>(a, s);
  }
}

}  // namespace
}  // namespace sv

extern "C" spec_status spec_test_inject_product_copy_timeout(int enable) {
  sv::g_more_bytes = enable ? 16u : 0u;
  return SPEC_OK;
}

extern "C" size_t spec_int4_product_workspace_size(int R, int V, int d, int group) {
  return sv::good_shape(R, V, d, group) ? sv::product_workspace(R) : 0;
}

extern "C" spec_status spec_int4_product(const spec_int4_product_args* a, cudaStream_t stream) {
  using namespace sv;
  NvtxRange nvtx_range("spec_int4_product");
  if (a == nullptr) return SPEC_EINVAL;
  if (a->out_dtype != SPEC_F32 && a->out_dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (!good_shape(a->R, a->V, a->d, a->group)) return SPEC_EINVAL;
  if (!a->x || !a->codes || !a->scales || !a->out) return SPEC_EINVAL;
  if (a->x_ld < a->d || a->x_ld % 8 || a->codes_ld < a->d / 2 || a->codes_ld % 16) return SPEC_EINVAL;
  if (a->scales_ld < a->V || a->out_ld < a->V || (a->zeros && a->zeros_ld < a->V)) return SPEC_EINVAL;
  if (!aligned(a->x, 16) || !aligned(a->codes, 16) || !aligned(a->scales, 2) ||
      !aligned(a->out, a->out_dtype == SPEC_F32 ? 4 : 2))
    return SPEC_EALIGN;
  if (!a->workspace || a->workspace_bytes < product_workspace(a->R) || !aligned(a->workspace, 256))
    return SPEC_EWORKSPACE;
  switch (rows_tile(a->R)) {
    case 16: return launch_product<16>(*a, stream);
    case 32: return launch_product<32>(*a, stream);
    case 64: return launch_product<64>(*a, stream);
    default: return launch_product<128>(*a, stream);
  }
}
