// Rows of a matrix that may start at any byte, copied in 16-byte blocks: which
// blocks lie within the matrix.  (Plain arithmetic, for the host as well.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SV_HOST_DEVICE inline
#endif

namespace sv {

// The blocks that the bytes [src, src + bytes) lie in, less those that reach
// out of the matrix's bytes [lo, hi): [begin, end), counted in bytes from the
// first block (src & ~15).  What of [src, src + bytes) lies outside them is
// copied byte by byte.
struct Blocks {
  unsigned begin, end;
};
SV_HOST_DEVICE Blocks blocks_within(uint64_t src, unsigned bytes, uint64_t lo, uint64_t hi) {
  const unsigned lead = static_cast<unsigned>(src) & 15u;
  Blocks b{0u, (lead + bytes + 15u) & ~15u};
  if (src - lead < lo) b.begin = 16u;
  if (src - lead + b.end > hi) b.end -= 16u;
  if (b.end < b.begin) b.end = b.begin;
  return b;
}

// Rows of V entries (of 1 or 2 bytes) are copied 128 entries [v0, v0 + 128) at a
// time, some rows per stage: whether blocks of a stage may reach out of the
// matrix, if that begins or ends within a block.  A block reaches at most 15
// bytes past what it is copied for: out of the front from the first row's first
// entries, out of the back from the last row's entries that fewer than 16
// follow; with fewer than 16 entries a row, from other rows as well.
SV_HOST_DEVICE bool blocks_may_stick_out(int V, int v0, bool first_rows, bool last_rows) {
  return V < 16 || (first_rows && v0 == 0) || (last_rows && V - v0 < 128 + 16);
}

}  // namespace sv
