// What the tcgen05 cross-attention kernels share: the walk over work items.
#pragma once

#include "cross.cuh"
#include "sm100_ptx.cuh"
#include "tcgen05.cuh"

namespace llsa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Byte offset of 16-byte chunk jj (0..7) of row r in a tile of 128-byte rows
// with 128-byte swizzle (the TMA layout of every tile here).
__device__ __forceinline__ uint32_t sw128(int r, int jj) { return (uint32_t)(r * 128 + ((jj ^ (r & 7)) << 4)); }

// A value that is the same in all lanes, where the compiler sees that it is:
// the operands of the MMAs and TMA copies then stay in uniform registers.
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// Descriptor of an operand tile at shared address a, given that of address 0
// (addresses stay below 2^18, so the field takes the sum).
__device__ __forceinline__ uint64_t desc_at(uint64_t desc0, uint32_t a) { return desc0 + (a >> 4); }

// The items of a CTA, in order: 256 query rows of one key head against one
// range of its key tiles.  Every warp role walks them by itself; rows are
// innermost, so items of the same keys follow one another (a run).
struct CrossItems {
  const CrossParams& p;
  int i, end, nqp, cap;
  int R;                       // query rows of a key head
  size_t rows;                 // and of all of them
  int bk, b, split, r0, len;   // the item: key head, batch entry, key range, first row, keys seen at the front
  int kt0, nkt;                // its key tiles
  bool act1;                   // whether its second tile of 128 rows has any
  bool new_run, last_of_run;
  bool resident;               // its key tiles fit in the ring: loaded once for the run

  __device__ __forceinline__ CrossItems(const CrossParams& p_, int items, int cap_) : p(p_), cap(cap_) {
    R = p.N;
    rows = (size_t)p.B * p.H * R;
    nqp = (R + 255) / 256;
    i = (int)((long long)items * blockIdx.x / gridDim.x) - 1;
    end = (int)((long long)items * (blockIdx.x + 1) / gridDim.x);
    bk = -1;
    split = -1;
  }
  __device__ __forceinline__ bool next() {
    if (++i >= end) return false;
    const int run = i / nqp, qp = i - run * nqp;
    const int nbk = run / p.nks, nsplit = run - nbk * p.nks;
    new_run = nbk != bk || nsplit != split;
    last_of_run = qp == nqp - 1 || i + 1 == end;
    if (new_run) {
      bk = nbk;
      split = nsplit;
      b = bk / p.H;
      len = cross_len(p, b);
      const int kt = (len + 127) / 128;
      kt0 = (int)((long long)kt * split / p.nks);
      nkt = (int)((long long)kt * (split + 1) / p.nks) - kt0;
      resident = nkt <= cap;
    }
    r0 = qp * 256;
    act1 = r0 + 128 < R;
    return true;
  }
  // 16-key steps of key tile j of the item
  __device__ __forceinline__ int steps(int j) const {
    const int n = len - (kt0 + j) * 128;
    return n >= 128 ? 8 : (n + 15) >> 4;
  }
};

}  // namespace llsa
