// What the tcgen05 cross-attention kernels share: tile addresses, barrier waits,
// rings of slots, hidden keys.
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

// mbar_wait_bounded in few instructions: these kernels wait in many places,
// and their warp roles share the instruction cache.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {  // a poll suspends the warp
    const uint64_t t = global_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitLimitNs) return false;
  }
  return true;
}

// Whether the phase is over, without waiting for it.
__device__ __forceinline__ bool mbar_look(uint32_t bar, uint32_t parity) {
  uint32_t over;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(over)
      : "r"(bar), "r"(parity)
      : "memory");
  return over != 0;
}

// A place in a ring of N and the parity of the round it is in.
template <int N>
struct Ring {
  uint32_t i = 0, parity = 0;
  __device__ __forceinline__ void next(uint32_t by = 1) {  // by <= N
    i += by;
    if (i >= N) {
      i -= N;
      parity ^= 1u;
    }
  }
  // of the barriers at `bars`, this place's
  __device__ __forceinline__ uint32_t at(uint32_t bars) const { return bars + 8u * i; }
};

// Puts `with` over the 16 scores (or dP) of a row at ts whose bit of `seen` is
// off.  Rare: tiles with keys that are not seen.
static __device__ __noinline__ void hide16(uint32_t ts, uint32_t seen, float with) {
  float x[16];
  tmem_ld16(ts, x);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = (seen >> i) & 1u ? x[i] : with;
  tmem_st16(ts, x);
  tmem_wait_st();
}

}  // namespace llsa
