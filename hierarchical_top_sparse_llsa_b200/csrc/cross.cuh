// Launch parameters of the cross-attention kernels (not part of the C ABI).
#pragma once

#include <cuda.h>

#include "llsa_internal.cuh"

namespace llsa {

struct CrossParams {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* kv_len;   // [B] or null
  const uint8_t* mask;     // [B, S] or null
  const void* o_in;        // bwd: O
  const void* res_in;      // bwd: bf16 residual of O or null
  const float* lse_in;     // bwd
  const void* dout;
  void* o;
  void* o_res;
  float* lse;
  void* dq;
  void* dk;
  void* dv;
  float* part_o;   // fwd, nks > 1: [nks][B H N][D], the splits' unnormalised O
  float2* part_ml; // fwd, nks > 1: [nks][B H N], their maxima (base 2) and sums
  float* delta;    // bwd: [B H N]
  float* part_dq;  // bwd, nks > 1: [nks][B H N][D]
  float* part_dqb; // bwd of bf16, nks > 1: the same again, and
  float4* part_s;  // [nks][B H N]: c, sum P, sum P (dP - c), whether the parts are written
  float* part_dk;  // bwd, nz > 1: [nz][B H S][D]; of bf16 [B H key tiles of 128][nz][128][D]
  float* part_dv;
  int32_t* alone;  // bwd: [B], whether the entry sees at most one key
  int32_t* status;
  // The query heads of a key head are neighbours in memory and see the same
  // keys: the kernels take them as one run of rows.
  int B, H;        // batch entries, key heads
  int N;           // query rows of a key head: (query heads / key heads) x query tokens
  int S, D;
  int nks;         // splits of the keys (fwd: of O; bwd: of dQ)
  int nz;          // bwd: segments of the query tiles (dK, dV)
  float scale;
};

// Key tokens that batch entry b sees at the front (the mask aside).
__device__ __forceinline__ int cross_len(const CrossParams& p, int b) {
  if (p.kv_len == nullptr) return p.S;
  const int n = p.kv_len[b];
  return n < 0 ? 0 : (n > p.S ? p.S : n);
}

// How the work is cut, from the sizes alone (workspace sizes follow from it).
struct CrossPlan {
  int nks, nz;
};
CrossPlan cross_simt_fwd_plan(long long BH, int N, int S);
CrossPlan cross_simt_bwd_plan(long long BH, int N, int S);
CrossPlan cross_tc_fwd_plan(long long BH, int N, int S);
CrossPlan cross_tc_bwd_plan(long long BH, int N, int S);

constexpr int kCrossSms = 148;  // SMs of a B200

// The second pass of the bf16 backward walks pairs of a key tile (128) and a
// tile of 64 query rows, the queries innermost; CTA c takes the pairs from
// begin(c) to begin(c + 1).  A key tile that several CTAs share has up to
// slots() parts.  Whole key tiles are given out (no parts) where there are
// many of them, at least four a CTA, or nothing to cut.
struct CrossPairs {
  long long nq, total;  // query tiles of a head; all pairs
  int grid;
  bool whole;
  __host__ __device__ __forceinline__ static long long tiles(long long n, int t) { return (n + t - 1) / t; }
  __host__ __device__ __forceinline__ CrossPairs(long long BH, int N, int S, int nz, int grid_)
      : nq(tiles(N, 64)), total(BH * tiles(S, 128) * nq), grid(grid_), whole(nz == 1) {}
  __host__ __device__ __forceinline__ long long begin(int c) const {
    return whole ? total / nq * c / grid * nq : total * c / grid;
  }
  // the CTA that has pair x (parts only)
  __host__ __device__ __forceinline__ int cta_of(long long x) const { return (int)(((x + 1) * grid - 1) / total); }
  static int slots(long long BH, int N, int S) {
    const long long nq = tiles(N, 64), units = BH * tiles(S, 128), total = units * nq;
    if (total == 0 || nq == 1 || units >= 4 * kCrossSms || units % kCrossSms == 0) return 1;
    // an interval of nq pairs meets at most ceil((nq - 1) / (total / grid)) + 1 CTAs
    return (int)(tiles(total < kCrossSms ? total : kCrossSms, (int)units) + 1);
  }
  static int grid_of(long long BH, int N, int S, int nz) {
    const long long units = BH * tiles(S, 128), n = nz == 1 ? units : units * tiles(N, 64);
    return (int)(n < kCrossSms ? n : kCrossSms);
  }
};

// maps: Q, K, V, O as 3D [B H, rows, D] bf16, box 128 rows x 64 columns, 128-byte swizzle
cudaError_t launch_cross_fwd_tc(const CrossParams& p, const CUtensorMap* maps, cudaStream_t s);
// q128, kv64, kv128, q64: (Q, dO) or (K, V) as above, boxes of 128 or 64 rows; q128[2]: dQ
cudaError_t launch_cross_bwd_tc(const CrossParams& p, const CUtensorMap* q128, const CUtensorMap* kv64,
                                const CUtensorMap* kv128, const CUtensorMap* q64, cudaStream_t s);
cudaError_t launch_cross_fwd_simt(const CrossParams& p, int dtype, cudaStream_t s);
cudaError_t launch_cross_bwd_simt(const CrossParams& p, int dtype, cudaStream_t s);
cudaError_t launch_cross_combine(const CrossParams& p, int dtype, cudaStream_t s);
cudaError_t launch_cross_delta(const CrossParams& p, int dtype, cudaStream_t s);
// out[i] = f * sum over z < n of part[z][i], i < total (a multiple of 8)
cudaError_t launch_cross_reduce(const float* part, void* out, int n, size_t total, float f, int dtype, cudaStream_t s);

}  // namespace llsa
