// Launch parameters of the cross-attention kernels (not part of the C ABI).
#pragma once

#include <cuda.h>

#include "llsa_internal.cuh"

namespace llsa {

// n items cut into one run per CTA, the first n % grid of them longer by one.
struct CrossRuns {
  int64_t each, more;
  __host__ __device__ __forceinline__ int64_t begin(int c) const { return each * c + (c < more ? c : more); }
  __host__ __device__ __forceinline__ int cta_of(int64_t x) const {
    const int64_t longer = more * (each + 1);
    return (int)(x < longer ? x / (each + 1) : more + (x - longer) / each);
  }
};
inline CrossRuns cross_runs(int64_t n, int grid) { return {n / grid, n % grid}; }
inline int64_t cross_tiles(int64_t n, int t) { return (n + t - 1) / t; }

struct CrossParams {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* kv_len;   // [B] or null
  const uint8_t* mask;     // [B, S] or null
  const void* o_in;        // bwd: O
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
  float* delta;    // bwd of bf16: [B H N]
  float* part_dq;  // bwd, nks > 1: [nks][B H N][D]
  float* part_dqb; // bwd of bf16, nks > 1: the same again, and
  float4* part_s;  // [nks][B H N]: c, sum P (dP - c), the sum of its rounded terms, whether the parts are written
  float* part_dk;  // bwd, nz > 1: [nz][B H S][D]; of bf16 [B H key tiles of 128][nz][128][D]
  float* part_dv;
  int32_t* alone;  // bwd of bf16: [B], whether the entry sees at most one key
  int32_t* status;
  // The query heads of a key head are neighbours in memory and see the same
  // keys: the kernels take them as one run of rows.
  int B, H;        // batch entries, key heads
  int N;           // query rows of a key head: (query heads / key heads) x query tokens
  int S, D;
  int nks;         // splits of the keys (fwd: of O; bwd: of dQ)
  int nz;          // bwd: segments of the query tiles (dK, dV)
  CrossRuns runs;  // bf16: what each CTA does
  int items;       // bwd of bf16: of the first pass
  float scale;
};

// Key tokens that batch entry b sees at the front (the mask aside).
__device__ __forceinline__ int cross_len(const CrossParams& p, int b) {
  if (p.kv_len == nullptr) return p.S;
  const int n = p.kv_len[b];
  return n < 0 ? 0 : (n > p.S ? p.S : n);
}

// Whether b sees at most one key (a whole warp asks).
__device__ __forceinline__ bool sees_one(const CrossParams& p, int b, int len) {
  if (p.mask == nullptr || len <= 1) return len <= 1;
  const uint8_t* m = p.mask + (size_t)b * p.S;
  const int lane = threadIdx.x & 31;
  int seen = 0;
  for (int k0 = 0; k0 < len && seen < 2; k0 += 256) {
    bool on[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + 32 * u + lane;
      on[u] = k < len && m[k] != 0;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) seen += __popc(__ballot_sync(0xffffffffu, on[u]));
  }
  return seen <= 1;
}

// How the work is cut, from the sizes alone (workspace sizes follow from it).
struct CrossPlan {
  int nks, nz;
};
CrossPlan cross_simt_fwd_plan(long long BH, int N, int S);
CrossPlan cross_simt_bwd_plan(long long BH, int N, int S);
CrossPlan cross_tc_fwd_plan(long long BH, int N, int S, int D);
CrossPlan cross_tc_bwd_plan(long long BH, int N, int S);

constexpr int kCrossSms = 148;  // SMs of a B200

// maps: Q, K, V, O as 3D [B H, rows, D] bf16, 128-byte swizzle, boxes of 64
// columns and 128 rows (K, V at D = 64: 64 rows)
cudaError_t launch_cross_fwd_tc(const CrossParams& p, const CUtensorMap* maps, cudaStream_t s);
// q128, kv64, kv128, q64: (Q, dO) or (K, V) as above, boxes of 128 or 64 rows; q128[2]: dQ
cudaError_t launch_cross_bwd_tc(const CrossParams& p, const CUtensorMap* q128, const CUtensorMap* kv64,
                                const CUtensorMap* kv128, const CUtensorMap* q64, cudaStream_t s);
cudaError_t launch_cross_fwd_simt(const CrossParams& p, cudaStream_t s);
cudaError_t launch_cross_bwd_simt(const CrossParams& p, cudaStream_t s);
cudaError_t launch_cross_combine(const CrossParams& p, int dtype, cudaStream_t s);

}  // namespace llsa
