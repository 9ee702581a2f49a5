// Launch parameters of the rotary-position kernels (not part of the C ABI).
#pragma once

#include "llsa_internal.cuh"

namespace llsa {

constexpr int kMaxRopeFreqs = 64;  // rot_dim / 2 <= 64

// the table's frequencies in turns per position, f_j / 2 pi, j < n, each the sum
// of two doubles: far positions multiply what one leaves off
struct RopeFreqs {
  double2 turns[kMaxRopeFreqs];
  int half;   // pairs per row, rot_dim / 2
  int n;      // pairs per axis
  int axes;
  float m;    // scale of cosine and sine
};

struct RopeParams {
  const void* x[3];  // q, k (and v for the pool)
  void* y[2];        // rotated q, k
  const float* table;
  int B, H, N, D, rot;
  int interleaved;
  int per_batch;     // the table has a row per (b, n), else per n
  int ntensor;       // tensors to rotate, 1 or 2
  int per;           // (tensor, head) rows per thread
  float sign;        // -1 for the adjoint
};

cudaError_t launch_rope_table(const RopeFreqs& f, int rows, const int32_t* pos, float* table, cudaStream_t s);
cudaError_t launch_rope(const RopeParams& p, int dtype, cudaStream_t s);
// whether the pool can be fused: every pair within a thread's two chunks
bool rope_pool_fused(int rot, bool interleaved, int dtype);
cudaError_t launch_rope_pool(const RopeParams& p, const PoolParams& o, int dtype, cudaStream_t s);

}  // namespace llsa
