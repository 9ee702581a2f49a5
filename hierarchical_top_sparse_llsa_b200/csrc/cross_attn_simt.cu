// Cross attention in fp32 on the CUDA cores: forward, dQ, and dK with dV, in
// tiles of 64 queries x 64 keys.
//
//   s = scale q k^T, P = e^(s - lse), O = P V / l
//   dV = P^T dO, dS = P (dO V^T - Delta), dQ = scale dS K, dK = scale dS^T Q
//
// Bound by the fp32 FMA rate: tensor-core formats hold too few bits for fp32
// inputs.  A thread holds a block of the tile in registers (8 x 4 scores in
// the forward) and feeds it with 16-byte shared-memory loads, rows padded so
// that the 16 keys a half warp reads sit in different banks.  Probabilities
// pass through shared memory, over the K tile that is no longer read.
// The forward is cut along the keys, dQ likewise, and dK with dV along the
// query tiles, where whole tiles would leave SMs idle; the parts are fp32 and
// joined in a fixed order.  A key that is not seen is stored as zeros and its
// probability set to zero, so what its memory holds has no effect.

#include <math.h>

#include "cross.cuh"

namespace llsa {

namespace {

constexpr int kT = 64;          // queries and keys per tile
constexpr int kFwdThreads = 128;
constexpr int kBwdThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

inline int tiles_of(int n) { return n / kT + (n % kT != 0); }

// rows r < nrows of src [.., D] (kept where keep is null or keep[r] != 0) as
// floats into dst rows of LD floats; the others as zeros
template <typename T, int D, int LD, int THREADS>
__device__ __forceinline__ void load_rows(float* dst, const T* src, int nrows, const uint8_t* keep) {
  constexpr int VEC = Vec16<T>::N;
  for (int e = threadIdx.x; e < kT * (D / VEC); e += THREADS) {
    const int r = e / (D / VEC), c = (e % (D / VEC)) * VEC;
    float x[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = 0.f;
    if (r < nrows && (keep == nullptr || keep[r] != 0)) Vec16<T>::load(src + (size_t)r * D + c, x);
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      *reinterpret_cast<float4*>(dst + r * LD + c + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  }
}

// keep[j] = whether key k0 + j is seen
__device__ __forceinline__ void load_keep(uint8_t* keep, const CrossParams& p, int b, int k0, int len) {
  if (threadIdx.x < kT) {
    const int j = k0 + threadIdx.x;
    keep[threadIdx.x] = j < len && (p.mask == nullptr || p.mask[(size_t)b * p.S + j] != 0);
  }
}

__device__ __forceinline__ float half_max(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float half_sum(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// acc[i][j] = a row (ty * R + i) . b row (tx + 16 j)
template <int D, int R>
__device__ __forceinline__ void dot_tile(float (&acc)[R][4], const float* a, const float* b, int ty, int tx) {
  constexpr int LD = D + 4;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 2
  for (int d = 0; d < D; d += 4) {
    float4 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(a + (ty * R + i) * LD + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(x.x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x.y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x.z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x.w, y[j].w, acc[i][j]);
      }
    }
  }
}

constexpr int kLP = kT + 4;  // row length of the probability tiles

// ----------------------------------------------------------------- forward
template <typename T, int D>
__global__ void __launch_bounds__(kFwdThreads)
cross_fwd_simt(CrossParams p, int qtiles) {
  constexpr int LD = D + 4;
  extern __shared__ __align__(16) float smf[];
  __shared__ uint8_t keep[kT];
  float* Q = smf;             // [64][LD]
  float* K = Q + kT * LD;     // [64][LD], then P [64][kLP]
  float* V = K + kT * LD;     // [64][D]
  float* P = K;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  long long id = blockIdx.x;
  const int qt = (int)(id % qtiles);
  id /= qtiles;
  const int split = (int)(id % p.nks);
  const int bh = (int)(id / p.nks);
  const int b = bh / p.H;
  const size_t kvrow = (size_t)bh * p.S;
  const int q0 = qt * kT, nq = min(kT, p.N - q0);
  const size_t row0 = (size_t)bh * p.N + q0;
  const int len = cross_len(p, b);
  const int ktiles = (len + kT - 1) / kT;
  const int kt0 = (int)((long long)ktiles * split / p.nks), kt1 = (int)((long long)ktiles * (split + 1) / p.nks);
  const float sc2 = p.scale * kLog2e;

  load_rows<T, D, LD, kFwdThreads>(Q, static_cast<const T*>(p.q) + row0 * D, nq, nullptr);
  float o[8][D / 16];
  float m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
  }
  for (int kt = kt0; kt < kt1; ++kt) {
    const int k0 = kt * kT;
    __syncthreads();  // the last tile is no longer read
    load_keep(keep, p, b, k0, len);
    __syncthreads();
    const int nk = min(kT, p.S - k0);
    load_rows<T, D, LD, kFwdThreads>(K, static_cast<const T*>(p.k) + (kvrow + k0) * D, nk, keep);
    load_rows<T, D, D, kFwdThreads>(V, static_cast<const T*>(p.v) + (kvrow + k0) * D, nk, keep);
    __syncthreads();
    float s[8][4];
    dot_tile<D, 8>(s, Q, K, ty, tx);
    bool on[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) on[j] = keep[tx + 16 * j] != 0;
    __syncthreads();  // K is read; P takes its place
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = on[j] ? s[i][j] * sc2 : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      const float mn = fmaxf(m[i], half_max(mx));
      const float mb = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m[i] - mb);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - mb);
        P[(ty * 8 + i) * kLP + tx + 16 * j] = e;
        sum += e;
      }
      l[i] = l[i] * corr + half_sum(sum);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[i][c] *= corr;
    }
    __syncwarp();  // a P row is written and read by one half warp
    for (int j = 0; j < kT; j += 4) {
      float4 pr[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pr[i] = *reinterpret_cast<const float4*>(P + (ty * 8 + i) * kLP + j);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(V + (j + jj) * D + c * 64 + tx * 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float w = jj == 0 ? pr[i].x : (jj == 1 ? pr[i].y : (jj == 2 ? pr[i].z : pr[i].w));
            o[i][4 * c] = fmaf(w, v.x, o[i][4 * c]);
            o[i][4 * c + 1] = fmaf(w, v.y, o[i][4 * c + 1]);
            o[i][4 * c + 2] = fmaf(w, v.z, o[i][4 * c + 2]);
            o[i][4 * c + 3] = fmaf(w, v.w, o[i][4 * c + 3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = ty * 8 + i;
    if (r >= nq) continue;
    const size_t row = row0 + r;
    if (p.nks > 1) {
      const size_t prow = (size_t)split * p.B * p.H * p.N + row;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        *reinterpret_cast<float4*>(p.part_o + prow * D + c * 64 + tx * 4) =
            make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
      if (tx == 0) p.part_ml[prow] = make_float2(m[i], l[i]);
    } else {
      const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;  // 0 without keys; NaN stays NaN
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const size_t at = row * D + (c / 4) * 64 + tx * 4 + (c % 4);
        const float x = o[i][c] * inv;
        T y;
        store_elem(&y, x);
        static_cast<T*>(p.o)[at] = y;
        if (sizeof(T) == 2 && p.o_res != nullptr) store_elem(static_cast<bf16*>(p.o_res) + at, x - to_f32(y));
      }
      if (tx == 0) p.lse[row] = l[i] != 0.f ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
    }
  }
}

// The splits of a row joined: one warp per row, in the order of the splits.
template <typename T, int D>
__global__ void __launch_bounds__(256)
cross_combine_kernel(CrossParams p) {
  constexpr int C = D / 32;
  const size_t rows = (size_t)p.B * p.H * p.N;
  const size_t row = (size_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float m = -INFINITY;
  for (int z = lane; z < p.nks; z += 32) m = fmaxf(m, p.part_ml[z * rows + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float mb = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
#pragma unroll 4
  for (int z = 0; z < p.nks; ++z) {
    const float2 ml = p.part_ml[z * rows + row];
    if (ml.x == -INFINITY) continue;  // a split without keys: its O may not be written
    const float w = exp2f(ml.x - mb);
    l = fmaf(ml.y, w, l);
    const float* src = p.part_o + (z * rows + row) * D + lane * C;
    if (C == 2) {
      const float2 v = *reinterpret_cast<const float2*>(src);
      acc[0] = fmaf(v.x, w, acc[0]);
      acc[1] = fmaf(v.y, w, acc[1]);
    } else {
      const float4 v = *reinterpret_cast<const float4*>(src);
      acc[0] = fmaf(v.x, w, acc[0]);
      acc[1] = fmaf(v.y, w, acc[1]);
      acc[C - 2] = fmaf(v.z, w, acc[C - 2]);
      acc[C - 1] = fmaf(v.w, w, acc[C - 1]);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const size_t at = row * D + lane * C + c;
    const float x = acc[c] * inv;
    T y;
    store_elem(&y, x);
    static_cast<T*>(p.o)[at] = y;
    if (sizeof(T) == 2 && p.o_res != nullptr) store_elem(static_cast<bf16*>(p.o_res) + at, x - to_f32(y));
  }
  if (lane == 0) p.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// ---------------------------------------------------------------- backward
// Delta = dO . (O + residual): a warp per row
template <typename T, int D>
__global__ void __launch_bounds__(256)
cross_delta_kernel(CrossParams p) {
  constexpr int C = D / 32;
  const size_t rows = (size_t)p.B * p.H * p.N;
  const size_t row = (size_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const size_t at = row * D + lane * C + c;
    float o = to_f32(static_cast<const T*>(p.o_in)[at]);
    if (sizeof(T) == 2 && p.res_in != nullptr) o += to_f32(static_cast<const bf16*>(p.res_in)[at]);
    s = fmaf(o, to_f32(static_cast<const T*>(p.dout)[at]), s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.delta[row] = s;
}

// The P and dS of a tile, written to shared memory [query][key].
template <int D>
__device__ __forceinline__ void p_and_ds(const float* Q, const float* K, const float* dO, const float* V, float* P,
                                         float* dS, const float* lse2, const float* del, const uint8_t* keep,
                                         float sc2, int ty, int tx) {
  float s[4][4], dp[4][4];
  dot_tile<D, 4>(s, Q, K, ty, tx);
  dot_tile<D, 4>(dp, dO, V, ty, tx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = tx + 16 * j;
      const float e = keep[c] != 0 ? exp2f(fmaf(s[i][j], sc2, -lse2[r])) : 0.f;
      P[r * kLP + c] = e;
      dS[r * kLP + c] = e * (dp[i][j] - del[r]);
    }
  }
}

// lse2[r], del[r] of 64 query rows; rows past the end take lse = +inf, so
// that their probabilities are zero
__device__ __forceinline__ void load_side(float* lse2, float* del, const CrossParams& p, size_t row0, int nq) {
  if (threadIdx.x < kT) {
    const bool on = (int)threadIdx.x < nq;
    lse2[threadIdx.x] = on ? p.lse_in[row0 + threadIdx.x] * kLog2e : INFINITY;
    del[threadIdx.x] = on ? p.delta[row0 + threadIdx.x] : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* dst, const float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) store_elem(dst + i, v[i]);
}

template <int D>
struct BwdSmem {
  static constexpr int LD = D + 4;
  static constexpr int kFloats = 4 * kT * LD + 2 * kT * kLP;
};

// dQ of one query tile over one split of the key tiles.
template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads)
cross_dq_simt(CrossParams p, int qtiles) {
  constexpr int LD = D + 4;
  extern __shared__ __align__(16) float smf[];
  __shared__ uint8_t keep[kT];
  __shared__ float lse2[kT], del[kT];
  float *Q = smf, *dO = Q + kT * LD, *K = dO + kT * LD, *V = K + kT * LD, *P = V + kT * LD, *dS = P + kT * kLP;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  long long id = blockIdx.x;
  const int qt = (int)(id % qtiles);
  id /= qtiles;
  const int split = (int)(id % p.nks);
  const int bh = (int)(id / p.nks);
  const int b = bh / p.H;
  const size_t kvrow = (size_t)bh * p.S;
  const int q0 = qt * kT, nq = min(kT, p.N - q0);
  const size_t row0 = (size_t)bh * p.N + q0;
  const int len = cross_len(p, b);
  const int ktiles = (len + kT - 1) / kT;
  const int kt0 = (int)((long long)ktiles * split / p.nks), kt1 = (int)((long long)ktiles * (split + 1) / p.nks);
  load_rows<T, D, LD, kBwdThreads>(Q, static_cast<const T*>(p.q) + row0 * D, nq, nullptr);
  load_rows<T, D, LD, kBwdThreads>(dO, static_cast<const T*>(p.dout) + row0 * D, nq, nullptr);
  load_side(lse2, del, p, row0, nq);
  float acc[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
  for (int kt = kt0; kt < kt1; ++kt) {
    const int k0 = kt * kT, nk = min(kT, p.S - k0);
    __syncthreads();
    load_keep(keep, p, b, k0, len);
    __syncthreads();
    load_rows<T, D, LD, kBwdThreads>(K, static_cast<const T*>(p.k) + (kvrow + k0) * D, nk, keep);
    load_rows<T, D, LD, kBwdThreads>(V, static_cast<const T*>(p.v) + (kvrow + k0) * D, nk, keep);
    __syncthreads();
    p_and_ds<D>(Q, K, dO, V, P, dS, lse2, del, keep, p.scale * kLog2e, ty, tx);
    __syncwarp();  // a dS row is written and read by one half warp
    for (int j = 0; j < kT; ++j) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = dS[(ty * 4 + i) * kLP + j];
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 k4 = *reinterpret_cast<const float4*>(K + j * LD + c * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][4 * c] = fmaf(w[i], k4.x, acc[i][4 * c]);
          acc[i][4 * c + 1] = fmaf(w[i], k4.y, acc[i][4 * c + 1]);
          acc[i][4 * c + 2] = fmaf(w[i], k4.z, acc[i][4 * c + 2]);
          acc[i][4 * c + 3] = fmaf(w[i], k4.w, acc[i][4 * c + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
    if (r >= nq) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const size_t at = (row0 + r) * D + c * 64 + tx * 4;
      if (p.nks > 1) {
        store4(p.part_dq + (size_t)split * p.B * p.H * p.N * D + at, &acc[i][4 * c]);
      } else {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = acc[i][4 * c + e] * p.scale;
        store4(static_cast<T*>(p.dq) + at, x);
      }
    }
  }
}

// dK and dV of one key tile over one segment of the query tiles.
template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads)
cross_dkv_simt(CrossParams p, int qtiles, int ktiles) {
  constexpr int LD = D + 4;
  extern __shared__ __align__(16) float smf[];
  __shared__ uint8_t keep[kT];
  __shared__ float lse2[kT], del[kT];
  float *Q = smf, *dO = Q + kT * LD, *K = dO + kT * LD, *V = K + kT * LD, *P = V + kT * LD, *dS = P + kT * kLP;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  long long id = blockIdx.x;
  const int kt = (int)(id % ktiles);
  id /= ktiles;
  const int z = (int)(id % p.nz);
  const int bh = (int)(id / p.nz);
  const int b = bh / p.H;
  const int k0 = kt * kT, nk = min(kT, p.S - k0);
  const size_t kvrow = (size_t)bh * p.S + k0;
  const int len = cross_len(p, b);
  load_keep(keep, p, b, k0, len);
  __syncthreads();
  load_rows<T, D, LD, kBwdThreads>(K, static_cast<const T*>(p.k) + kvrow * D, nk, keep);
  load_rows<T, D, LD, kBwdThreads>(V, static_cast<const T*>(p.v) + kvrow * D, nk, keep);
  float ak[4][D / 16], av[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) ak[i][c] = av[i][c] = 0.f;
  int qt = (int)((long long)qtiles * z / p.nz);
  const int qt1 = k0 < len ? (int)((long long)qtiles * (z + 1) / p.nz) : qt;  // a tile past the end gets zeros
  for (; qt < qt1; ++qt) {
    const int q0 = qt * kT, nq = min(kT, p.N - q0);
    const size_t row0 = (size_t)bh * p.N + q0;
    __syncthreads();
    load_rows<T, D, LD, kBwdThreads>(Q, static_cast<const T*>(p.q) + row0 * D, nq, nullptr);
    load_rows<T, D, LD, kBwdThreads>(dO, static_cast<const T*>(p.dout) + row0 * D, nq, nullptr);
    load_side(lse2, del, p, row0, nq);
    __syncthreads();
    p_and_ds<D>(Q, K, dO, V, P, dS, lse2, del, keep, p.scale * kLog2e, ty, tx);
    __syncthreads();
    for (int r = 0; r < kT; ++r) {
      const float4 w = *reinterpret_cast<const float4*>(P + r * kLP + ty * 4);
      const float4 u = *reinterpret_cast<const float4*>(dS + r * kLP + ty * 4);
      const float wv[4] = {w.x, w.y, w.z, w.w}, uv[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 g = *reinterpret_cast<const float4*>(dO + r * LD + c * 64 + tx * 4);
        const float4 q = *reinterpret_cast<const float4*>(Q + r * LD + c * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          av[i][4 * c] = fmaf(wv[i], g.x, av[i][4 * c]);
          av[i][4 * c + 1] = fmaf(wv[i], g.y, av[i][4 * c + 1]);
          av[i][4 * c + 2] = fmaf(wv[i], g.z, av[i][4 * c + 2]);
          av[i][4 * c + 3] = fmaf(wv[i], g.w, av[i][4 * c + 3]);
          ak[i][4 * c] = fmaf(uv[i], q.x, ak[i][4 * c]);
          ak[i][4 * c + 1] = fmaf(uv[i], q.y, ak[i][4 * c + 1]);
          ak[i][4 * c + 2] = fmaf(uv[i], q.z, ak[i][4 * c + 2]);
          ak[i][4 * c + 3] = fmaf(uv[i], q.w, ak[i][4 * c + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
    if (r >= nk) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const size_t at = (kvrow + r) * D + c * 64 + tx * 4;
      if (p.nz > 1) {
        const size_t off = (size_t)z * p.B * p.H * p.S * D + at;
        store4(p.part_dk + off, &ak[i][4 * c]);
        store4(p.part_dv + off, &av[i][4 * c]);
      } else {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = ak[i][4 * c + e] * p.scale;
        store4(static_cast<T*>(p.dk) + at, x);
        store4(static_cast<T*>(p.dv) + at, &av[i][4 * c]);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
cross_reduce_kernel(const float* __restrict__ part, T* __restrict__ out, int n, size_t total, float f) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= total) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int z = 0; z < n; ++z) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(part + (size_t)z * total + i));
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  const float x[4] = {a.x * f, a.y * f, a.z * f, a.w * f};
  store4(out + i, x);
}

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int D>
cudaError_t fwd_typed(const CrossParams& p, cudaStream_t s) {
  const int qt = tiles_of(p.N);
  const long long blocks = (long long)p.B * p.H * p.nks * qt;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t smem = (size_t)(2 * kT * (D + 4) + kT * D) * sizeof(float);
  cudaError_t e = allow_smem(cross_fwd_simt<T, D>, smem);
  if (e != cudaSuccess) return e;
  cross_fwd_simt<T, D><<<(unsigned)blocks, kFwdThreads, smem, s>>>(p, qt);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd_typed(const CrossParams& p, cudaStream_t s) {
  const int qt = tiles_of(p.N), kt = tiles_of(p.S);
  const long long b1 = (long long)p.B * p.H * p.nks * qt, b2 = (long long)p.B * p.H * p.nz * kt;
  if (b1 > 0x7fffffffLL || b2 > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t smem = BwdSmem<D>::kFloats * sizeof(float);
  cudaError_t e = allow_smem(cross_dq_simt<T, D>, smem);
  if (e == cudaSuccess) e = allow_smem(cross_dkv_simt<T, D>, smem);
  if (e != cudaSuccess) return e;
  cross_dq_simt<T, D><<<(unsigned)b1, kBwdThreads, smem, s>>>(p, qt);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.S == 0) return e;
  cross_dkv_simt<T, D><<<(unsigned)b2, kBwdThreads, smem, s>>>(p, qt, kt);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t rows_typed(const CrossParams& p, bool combine, cudaStream_t s) {
  const size_t blocks = ((size_t)p.B * p.H * p.N + 7) / 8;
  if (blocks > 0x7fffffffULL) return cudaErrorInvalidValue;
  if (combine) cross_combine_kernel<T, D><<<(unsigned)blocks, 256, 0, s>>>(p);
  else cross_delta_kernel<T, D><<<(unsigned)blocks, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t rows_dispatch(const CrossParams& p, int dtype, bool combine, cudaStream_t s) {
  if (dtype == LLSA_BF16) return p.D == 64 ? rows_typed<bf16, 64>(p, combine, s) : rows_typed<bf16, 128>(p, combine, s);
  return p.D == 64 ? rows_typed<float, 64>(p, combine, s) : rows_typed<float, 128>(p, combine, s);
}

// parts of n tiles so that units * parts reaches about two blocks per SM
int parts_for(long long units, int n) {
  if (n < 1) return 1;
  long long parts = (2LL * kCrossSms + units - 1) / units;
  if (parts > n) parts = n;
  return parts < 1 ? 1 : (int)parts;
}

}  // namespace

CrossPlan cross_simt_fwd_plan(long long BH, int N, int S) { return {parts_for(BH * tiles_of(N), tiles_of(S)), 1}; }

CrossPlan cross_simt_bwd_plan(long long BH, int N, int S) {
  return {parts_for(BH * tiles_of(N), tiles_of(S)), parts_for(BH * (S > 0 ? tiles_of(S) : 1), tiles_of(N))};
}

cudaError_t launch_cross_fwd_simt(const CrossParams& p, int dtype, cudaStream_t s) {
  if (dtype == LLSA_BF16) return p.D == 64 ? fwd_typed<bf16, 64>(p, s) : fwd_typed<bf16, 128>(p, s);
  return p.D == 64 ? fwd_typed<float, 64>(p, s) : fwd_typed<float, 128>(p, s);
}

cudaError_t launch_cross_bwd_simt(const CrossParams& p, int dtype, cudaStream_t s) {
  if (dtype == LLSA_BF16) return p.D == 64 ? bwd_typed<bf16, 64>(p, s) : bwd_typed<bf16, 128>(p, s);
  return p.D == 64 ? bwd_typed<float, 64>(p, s) : bwd_typed<float, 128>(p, s);
}

cudaError_t launch_cross_combine(const CrossParams& p, int dtype, cudaStream_t s) {
  return rows_dispatch(p, dtype, true, s);
}

cudaError_t launch_cross_delta(const CrossParams& p, int dtype, cudaStream_t s) {
  return rows_dispatch(p, dtype, false, s);
}

cudaError_t launch_cross_reduce(const float* part, void* out, int n, size_t total, float f, int dtype,
                                cudaStream_t s) {
  if (total == 0) return cudaSuccess;
  const size_t blocks = (total / 4 + 255) / 256;
  if (blocks > 0x7fffffffULL) return cudaErrorInvalidValue;
  if (dtype == LLSA_BF16)
    cross_reduce_kernel<bf16><<<(unsigned)blocks, 256, 0, s>>>(part, static_cast<bf16*>(out), n, total, f);
  else
    cross_reduce_kernel<float><<<(unsigned)blocks, 256, 0, s>>>(part, static_cast<float*>(out), n, total, f);
  return cudaGetLastError();
}

}  // namespace llsa
