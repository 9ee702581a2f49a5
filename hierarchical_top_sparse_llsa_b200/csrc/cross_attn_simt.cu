// Cross attention in fp32 on the CUDA cores: forward, dQ, and dK with dV, in
// tiles of 64 queries (16 in a short forward) x 64 keys.
//
//   s = scale q k^T, P = e^(s - lse), O = P V / l
//   dV = P^T dO, dS = P (dO V^T - Delta), dQ = scale dS K, dK = scale dS^T Q
//
// Tensor-core formats hold too few bits for fp32 inputs.  A thread holds a block
// of the tile in registers (8 x 4 scores in the forward) and feeds it with 16-byte
// shared-memory loads, rows padded so that the 16 keys a half warp reads sit in
// different banks.  Probabilities pass through shared memory, over the K tile that
// is no longer read.  19 to 22 TFLOP/s at 16384 queries x 256 keys, of about 74: by
// count the FMAs wait for the loads from shared memory (16 bytes a thread take 9
// cycles an SM).
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

inline int tiles_of(int n, int t = kT) { return n / t + (n % t != 0); }

// rows r < nrows of src [.., D] (kept where keep is null or keep[r] != 0) into
// `rows` dst rows of LD floats; the others as zeros
template <int D, int LD, int THREADS>
__device__ __forceinline__ void load_rows(float* dst, const void* src, int nrows, const uint8_t* keep, int rows = kT) {
#pragma unroll 4
  for (int e = threadIdx.x; e < rows * (D / 4); e += THREADS) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nrows && (keep == nullptr || keep[r] != 0))
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + (size_t)r * D + c);
    *reinterpret_cast<float4*>(dst + r * LD + c) = x;
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

// of the columns j < J
template <int D, int R, int J>
__device__ __forceinline__ void dot_part(float (&acc)[R][4], const float* a, const float* b, int ty, int tx) {
  constexpr int LD = D + 4;
#pragma unroll 2
  for (int d = 0; d < D; d += 4) {
    float4 y[J];
#pragma unroll
    for (int j = 0; j < J; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(a + (ty * R + i) * LD + d);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        acc[i][j] = fmaf(x.x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x.y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x.z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x.w, y[j].w, acc[i][j]);
      }
    }
  }
}

// acc[i][j] = a row (ty * R + i) . b row (tx + 16 j), of the first n rows of b
// (16 more at a time)
template <int D, int R>
__device__ __forceinline__ void dot_tile(float (&acc)[R][4], const float* a, const float* b, int n, int ty, int tx) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  if (n > 32) dot_part<D, R, 4>(acc, a, b, ty, tx);
  else if (n > 16) dot_part<D, R, 2>(acc, a, b, ty, tx);
  else dot_part<D, R, 1>(acc, a, b, ty, tx);
}

constexpr int kLP = kT + 4;  // row length of the probability tiles

// Rows that the forward's key tiles hold: what dot_tile and the product read of
// a short sequence's only tile, so that more CTAs fit on an SM (9 heads of 29127
// queries, us, against 64 rows always: D = 128, one key 158 and 166, 16 keys 194
// and 205, 32 keys 258 and 268; D = 64, 90 and 94, 108 and 113, 144 and 148).
__host__ __device__ inline int key_rows(int S) { return S > 32 ? kT : (S > 16 ? 32 : 16); }

// ----------------------------------------------------------------- forward
// R query rows a thread, 8 R a tile
template <int D, int R>
__global__ void __launch_bounds__(kFwdThreads)
cross_fwd_simt(CrossParams p, int qtiles) {
  constexpr int LD = D + 4;
  extern __shared__ __align__(16) float smf[];
  __shared__ uint8_t keep[kT];
  constexpr int kQ = 8 * R;
  float* Q = smf;             // [kQ][LD]
  const int kr = key_rows(p.S);
  float* K = Q + kQ * LD;     // [kr][LD], then P [kQ][kLP]
  float* V = K + max(kr * LD, kQ * kLP);  // [kr][D]
  float* P = K;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  long long id = blockIdx.x;
  const int qt = (int)(id % qtiles);
  id /= qtiles;
  const int split = (int)(id % p.nks);
  const int bh = (int)(id / p.nks);
  const int b = bh / p.H;
  const size_t kvrow = (size_t)bh * p.S;
  const int q0 = qt * kQ, nq = min(kQ, p.N - q0);
  const size_t row0 = (size_t)bh * p.N + q0;
  const int len = cross_len(p, b);
  const int ktiles = (len + kT - 1) / kT;
  const int kt0 = (int)((long long)ktiles * split / p.nks), kt1 = (int)((long long)ktiles * (split + 1) / p.nks);
  const float sc2 = p.scale * kLog2e;

  load_rows<D, LD, kFwdThreads>(Q, static_cast<const float*>(p.q) + row0 * D, nq, nullptr, kQ);
  float o[R][D / 16];
  float m[R], l[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
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
    load_rows<D, LD, kFwdThreads>(K, static_cast<const float*>(p.k) + (kvrow + k0) * D, nk, keep, kr);
    load_rows<D, D, kFwdThreads>(V, static_cast<const float*>(p.v) + (kvrow + k0) * D, nk, keep, kr);
    __syncthreads();
    float s[R][4];
    dot_tile<D, R>(s, Q, K, nk, ty, tx);
    bool on[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) on[j] = keep[tx + 16 * j] != 0;
    __syncthreads();  // K is read; P takes its place
#pragma unroll
    for (int i = 0; i < R; ++i) {
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
        P[(ty * R + i) * kLP + tx + 16 * j] = e;
        sum += e;
      }
      l[i] = l[i] * corr + half_sum(sum);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[i][c] *= corr;
    }
    __syncwarp();  // a P row is written and read by one half warp
    for (int j = 0; j < nk; j += 4) {
      float4 pr[R];
#pragma unroll
      for (int i = 0; i < R; ++i) pr[i] = *reinterpret_cast<const float4*>(P + (ty * R + i) * kLP + j);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(V + (j + jj) * D + c * 64 + tx * 4);
#pragma unroll
          for (int i = 0; i < R; ++i) {
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
  for (int i = 0; i < R; ++i) {
    const int r = ty * R + i;
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
      for (int c = 0; c < D / 64; ++c)
        *reinterpret_cast<float4*>(static_cast<float*>(p.o) + row * D + c * 64 + tx * 4) =
            make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv);
      if (tx == 0) p.lse[row] = l[i] != 0.f ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
    }
  }
}

// The splits of a row joined, in a fixed order: by a warp, or (kWarps = 8, for
// eight splits or more) by a block whose warps take every eighth.
template <typename T, int D, int kWarps>
__global__ void __launch_bounds__(256)
cross_combine_kernel(CrossParams p) {
  constexpr int C = D / 32;
  __shared__ float part[kWarps][D + 1];
  const size_t rows = (size_t)p.B * p.H * p.N;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const size_t row = kWarps == 1 ? (size_t)blockIdx.x * 8 + warp : (size_t)blockIdx.x;
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
  for (int z = kWarps == 1 ? 0 : warp; z < p.nks; z += kWarps) {
    const float2 ml = p.part_ml[z * rows + row];
    // a split without keys: its O may not be written.  By the sum, for a split
    // whose scores are all NaN has no maximum either, and must show.
    if (ml.y == 0.f) continue;
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
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) part[warp][lane * C + c] = acc[c];
    if (lane == 0) part[warp][D] = l;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int u = 1; u < kWarps; ++u) {
      l += part[u][D];
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] += part[u][lane * C + c];
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
// The P and dS of a tile, written to shared memory [query][key].
template <int D>
__device__ __forceinline__ void p_and_ds(const float* Q, const float* K, const float* dO, const float* V, float* P,
                                         float* dS, const float* lse2, const float* del, const uint8_t* keep,
                                         float sc2, bool one, int nk, int ty, int tx) {
  float s[4][4], dp[4][4];
  dot_tile<D, 4>(s, Q, K, nk, ty, tx);
  dot_tile<D, 4>(dp, dO, V, nk, ty, tx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = tx + 16 * j;
      const float e = keep[c] != 0 ? exp2f(fmaf(s[i][j], sc2, -lse2[r])) : 0.f;
      P[r * kLP + c] = e;
      dS[r * kLP + c] = one ? 0.f : e * (dp[i][j] - del[r]);
    }
  }
}

// lse2[r] and del[r] = dO . O of 64 query rows, four threads a row; rows past
// the end take lse = +inf, so that their probabilities are zero.  dO: the tile.
template <int D>
__device__ __forceinline__ void load_side(float* lse2, float* del, const float* dO, const CrossParams& p, size_t row0,
                                          int nq) {
  const int r = threadIdx.x / 4, q = threadIdx.x % 4;
  float s = 0.f;
  if (r < nq) {
    const float* o = static_cast<const float*>(p.o_in) + (row0 + r) * D;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const float4 x = *reinterpret_cast<const float4*>(o + (4 * c + q) * 4);
      const float4 y = *reinterpret_cast<const float4*>(dO + r * (D + 4) + (4 * c + q) * 4);
      s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
    }
  }
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  if (q == 0) {
    const float l = r < nq ? p.lse_in[row0 + r] : INFINITY;
    lse2[r] = l == -INFINITY ? INFINITY : l * kLog2e;  // without keys too
    del[r] = s;
  }
}

__device__ __forceinline__ void store4(float* dst, const float* v) {
  *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
}

template <int D>
struct BwdSmem {
  static constexpr int LD = D + 4;
  static constexpr int kFloats = 4 * kT * LD + 2 * kT * kLP;
};

struct BwdSide {
  uint8_t keep[kT];
  float lse2[kT], del[kT];
};

// dQ of one query tile over one split of the key tiles.
template <int D>
__device__ __forceinline__ void dq_tile(const CrossParams& p, int qtiles, long long id, float* smf, BwdSide& S) {
  constexpr int LD = D + 4;
  uint8_t* keep = S.keep;
  float *lse2 = S.lse2, *del = S.del;
  float *Q = smf, *dO = Q + kT * LD, *K = dO + kT * LD, *V = K + kT * LD, *P = V + kT * LD, *dS = P + kT * kLP;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
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
  const bool one = sees_one(p, b, len);
  load_rows<D, LD, kBwdThreads>(Q, static_cast<const float*>(p.q) + row0 * D, nq, nullptr);
  load_rows<D, LD, kBwdThreads>(dO, static_cast<const float*>(p.dout) + row0 * D, nq, nullptr);
  __syncthreads();
  load_side<D>(lse2, del, dO, p, row0, nq);
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
    load_rows<D, LD, kBwdThreads>(K, static_cast<const float*>(p.k) + (kvrow + k0) * D, nk, keep);
    load_rows<D, LD, kBwdThreads>(V, static_cast<const float*>(p.v) + (kvrow + k0) * D, nk, keep);
    __syncthreads();
    p_and_ds<D>(Q, K, dO, V, P, dS, lse2, del, keep, p.scale * kLog2e, one, nk, ty, tx);
    __syncwarp();  // a dS row is written and read by one half warp
    for (int j = 0; j < nk; ++j) {
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
        store4(static_cast<float*>(p.dq) + at, x);
      }
    }
  }
}

// dK and dV of one key tile over one segment of the query tiles.
template <int D>
__device__ __forceinline__ void dkv_tile(const CrossParams& p, int qtiles, int ktiles, long long id, float* smf,
                                         BwdSide& S) {
  constexpr int LD = D + 4;
  uint8_t* keep = S.keep;
  float *lse2 = S.lse2, *del = S.del;
  float *Q = smf, *dO = Q + kT * LD, *K = dO + kT * LD, *V = K + kT * LD, *P = V + kT * LD, *dS = P + kT * kLP;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int kt = (int)(id % ktiles);
  id /= ktiles;
  const int z = (int)(id % p.nz);
  const int bh = (int)(id / p.nz);
  const int b = bh / p.H;
  const int k0 = kt * kT, nk = min(kT, p.S - k0);
  const size_t kvrow = (size_t)bh * p.S + k0;
  const int len = cross_len(p, b);
  const bool one = sees_one(p, b, len);
  load_keep(keep, p, b, k0, len);
  __syncthreads();
  load_rows<D, LD, kBwdThreads>(K, static_cast<const float*>(p.k) + kvrow * D, nk, keep);
  load_rows<D, LD, kBwdThreads>(V, static_cast<const float*>(p.v) + kvrow * D, nk, keep);
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
    load_rows<D, LD, kBwdThreads>(Q, static_cast<const float*>(p.q) + row0 * D, nq, nullptr);
    load_rows<D, LD, kBwdThreads>(dO, static_cast<const float*>(p.dout) + row0 * D, nq, nullptr);
    __syncthreads();
    load_side<D>(lse2, del, dO, p, row0, nq);
    __syncthreads();
    p_and_ds<D>(Q, K, dO, V, P, dS, lse2, del, keep, p.scale * kLog2e, one, nk, ty, tx);
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
        store4(static_cast<float*>(p.dk) + at, x);
        store4(static_cast<float*>(p.dv) + at, &av[i][4 * c]);
      }
    }
  }
}

// The blocks of dK and dV, which are the longer ones, then those of dQ: one
// launch, for neither alone fills the GPU in a short problem.
template <int D>
__global__ void __launch_bounds__(kBwdThreads)
cross_bwd_simt(CrossParams p, int qtiles, int ktiles, int dkv_blocks) {
  extern __shared__ __align__(16) float smf[];
  __shared__ BwdSide S;
  const long long id = blockIdx.x;
  if (id < dkv_blocks) dkv_tile<D>(p, qtiles, ktiles, id, smf, S);
  else dq_tile<D>(p, qtiles, id - dkv_blocks, smf, S);
}

// The parts of dQ, dK and dV (blockIdx.y, from `first`) summed in order.
__global__ void __launch_bounds__(256)
cross_reduce_kernel(CrossParams p, int first) {
  const int which = first + blockIdx.y;
  const size_t total = (size_t)p.B * p.H * (which == 0 ? p.N : p.S) * p.D;
  const float* part = which == 0 ? p.part_dq : (which == 1 ? p.part_dk : p.part_dv);
  float* out = static_cast<float*>(which == 0 ? p.dq : (which == 1 ? p.dk : p.dv));
  const int n = which == 0 ? p.nks : p.nz;
  const float f = which == 2 ? 1.f : p.scale;
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
  *reinterpret_cast<float4*>(out + i) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
}

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Query rows a thread of the forward: tiles of 16 rows where 64 would be mostly
// empty, or would leave SMs without a block however the keys are cut.
inline int fwd_rows(long long BH, int N, int S) {
  return N <= 32 || BH * tiles_of(N) * ((tiles_of(S) + 1) / 2) < kCrossSms ? 2 : 8;
}

template <int D, int R>
cudaError_t fwd_typed(const CrossParams& p, cudaStream_t s) {
  const int qt = tiles_of(p.N, 8 * R);
  const long long blocks = (long long)p.B * p.H * p.nks * qt;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int kr = key_rows(p.S), kq = 8 * R;
  const size_t smem = (size_t)(kq * (D + 4) + max(kr * (D + 4), kq * kLP) + kr * D) * sizeof(float);
  cudaError_t e = allow_smem(cross_fwd_simt<D, R>, smem);
  if (e != cudaSuccess) return e;
  cross_fwd_simt<D, R><<<(unsigned)blocks, kFwdThreads, smem, s>>>(p, qt);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd_typed(const CrossParams& p, cudaStream_t s) {
  const int qt = tiles_of(p.N), kt = tiles_of(p.S);
  const long long b1 = (long long)p.B * p.H * p.nks * qt, b2 = (long long)p.B * p.H * p.nz * kt;
  if (b1 + b2 > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t smem = BwdSmem<D>::kFloats * sizeof(float);
  cudaError_t e = allow_smem(cross_bwd_simt<D>, smem);
  if (e != cudaSuccess) return e;
  cross_bwd_simt<D><<<(unsigned)(b1 + b2), kBwdThreads, smem, s>>>(p, qt, kt, (int)b2);
  e = cudaGetLastError();
  const int first = p.nks > 1 ? 0 : 1, last = p.nz > 1 ? 2 : 0;
  if (e != cudaSuccess || first > last) return e;
  const size_t rows = first == 0 && last == 2 ? (size_t)max(p.N, p.S) : (size_t)(first == 0 ? p.N : p.S);
  const size_t blocks = (p.B * (size_t)p.H * rows * p.D / 4 + 255) / 256;
  if (blocks > 0x7fffffffULL) return cudaErrorInvalidValue;
  cross_reduce_kernel<<<dim3((unsigned)blocks, last - first + 1), 256, 0, s>>>(p, first);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t combine_typed(const CrossParams& p, cudaStream_t s) {
  const size_t rows = (size_t)p.B * p.H * p.N;
  if (p.nks >= 8) cross_combine_kernel<T, D, 8><<<(unsigned)rows, 256, 0, s>>>(p);
  else cross_combine_kernel<T, D, 1><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(p);
  return cudaGetLastError();
}

// parts of n tiles, two tiles or more in each, so that units * parts reaches
// about two blocks per SM
int parts_for(long long units, int n) {
  long long parts = 2LL * kCrossSms / units;
  if (parts > (n + 1) / 2) parts = (n + 1) / 2;
  return parts < 1 ? 1 : (int)parts;
}

}  // namespace

CrossPlan cross_simt_fwd_plan(long long BH, int N, int S) {
  return {parts_for(BH * tiles_of(N, 8 * fwd_rows(BH, N, S)), tiles_of(S)), 1};
}

CrossPlan cross_simt_bwd_plan(long long BH, int N, int S) {
  if (S == 0) return {1, 1};  // no dK and dV to cut or to join
  return {parts_for(BH * tiles_of(N), tiles_of(S)), parts_for(BH * tiles_of(S), tiles_of(N))};
}

cudaError_t launch_cross_fwd_simt(const CrossParams& p, cudaStream_t s) {
  const bool few = fwd_rows((long long)p.B * p.H, p.N, p.S) == 2;
  if (p.D == 64) return few ? fwd_typed<64, 2>(p, s) : fwd_typed<64, 8>(p, s);
  return few ? fwd_typed<128, 2>(p, s) : fwd_typed<128, 8>(p, s);
}

cudaError_t launch_cross_bwd_simt(const CrossParams& p, cudaStream_t s) {
  return p.D == 64 ? bwd_typed<64>(p, s) : bwd_typed<128>(p, s);
}

cudaError_t launch_cross_combine(const CrossParams& p, int dtype, cudaStream_t s) {
  if (dtype == LLSA_BF16) return p.D == 64 ? combine_typed<bf16, 64>(p, s) : combine_typed<bf16, 128>(p, s);
  return p.D == 64 ? combine_typed<float, 64>(p, s) : combine_typed<float, 128>(p, s);
}

}  // namespace llsa
