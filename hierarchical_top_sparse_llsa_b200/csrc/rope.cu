// Rotary positions: the cosine/sine table, the rotation of Q and K (and its
// adjoint for dQ and dK), and the rotation with the hierarchical compression
// (Step 1 of the howistudyai explainer of "Trainable Log-linear Sparse
// Attention for Efficient Diffusion Transformers") of the rotated tensors.
//
// A pair (a, b) of a head's channels turns by its token's angle:
//   (a c - b s, b c + a s)         adjoint: (a c + b s, b c - a s)
// Products and sums are rounded one by one in fp32 (no FMA), then once to the
// stored type, so the fused and the separate calls agree bit for bit.
//
// All three kernels are bound by memory.  The rotation reads and writes each
// element once; the table (rot_dim / 2 pairs of fp32, twice a bf16 head row)
// would be as much traffic again if it were read per head, so a thread keeps
// the cosines and sines of its token and channels in registers and walks the
// heads of Q and K with them.

#include "llsa_internal.cuh"
#include "rope.cuh"

namespace llsa {

namespace {

constexpr int kSms = 148;

// ---------------------------------------------------------------- the table
constexpr int kTableThreads = 256;

// the low 32 bits' even-position bits packed into the low 16 (bit 2b -> bit b)
__device__ __forceinline__ uint32_t even_bits(uint32_t v) {
  v &= 0x55555555u;
  v = (v | (v >> 1)) & 0x33333333u;
  v = (v | (v >> 2)) & 0x0f0f0f0fu;
  v = (v | (v >> 4)) & 0x00ff00ffu;
  v = (v | (v >> 8)) & 0x0000ffffu;
  return v;
}

// Cosine and sine, times m, of position x at turns.x + turns.y turns a position.
// The angle is held in turns: its whole turns come off the exact product in one
// fp64 step, the frequency's rest is added, and only the remainder in [-1/2, 1/2]
// is rounded to fp32 (sincospi of twice it), so the angle's error is 2^-24 of a
// half turn at any position.  (Whole turns off the rounded product, without the
// rest: 2^-22 more near 2^31, and no faster.)
__device__ __forceinline__ float2 turn_of(int x, double2 turns, float m) {
  const double p = (double)x;
  float s, c;
  sincospif(2.0f * (float)fma(p, turns.y, fma(p, turns.x, -rint(p * turns.x))), &s, &c);
  return make_float2(c * m, s * m);
}

// Pairs 2 j and 2 j + 1 of a row (a lone last pair is given twice).
__device__ __forceinline__ void store_turns(float* row, int half, int p0, float2 a, float2 b) {
  float* dst = row + 2 * p0;
  if ((half & 1) == 0) {  // whole rows are 16-byte aligned
    *reinterpret_cast<float4*>(dst) = make_float4(a.x, a.y, b.x, b.y);
  } else {
    *reinterpret_cast<float2*>(dst) = a;
    if (p0 + 1 < half) *reinterpret_cast<float2*>(dst + 2) = b;
  }
}

// Thread (r, j): pairs 2 j and 2 j + 1 of rows r, r + step, ...
__global__ void __launch_bounds__(kTableThreads)
rope_table_kernel(RopeFreqs f, int rows, const int32_t* __restrict__ pos, float* __restrict__ table) {
  // Lanes of unlike frequencies take the parameters' constant bank one after the
  // other, so each is read from there once a CTA.
  __shared__ double2 turns[kMaxRopeFreqs];
  if (threadIdx.x < f.n) turns[threadIdx.x] = f.turns[threadIdx.x];
  __syncthreads();
  const int hp = (f.half + 1) / 2;  // threads per row
  const int per = kTableThreads / hp;
  const int r0 = threadIdx.x / hp, j = threadIdx.x % hp;
  if (r0 >= per) return;
  const int p0 = 2 * j, p1 = min(2 * j + 1, f.half - 1);
  const int a0 = p0 / f.n, a1 = p1 / f.n;
  const double2 f0 = turns[p0 % f.n], f1 = turns[p1 % f.n];
  for (long long r = (long long)blockIdx.x * per + r0; r < rows; r += (long long)gridDim.x * per) {
    int x0, x1;
    if (pos != nullptr) {
      x0 = pos[r * f.axes + a0];
      x1 = pos[r * f.axes + a1];
    } else if (f.axes == 2) {  // Z-order
      x0 = (int)even_bits((uint32_t)r >> a0);
      x1 = (int)even_bits((uint32_t)r >> a1);
    } else {
      x0 = x1 = (int)r;
    }
    store_turns(table + r * f.half * 2, f.half, p0, turn_of(x0, f0, f.m), turn_of(x1, f1, f.m));
  }
}

// Two axes, positions from the Z-order: 256 consecutive tokens are a square of
// 16 x 16 pixels, so a CTA forms the turns of its 16 + 16 coordinates and
// writes each 16 times.  Chosen where more than half of the SMs have a square: its coordinates
// come before its first store, which only other CTAs can cover.  Computing every
// entry against this, us a launch, back to back: rot_dim 64, 256 rows 1.7 and 3.6,
// 16384 rows 3.5 and 3.7, 65536 rows 8.3 and 5.3; rot_dim 128, 2.1 and 6.2, 6.2
// and 6.4, 13.1 and 9.5.
constexpr int kSquare = 256;
__global__ void __launch_bounds__(kTableThreads)
rope_table_square_kernel(RopeFreqs f, int rows, float* __restrict__ table) {
  __shared__ float2 turns[2][16][kMaxRopeFreqs / 2 + 1];  // axis, coordinate, frequency
  const int r0 = blockIdx.x * kSquare;
  const int x0 = (int)even_bits((uint32_t)r0), y0 = (int)even_bits((uint32_t)r0 >> 1);
  for (int i = threadIdx.x; i < 32 * f.n; i += kTableThreads) {
    const int k = i & 31, w = i >> 5;  // a warp has one frequency
    turns[k >> 4][k & 15][w] = turn_of((k < 16 ? x0 : y0) + (k & 15), f.turns[w], f.m);
  }
  __syncthreads();
  const int hp = (f.half + 1) / 2;
  for (int i = threadIdx.x; i < kSquare * hp; i += kTableThreads) {
    const int r = i / hp, p0 = 2 * (i - r * hp), p1 = min(p0 + 1, f.half - 1);
    if (r0 + r >= rows) return;
    const int c[2] = {(int)even_bits((uint32_t)r), (int)even_bits((uint32_t)r >> 1)};
    const int a0 = p0 >= f.n, a1 = p1 >= f.n;
    store_turns(table + (size_t)(r0 + r) * f.half * 2, f.half, p0, turns[a0][a0 ? c[1] : c[0]][p0 - a0 * f.n],
                turns[a1][a1 ? c[1] : c[0]][p1 - a1 * f.n]);
  }
}

// ------------------------------------------------------------- the rotation
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const float* v);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* v) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<bf16>(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A slot is two 16-byte chunks of a head row that hold whole pairs: in the
// interleaved layout chunks 2 s and 2 s + 1, in the half layout chunk s and
// its partner rot_dim / 2 channels on (or, past the rotated channels, two
// neighbouring ones).  Needs rot_dim / 2 to be a multiple of a chunk in the
// half layout.
template <typename T>
struct Slot {
  static constexpr int VEC = Vec16<T>::N;
  int c0, c1;  // its chunks
  int pair0;   // its first pair
  int nrot;    // how many of its VEC pairs turn
  __device__ __forceinline__ Slot(int s, int half, bool interleaved) {
    if (interleaved) {
      c0 = 2 * s;
      c1 = 2 * s + 1;
      pair0 = s * VEC;
      nrot = min(max(half - pair0, 0), VEC);
    } else {
      const int hc = half / VEC;  // chunks of the first half
      const bool rot = s < hc;
      c0 = rot ? s : 2 * s;
      c1 = rot ? s + hc : 2 * s + 1;
      pair0 = rot ? s * VEC : 0;
      nrot = rot ? VEC : 0;
    }
  }
};

// cosines and sines of a slot's pairs (those that do not turn are not read)
template <int VEC>
__device__ __forceinline__ void load_turns(const float* __restrict__ row, int pair0, int nrot, float sign, float* c,
                                           float* s) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float2 t = make_float2(1.f, 0.f);
    if (e < nrot) t = __ldg(reinterpret_cast<const float2*>(row) + pair0 + e);
    c[e] = t.x;
    s[e] = sign * t.y;
  }
}

// The slot's two chunks, turned; what does not turn keeps its bits.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void turn_slot(uint4 (&v)[2], const float* c, const float* s, int nrot) {
  constexpr int VEC = Vec16<T>::N;
  float x[2 * VEC];
  Vec16<T>::unpack(v[0], x);
  Vec16<T>::unpack(v[1], x + VEC);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if (kInterleaved) turn(x[2 * e], x[2 * e + 1], c[e], s[e]);
    else turn(x[e], x[VEC + e], c[e], s[e]);
  }
  // word i of the two chunks belongs to pair i VEC / 8 (in the half layout a
  // slot turns as a whole or not at all)
  const uint4 w0 = pack16<T>(x), w1 = pack16<T>(x + VEC);
  if (0 * VEC / 8 < nrot) v[0].x = w0.x;
  if (1 * VEC / 8 < nrot) v[0].y = w0.y;
  if (2 * VEC / 8 < nrot) v[0].z = w0.z;
  if (3 * VEC / 8 < nrot) v[0].w = w0.w;
  if (4 * VEC / 8 < nrot) v[1].x = w1.x;
  if (5 * VEC / 8 < nrot) v[1].y = w1.y;
  if (6 * VEC / 8 < nrot) v[1].z = w1.z;
  if (7 * VEC / 8 < nrot) v[1].w = w1.w;
}

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;

// Thread: one slot of one token, over `per` of the (tensor, head) rows that
// share the token's table row.  Every element is read and written by one
// thread, the reads first, so the outputs may be the inputs.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(RopeParams p) {
  constexpr int VEC = Vec16<T>::N;
  const int slots = p.D / (2 * VEC);
  const int half = p.rot / 2;
  const long long e = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const long long tok = e / slots;  // b * N + n
  if (tok >= (long long)p.B * p.N) return;
  const long long b = tok / p.N, n = tok - b * p.N;
  const Slot<T> sl((int)(e - tok * slots), half, kInterleaved);
  float c[VEC], s[VEC];
  load_turns<VEC>(p.table + (p.per_batch ? tok : n) * (2 * half), sl.pair0, sl.nrot, p.sign, c, s);
  const int rows = p.H * p.ntensor;
  const int i0 = blockIdx.y * p.per, i1 = min(rows, i0 + p.per);
  for (int i = i0; i < i1; i += kRopeUnroll) {
    uint4 v[kRopeUnroll][2];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (i + u < i1) {
        const int t = (i + u) / p.H, h = (i + u) - t * p.H;
        const uint4* src = static_cast<const uint4*>(p.x[t]) + ((b * p.H + h) * p.N + n) * (p.D / VEC);
        v[u][0] = src[sl.c0];
        v[u][1] = src[sl.c1];
      }
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (i + u < i1) {
        const int t = (i + u) / p.H, h = (i + u) - t * p.H;
        uint4* dst = static_cast<uint4*>(p.y[t]) + ((b * p.H + h) * p.N + n) * (p.D / VEC);
        turn_slot<T, kInterleaved>(v[u], c, s, sl.nrot);
        dst[sl.c0] = v[u][0];
        dst[sl.c1] = v[u][1];
      }
    }
  }
}

// The half layout where a partner sits off the 16-byte chunks: a thread per
// pair (or per two channels that pass through), element by element.  Q and K of
// 24 heads, 16384 tokens of bf16, with 12 or 30 pairs 141 and 131 us, 45 in chunks.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads)
rope_ragged_kernel(RopeParams p) {
  const int half = p.rot / 2, slots = p.D / 2;
  const long long e = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const long long tok = e / slots;
  if (tok >= (long long)p.B * p.N) return;
  const long long b = tok / p.N, n = tok - b * p.N;
  const int s = (int)(e - tok * slots);
  const bool rot = s < half;
  const int d0 = rot ? s : 2 * s, d1 = rot ? s + half : 2 * s + 1;
  float2 t = make_float2(1.f, 0.f);
  if (rot) t = __ldg(reinterpret_cast<const float2*>(p.table + (p.per_batch ? tok : n) * (2 * half)) + s);
  t.y *= p.sign;
  const int rows = p.H * p.ntensor;
  const int i1 = min(rows, (int)(blockIdx.y + 1) * p.per);
  for (int i = blockIdx.y * p.per; i < i1; ++i) {
    const int k = i / p.H, h = i - k * p.H;
    const long long row = ((b * p.H + h) * p.N + n) * p.D;
    const T* src = static_cast<const T*>(p.x[k]) + row;
    T* dst = static_cast<T*>(p.y[k]) + row;
    if (rot) {
      float x = to_f32(src[d0]), y = to_f32(src[d1]);
      turn(x, y, t.x, t.y);
      store_elem(dst + d0, x);
      store_elem(dst + d1, y);
    } else {
      const T x = src[d0], y = src[d1];
      dst[d0] = x;
      dst[d1] = y;
    }
  }
}

template <typename T>
cudaError_t launch_rope_typed(RopeParams p, cudaStream_t s) {
  const int half = p.rot / 2;
  constexpr int VEC = Vec16<T>::N;
  const bool ragged = !p.interleaved && half % VEC != 0;
  const int slots = ragged ? p.D / 2 : p.D / (2 * VEC);
  const long long threads = (long long)p.B * p.N * slots;
  const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  // rows a thread walks: all that share its table row, fewer when that leaves
  // the SMs (8 blocks each) without work
  const int rows = p.H * p.ntensor;
  const long long want = 8LL * kSms;
  long long parts = (want + blocks - 1) / blocks;
  if (parts > rows) parts = rows;
  p.per = (int)((rows + parts - 1) / parts);
  const dim3 grid((unsigned)blocks, (unsigned)((rows + p.per - 1) / p.per));
  if (ragged) rope_ragged_kernel<T><<<grid, kRopeThreads, 0, s>>>(p);
  else if (p.interleaved) rope_kernel<T, true><<<grid, kRopeThreads, 0, s>>>(p);
  else rope_kernel<T, false><<<grid, kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------ the rotation with the pool
// One CTA: 256 tokens of one (b, h) of Q and K, or of V; thread (t1, slot)
// turns and sums the 16 rows of level-1 token t1 (16 rows of two chunks), left
// to right, as the pool kernel does; level 2 from the level-1 means in shared
// memory.  Q and K share the table's row, which is as large as a bf16 head's
// row of both and comes from the L2 cache for every head but the first.
// Rows, and the table's, are copied to shared memory kDepth ahead (cp.async;
// each thread its own chunks, so nothing is synchronised): up to 64 KB a CTA
// are in flight, without the registers that would cost.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the last n groups have landed
template <int n>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

template <typename T, int D>
struct PoolShape {
  static constexpr int kThreads = 16 * D / (2 * Vec16<T>::N);
  // a thread's part of a row: two chunks of Q and of K, its pairs' turns
  static constexpr int kTurns = Vec16<T>::N * 8, kPart = 64 + kTurns;
  // rows ahead: what hides the latency with several CTAs an SM.  At 256x256
  // pixels (64 threads): three 166 us, four 165, five 171, eight 174, sixteen
  // 302.  With a CTA an SM or fewer, every row that fits in flight gains
  // nothing (10.3 us with four, 10.8 with all; 144 CTAs, bf16, D = 64).
  static constexpr int kDepth = kThreads <= 64 ? 4 : 512 / kThreads;
  static constexpr int kSmem = kDepth * kPart * kThreads + 2 * 16 * D * 4;
};

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(PoolShape<T, D>::kThreads)
rope_pool_kernel(RopeParams p, PoolParams o) {
  using P = PoolShape<T, D>;
  constexpr int VEC = Vec16<T>::N;
  constexpr int SL = D / (2 * VEC);  // slots per row
  constexpr int kRow = D / VEC;      // chunks of a row
  extern __shared__ __align__(16) unsigned char smem[];
  // ring: [kDepth][chunk of Q, Q, K, K, turns ...][thread] of 16 bytes
  float* m1 = reinterpret_cast<float*>(smem + P::kDepth * P::kPart * P::kThreads);  // [tensor][16][D]
  const int kinds = o.L >= 2 ? 2 : 1;  // V has no level-1 output
  long long id = blockIdx.x;
  const bool is_v = kinds == 2 && (id & 1) != 0;
  id /= kinds;
  const int bh = (int)(id % o.BH);
  const int chunk = (int)(id / o.BH);
  const int tid = threadIdx.x, t1 = tid / SL;
  const int n1 = o.N / kBlock;
  const int g1 = chunk * 16 + t1;
  const int half = p.rot / 2;
  const Slot<T> sl(tid % SL, half, kInterleaved);
  const int nt = is_v ? 1 : 2;
  if (g1 < n1) {
    const size_t row0 = ((size_t)bh * o.N + (size_t)g1 * kBlock) * kRow;
    const uint4* src0 = static_cast<const uint4*>(is_v ? p.x[2] : p.x[0]) + row0;
    const uint4* src1 = static_cast<const uint4*>(p.x[1]) + row0;
    uint4* dst0 = static_cast<uint4*>(p.y[0]) + row0;
    uint4* dst1 = static_cast<uint4*>(p.y[1]) + row0;
    const size_t trow = (p.per_batch ? (size_t)(bh / p.H) * o.N : 0) + (size_t)g1 * kBlock;
    const float* tab = p.table + trow * (2 * half);
    constexpr int kLine = P::kThreads * 16;
    unsigned char* mine = smem + tid * 16;
    const bool wide = half % 2 == 0 && sl.nrot == VEC;  // turns in pieces of 16 bytes, else of 8
    auto fetch = [&](int j) {
      if (j < kBlock) {
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(mine) + (uint32_t)((j % P::kDepth) * P::kPart * P::kThreads);
        const float* turns = tab + (size_t)j * (2 * half) + 2 * sl.pair0;
        if (is_v) {
        } else if (wide) {
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) copy16(at + (4 + e) * kLine, turns + 4 * e);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (e < sl.nrot) copy8(at + (4 + e / 2) * kLine + (e & 1) * 8, turns + 2 * e);
        }
        copy16(at, src0 + j * kRow + sl.c0);
        copy16(at + kLine, src0 + j * kRow + sl.c1);
        if (!is_v) {
          copy16(at + 2 * kLine, src1 + j * kRow + sl.c0);
          copy16(at + 3 * kLine, src1 + j * kRow + sl.c1);
        }
      }
      copies_issued();
    };
#pragma unroll 1
    for (int j = 0; j < P::kDepth; ++j) fetch(j);
    float acc[2][2 * VEC];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 2 * VEC; ++e) acc[t][e] = 0.f;
#pragma unroll 2
    for (int j = 0; j < kBlock; ++j) {
      copies_wait<P::kDepth - 1>();
      const unsigned char* at = mine + (j % P::kDepth) * P::kPart * P::kThreads;
      float c[VEC], s[VEC];
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float4 t = *reinterpret_cast<const float4*>(at + (4 + e) * kLine);
        const bool on0 = 2 * e < sl.nrot, on1 = 2 * e + 1 < sl.nrot;
        c[2 * e] = on0 ? t.x : 1.f;
        s[2 * e] = on0 ? t.y : 0.f;
        c[2 * e + 1] = on1 ? t.z : 1.f;
        s[2 * e + 1] = on1 ? t.w : 0.f;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t == 1 && is_v) break;
        uint4 v[2] = {*reinterpret_cast<const uint4*>(at + 2 * t * kLine),
                      *reinterpret_cast<const uint4*>(at + (2 * t + 1) * kLine)};
        if (!is_v) {
          turn_slot<T, kInterleaved>(v, c, s, sl.nrot);
          uint4* dst = (t == 0 ? dst0 : dst1) + j * kRow;
          dst[sl.c0] = v[0];
          dst[sl.c1] = v[1];
        }
        float x[2 * VEC];  // the means are of the stored values
        Vec16<T>::unpack(v[0], x);
        Vec16<T>::unpack(v[1], x + VEC);
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) acc[t][e] = j == 0 ? x[e] : __fadd_rn(acc[t][e], x[e]);
      }
      fetch(j + P::kDepth);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t == 1 && is_v) break;
      float* o1 = is_v ? nullptr : (t == 0 ? o.lvl[0][1] : o.lvl[1][1]);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int d = (w ? sl.c1 : sl.c0) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          float4 m;
          m.x = __fmul_rn(acc[t][w * VEC + e], 0.0625f);
          m.y = __fmul_rn(acc[t][w * VEC + e + 1], 0.0625f);
          m.z = __fmul_rn(acc[t][w * VEC + e + 2], 0.0625f);
          m.w = __fmul_rn(acc[t][w * VEC + e + 3], 0.0625f);
          *reinterpret_cast<float4*>(m1 + (t * 16 + t1) * D + d + e) = m;
          if (o1 != nullptr) *reinterpret_cast<float4*>(o1 + ((size_t)bh * n1 + g1) * D + d + e) = m;
        }
      }
    }
  }
  if (o.L < 2) return;
  __syncthreads();
  // level 2: one level-2 token per CTA (N is a multiple of 256 when L >= 2)
  for (int i = tid; i < nt * D; i += P::kThreads) {
    const int t = i / D, d = i - t * D;
    const float* m = m1 + t * 16 * D + d;
    float a = m[0];
#pragma unroll
    for (int k = 1; k < 16; ++k) a = __fadd_rn(a, m[k * D]);
    float* o2 = is_v ? o.lvl[2][2] : (t == 0 ? o.lvl[0][2] : o.lvl[1][2]);
    o2[((size_t)bh * (o.N >> 8) + chunk) * D + d] = __fmul_rn(a, 0.0625f);
  }
}

template <typename T, int D, bool kInterleaved>
cudaError_t launch_rope_pool_as(const RopeParams& p, const PoolParams& o, long long blocks, cudaStream_t s) {
  using P = PoolShape<T, D>;
  const cudaError_t e = cudaFuncSetAttribute(rope_pool_kernel<T, D, kInterleaved>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (e != cudaSuccess) return e;
  rope_pool_kernel<T, D, kInterleaved><<<(unsigned)blocks, P::kThreads, P::kSmem, s>>>(p, o);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rope_pool_typed(const RopeParams& p, const PoolParams& o, cudaStream_t s) {
  const long long blocks = (long long)((o.N / kBlock + 15) / 16) * o.BH * (o.L >= 2 ? 2 : 1);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return p.interleaved ? launch_rope_pool_as<T, D, true>(p, o, blocks, s)
                       : launch_rope_pool_as<T, D, false>(p, o, blocks, s);
}

}  // namespace

cudaError_t launch_rope_table(const RopeFreqs& f, int rows, const int32_t* pos, float* table, cudaStream_t s) {
  if (pos == nullptr && f.axes == 2 && (rows - 1) / kSquare >= kSms / 2) {
    rope_table_square_kernel<<<(rows - 1) / kSquare + 1, kTableThreads, 0, s>>>(f, rows, table);
    return cudaGetLastError();
  }
  const int per = kTableThreads / ((f.half + 1) / 2);
  long long blocks = ((long long)rows + per - 1) / per;
  if (blocks > 16LL * kSms) blocks = 16LL * kSms;
  rope_table_kernel<<<(int)blocks, kTableThreads, 0, s>>>(f, rows, pos, table);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeParams& p, int dtype, cudaStream_t s) {
  return dtype == LLSA_BF16 ? launch_rope_typed<bf16>(p, s) : launch_rope_typed<float>(p, s);
}

bool rope_pool_fused(int rot, bool interleaved, int dtype) {
  return interleaved || (rot / 2) % (dtype == LLSA_BF16 ? 8 : 4) == 0;
}

cudaError_t launch_rope_pool(const RopeParams& p, const PoolParams& o, int dtype, cudaStream_t s) {
  cudaError_t e;
  if (dtype == LLSA_BF16)
    e = o.D == 64 ? launch_rope_pool_typed<bf16, 64>(p, o, s) : launch_rope_pool_typed<bf16, 128>(p, o, s);
  else
    e = o.D == 64 ? launch_rope_pool_typed<float, 64>(p, o, s) : launch_rope_pool_typed<float, 128>(p, o, s);
  if (e != cudaSuccess) return e;
  return launch_pool_up(o, s);
}

}  // namespace llsa
