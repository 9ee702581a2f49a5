// Cross attention backward on the 5th-generation tensor cores (tcgen05), bf16,
// D = 64 or 128:
//   P = e^(scale S - lse),  S = Q K^T,      dP = dO V^T
//   Delta_i = sum_j P_ij dP_ij,             dS = P (dP - Delta)
//   dQ = scale dS K,  dK = scale dS^T Q,    dV = P^T dO
// in two passes of one kernel: the first (kDq) walks the keys for 128 queries
// and gives dQ and Delta, the second walks the queries for 128 keys and gives
// dK and dV.  Both have the same shape.  With A1, A2 the 128 rows that stay
// (Q, dO; K, V) and N1, N2 the 64 rows that stream by (K, V; Q, dO):
//   S = A1 N1^T, dP = A2 N2^T     into tensor memory,
//   P and dS                      bf16, over them in tensor memory,
//   accA += dS N1, accB += P N1 (first pass) or P N2 (second pass),
// so neither P nor dS goes through shared memory.
//
// Delta is formed from unrounded terms and in the same walk as dQ.  With any
// number c per row, dS = P (dP - c) + P (c - Delta), so
//   dQ = scale (sum_j P (dP - c) K + f sum_j P K),    f = c - Delta,
//   Delta = c + sum_j P (dP - c),
// as sum_j P = 1 (but for the rounding of lse, which only scales f).  c is dO . O
// with O as the forward stored it, rounded to bf16 on top, which is near Delta in
// every row, so that f, and with it the rounding of P, is small.  (Delta from the
// stored O would carry O's rounding to bf16, which the keys' common part lifts
// above the gradient where many keys share a row.)
// The sum over j of dS is zero, so what the keys have in common leaves dQ, but
// roundings do not add up to zero: f is the sum of the rounded P (dP - c), negated,
// so that the weights of K do.  dQ is off by 2.3e-3 of its norm then, as dK is, and
// by 2.8e-3 where keys and values lie around 16 (2.8e-2 with f = c - Delta).  dS as
// two bf16 and three products a step: 1.7e-3, but 360 us for both passes at 256x256
// pixels, 346 so.
// A query that sees one key alone has dS = 0: P is 1 whatever the score.
//
// S and dP have kStages stages in tensor memory, each with a group of four
// warps, one thread per row; the tensor cores fill one while the exponentials
// of the others are computed.  Warps:
//   the groups' first;
//   four for the epilogue, so that the groups go on with the next item;
//   load    TMA loads of A (two buffers) and N (a ring);
//   mma     issues S and dP; prod the products.  One warp for both would leave
//           the tensor cores idle between its waits;
//   dot     (four or eight) first pass: c;
//   aux     first pass: with lengths or a mask, the bits of the keys seen and
//           zeros over the K rows that are not (their dS is zero, and zero
//           times NaN is NaN); second pass: lse and Delta of the queries that
//           stream by.
// The second pass cuts all its (key tile, query tile) pairs into equal runs,
// one per SM; a key tile that several SMs share is summed by a last kernel, in
// a fixed order.  The first pass cuts the keys where there are few rows.
// 32768 queries x 16 heads x 256 keys, D = 64: 106 us and 82 us, the tensor
// cores busy for 33% and 51%, the special-function units for 35% and 45%.  With
// row work, MMAs and loads left out 63% and 47% of the cycles remained (before O
// was read): the chain of waits (scores, row work, products, scores) is the
// largest part.
// Every wait is bounded; a time-out is reported as LLSA_DEV_TIMEOUT.

#include <math.h>

#include <type_traits>

#include "cross.cuh"
#include "cross_tc.cuh"

namespace llsa {

namespace {

template <int D>
struct Sizes {
  // tensor memory has 512 columns: accA and accB take 2 D, a stage 128
  static constexpr int kStages = (D == 64) ? 3 : 2;
  static constexpr int kEpi = kStages * 4;  // first epilogue warp
  static constexpr int kLoad = kEpi + 4, kMma = kLoad + 1, kProd = kMma + 1, kAux = kProd + 1;
  // Each aux warp has every kAuxWarps-th tile.  kAuxWarps divides kSlots, so a
  // warp sees every round of its slots: a barrier is not waited for before the
  // round before has been seen, which its parity would not tell apart.
  static constexpr int kAuxWarps = 3;
  // First pass: sets of four warps for c, which take turns.  Two where registers
  // allow: D = 128 against 80 keys 196 us, 208 with one.
  static constexpr int kDot = kAux + kAuxWarps;
  static constexpr int kDotSets = (D == 64) ? 1 : 2;
  static constexpr int kA = 128 * D * 2;   // a tile of A1 or A2
  static constexpr int kN = 64 * D * 2;    // a tile of N1 or N2
  static constexpr int kSlots = (D == 64) ? 6 : 3;
  static_assert(kSlots % kAuxWarps == 0, "a slot belongs to one aux warp");
  static constexpr uint32_t kColAcc = 128 * kStages;  // S | dP of each stage, accA | accB
};

template <typename C>
struct Shared {
  uint64_t a_full[C::kBufs], a_empty[C::kBufs], n_full[C::kSlots], n_empty[C::kSlots], n_aux[C::kSlots];
  uint64_t s_full[C::kStages], p_full[C::kStages], acc_full, acc_free, staged, done;
  uint64_t c_full[2], c_read[2], x_full[C::kSums], x_read[C::kSums];
  uint32_t tmem_base;
  uint32_t bits[C::kSlots][2];  // first pass: keys seen, by slot
  typename C::Side side;
};

// First pass: of the rows of an item (the sums of two of them where there is room).
template <int kSums, int kStages>
struct RowSums {
  static constexpr int kHeld = kSums;
  bf16 c[2][128];
  float2 sums[kSums][kStages][128];  // each group's sum P (dP - c), and of the rounded terms
};

// Second pass: one more step of 16 along the heads' dimension adds -lse /
// scale to S and -Delta to dP.  Its left side is all ones, its right side a
// query's number in three bf16 terms and 13 zeros; both without a swizzle, 32
// bytes a row.  (Read from shared memory by every thread, the two numbers of
// each query would cost more cycles than the exponentials.)
template <int kSlots>
struct ColumnTerms {
  static constexpr int kHeld = 1;
  alignas(128) unsigned char ones[4096];
  unsigned char terms[kSlots][2][2048];
};

template <int D, bool kDq>
struct Cfg : Sizes<D> {
  using Z = Sizes<D>;
  static constexpr int kThreads = (Z::kDot + (kDq ? 4 * Z::kDotSets : 0)) * 32;
  // buffers of A1, A2: the second pass has few items
  static constexpr int kBufs = (D == 64 || kDq) ? 2 : 1;
  static constexpr int kOffN = kBufs * 2 * Z::kA;
  static constexpr int kEnd = kOffN + Z::kSlots * 2 * Z::kN;
  using Side = std::conditional_t<kDq, RowSums<(D == 64) ? 2 : 1, Z::kStages>, ColumnTerms<Z::kSlots>>;
  static constexpr int kSums = Side::kHeld;
};

// The items of a CTA, in order.  First pass: 128 query rows against one range
// of the keys, every grid-th item, so that batch entries of unlike lengths are
// shared out.  Second pass: 128 keys (a key tile) against one range of the
// queries.  There the CTA's run is of pairs of a key tile and a tile of 64
// queries, the queries innermost, or of key tiles (nz == 1).
template <bool kDq>
struct BwdItems {
  const CrossParams& p;
  int i, end, nt, nq;          // kDq: items; else key tiles; nt: row tiles per head; nq: query tiles of a head
  int64_t beg, fin;            // second pass: the CTA's pairs
  int step_runs, step_tiles;   // first pass: grid in row tiles
  int run, bk, b, split, tile, r0, len;
  int n0, n;                   // first tile of 64 streamed rows, how many
  bool started;

  __device__ __forceinline__ BwdItems(const CrossParams& p_) : p(p_), b(-1), started(false) {
    nq = (p.N + 63) / 64;
    nt = ((kDq ? p.N : p.S) + 127) / 128;
    if (kDq) {
      i = blockIdx.x;
      end = p.items;
      step_runs = gridDim.x / nt;
      step_tiles = gridDim.x - step_runs * nt;
    } else {
      beg = p.runs.begin(blockIdx.x);
      fin = p.runs.begin(blockIdx.x + 1);
      i = (int)(p.nz > 1 ? beg / nq : beg);
      end = (int)(p.nz > 1 ? (fin + nq - 1) / nq : fin);
    }
    run = i / nt;
    tile = i - run * nt;
    if (i < end) range();
  }
  // what the head and the range of the keys settle
  __device__ __forceinline__ void range() {
    bk = kDq && p.nks > 1 ? run / p.nks : run;
    split = run - bk * (kDq ? p.nks : 1);
    const int nb = bk / p.H;
    if (nb != b) {
      b = nb;
      len = cross_len(p, b);
    }
    if (kDq) {
      n0 = 0;
      n = (len + 63) / 64;
      if (p.nks > 1) {  // the first n % nks ranges are longer by one
        const int each = n / p.nks, more = n - each * p.nks;
        n0 = each * split + min(split, more);
        n = each + (split < more);
      }
    }
  }
  __device__ __forceinline__ bool next() {
    if (started) {
      const int last = run;
      i += kDq ? gridDim.x : 1;
      run += kDq ? step_runs : 0;
      tile += kDq ? step_tiles : 1;
      if (tile >= nt) {
        tile -= nt;
        ++run;
      }
      if (i < end && run != last) range();
    }
    started = true;
    if (i >= end) return false;
    r0 = tile * 128;
    if (!kDq) {
      n0 = 0;
      n = nq;
      if (p.nz > 1) {
        const int64_t u = (int64_t)i * nq;
        if (beg > u) n0 = (int)(beg - u);
        if (fin < u + nq) n = (int)(fin - u);
        n -= n0;
      }
      if (r0 >= len) n = 0;  // no key of the tile is seen
    }
    return true;
  }
  // first pass: the query row that row r of the item after this one is (of the
  // first item, before the first next()); any row where there is none
  __device__ __forceinline__ size_t peek(int r) const {
    int ti = tile, ru = run;
    if (started) {
      ti += step_tiles;
      ru += step_runs;
      if (ti >= nt) {
        ti -= nt;
        ++ru;
      }
      if (i + (int)gridDim.x >= end) return 0;
    }
    const int row = ti * 128 + r;
    return (size_t)(p.nks > 1 ? ru / p.nks : ru) * p.N + (row < p.N ? row : 0);
  }
  // 16-row steps of the item's tile j
  __device__ __forceinline__ int steps(int j) const {
    if (!kDq) return 4;
    const int m = len - (n0 + j) * 64;
    return m >= 64 ? 4 : (m + 15) >> 4;
  }
};

using bf16x2 = __nv_bfloat162;
__device__ __forceinline__ bf16x2 as_bf16x2(uint32_t x) { return *reinterpret_cast<bf16x2*>(&x); }

// -lse in units of log2; without keys (lse = -inf) every probability is zero.
__device__ __forceinline__ float neg_lse2(float lse) { return lse == -INFINITY ? lse : -lse * kLog2e; }

// x as the sum of three bf16 (infinities and NaN as they are), and a zero.
__device__ __forceinline__ uint2 three_terms(float x) {
  const float h = bf16x2_lo(pack_bf16(x, 0.f));
  const float m0 = fabsf(h) < INFINITY ? x - h : 0.f;
  const float m = bf16x2_lo(pack_bf16(m0, 0.f));
  return make_uint2(pack_bf16(h, m), pack_bf16(m0 - m, 0.f));
}

template <int D, bool kDq>
__global__ void __launch_bounds__(Cfg<D, kDq>::kThreads, 1)
cross_bwd_tc_kernel(const __grid_constant__ CUtensorMap ta1, const __grid_constant__ CUtensorMap ta2,
                    const __grid_constant__ CUtensorMap tn1, const __grid_constant__ CUtensorMap tn2,
                    const __grid_constant__ CUtensorMap tdq, CrossParams p) {
  using C = Cfg<D, kDq>;
  constexpr int H = D / 64;  // 64-column halves of a tile
  constexpr int NS = C::kSlots, NG = C::kStages;
  extern __shared__ __align__(1024) unsigned char sm[];
  Shared<C>& S = *reinterpret_cast<Shared<C>*>(sm + C::kEnd);
  const uint32_t base = smem_u32(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const bool clean = kDq && (p.mask != nullptr || p.kv_len != nullptr);
  bool ok = true;

  if (warp == C::kMma) {
    tmem_alloc(smem_u32(&S.tmem_base), 512);
    tmem_relinquish();
  } else if (tid == 0) {
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(smem_u32(&S.a_full[i]), 1);
      mbar_init(smem_u32(&S.a_empty[i]), 1);
    }
    for (int i = 0; i < NG; ++i) {
      mbar_init(smem_u32(&S.s_full[i]), 1);
      mbar_init(smem_u32(&S.p_full[i]), 128);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&S.n_full[i]), 1);
      mbar_init(smem_u32(&S.n_empty[i]), 1);
      mbar_init(smem_u32(&S.n_aux[i]), 1);
    }
    mbar_init(smem_u32(&S.acc_full), 1);
    mbar_init(smem_u32(&S.acc_free), 128);
    mbar_init(smem_u32(&S.staged), 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&S.c_full[i]), 128);
      mbar_init(smem_u32(&S.c_read[i]), (NG + 1) * 128);
    }
    for (int i = 0; i < C::kSums; ++i) {
      mbar_init(smem_u32(&S.x_full[i]), NG * 128);
      mbar_init(smem_u32(&S.x_read[i]), 128);
    }
    mbar_init(smem_u32(&S.done), 2);
    fence_mbar_init();
  }
  if constexpr (!kDq) {
    uint32_t* x = reinterpret_cast<uint32_t*>(&S.side);
    for (int i = tid; i < (int)sizeof(S.side) / 4; i += C::kThreads) x[i] = i < 1024 ? 0x3f803f80u : 0u;
    fence_proxy_async_smem();  // generic writes -> MMA operand reads
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = uniform(S.tmem_base);
  auto abuf = [&](uint32_t i) { return base + i * 2 * C::kA; };
  auto nslot = [&](uint32_t i) { return base + C::kOffN + i * 2 * C::kN; };
  const uint32_t a_full = smem_u32(S.a_full), a_empty = smem_u32(S.a_empty), n_full = smem_u32(S.n_full),
                 n_empty = smem_u32(S.n_empty), n_aux = smem_u32(S.n_aux), s_full = smem_u32(S.s_full),
                 p_full = smem_u32(S.p_full), acc_full = smem_u32(&S.acc_full), acc_free = smem_u32(&S.acc_free),
                 c_full = smem_u32(S.c_full), c_read = smem_u32(S.c_read), x_full = smem_u32(S.x_full), x_read = smem_u32(S.x_read);
  // Waits of whole warps.  A look at a barrier takes 150 cycles even where its
  // phase is over: where it can, a warp looks before it does something else
  // (or at two barriers at once) and takes the answer afterwards.
  auto wait = [&](uint32_t bar, uint32_t parity) { return ok = __all_sync(0xffffffffu, mbar_wait(bar, parity)); };
  auto look = [&](uint32_t bar, uint32_t parity) { return mbar_look(bar, parity); };
  auto finish = [&](bool seen, uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, seen) || wait(bar, parity);
  };
  BwdItems<kDq> it(p);

  if (warp == C::kLoad) {
    if (lane == 0) {
      Ring<C::kBufs> ra;
      Ring<NS> rn;
      // a buffer's first round waits for the phase before the first, which is over
      for (; ok && it.next();) {
        if (it.n == 0) continue;
        ok = mbar_wait(ra.at(a_empty), ra.parity ^ 1u);
        if (!ok) break;
        mbar_arrive_expect_tx(ra.at(a_full), 2 * C::kA);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          tma_load_3d(abuf(ra.i) + h * 16384, &ta1, 64 * h, it.r0, it.bk, ra.at(a_full));
          tma_load_3d(abuf(ra.i) + C::kA + h * 16384, &ta2, 64 * h, it.r0, it.bk, ra.at(a_full));
        }
        ra.next();
        for (int j = 0; j < it.n; ++j) {
          ok = mbar_wait(rn.at(n_empty), rn.parity ^ 1u);
          if (!ok) break;
          mbar_arrive_expect_tx(rn.at(n_full), 2 * C::kN);
#pragma unroll
          for (int h = 0; h < H; ++h) {
            tma_load_3d(nslot(rn.i) + h * 8192, &tn1, 64 * h, (it.n0 + j) * 64, it.bk, rn.at(n_full));
            tma_load_3d(nslot(rn.i) + C::kN + h * 8192, &tn2, 64 * h, (it.n0 + j) * 64, it.bk, rn.at(n_full));
          }
          rn.next();
        }
      }
      // no copy may still be landing when the CTA exits: of every place, the
      // last round that was begun
      for (int i = 0; i < C::kBufs; ++i, ra.next())
        if (!mbar_wait(ra.at(a_full), ra.parity ^ 1u)) ok = false;
      for (int i = 0; i < NS; ++i, rn.next())
        if (!mbar_wait(rn.at(n_full), rn.parity ^ 1u)) ok = false;
    }
  } else if (warp == C::kMma) {
    // S and dP; the whole warp walks, one lane issues
    const uint64_t kmaj = smem_desc_sw128(0, 16, 1024);
    const uint32_t lead = elect_lane();
    Ring<C::kBufs> ra;
    Ring<NS> rn, pn;  // tiles; and the tiles NG before, whose stages these take
    Ring<NG> rs;
    int fresh = NG;   // stages not used yet
    // of the next tile: whether it has been loaded, and the products that read
    // its stage are done
    bool n_seen = false, e_seen = false;
    for (; ok && it.next();) {
      const int n = uniform(it.n);
      if (n == 0) continue;
      if (!wait(ra.at(a_full), ra.parity)) break;
      const uint64_t a1 = desc_at(kmaj, abuf(ra.i));
      for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, n_seen)) {
          if (!wait(rn.at(n_full), rn.parity)) break;
          if (!kDq && !wait(rn.at(n_aux), rn.parity)) break;
        }
        if (fresh == 0) {
          if (!finish(e_seen, pn.at(n_empty), pn.parity)) break;
          pn.next();
        } else {
          --fresh;
        }
        const uint32_t slot = rn.i;
        rn.next();
        n_seen = look(rn.at(n_full), rn.parity) && (kDq || look(rn.at(n_aux), rn.parity));
        e_seen = look(pn.at(n_empty), pn.parity);
        tc_fence_after();
        const uint32_t ts = tbase + rs.i * 128;
        const uint32_t idesc_s = idesc_bf16_f32(128, 16 * (kDq ? uniform(it.steps(j)) : 4), 0, 0);
        const uint64_t n1 = desc_at(kmaj, nslot(slot));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int w = 0; w < 2; ++w)
            tc_mma_f16_by(lead, ts + 64 * w, desc_at(a1, w * C::kA + (ks >> 2) * 16384 + (ks & 3) * 32),
                          desc_at(n1, w * C::kN + (ks >> 2) * 8192 + (ks & 3) * 32), idesc_s, ks > 0);
        if constexpr (!kDq) {
          const uint64_t x = smem_desc_plain(smem_u32(S.side.ones), 128, 256);
#pragma unroll
          for (int w = 0; w < 2; ++w)
            tc_mma_f16_by(lead, ts + 64 * w, x, desc_at(x, 4096 + slot * 4096 + w * 2048), idesc_s, 1);
        }
        tc_commit_by(lead, rs.at(s_full));
        rs.next();
      }
      if (!ok) break;
      if (!kDq) tc_commit_by(lead, ra.at(a_empty));
      ra.next();
    }
    // every MMA of this CTA has completed before tensor memory is freed
    tc_commit_by(lead, smem_u32(&S.done));
    if (!mbar_wait(smem_u32(&S.done), 0)) ok = false;
  } else if (warp == C::kProd) {
    // accA (+)= dS N1, accB (+)= P N1 or N2
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, D, 1, 0);
    constexpr uint32_t kSecond = kDq ? 0 : C::kN;
    const uint64_t nmaj = smem_desc_sw128(0, 8192, 1024);
    const uint32_t lead = elect_lane();
    Ring<NS> rn;
    Ring<NG> rs;
    uint32_t acc_par = 1;  // of acc_free: the phase before the first is over
    for (; ok && it.next();) {
      const int n = uniform(it.n);
      if (n == 0) continue;
      for (int j = 0; j < n; ++j) {
        if (kDq && clean && !wait(rn.at(n_aux), rn.parity)) break;
        if (j == 0 && !wait(acc_free, acc_par)) break;
        if (!wait(rs.at(p_full), rs.parity)) break;
        tc_fence_after();
        const uint32_t ts = tbase + rs.i * 128;
        const int nt = kDq ? uniform(it.steps(j)) : 4;
        const uint64_t n1 = desc_at(nmaj, nslot(rn.i)), n2 = desc_at(n1, kSecond);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= nt) break;
          const uint32_t add = j > 0 || k > 0;
          tc_mma_f16_ts_by(lead, tbase + C::kColAcc + D, ts + k * 8, desc_at(n2, k * 2048), idesc_acc, add);
          tc_mma_f16_ts_by(lead, tbase + C::kColAcc, ts + 64 + k * 8, desc_at(n1, k * 2048), idesc_acc, add);
        }
        tc_commit_by(lead, rn.at(n_empty));
        rn.next();
        rs.next();
      }
      if (!ok) break;
      acc_par ^= 1u;
      tc_commit_by(lead, acc_full);
    }
    tc_commit_by(lead, smem_u32(&S.done));
    if (!mbar_wait(smem_u32(&S.done), 0)) ok = false;
  } else if (kDq && warp >= C::kDot) {
    // c of an item's rows, 32 a warp: L lanes a row, 16 bytes of it each, and L
    // such steps, whose sums over the lanes then end in one lane each.  A lane
    // adds its eight products in bf16: any c is right, and this one as near.  dO
    // is read again rather than taken from its tile, so that c does not wait for
    // that (336 us against 340 at 256x256 pixels, D = 128 182 against 188).  Reading
    // O is what the pass takes longer for where it is bound by memory.
    if constexpr (kDq) {
      constexpr int L = D / 8, kRows = 32 / L;
      const int first = 32 * ((warp - C::kDot) & 3) + lane / L, chunk = lane % L;
      Ring<2> rc;
      int turn = (warp - C::kDot) >> 2;  // items of the other set before this one's next
      rc.next(turn);
      for (; ok && it.next();) {
        if (it.n == 0) continue;
        if (C::kDotSets > 1 && turn-- > 0) continue;
        turn = C::kDotSets - 1;
        const size_t at = ((size_t)it.bk * p.N + it.r0 + first) * L + chunk;
        const uint4 *o = static_cast<const uint4*>(p.o_in) + at, *g = static_cast<const uint4*>(p.dout) + at;
        float s[L];
#pragma unroll
        for (int i0 = 0; i0 < L; i0 += 4) {  // eight loads in flight
          uint4 x[4], y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = y[i] = make_uint4(0, 0, 0, 0);
            if (it.r0 + first + (i0 + i) * kRows < p.N) {
              x[i] = __ldg(o + (i0 + i) * 32);
              y[i] = __ldg(g + (i0 + i) * 32);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, b[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
            bf16x2 t = __hmul2(as_bf16x2(a[0]), as_bf16x2(b[0]));
#pragma unroll
            for (int e = 1; e < 4; ++e) t = __hfma2(as_bf16x2(a[e]), as_bf16x2(b[e]), t);
            s[i0 + i] = __low2float(t) + __high2float(t);
          }
        }
#pragma unroll
        for (int m = L / 2; m > 0; m /= 2) {
          const bool up = (chunk & m) != 0;
#pragma unroll
          for (int i = 0; i < m; ++i) {
            const float keep = up ? s[i + m] : s[i], send = up ? s[i] : s[i + m];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
          }
        }
        if (!wait(rc.at(c_read), rc.parity ^ 1u)) break;
        S.side.c[rc.i][first + chunk * kRows] = __float2bfloat16_rn(fabsf(s[0]) < 3e38f ? s[0] : 0.f);
        mbar_arrive(rc.at(c_full));
        rc.next(C::kDotSets);
      }
    }
  } else if (warp >= C::kAux) {
    constexpr int NA = C::kAuxWarps;
    Ring<NS> rn;
    rn.next(warp - C::kAux);
    int j = warp - C::kAux;  // this warp's next tile of the item
    if constexpr (kDq) {
      for (; ok && clean && it.next(); j -= it.n) {
        for (; j < it.n; j += NA, rn.next(NA)) {
          uint32_t word[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int key = (it.n0 + j) * 64 + 32 * c + lane;
            const bool on = key < it.len && (p.mask == nullptr || p.mask[(size_t)it.b * p.S + key] != 0);
            word[c] = __ballot_sync(0xffffffffu, on);
          }
          if (!wait(rn.at(n_full), rn.parity)) break;
          const int rows = 16 * it.steps(j);
          unsigned char* k = sm + (nslot(rn.i) - base);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (lane == 0) S.bits[rn.i][c] = word[c];
            for (uint32_t off = ~word[c]; off != 0u; off &= off - 1) {  // one row at a time, 16 bytes a lane
              const int r = 32 * c + __ffs(off) - 1;
              if (r >= rows) break;
              if (lane < D / 8)
                *reinterpret_cast<uint4*>(k + (lane >> 3) * 8192 + sw128(r, lane & 7)) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();  // generic writes -> MMA operand reads
          __syncwarp();
          if (lane == 0) mbar_arrive(rn.at(n_aux));
        }
        if (!ok) break;
      }
    } else {
      const float over = -1.f / p.scale;
      for (; ok && it.next(); j -= it.n) {
        const size_t g0 = (size_t)it.bk * p.N;
        float l[2], de[2];
        auto load = [&]() {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = (it.n0 + j) * 64 + 32 * i + lane;
            const bool on = j < it.n && row < p.N;  // rows past the end: probability zero
            l[i] = on ? p.lse_in[g0 + row] : -INFINITY;
            de[i] = on ? p.delta[g0 + row] : 0.f;
          }
        };
        load();
        while (j < it.n) {
          uint2 x[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[0][i] = three_terms(l[i] == -INFINITY ? -INFINITY : l[i] * over);  // no keys: probability zero
            x[1][i] = three_terms(-de[i]);
          }
          if (!wait(rn.at(n_empty), rn.parity ^ 1u)) break;
          j += NA;
          load();
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = 32 * i + lane;
              *reinterpret_cast<uint2*>(S.side.terms[rn.i][w] + (r >> 3) * 256 + (r & 7) * 16) = x[w][i];
            }
          fence_proxy_async_smem();  // generic writes -> MMA operand reads
          __syncwarp();
          if (lane == 0) mbar_arrive(rn.at(n_aux));
          rn.next(NA);
        }
        if (!ok) break;
      }
    }
  } else if (warp >= C::kEpi) {
    // ------------------------------------------------------------- epilogue
    const int q4 = warp & 3, r = q4 * 32 + lane;  // row of A = TMEM lane
    const uint32_t tacc = tbase + ((uint32_t)(q4 * 32) << 16) + C::kColAcc;
    int last_b = -1;
    bool one = false;
    Ring<C::kBufs> ra;
    Ring<C::kSums> rx;
    Ring<2> rc;
    uint32_t par = 0;  // of acc_full and staged: the item's
    for (; ok && it.next(); ) {
      const int row = it.r0 + r;
      const bool new_b = it.b != last_b;
      last_b = it.b;
      if constexpr (kDq) {
        const bool valid = row < p.N;
        const size_t grow = (size_t)it.bk * p.N + row;
        const size_t rows = (size_t)p.B * p.H * p.N;
        if (new_b) {
          one = sees_one(p, it.b, it.len);
          if (r == 0) p.alone[it.b] = one;
        }
        if (it.n == 0) {  // no keys (in this range)
          if (valid) {
            if (p.nks > 1) {
              p.part_s[it.split * rows + grow] = make_float4(0.f, 0.f, 0.f, 0.f);
            } else {
              for (int c = 0; c < D / 8; ++c)
                reinterpret_cast<uint4*>(static_cast<bf16*>(p.dq) + grow * D)[c] = make_uint4(0, 0, 0, 0);
              p.delta[grow] = 0.f;
            }
          }
          continue;
        }
        if (!wait(rc.at(c_full), rc.parity)) break;
        const float c0 = __bfloat162float(S.side.c[rc.i][r]);
        mbar_arrive(rc.at(c_read));
        rc.next();
        if (!wait(rx.at(x_full), rx.parity)) break;
        float sd = 0.f, sr = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float2 x = S.side.sums[rx.i][g][r];
          sd += x.x;
          sr += x.y;
        }
        mbar_arrive(rx.at(x_read));
        rx.next();
        const float f = -sr;
        if (valid) {
          if (p.nks > 1) p.part_s[it.split * rows + grow] = make_float4(c0, sd, sr, 1.f);
          else p.delta[grow] = c0 + sd;
        }
        if (!wait(acc_full, par)) break;
        tc_fence_after();
        unsigned char* stage = sm + (abuf(ra.i) - base);  // A1, which no MMA reads any more
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float x[16], y[16];
          tmem_ld16(tacc + c, x);
          tmem_ld16(tacc + D + c, y);
          tmem_wait_ld();
          if (p.nks > 1) {
            const size_t at = (it.split * rows + grow) * D + c;
            if (valid) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                *reinterpret_cast<float4*>(p.part_dq + at + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                *reinterpret_cast<float4*>(p.part_dqb + at + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = one ? 0.f : fmaf(f, y[i], x[i]) * p.scale;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int cc = c / 8 + i;
              *reinterpret_cast<uint4*>(stage + (cc >> 3) * 16384 + sw128(r, cc & 7)) =
                  make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                             pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
            }
          }
        }
        tc_fence_before();
        mbar_arrive(acc_free);
        fence_proxy_async_smem();  // generic writes -> TMA store
        mbar_arrive(smem_u32(&S.staged));
        if (q4 == 0) {
          if (!wait(smem_u32(&S.staged), par)) break;
          if (lane == 0) {
            if (p.nks == 1) {
#pragma unroll
              for (int h = 0; h < H; ++h) tma_store_3d(&tdq, 64 * h, it.r0, it.bk, abuf(ra.i) + h * 16384);
              bulk_commit_group();
              bulk_wait_read_all();
            }
            mbar_arrive(ra.at(a_empty));
          }
        }
        ra.next();
        par ^= 1u;
      } else {
        // keys that are not seen: whatever their rows hold, it stays in them
        const bool seen = row < it.len && (p.mask == nullptr || p.mask[(size_t)it.b * p.S + row] != 0);
        const size_t at = ((size_t)it.bk * p.S + row) * D;
        if (it.n == 0) {
          if (p.nz == 1 && row < p.S)
            for (int c = 0; c < D / 8; ++c) {
              reinterpret_cast<uint4*>(static_cast<bf16*>(p.dk) + at)[c] = make_uint4(0, 0, 0, 0);
              reinterpret_cast<uint4*>(static_cast<bf16*>(p.dv) + at)[c] = make_uint4(0, 0, 0, 0);
            }
          continue;
        }
        const float fk = p.alone[it.b] != 0 ? 0.f : p.scale;
        size_t part_row = 0;  // of the parts
        if (p.nz > 1) {
          const int slot = (int)blockIdx.x - p.runs.cta_of((int64_t)it.i * it.nq);
          part_row = ((size_t)it.i * p.nz + slot) * 128 + r;
        }
        if (!wait(acc_full, par)) break;
        par ^= 1u;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 2 * D; c += 32) {  // accA is dK, accB dV
          float x[32];
          tmem_ld32(tacc + c, x);
          tmem_wait_ld();
          if (row >= p.S) continue;
          const bool is_k = c < D;
          if (p.nz > 1) {
            float4* to = reinterpret_cast<float4*>((is_k ? p.part_dk : p.part_dv) +
                                                   part_row * D + c % D);
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          } else {
            uint4* to = reinterpret_cast<uint4*>(static_cast<bf16*>(is_k ? p.dk : p.dv) + at + c % D);
            const float f = is_k ? fk : 1.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = seen && f != 0.f ? x[i] * f : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              to[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                                 pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
          }
        }
        tc_fence_before();
        mbar_arrive(acc_free);
      }
    }
    if (kDq && r == 0) bulk_wait_all();
  } else {
    // ----------------------------------------------------------- P and dS
    const int g = warp >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t ts = tbase + ((uint32_t)(q4 * 32) << 16) + (uint32_t)g * 128;
    const float sc2 = p.scale * kLog2e;
    const uint64_t sc2x2 = f2_make(sc2, sc2);
    Ring<NS> rn;          // of this group's tiles
    rn.next(g);
    uint32_t turn = 0;    // parity of its stage
    int j = g;            // its next tile of the item
    Ring<C::kSums> rx;
    Ring<2> rc;
    float lse_next = 0.f;
    if (kDq) lse_next = p.lse_in[it.peek(r)];
    for (; ok && it.next();) {
      if constexpr (kDq) {
        const float lse = lse_next;
        lse_next = p.lse_in[it.peek(r)];
        if (it.n == 0) continue;
        const float nl = it.r0 + r < p.N ? neg_lse2(lse) : -INFINITY;  // rows past the end: probability zero
        const uint64_t nl2 = f2_make(nl, nl);
        bool have_c = false;
        uint64_t c2 = 0, ds = 0, rs = 0;
        const bool c_seen = look(rc.at(c_full), rc.parity);
        auto take_c = [&]() {
          have_c = true;
          if (!finish(c_seen, rc.at(c_full), rc.parity)) return false;
          const float c0 = __bfloat162float(S.side.c[rc.i][r]);
          c2 = f2_make(c0, c0);
          mbar_arrive(rc.at(c_read));
          rc.next();
          return true;
        };
        for (; j < it.n; j += NG, rn.next(NG), turn ^= 1u) {
          // S first: it tells that the round before of n_aux is over, which this
          // group may not have seen
          if (!wait(s_full + 8 * g, turn)) break;
          const bool x_seen = !clean || look(rn.at(n_aux), rn.parity);
          if (!have_c && !take_c()) break;
          if (!finish(x_seen, rn.at(n_aux), rn.parity)) break;
          tc_fence_after();
          const int nt = it.steps(j), left = it.len - (it.n0 + j) * 64;
          if (clean || left < 64) {
#pragma unroll 1
            for (int c = 0; c < nt; ++c) {
              const uint32_t bits = clean ? (S.bits[rn.i][c >> 1] >> (16 * (c & 1))) & 0xffffu
                                          : (left - 16 * c >= 16 ? 0xffffu : (1u << (left - 16 * c)) - 1u);
              if (bits == 0xffffu) continue;
              hide16(ts + 16 * c, bits, -INFINITY);
              hide16(ts + 64 + 16 * c, bits, 0.f);
            }
          }
#pragma unroll 1
          for (int c = 0; c < nt; ++c) {  // 16 keys
            float x[16], d[16];
            tmem_ld16(ts + 16 * c, x);
            tmem_ld16(ts + 64 + 16 * c, d);
            tmem_wait_ld();
            uint32_t pk[8], dk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 e = f2_split(f2_fma(f2_make(x[2 * i], x[2 * i + 1]), sc2x2, nl2));
              const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
              const uint64_t pp = f2_make(p0, p1);
              const uint64_t t = f2_mul(pp, f2_sub(f2_make(d[2 * i], d[2 * i + 1]), c2));
              ds = f2_add(ds, t);
              const float2 tt = f2_split(t);
              pk[i] = pack_bf16(p0, p1);
              dk[i] = pack_bf16(tt.x, tt.y);
              rs = f2_add(rs, f2_make(bf16x2_lo(dk[i]), bf16x2_hi(dk[i])));
            }
            tmem_st8u(ts + 8 * c, pk);
            tmem_st8u(ts + 64 + 8 * c, dk);
          }
          if (!ok) break;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_full + 8 * g);
        }
        if (!ok || (!have_c && !take_c())) break;
        j -= it.n;
        if (!wait(rx.at(x_read), rx.parity ^ 1u)) break;
        const float2 d2 = f2_split(ds), r2 = f2_split(rs);
        S.side.sums[rx.i][g][r] = make_float2(d2.x + d2.y, r2.x + r2.y);
        mbar_arrive(rx.at(x_full));
        rx.next();
      } else {
        for (; j < it.n; j += NG, turn ^= 1u) {
          if (!wait(s_full + 8 * g, turn)) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {  // 16 queries
            float x[16], d[16];
            tmem_ld16(ts + 16 * c, x);
            tmem_ld16(ts + 64 + 16 * c, d);
            tmem_wait_ld();
            uint32_t pk[8], dk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 e = f2_split(f2_mul(f2_make(x[2 * i], x[2 * i + 1]), sc2x2));
              const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
              const float2 q = f2_split(f2_mul(f2_make(p0, p1), f2_make(d[2 * i], d[2 * i + 1])));
              pk[i] = pack_bf16(p0, p1);
              dk[i] = pack_bf16(q.x, q.y);
            }
            tmem_st8u(ts + 8 * c, pk);
            tmem_st8u(ts + 64 + 8 * c, dk);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_full + 8 * g);
        }
        j -= it.n;
      }
    }
  }

  if (!ok) report_status(p.status, LLSA_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMma) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// The first pass's splits of a row joined: a warp per row.
template <int D>
__global__ void __launch_bounds__(256)
cross_dq_join(CrossParams p) {
  constexpr int C = D / 32;
  const size_t rows = (size_t)p.B * p.H * p.N;
  const size_t row = (size_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float c0 = 0.f, sd = 0.f, f = 0.f;
  for (int z = 0; z < p.nks; ++z) {
    const float4 s = p.part_s[z * rows + row];
    if (s.w != 0.f) c0 = s.x;  // the row's, in every split that has keys
    sd += s.y;
    f -= s.z;
  }
  float acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  for (int z = 0; z < p.nks; ++z) {
    if (p.part_s[z * rows + row].w == 0.f) continue;  // a split without keys: its parts are not written
    const size_t at = (z * rows + row) * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] += fmaf(f, p.part_dqb[at + c], p.part_dq[at + c]);
  }
  const bool one = p.alone[row / ((size_t)p.H * p.N)] != 0;
#pragma unroll
  for (int c = 0; c < C; ++c)
    store_elem(static_cast<bf16*>(p.dq) + row * D + lane * C + c, one ? 0.f : acc[c] * p.scale);
  if (lane == 0) p.delta[row] = c0 + sd;
}

// The second pass's shares of a key tile summed: D / 4 threads per key and
// tensor (blockIdx.y: dV, dK).
template <int D>
__global__ void __launch_bounds__(256)
cross_dkv_join(CrossParams p) {
  constexpr int T = D / 4;
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t krow = at / T;
  const int c = (int)(at % T) * 4;
  if (krow >= (size_t)p.B * p.H * p.S) return;
  const int bk = (int)(krow / p.S), key = (int)(krow - (size_t)bk * p.S), b = bk / p.H;
  const bool is_k = blockIdx.y != 0;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (key < cross_len(p, b) && (p.mask == nullptr || p.mask[(size_t)b * p.S + key] != 0) &&
      !(is_k && p.alone[b] != 0)) {
    const int nq = (p.N + 63) / 64;
    const int64_t u = (int64_t)bk * ((p.S + 127) / 128) + key / 128;
    const int n = p.runs.cta_of(u * nq + nq - 1) - p.runs.cta_of(u * nq) + 1;
    const float* src = (is_k ? p.part_dk : p.part_dv) + ((size_t)u * p.nz * 128 + key % 128) * D + c;
    for (int z = 0; z < n; ++z) {
      const float4 x = *reinterpret_cast<const float4*>(src + (size_t)z * 128 * D);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    const float f = is_k ? p.scale : 1.f;
    s.x *= f;
    s.y *= f;
    s.z *= f;
    s.w *= f;
  }
  uint2* dst = reinterpret_cast<uint2*>(static_cast<bf16*>(is_k ? p.dk : p.dv) + krow * D + c);
  *dst = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

template <int D, bool kDq>
cudaError_t launch_pass(const CrossParams& p, const CUtensorMap* a, const CUtensorMap* n, const CUtensorMap& dq,
                        int grid, cudaStream_t s) {
  using C = Cfg<D, kDq>;
  constexpr size_t smem = C::kEnd + sizeof(Shared<C>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  cudaError_t e =
      cudaFuncSetAttribute(cross_bwd_tc_kernel<D, kDq>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cross_bwd_tc_kernel<D, kDq><<<grid, C::kThreads, smem, s>>>(a[0], a[1], n[0], n[1], dq, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_typed(CrossParams p, const CUtensorMap* q128, const CUtensorMap* kv64, const CUtensorMap* kv128,
                         const CUtensorMap* q64, cudaStream_t s) {
  const int64_t items = (int64_t)p.B * p.H * p.nks * cross_tiles(p.N, 128);
  int grid = (int)(items < kCrossSms ? items : kCrossSms);
  if (items > 0x7fffff00LL) return cudaErrorInvalidValue;  // and the grid on top
  p.items = (int)items;
  cudaError_t e = launch_pass<D, true>(p, q128, kv64, q128[2], grid, s);
  const size_t rows = (size_t)p.B * p.H * p.N;
  if (e == cudaSuccess && p.nks > 1) {
    cross_dq_join<D><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || p.S == 0) return e;
  const int64_t pairs = (int64_t)p.B * p.H * cross_tiles(p.S, 128) * (p.nz > 1 ? cross_tiles(p.N, 64) : 1);
  grid = (int)(pairs < kCrossSms ? pairs : kCrossSms);
  p.runs = cross_runs(pairs, grid);
  e = launch_pass<D, false>(p, kv128, q64, q128[2], grid, s);
  if (e == cudaSuccess && p.nz > 1) {
    const size_t threads = (size_t)p.B * p.H * p.S * (D / 4);
    cross_dkv_join<D><<<dim3((unsigned)((threads + 255) / 256), 2), 256, 0, s>>>(p);
    e = cudaGetLastError();
  }
  return e;
}

// Parts of a key tile: as many as its query tiles' pairs meet CTAs.  Whole key
// tiles are given out where there are many of them, at least four a CTA, or
// nothing to cut.
int parts_of_key_tile(int64_t BH, int N, int S) {
  const int64_t nq = cross_tiles(N, 64), units = BH * cross_tiles(S, 128), total = units * nq;
  if (total == 0 || nq == 1 || units >= 4 * kCrossSms || units % kCrossSms == 0) return 1;
  // a run has at least floor(total / grid) pairs, and an interval of nq pairs
  // meets at most ceil((nq - 1) / that) + 1 runs
  const int64_t grid = total < kCrossSms ? total : kCrossSms;
  return (int)(cross_tiles(nq - 1, (int)(total / grid > nq ? nq : total / grid)) + 1);
}

}  // namespace

CrossPlan cross_tc_bwd_plan(long long BH, int N, int S) {
  const int64_t units = BH * cross_tiles(N, 128), kt = cross_tiles(S, 64);
  int64_t nks = kCrossSms / units;
  if (nks > kt) nks = kt;
  return {nks < 1 ? 1 : (int)nks, parts_of_key_tile(BH, N, S)};
}

cudaError_t launch_cross_bwd_tc(const CrossParams& p, const CUtensorMap* q128, const CUtensorMap* kv64,
                                const CUtensorMap* kv128, const CUtensorMap* q64, cudaStream_t s) {
  return p.D == 64 ? launch_typed<64>(p, q128, kv64, kv128, q64, s) : launch_typed<128>(p, q128, kv64, kv128, q64, s);
}

}  // namespace llsa
