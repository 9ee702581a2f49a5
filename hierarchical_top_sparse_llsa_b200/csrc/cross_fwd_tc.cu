// Cross attention forward on the 5th-generation tensor cores (tcgen05), bf16,
// D = 64 or 128:
//   S = Q K^T,  P = e^(scale S - m),  O = P V / l,  lse = scale m + ln l
// with the running maximum m and sum l of the softmax, in one pass over the
// keys.
//
// The query heads of a key head are neighbours in memory, so their queries
// are one run of R rows against the same keys.  A work item is kNq tiles of
// 128 of these rows (the M of an MMA) against a range of key tiles; a
// persistent CTA per SM walks a contiguous range of items.  Warps:
//   four per query tile: its softmax, one thread per row;
//   load   TMA loads: Q tiles into a ring of slots for each mma warp, K and V
//          tiles into another.  Key tiles that fit in the ring are loaded
//          once and stay for all items of the same keys;
//   mma    (one for every query tile) issues S_w = Q_w K^T into tensor
//          memory, and O_w += P_w V with P_w read from tensor memory (over
//          S_w, which the softmax has read);
//   clean  with lengths or a mask: the bits of the keys seen in each tile,
//          and zeros over the V rows that are not seen (their probability is
//          zero, and zero times NaN is NaN);
//   store  TMA stores of the finished O tiles, staged over their Q.
// The query tiles take turns: the tensor cores work on some while the
// exponentials of the others are computed (one per score; 16 a clock and SM).
// 65536 queries x 16 heads x 256 keys of D = 64 take 136 to 139 us (42 us of
// memory, 60 of exponentials): the special-function units are busy for 50% of
// the time, the tensor cores for 24%, the rest is waits between the warps.
// At D = 64 four query tiles are in flight, each
// against 64 keys at a time; at D = 128 tensor memory holds two, and they take
// 128 keys, an N that the tensor cores run at full rate (two tiles of 128 keys at
// D = 64: 151 us against 127).  The next item's
// first S is issued before this item's epilogue.  Few rows: the keys are cut
// into ranges, each a work item of its own, whose fp32 parts are joined by
// another kernel.
// P is rounded to bf16 for the product (the exact running maximum is kept, so
// a row's largest probability is 1 and rounds exactly); m, l and O are fp32.
// Every wait is bounded; a time-out is reported as LLSA_DEV_TIMEOUT.

#include <math.h>

#include "cross.cuh"
#include "cross_tc.cuh"

namespace llsa {

namespace {

template <int D>
struct Cfg {
  static constexpr int kNq = (D == 64) ? 4 : 2;         // query tiles of an item
  static constexpr int kKeys = (D == 64) ? 64 : 128;    // keys of a tile
  static constexpr int kPer = 2;                        // query tiles of an mma warp
  static constexpr int kMmaWarps = kNq / kPer;
  static constexpr int kLoad = kNq * 4, kMma = kLoad + 1, kClean = kMma + kMmaWarps, kStore = kClean + 1;
  static constexpr int kThreads = (kStore + 1) * 32;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kKvTile = kKeys * D * 2;
  // Q slots: a ring of kQr for the tiles of each mma warp, which so waits for
  // every round of its slots, in order
  static constexpr int kQ = (D == 64) ? 8 : 3;
  static constexpr int kQr = kQ / kMmaWarps;
  static constexpr int kKv = (D == 64) ? 12 : 4;        // K and V slots
  static constexpr int kOffKv = kQ * kQTile;
  static constexpr int kEnd = kOffKv + kKv * kKvTile;
  static constexpr int kColO = 256;                     // S of each tile, O of each tile
};

template <typename C>
struct Shared {
  uint64_t q_full[C::kMmaWarps][C::kQr], q_empty[C::kMmaWarps][C::kQr];
  uint64_t kv_full[C::kKv], kv_empty[C::kKv], kv_clean[C::kKv];
  uint64_t s_full[C::kNq], p_full[C::kNq], o_full[C::kNq], o_staged[C::kNq], done;
  uint32_t bits[C::kKv][C::kKeys / 32];  // keys seen, by V slot
  uint32_t tmem_base;
};

// The items of a CTA, in order: kNq * 128 query rows of one key head against
// one range of its key tiles.  Every warp role walks them by itself; rows are
// innermost, so items of the same keys follow one another (a run).
template <typename C>
struct FwdItems {
  const CrossParams& p;
  int i, end, nt;
  int R;                       // query rows of a key head
  size_t rows;                 // and of all of them
  int bk, b, split, tile, r0, len;  // the item: key head, batch entry, key range, rows, keys seen at the front
  int kt0, nkt;                // its key tiles
  int nact;                    // its query tiles that have rows
  bool first, new_run, last_of_run;
  bool resident;               // its key tiles fit in the ring: loaded once for the run

  __device__ __forceinline__ FwdItems(const CrossParams& p_) : p(p_), b(-1) {
    R = p.N;
    rows = (size_t)p.B * p.H * R;
    nt = (R + C::kNq * 128 - 1) / (C::kNq * 128);
    i = (int)p.runs.begin(blockIdx.x) - 1;
    end = (int)p.runs.begin(blockIdx.x + 1);
    const int run = (i + 1) / nt;
    tile = i - run * nt;  // of the item before the first
    bk = run / p.nks;
    split = run - bk * p.nks;
    range();
    first = true;
  }
  __device__ __forceinline__ void range() {
    const int nb = bk / p.H;
    if (nb >= p.B) return;  // past the last item
    if (nb != b) {
      b = nb;
      len = cross_len(p, b);
    }
    kt0 = 0;
    nkt = (len + C::kKeys - 1) / C::kKeys;
    if (p.nks > 1) {  // the first nkt % nks ranges are longer by one
      const int each = nkt / p.nks, more = nkt - each * p.nks;
      kt0 = each * split + min(split, more);
      nkt = each + (split < more);
    }
    resident = 2 * nkt <= C::kKv;
  }
  __device__ __forceinline__ bool next() {
    if (i + 1 >= end) return false;
    new_run = first;
    first = false;
    ++i;
    if (++tile == nt) {
      tile = 0;
      new_run = true;
      if (++split == p.nks) {
        split = 0;
        ++bk;
      }
      range();
    }
    last_of_run = tile == nt - 1 || i + 1 == end;
    r0 = tile * C::kNq * 128;
    nact = min(C::kNq, (R - r0 + 127) / 128);
    return true;
  }
  // whether the item's keys are loaded for it
  __device__ __forceinline__ bool loads() const { return !resident || new_run; }
  // 16-key steps of key tile j of the item
  __device__ __forceinline__ int steps(int j) const {
    const int n = len - (kt0 + j) * C::kKeys;
    return n >= C::kKeys ? C::kKeys / 16 : (n + 15) >> 4;
  }
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
cross_fwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to, CrossParams p) {
  using C = Cfg<D>;
  constexpr int H = D / 64;  // 64-column halves of a tile
  constexpr int kKvHalf = C::kKeys * 128;
  extern __shared__ __align__(1024) unsigned char sm[];
  Shared<C>& S = *reinterpret_cast<Shared<C>*>(sm + C::kEnd);
  const uint32_t base = smem_u32(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const bool clean = p.mask != nullptr || p.kv_len != nullptr;
  bool ok = true;

  if (warp == C::kMma) {
    tmem_alloc(smem_u32(&S.tmem_base), 512);
    tmem_relinquish();
  } else if (tid == 0) {
    for (int i = 0; i < C::kQ; ++i) {
      mbar_init(smem_u32(&S.q_full[i / C::kQr][i % C::kQr]), 1);
      mbar_init(smem_u32(&S.q_empty[i / C::kQr][i % C::kQr]), 1);
    }
    for (int i = 0; i < C::kKv; ++i) {
      mbar_init(smem_u32(&S.kv_full[i]), 1);
      mbar_init(smem_u32(&S.kv_empty[i]), C::kMmaWarps);
      mbar_init(smem_u32(&S.kv_clean[i]), 1);
    }
    for (int w = 0; w < C::kNq; ++w) {
      mbar_init(smem_u32(&S.s_full[w]), 1);
      mbar_init(smem_u32(&S.p_full[w]), 128);
      mbar_init(smem_u32(&S.o_full[w]), 1);
      mbar_init(smem_u32(&S.o_staged[w]), 128);
    }
    mbar_init(smem_u32(&S.done), C::kMmaWarps);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = uniform(S.tmem_base);
  // Q slots and their barriers, by ring (the mma warp whose tiles take it) and place
  auto qslot = [&](int ring, uint32_t i) { return base + (ring * C::kQr + i) * C::kQTile; };
  auto kvslot = [&](uint32_t i) { return base + C::kOffKv + i * C::kKvTile; };
  auto q_full = [&](int ring) { return smem_u32(S.q_full[ring]); };
  auto q_empty = [&](int ring) { return smem_u32(S.q_empty[ring]); };
  const uint32_t kv_full = smem_u32(S.kv_full), kv_empty = smem_u32(S.kv_empty), kv_clean = smem_u32(S.kv_clean),
                 s_full = smem_u32(S.s_full), p_full = smem_u32(S.p_full), o_full = smem_u32(S.o_full),
                 o_staged = smem_u32(S.o_staged);
  auto wait = [&](uint32_t bar, uint32_t parity) { return ok = __all_sync(0xffffffffu, mbar_wait(bar, parity)); };
  FwdItems<C> it(p);

  if (warp == C::kLoad) {
    if (lane == 0) {
      Ring<C::kQr> rq[C::kMmaWarps];
      Ring<C::kKv> rk;
      // a slot's first round waits for the phase before the first, which is over
      auto load = [&](uint32_t dst, uint32_t half, const CUtensorMap* map, int row, uint32_t full, uint32_t bytes) {
        mbar_arrive_expect_tx(full, bytes);
#pragma unroll
        for (int h = 0; h < H; ++h) tma_load_3d(dst + h * half, map, 64 * h, row, it.bk, full);
      };
      auto load_q = [&](int w) {
        const int u = w / C::kPer;
        Ring<C::kQr>& r = rq[u];
        if (ok) ok = mbar_wait(r.at(q_empty(u)), r.parity ^ 1u);
        if (!ok) return;
        load(qslot(u, r.i), 16384, &tq, it.r0 + 128 * w, r.at(q_full(u)), C::kQTile);
        r.next();
      };
      auto load_kv = [&](const CUtensorMap* map, int j) {
        if (ok) ok = mbar_wait(rk.at(kv_empty), rk.parity ^ 1u);
        if (!ok) return;
        load(kvslot(rk.i), kKvHalf, map, (it.kt0 + j) * C::kKeys, rk.at(kv_full), C::kKvTile);
        rk.next();
      };
      for (; ok && it.next();) {
        if (it.nkt == 0) continue;
        const int n = it.loads() ? it.nkt : 0;
        load_q(0);
        if (n > 0) load_kv(&tk, 0);
#pragma unroll
        for (int w = 1; w < C::kNq; ++w)
          if (w < it.nact) load_q(w);
        if (n > 0) load_kv(&tv, 0);
        for (int j = 1; j < n && ok; ++j) {
          load_kv(&tk, j);
          load_kv(&tv, j);
        }
      }
      // no copy may still be landing when the CTA exits: of every slot, the
      // last round that was begun
#pragma unroll
      for (int u = 0; u < C::kMmaWarps; ++u)
        for (int i = 0; i < C::kQr; ++i, rq[u].next())
          if (!mbar_wait(rq[u].at(q_full(u)), rq[u].parity ^ 1u)) ok = false;
      for (int i = 0; i < C::kKv; ++i, rk.next())
        if (!mbar_wait(rk.at(kv_full), rk.parity ^ 1u)) ok = false;
    }
  } else if (warp >= C::kMma && warp < C::kClean) {
    // query tiles w0 .. w0 + kPer - 1; the whole warp walks, one lane issues
    const int ring = warp - C::kMma, w0 = C::kPer * ring;
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1, 0);
    const uint64_t kmaj = smem_desc_sw128(0, 16, 1024), nmaj = smem_desc_sw128(0, kKvHalf, 1024);
    const uint32_t lead = elect_lane();
    Ring<C::kQr> rq;               // of the first of them
    Ring<C::kKv> run, kv, pv_at;   // the run's first tile, this step's K, the pending products' V
    uint32_t turn[C::kPer] = {};   // parity of p_full
    bool pend[C::kPer] = {};
    int pnt = 0;                   // the pending products' 16-key steps
    bool pfirst = false, plast = false, pfree = false, held = false;
    // O_w (+)= P_w V of the previous step.  V is waited for by every issuing
    // warp at every step, also for tiles without rows: its slots are then freed
    // only after it has been seen, and who waits for S of the next step knows
    // that V of every step before is there (a barrier tells rounds apart by
    // parity, so no wait for one may begin before the round before is over).
    auto products = [&](int u) {
      if (u == 0 && held) {
        held = false;
        if (clean ? !wait(pv_at.at(kv_clean), pv_at.parity) : !wait(pv_at.at(kv_full), pv_at.parity)) return;
      }
      if (!pend[u]) return;
      pend[u] = false;
      const int w = w0 + u;
      if (!wait(p_full + 8 * w, turn[u])) return;
      turn[u] ^= 1u;
      tc_fence_after();
      const uint64_t v = desc_at(nmaj, kvslot(pv_at.i));
#pragma unroll
      for (int k = 0; k < C::kKeys / 16; ++k) {
        if (k >= pnt) break;
        tc_mma_f16_ts_by(lead, tbase + C::kColO + w * D, tbase + w * C::kKeys + k * 8, desc_at(v, k * 2048), idesc_pv,
                         !pfirst || k > 0);
      }
      if (plast) tc_commit_by(lead, o_full + 8 * w);
    };
    for (; ok && it.next();) {
      const int nkt = uniform(it.nkt), nact = uniform(it.nact);
      if (nkt == 0) continue;
      const bool loads = 2 * nkt > C::kKv || it.new_run, free = 2 * nkt > C::kKv || it.last_of_run;
      if (loads) {
        run = kv;
      } else {
        kv = run;
      }
      for (int j = 0; j < nkt && ok; ++j) {
        const int nt = uniform(it.steps(j));
        const uint32_t idesc_s = idesc_bf16_f32(128, 16 * nt, 0, 0);
        const uint64_t k = desc_at(kmaj, kvslot(kv.i));
        if (!wait(kv.at(kv_full), kv.parity)) break;
#pragma unroll
        for (int u = 0; u < C::kPer; ++u) {
          if (ok) products(u);
          const int w = w0 + u;
          if (!ok || w >= nact) continue;
          Ring<C::kQr> at = rq;
          at.next(u);
          if (j == 0 && !wait(at.at(q_full(ring)), at.parity)) continue;
          tc_fence_after();
          const uint64_t q = desc_at(kmaj, qslot(ring, at.i));
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc_mma_f16_by(lead, tbase + w * C::kKeys, desc_at(q, (ks >> 2) * 16384 + (ks & 3) * 32),
                          desc_at(k, (ks >> 2) * kKvHalf + (ks & 3) * 32), idesc_s, ks > 0);
          tc_commit_by(lead, s_full + 8 * w);
          pend[u] = true;
        }
        if (!ok) break;
        if (pfree) tc_commit_by(lead, pv_at.at(kv_empty));
        if (free) tc_commit_by(lead, kv.at(kv_empty));
        pv_at = kv;
        pv_at.next();
        pnt = nt;
        pfirst = j == 0;
        plast = j == nkt - 1;
        pfree = free;
        held = true;
        kv.next(2);
      }
      rq.next(min(max(nact - w0, 0), C::kPer));
    }
#pragma unroll
    for (int u = 0; u < C::kPer; ++u)
      if (ok) products(u);
    // every MMA of this CTA has completed before tensor memory is freed
    tc_commit_by(lead, smem_u32(&S.done));
    if (!mbar_wait(smem_u32(&S.done), 0)) ok = false;
  } else if (warp == C::kClean) {
    Ring<C::kKv> rv;  // of V
    rv.next();
    for (; ok && clean && it.next();) {
      if (!it.loads()) continue;
      for (int j = 0; j < it.nkt; ++j, rv.next(2)) {
        const int k0 = (it.kt0 + j) * C::kKeys;
        uint32_t word[C::kKeys / 32];
#pragma unroll
        for (int c = 0; c < C::kKeys / 32; ++c) {
          const int key = k0 + 32 * c + lane;
          const bool on = key < it.len && (p.mask == nullptr || p.mask[(size_t)it.b * p.S + key] != 0);
          word[c] = __ballot_sync(0xffffffffu, on);
        }
        if (!wait(rv.at(kv_full), rv.parity)) break;
        const int rows = 16 * it.steps(j);
        unsigned char* v = sm + (kvslot(rv.i) - base);
#pragma unroll
        for (int c = 0; c < C::kKeys / 32; ++c) {
          if (lane == 0) S.bits[rv.i][c] = word[c];
          for (uint32_t off = ~word[c]; off != 0u; off &= off - 1) {  // one row at a time, 16 bytes a lane
            const int r = 32 * c + __ffs(off) - 1;
            if (r >= rows) break;
            if (lane < D / 8)
              *reinterpret_cast<uint4*>(v + (lane >> 3) * kKvHalf + sw128(r, lane & 7)) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();  // generic writes -> MMA operand reads
        __syncwarp();
        if (lane == 0) mbar_arrive(rv.at(kv_clean));
      }
    }
  } else if (warp == C::kStore) {
    if (lane == 0) {
      Ring<C::kQr> rq[C::kMmaWarps];
      uint32_t turn = 0;  // parities of o_staged, a bit each
      for (; ok && it.next();) {
        if (it.nkt == 0) continue;
#pragma unroll
        for (int w = 0; w < C::kNq; ++w) {
          if (!ok || w >= it.nact) break;
          ok = mbar_wait(o_staged + 8 * w, (turn >> w) & 1u);
          if (!ok) break;
          turn ^= 1u << w;
          const int u = w / C::kPer;
          if (p.nks == 1) {
#pragma unroll
            for (int h = 0; h < H; ++h) tma_store_3d(&to, 64 * h, it.r0 + 128 * w, it.bk, qslot(u, rq[u].i) + h * 16384);
            bulk_commit_group();
            bulk_wait_read_all();
          }
          mbar_arrive(rq[u].at(q_empty(u)));
          rq[u].next();
        }
      }
      bulk_wait_all();
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int w = warp >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t trow = tbase + ((uint32_t)(q4 * 32) << 16);
    const uint32_t ts = trow + (uint32_t)(w * C::kKeys), tO = trow + C::kColO + (uint32_t)w * D;
    const float sc2 = p.scale * kLog2e;
    const uint64_t sc2x2 = f2_make(sc2, sc2);
    const int ring = w / C::kPer, w0 = C::kPer * ring;
    Ring<C::kQr> rq;       // of the first of the ring's tiles
    Ring<C::kKv> run, rv;  // of V
    rv.next();
    uint32_t s_turn = 0, o_turn = 0;
    Ring<C::kQr> last;     // the slot of this tile's last item
    bool staged = false;
    for (; ok && it.next();) {
      const int row = it.r0 + 128 * w + r;
      const size_t grow = (size_t)it.bk * it.R + row;
      if (it.nkt == 0) {  // no keys (in this range): nothing to wait for
        if (row < it.R) {
          if (p.nks > 1) {
            p.part_ml[(size_t)it.split * it.rows + grow] = make_float2(-INFINITY, 0.f);
          } else {
            for (int c = 0; c < D / 8; ++c) {
              reinterpret_cast<uint4*>(static_cast<bf16*>(p.o) + grow * D)[c] = make_uint4(0, 0, 0, 0);
              if (p.o_res != nullptr)
                reinterpret_cast<uint4*>(static_cast<bf16*>(p.o_res) + grow * D)[c] = make_uint4(0, 0, 0, 0);
            }
            p.lse[grow] = -INFINITY;
          }
        }
        continue;
      }
      if (it.loads()) run = rv;
      else rv = run;
      Ring<C::kQr> at = rq;
      at.next(w - w0);
      rq.next(min(max(it.nact - w0, 0), C::kPer));
      if (w >= it.nact) {
        for (int j = 0; j < it.nkt; ++j) rv.next(2);
        continue;
      }
      float m = -INFINITY;  // running maximum, in units of log2
      float l = 0.f;
      for (int j = 0; j < it.nkt; ++j, rv.next(2)) {
        const int nch = (it.steps(j) + 1) / 2;  // chunks of 32 keys
        if (!wait(s_full + 8 * w, s_turn)) break;
        s_turn ^= 1u;
        if (clean && !wait(rv.at(kv_clean), rv.parity)) break;
        tc_fence_after();
        const int left = it.len - (it.kt0 + j) * C::kKeys;
        if (clean || left < C::kKeys) {
#pragma unroll 1
          for (int c = 0; c < 2 * nch; ++c) {
            const uint32_t bits = clean ? (S.bits[rv.i][c >> 1] >> (16 * (c & 1))) & 0xffffu
                                        : (1u << min(max(left - 16 * c, 0), 16)) - 1u;
            if (bits != 0xffffu) hide16(ts + 16 * c, bits, -INFINITY);
          }
        }
        // the row's maximum
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
          float x[32];
          tmem_ld32(ts + 32 * c, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], x[i]);
        }
        const float mt = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sc2;
        const float mn = fmaxf(m, mt);
        const bool need = m != -INFINITY && mn > m;
        const float corr = need ? ex2_approx(m - mn) : 1.f;
        m = mn;
        const float mb = m == -INFINITY ? 0.f : m;
        if (__any_sync(0xffffffffu, need)) {  // O of the tiles so far: S of this one came after it
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= corr;
            tmem_st32(tO + c, o);
          }
        }
        // P = 2^(s sc2 - m), over the S columns already read
        const uint64_t nm2 = f2_make(-mb, -mb);
        uint64_t sum[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
          float x[32];
          tmem_ld32(ts + 32 * c, x);
          tmem_wait_ld();
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 d = f2_split(f2_fma(f2_make(x[2 * i], x[2 * i + 1]), sc2x2, nm2));
            const float p0 = ex2_approx(d.x), p1 = ex2_approx(d.y);
            pk[i] = pack_bf16(p0, p1);
            sum[i & 1] = f2_add(sum[i & 1], f2_make(p0, p1));
          }
          tmem_st16u(ts + 16 * c, pk);
        }
        const float2 s2 = f2_split(f2_add(sum[0], sum[1]));
        l = l * corr + (s2.x + s2.y);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + 8 * w);
      }
      if (!ok) break;
      // ------------------------------------------------------------ epilogue
      if (!wait(o_full + 8 * w, o_turn)) break;
      o_turn ^= 1u;
      tc_fence_after();
      const bool valid = row < it.R;
      const float inv = l != 0.f ? 1.f / l : 0.f;  // 0 without keys; NaN stays NaN
      unsigned char* stage = sm + (qslot(ring, at.i) - base);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(tO + c, o);
        tmem_wait_ld();
        if (p.nks > 1) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + ((size_t)it.split * it.rows + grow) * D + c);
          if (valid) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= inv;
          uint4* rdst = p.o_res != nullptr && valid
                            ? reinterpret_cast<uint4*>(static_cast<bf16*>(p.o_res) + grow * D + c) : nullptr;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float* a = o + 8 * g;
            const uint4 u = make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]),
                                       pack_bf16(a[6], a[7]));
            const int cc = c / 8 + g;
            *reinterpret_cast<uint4*>(stage + (cc >> 3) * 16384 + sw128(r, cc & 7)) = u;
            if (rdst != nullptr)
              rdst[g] = make_uint4(pack_bf16(a[0] - bf16x2_lo(u.x), a[1] - bf16x2_hi(u.x)),
                                   pack_bf16(a[2] - bf16x2_lo(u.y), a[3] - bf16x2_hi(u.y)),
                                   pack_bf16(a[4] - bf16x2_lo(u.z), a[5] - bf16x2_hi(u.z)),
                                   pack_bf16(a[6] - bf16x2_lo(u.w), a[7] - bf16x2_hi(u.w)));
          }
        }
      }
      fence_proxy_async_smem();  // generic writes -> TMA store
      tc_fence_before();
      // the store warp has taken the last one, else this phase could pass it by
      if (staged && !wait(last.at(q_empty(ring)), last.parity)) break;
      last = at;
      staged = true;
      mbar_arrive(o_staged + 8 * w);
      if (valid) {
        if (p.nks > 1) p.part_ml[(size_t)it.split * it.rows + grow] = make_float2(m, l);
        else p.lse[grow] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
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

template <int D>
cudaError_t launch_typed(CrossParams p, const CUtensorMap* maps, cudaStream_t s) {
  using C = Cfg<D>;
  constexpr size_t smem = C::kEnd + sizeof(Shared<C>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(cross_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.B * p.H * p.nks * cross_tiles(p.N, C::kNq * 128);
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int grid = (int)(items < kCrossSms ? items : kCrossSms);
  p.runs = cross_runs(items, grid);
  cross_fwd_tc_kernel<D><<<grid, C::kThreads, smem, s>>>(maps[0], maps[1], maps[2], maps[3], p);
  return cudaGetLastError();
}

}  // namespace

CrossPlan cross_tc_fwd_plan(long long BH, int N, int S, int D) {
  // cut the keys where the row tiles leave SMs without an item
  const int rows = (D == 64 ? Cfg<64>::kNq : Cfg<128>::kNq) * 128, keys = D == 64 ? Cfg<64>::kKeys : Cfg<128>::kKeys;
  const int64_t units = BH * cross_tiles(N, rows), kt = cross_tiles(S, keys);
  int64_t nks = kCrossSms / units;
  if (nks > kt) nks = kt;
  return {nks < 1 ? 1 : (int)nks, 1};
}

cudaError_t launch_cross_fwd_tc(const CrossParams& p, const CUtensorMap* maps, cudaStream_t s) {
  return p.D == 64 ? launch_typed<64>(p, maps, s) : launch_typed<128>(p, maps, s);
}

}  // namespace llsa
