// Cross attention forward on the 5th-generation tensor cores (tcgen05), bf16,
// D = 64 or 128:
//   S = Q K^T,  P = e^(scale S - m),  O = P V / l,  lse = scale m + ln l
// with the running maximum m and sum l of the softmax, in one pass over the
// keys.
//
// The query heads of a key head are neighbours in memory, so their queries
// are one run of R rows against the same keys.  A work item is 256 of these
// rows (two tiles of 128, the M of an MMA) against a range of key tiles of
// 128; a persistent CTA per SM walks a contiguous range of items:
//   warps 0-3, 4-7  softmax of the two query tiles, one thread per row;
//   warp 8          TMA loads: Q tiles into a ring of slots, K and V tiles
//                   into another.  Key tiles that fit in the ring are loaded
//                   once and stay for all items of the same keys;
//   warp 9          issues the MMAs: S_w = Q_w K^T into tensor
//                   memory, and O_w += P_w V with P_w read from tensor memory
//                   (over S_w, which the softmax has read);
//   warp 10         with lengths or a mask: the bits of the keys seen in each
//                   tile, and zeros over the V rows that are not seen (their
//                   probability is zero, and zero times NaN is NaN);
//   warp 11         TMA stores of the finished O tiles, staged over their Q.
// The two query tiles take turns: the tensor cores work on one while the
// exponentials of the other are computed, which bound the kernel (one per
// score; 16 a clock and SM).  The next item's first S is issued before this
// item's epilogue.  Few rows: the keys are cut into ranges, each a work item
// of its own, whose fp32 parts are joined by another kernel.
// P is rounded to bf16 for the product (the exact running maximum is kept, so
// a row's largest probability is 1 and rounds exactly); m, l and O are fp32.
// Every wait is bounded; a time-out is reported as LLSA_DEV_TIMEOUT.

#include <math.h>

#include "cross.cuh"
#include "cross_tc.cuh"

namespace llsa {

namespace {

constexpr int kThreads = 384;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpClean = 10, kWarpStore = 11;

template <int D>
struct Cfg {
  static constexpr int kTile = 128 * D * 2;             // a Q, K or V tile
  static constexpr int kQ = (D == 64) ? 4 : 3;          // Q slots
  static constexpr int kKv = (D == 64) ? 8 : 4;         // K and V slots
  static constexpr int kEnd = (kQ + kKv) * kTile;
  static constexpr uint32_t kColO = 256;                // S_0 | S_1 | O_0 | O_1
};

struct Shared {
  uint64_t q_full[4], q_empty[4], kv_full[8], kv_empty[8], kv_clean[8];
  uint64_t s_full[2], p_full[2], o_full[2], o_staged[2], done;
  uint32_t bits[8][4];  // keys seen, by V slot
  uint32_t tmem_base;
};

// The items of a CTA, in order: 256 query rows of one key head against one
// range of its key tiles.  Every warp role walks them by itself; rows are
// innermost, so items of the same keys follow one another (a run).
struct FwdItems {
  const CrossParams& p;
  int i, end, nt, cap;
  int R;                       // query rows of a key head
  size_t rows;                 // and of all of them
  int bk, b, split, tile, r0, len;  // the item: key head, batch entry, key range, rows, keys seen at the front
  int kt0, nkt;                // its key tiles
  bool act1;                   // whether its second tile of 128 rows has any
  bool first, new_run, last_of_run;
  bool resident;               // its key tiles fit in the ring: loaded once for the run

  __device__ __forceinline__ FwdItems(const CrossParams& p_, int cap_) : p(p_), cap(cap_), b(-1) {
    R = p.N;
    rows = (size_t)p.B * p.H * R;
    nt = (R + 255) / 256;
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
    nkt = (len + 127) / 128;
    if (p.nks > 1) {  // the first nkt % nks ranges are longer by one
      const int each = nkt / p.nks, more = nkt - each * p.nks;
      kt0 = each * split + min(split, more);
      nkt = each + (split < more);
    }
    resident = nkt <= cap;
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
    r0 = tile * 256;
    act1 = r0 + 128 < R;
    return true;
  }
  // 16-key steps of key tile j of the item
  __device__ __forceinline__ int steps(int j) const {
    const int n = len - (kt0 + j) * 128;
    return n >= 128 ? 8 : (n + 15) >> 4;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_fwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to, CrossParams p) {
  using C = Cfg<D>;
  constexpr int H = D / 64;  // 64-column halves of a tile
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Shared& S = *reinterpret_cast<Shared*>(sm + C::kEnd);
  const uint32_t base = smem_u32(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const bool clean = p.mask != nullptr || p.kv_len != nullptr;
  bool ok = true;

  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&S.tmem_base), 512);
    tmem_relinquish();
  } else if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&S.q_full[i]), 1);
      mbar_init(smem_u32(&S.q_empty[i]), 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&S.kv_full[i]), 1);
      mbar_init(smem_u32(&S.kv_empty[i]), 1);
      mbar_init(smem_u32(&S.kv_clean[i]), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&S.s_full[w]), 1);
      mbar_init(smem_u32(&S.p_full[w]), 128);
      mbar_init(smem_u32(&S.o_full[w]), 1);
      mbar_init(smem_u32(&S.o_staged[w]), 128);
    }
    mbar_init(smem_u32(&S.done), 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = uniform(S.tmem_base);
  auto qslot = [&](int t) { return base + (uint32_t)(t % C::kQ) * C::kTile; };
  auto kvslot = [&](int f) { return base + (uint32_t)(C::kQ + f % C::kKv) * C::kTile; };
  FwdItems it(p, C::kKv / 2);

  if (warp == kWarpLoad) {
    if (lane == 0) {
      int t = 0, f = 0;  // Q tiles and K/V tiles loaded so far
      auto load = [&](uint32_t dst, const CUtensorMap* map, int row, int bk, uint64_t* bar) {
        mbar_arrive_expect_tx(smem_u32(bar), C::kTile);
#pragma unroll
        for (int h = 0; h < H; ++h) tma_load_3d(dst + h * 16384, map, 64 * h, row, bk, smem_u32(bar));
      };
      auto load_q = [&](int w) {
        if (t >= C::kQ) ok = mbar_wait(smem_u32(&S.q_empty[t % C::kQ]), (uint32_t)((t / C::kQ - 1) & 1));
        if (!ok) return;
        load(qslot(t), &tq, it.r0 + 128 * w, it.bk, &S.q_full[t % C::kQ]);
        ++t;
      };
      for (; ok && it.next();) {
        if (it.nkt == 0) continue;
        // the second Q tile goes before the keys that have to wait for it to
        // be used: every step needs both
        load_q(0);
        const int nkv = (!it.resident || it.new_run) ? 2 * it.nkt : 0;
        for (int j = 0; j < nkv && ok; ++j) {
          if (j == 2 && it.act1) load_q(1);
          if (f >= C::kKv && ok)
            ok = mbar_wait(smem_u32(&S.kv_empty[f % C::kKv]), (uint32_t)((f / C::kKv - 1) & 1));
          if (!ok) break;
          load(kvslot(f), (j & 1) ? &tv : &tk, (it.kt0 + j / 2) * 128, it.bk, &S.kv_full[f % C::kKv]);
          ++f;
        }
        if (ok && it.act1 && nkv <= 2) load_q(1);
      }
      // no copy may still be landing when the CTA exits
      for (int i = t > C::kQ ? t - C::kQ : 0; i < t; ++i)
        if (!mbar_wait(smem_u32(&S.q_full[i % C::kQ]), (uint32_t)((i / C::kQ) & 1))) ok = false;
      for (int i = f > C::kKv ? f - C::kKv : 0; i < f; ++i)
        if (!mbar_wait(smem_u32(&S.kv_full[i % C::kKv]), (uint32_t)((i / C::kKv) & 1))) ok = false;
    }
  } else if (warp == kWarpMma) {
    // the whole warp walks; one lane issues
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1, 0);
    const uint64_t kmaj = smem_desc_sw128(0, 16, 1024), nmaj = smem_desc_sw128(0, 16384, 1024);
    const uint32_t lead = elect_lane();
    int t = 0, f = 0, frun = 0;
    int np[2] = {0, 0};      // P tiles taken
    bool pend[2] = {false, false};
    int pf = 0, pnt = 0;     // the pending product's V tile and its 16-key steps
    bool pfirst = false, plast = false, pfree = false;
    auto wait = [&](uint64_t* bar, int phase) {
      return ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), (uint32_t)(phase & 1)));
    };
    auto pv = [&](int w) {   // O_w (+)= P_w V of the previous step
      if (!pend[w]) return;
      pend[w] = false;
      if (!wait(&S.kv_full[pf % C::kKv], pf / C::kKv)) return;
      if (clean && !wait(&S.kv_clean[pf % C::kKv], pf / C::kKv)) return;
      if (!wait(&S.p_full[w], np[w])) return;
      ++np[w];
      tc_fence_after();
      const uint64_t v = desc_at(nmaj, kvslot(pf));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= pnt) break;
        tc_mma_f16_ts_by(lead, tbase + C::kColO + w * D, tbase + w * 128 + k * 8, desc_at(v, k * 2048), idesc_pv,
                         !pfirst || k > 0);
      }
      if (plast) tc_commit_by(lead, smem_u32(&S.o_full[w]));
    };
    for (; ok && it.next();) {
      const int nkt = uniform(it.nkt);
      if (nkt == 0) continue;
      const bool resident = nkt <= it.cap;
      if (!resident || it.new_run) {
        frun = f;
        f += 2 * nkt;
      }
      const int t0 = t;
      t += it.act1 ? 2 : 1;
      for (int j = 0; j < nkt && ok; ++j) {
        const int fk = frun + 2 * j;
        const int nt = uniform(it.steps(j));
        const uint32_t idesc_s = idesc_bf16_f32(128, 16 * nt, 0, 0);
        const uint64_t k = desc_at(kmaj, kvslot(fk));
        if (!wait(&S.kv_full[fk % C::kKv], fk / C::kKv)) break;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (ok) pv(w);
          if (!ok || (w == 1 && !it.act1)) continue;
          const int tw = t0 + w;
          if (j == 0 && !wait(&S.q_full[tw % C::kQ], tw / C::kQ)) continue;
          tc_fence_after();
          const uint64_t q = desc_at(kmaj, qslot(tw));
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc_mma_f16_by(lead, tbase + w * 128, desc_at(q, (ks >> 2) * 16384 + (ks & 3) * 32),
                          desc_at(k, (ks >> 2) * 16384 + (ks & 3) * 32), idesc_s, ks > 0);
          tc_commit_by(lead, smem_u32(&S.s_full[w]));
          pend[w] = true;
        }
        if (!ok) break;
        if (pfree) tc_commit_by(lead, smem_u32(&S.kv_empty[pf % C::kKv]));
        pf = fk + 1;
        pnt = nt;
        pfirst = j == 0;
        plast = j == nkt - 1;
        pfree = !resident || it.last_of_run;
        if (pfree) tc_commit_by(lead, smem_u32(&S.kv_empty[fk % C::kKv]));
      }
    }
    for (int w = 0; w < 2 && ok; ++w) pv(w);
    // every MMA of this CTA has completed before tensor memory is freed
    tc_commit_by(lead, smem_u32(&S.done));
    if (!mbar_wait(smem_u32(&S.done), 0)) ok = false;
  } else if (warp == kWarpClean) {
    if (clean) {
      int f = 0;
      for (; ok && it.next();) {
        if (it.nkt == 0 || (it.resident && !it.new_run)) continue;
        for (int j = 0; j < it.nkt && ok; ++j, f += 2) {
          const int slot = (f + 1) % C::kKv;
          const int k0 = (it.kt0 + j) * 128;
          uint32_t word[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = k0 + 32 * c + lane;
            const bool on = key < it.len && (p.mask == nullptr || p.mask[(size_t)it.b * p.S + key] != 0);
            word[c] = __ballot_sync(0xffffffffu, on);
          }
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S.kv_full[slot]), (uint32_t)(((f + 1) / C::kKv) & 1)));
          if (!ok) break;
          const int rows = 16 * it.steps(j);
          unsigned char* v = sm + (kvslot(f + 1) - base);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (lane == 0) S.bits[slot][c] = word[c];
            for (uint32_t off = ~word[c]; off != 0u; off &= off - 1) {  // one row at a time, 16 bytes a lane
              const int r = 32 * c + __ffs(off) - 1;
              if (r >= rows) break;
              if (lane < D / 8)
                *reinterpret_cast<uint4*>(v + (lane >> 3) * 16384 + sw128(r, lane & 7)) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();  // generic writes -> MMA operand reads
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&S.kv_clean[slot]));
        }
      }
    }
  } else if (warp == kWarpStore) {
    if (lane == 0) {
      int t = 0, n[2] = {0, 0};
      for (; ok && it.next();) {
        if (it.nkt == 0) continue;
        for (int w = 0; w < (it.act1 ? 2 : 1) && ok; ++w, ++t) {
          ok = mbar_wait(smem_u32(&S.o_staged[w]), (uint32_t)(n[w] & 1));
          if (!ok) break;
          ++n[w];
          if (p.nks == 1) {
#pragma unroll
            for (int h = 0; h < H; ++h) tma_store_3d(&to, 64 * h, it.r0 + 128 * w, it.bk, qslot(t) + h * 16384);
            bulk_commit_group();
            bulk_wait_read_all();
          }
          mbar_arrive(smem_u32(&S.q_empty[t % C::kQ]));
        }
      }
      bulk_wait_all();
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int w = warp >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t trow = tbase + ((uint32_t)(q4 * 32) << 16);
    const uint32_t ts = trow + (uint32_t)w * 128, tO = trow + C::kColO + (uint32_t)w * D;
    const float sc2 = p.scale * kLog2e;
    const uint64_t sc2x2 = f2_make(sc2, sc2);
    int t = 0, ns = 0, no = 0, f = 0, frun = 0;
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
      if (!it.resident || it.new_run) {
        frun = f;
        f += 2 * it.nkt;
      }
      const int tw = t + w;
      t += it.act1 ? 2 : 1;
      if (w == 1 && !it.act1) continue;
      float m = -INFINITY;  // running maximum, in units of log2
      float l = 0.f;
      for (int j = 0; j < it.nkt && ok; ++j, ++ns) {
        const int nch = (it.steps(j) + 1) / 2;  // chunks of 32 keys
        const int slot = (frun + 2 * j + 1) % C::kKv;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S.s_full[w]), (uint32_t)(ns & 1)));
        if (ok && clean)
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S.kv_clean[slot]),
                                                         (uint32_t)(((frun + 2 * j + 1) / C::kKv) & 1)));
        if (!ok) break;
        tc_fence_after();
        const int left = it.len - (it.kt0 + j) * 128;
        if (clean || left < 128) {
#pragma unroll 1
          for (int c = 0; c < 2 * nch; ++c) {
            const uint32_t bits = clean ? (S.bits[slot][c >> 1] >> (16 * (c & 1))) & 0xffffu
                                        : (left - 16 * c >= 16 ? 0xffffu : (left <= 16 * c ? 0u : (1u << (left - 16 * c)) - 1u));
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
        mbar_arrive(smem_u32(&S.p_full[w]));
      }
      if (!ok) break;
      // ------------------------------------------------------------ epilogue
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S.o_full[w]), (uint32_t)(no & 1)));
      if (!ok) break;
      ++no;
      tc_fence_after();
      const bool valid = row < it.R;
      const float inv = l != 0.f ? 1.f / l : 0.f;  // 0 without keys; NaN stays NaN
      unsigned char* stage = sm + (qslot(tw) - base);
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
          for (int i = 0; i < 32; ++i) o[i] = l != 0.f ? o[i] * inv : 0.f;
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
      mbar_arrive(smem_u32(&S.o_staged[w]));
      if (valid) {
        if (p.nks > 1) p.part_ml[(size_t)it.split * it.rows + grow] = make_float2(m, l);
        else p.lse[grow] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
  }

  if (!ok) report_status(p.status, LLSA_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D>
cudaError_t launch_typed(CrossParams p, const CUtensorMap* maps, cudaStream_t s) {
  constexpr size_t smem = 1024 + Cfg<D>::kEnd + sizeof(Shared);
  cudaError_t e = cudaFuncSetAttribute(cross_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.B * p.H * p.nks * cross_tiles(p.N, 256);
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int grid = (int)(items < kCrossSms ? items : kCrossSms);
  p.runs = cross_runs(items, grid);
  cross_fwd_tc_kernel<D><<<grid, kThreads, smem, s>>>(maps[0], maps[1], maps[2], maps[3], p);
  return cudaGetLastError();
}

}  // namespace

CrossPlan cross_tc_fwd_plan(long long BH, int N, int S) {
  // cut the keys where the row tiles leave SMs without an item
  const int64_t units = BH * cross_tiles(N, 256), kt = cross_tiles(S, 128);
  int64_t nks = kCrossSms / units;
  if (nks > kt) nks = kt;
  return {nks < 1 ? 1 : (int)nks, 1};
}

cudaError_t launch_cross_fwd_tc(const CrossParams& p, const CUtensorMap* maps, cudaStream_t s) {
  return p.D == 64 ? launch_typed<64>(p, maps, s) : launch_typed<128>(p, maps, s);
}

}  // namespace llsa
