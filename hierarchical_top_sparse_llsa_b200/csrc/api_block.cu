// Host side of the C ABI's calls around the self-attention: rotary positions
// and cross attention (argument checks, workspace layouts, dispatch).  No
// allocation, no state.

#include <math.h>
#include <string.h>

#include "api_common.cuh"
#include "cross.cuh"
#include "llsa_internal.cuh"
#include "rope.cuh"

using namespace llsa;

namespace {

inline int launch_status(cudaError_t e) { return e == cudaSuccess ? LLSA_OK : LLSA_ERR_LAUNCH; }

inline bool aligned(const void* ptr, size_t n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) == 0; }

// ----------------------------------------------------------- rotary positions
int check_rope(const llsa_rope_desc* r) {
  if (r == nullptr) return LLSA_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim % 2 != 0) return LLSA_ERR_INVALID_ARG;
  if (r->rot_dim > 2 * kMaxRopeFreqs) return LLSA_ERR_UNSUPPORTED;
  if (r->layout != LLSA_ROPE_HALF && r->layout != LLSA_ROPE_INTERLEAVED) return LLSA_ERR_INVALID_ARG;
  if ((r->axes != 1 && r->axes != 2) || (r->rot_dim / 2) % r->axes != 0) return LLSA_ERR_INVALID_ARG;
  if (r->scaling < LLSA_ROPE_SCALE_NONE || r->scaling > LLSA_ROPE_SCALE_YARN) return LLSA_ERR_INVALID_ARG;
  if (!(r->mscale >= 0.f) || isinf(r->mscale)) return LLSA_ERR_INVALID_ARG;
  if (r->base != 0.0 && (!(r->base > 1.0) || isinf(r->base))) return LLSA_ERR_INVALID_ARG;
  if (r->factor != 0.0 && (!(r->factor >= 1.0) || isinf(r->factor))) return LLSA_ERR_INVALID_ARG;
  if (r->scaling == LLSA_ROPE_SCALE_YARN) {
    const double fast = r->beta_fast != 0.0 ? r->beta_fast : 32.0, slow = r->beta_slow != 0.0 ? r->beta_slow : 1.0;
    if (r->orig_len < 1 || !(slow > 0.0) || !(fast > slow) || isinf(fast)) return LLSA_ERR_INVALID_ARG;
  }
  return LLSA_OK;
}

// The frequencies of a checked descriptor, in turns per position.
RopeFreqs rope_freqs(const llsa_rope_desc* r) {
  constexpr long double kTwoPiL = 6.283185307179586476925286766559006L;
  constexpr double kTwoPi = (double)kTwoPiL;
  RopeFreqs f;
  memset(&f, 0, sizeof(f));
  f.half = r->rot_dim / 2;
  f.axes = r->axes;
  f.n = f.half / f.axes;
  const double n = (double)f.n;
  const double factor = r->factor != 0.0 ? r->factor : 1.0;
  const double base = r->base != 0.0 ? r->base : 10000.0;
  long double wide = base;  // the powers in the long double that this host has
  if (r->scaling == LLSA_ROPE_SCALE_NTK && f.n > 1) wide *= powl(factor, (long double)f.n / (f.n - 1));
  double lo = 0.0, hi = 0.0;
  if (r->scaling == LLSA_ROPE_SCALE_YARN) {
    const double fast = r->beta_fast != 0.0 ? r->beta_fast : 32.0, slow = r->beta_slow != 0.0 ? r->beta_slow : 1.0;
    lo = fmax(floor(n * log((double)r->orig_len / (fast * kTwoPi)) / log(base)), 0.0);
    // up to the axis's channels less one, not its pairs: where even the slowest
    // pair turns within orig_len the ramp's end lies past the last pair
    hi = fmin(ceil(n * log((double)r->orig_len / (slow * kTwoPi)) / log(base)), 2.0 * n - 1.0);
  }
  for (int j = 0; j < f.n; ++j) {
    long double w = powl(wide, -(long double)j / f.n);
    if (r->scaling == LLSA_ROPE_SCALE_LINEAR) w /= factor;
    if (r->scaling == LLSA_ROPE_SCALE_YARN) {
      const double ramp = fmin(fmax(((double)j - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
      w = w / factor * ramp + w * (1.0 - ramp);
    }
    w /= kTwoPiL;
    f.turns[j].x = (double)w;
    f.turns[j].y = (double)(w - f.turns[j].x);
  }
  f.m = r->mscale > 0.f ? r->mscale
                        : (r->scaling == LLSA_ROPE_SCALE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f);
  return f;
}

inline bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + bytes && y < x + bytes;
}

// Whether each output is its own input or disjoint from every tensor given.
// in[i] for i < n are inputs, out[i] for i < m the outputs of the first m.
bool outputs_apart(const void* const* in, int n, void* const* out, int m, size_t bytes) {
  for (int i = 0; i < m; ++i) {
    for (int j = 0; j < n; ++j)
      if (overlap(out[i], in[j], bytes) && !(i == j && out[i] == in[j])) return false;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j], bytes)) return false;
  }
  return true;
}

// A buffer of a call, for the check that outputs overlap nothing.
struct Span {
  const void* ptr;
  size_t bytes;
};

bool spans_meet(const Span& a, const Span& b) {
  if (a.ptr == nullptr || b.ptr == nullptr) return false;
  const uintptr_t x = (uintptr_t)a.ptr, y = (uintptr_t)b.ptr;
  return x < y + b.bytes && y < x + a.bytes;
}

// Whether the first `outs` spans overlap neither each other nor the rest.
bool spans_apart(const Span* s, int n, int outs) {
  for (int i = 0; i < outs; ++i)
    for (int j = 0; j < n; ++j)
      if (j != i && spans_meet(s[i], s[j])) return false;
  return true;
}

Span table_span(const llsa_rope_desc* r, const float* table, int rows) {
  return {table, (size_t)rows * r->rot_dim * sizeof(float)};
}

RopeParams rope_params(const llsa_rope_desc* r, int B, int H, int N, int D, const float* table, int table_rows) {
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.table = table;
  p.B = B;
  p.H = H;
  p.N = N;
  p.D = D;
  p.rot = r->rot_dim;
  p.interleaved = r->layout == LLSA_ROPE_INTERLEAVED;
  p.per_batch = table_rows != N;
  p.sign = 1.f;
  return p;
}

// -------------------------------------------------------------- cross attention
int check_cross(const llsa_cross_desc* d) {
  if (d == nullptr) return LLSA_ERR_INVALID_ARG;
  if (d->B < 1 || d->H < 1 || d->Hkv < 1 || d->N < 1 || d->S < 0 || d->D < 1) return LLSA_ERR_INVALID_ARG;
  if (d->H % d->Hkv != 0 || d->flags != 0) return LLSA_ERR_INVALID_ARG;
  if (d->dtype != LLSA_F32 && d->dtype != LLSA_BF16) return LLSA_ERR_INVALID_ARG;
  if (!(d->sm_scale >= 0.f) || isinf(d->sm_scale)) return LLSA_ERR_INVALID_ARG;
  if (d->D != 64 && d->D != 128) return LLSA_ERR_UNSUPPORTED;
  if ((long long)d->B * d->H > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
  if ((long long)d->B * d->H * d->N > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;    // rows are int32
  if ((long long)d->B * d->Hkv * d->S > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
  return LLSA_OK;
}

struct CrossWs {
  CrossPlan plan;
  // a: O or dQ parts, a2, s: more of dQ's, b: (m, l) or dK parts, c: dV parts
  size_t delta = 0, alone = 0, a = 0, a2 = 0, s = 0, b = 0, c = 0, total = 0;
};

inline size_t take(size_t* off, size_t bytes) {
  const size_t at = *off;
  *off += (bytes + 255) & ~(size_t)255;
  return at;
}

// Query rows of a key head.
inline int rows_per_key_head(const llsa_cross_desc* d) { return d->H / d->Hkv * d->N; }

CrossWs cross_fwd_ws(const llsa_cross_desc* d) {
  CrossWs w;
  const long long BH = (long long)d->B * d->Hkv;
  w.plan = d->dtype == LLSA_BF16 ? cross_tc_fwd_plan(BH, rows_per_key_head(d), d->S, d->D)
                                 : cross_simt_fwd_plan(BH, rows_per_key_head(d), d->S);
  const size_t rows = (size_t)d->B * d->H * d->N;
  if (w.plan.nks > 1) {
    w.a = take(&w.total, w.plan.nks * rows * d->D * sizeof(float));
    w.b = take(&w.total, w.plan.nks * rows * sizeof(float2));
  }
  return w;
}

CrossWs cross_bwd_ws(const llsa_cross_desc* d) {
  CrossWs w;
  const bool tc = d->dtype == LLSA_BF16;
  const long long BH = (long long)d->B * d->Hkv;
  w.plan = (tc ? cross_tc_bwd_plan : cross_simt_bwd_plan)(BH, rows_per_key_head(d), d->S);
  const size_t rows = (size_t)d->B * d->H * d->N;
  // keys, in whole tiles where the parts are
  const size_t keys = (size_t)BH * (tc ? ((size_t)d->S + 127) / 128 * 128 : (size_t)d->S);
  if (tc) {  // what the first pass leaves the second
    w.delta = take(&w.total, rows * sizeof(float));
    w.alone = take(&w.total, (size_t)d->B * sizeof(int32_t));
  }
  if (w.plan.nks > 1) {
    w.a = take(&w.total, w.plan.nks * rows * d->D * sizeof(float));
    if (tc) {
      w.a2 = take(&w.total, w.plan.nks * rows * d->D * sizeof(float));
      w.s = take(&w.total, w.plan.nks * rows * sizeof(float4));
    }
  }
  if (w.plan.nz > 1) {
    w.b = take(&w.total, w.plan.nz * keys * d->D * sizeof(float));
    w.c = take(&w.total, w.plan.nz * keys * d->D * sizeof(float));
  }
  return w;
}

// A bf16 [heads, rows, D] tensor seen by TMA as boxes of `box_rows` rows
// x 64 columns (128 bytes) of one head with 128-byte swizzle; rows past a head's
// last read as zeros and are not written.
int make_head_map(CUtensorMap* map, const void* ptr, long long heads, int rows, int D, int box_rows) {
  EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return LLSA_ERR_LAUNCH;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)rows * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  const cuuint32_t estride[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estride,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? LLSA_OK : LLSA_ERR_LAUNCH;
}

// Maps of n tensors of the queries' rows.
int make_query_maps(CUtensorMap* maps, const llsa_cross_desc* d, const void* const* tensors, int n, int box_rows) {
  for (int i = 0; i < n; ++i) {
    const int st = make_head_map(&maps[i], tensors[i], (long long)d->B * d->Hkv, rows_per_key_head(d), d->D, box_rows);
    if (st != LLSA_OK) return st;
  }
  return LLSA_OK;
}

// Maps of K and V.  Without keys they are never read: q stands in.
int make_key_maps(CUtensorMap* maps, const llsa_cross_desc* d, const void* k, const void* v, const void* q,
                  int box_rows) {
  const void* const tensors[2] = {d->S > 0 ? k : q, d->S > 0 ? v : q};
  for (int i = 0; i < 2; ++i) {
    const int st = make_head_map(&maps[i], tensors[i], (long long)d->B * d->Hkv, d->S > 0 ? d->S : 1, d->D, box_rows);
    if (st != LLSA_OK) return st;
  }
  return LLSA_OK;
}

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return LLSA_OK;
  if (ws == nullptr || !aligned(ws, 256)) return LLSA_ERR_INVALID_ARG;
  return ws_bytes < need ? LLSA_ERR_WORKSPACE : LLSA_OK;
}

CrossParams cross_params(const llsa_cross_desc* d, const void* q, const void* k, const void* v,
                         const int32_t* kv_len, const uint8_t* mask, int32_t* status, const CrossPlan& plan) {
  CrossParams p;
  memset(&p, 0, sizeof(p));
  p.q = q;
  p.k = k;
  p.v = v;
  p.kv_len = kv_len;
  p.mask = mask;
  p.status = status;
  p.B = d->B;
  p.H = d->Hkv;
  p.N = rows_per_key_head(d);
  p.S = d->S;
  p.D = d->D;
  p.nks = plan.nks;
  p.nz = plan.nz;
  p.scale = d->sm_scale > 0.f ? d->sm_scale : 1.0f / sqrtf((float)d->D);
  return p;
}

}  // namespace

extern "C" {

int llsa_rope_table(const llsa_rope_desc* rope, int rows, const int32_t* pos, float* table, void* stream) {
  const int st = check_rope(rope);
  if (st != LLSA_OK) return st;
  if (rows < 1 || table == nullptr || !aligned(table, 16) || !aligned(pos, 4)) return LLSA_ERR_INVALID_ARG;
  if (spans_meet(table_span(rope, table, rows), {pos, (size_t)rows * rope->axes * sizeof(int32_t)}))
    return LLSA_ERR_INVALID_ARG;
  return launch_status(launch_rope_table(rope_freqs(rope), rows, pos, table, (cudaStream_t)stream));
}

int llsa_rope(const llsa_rope_desc* rope, int B, int H, int N, int D, int dtype, const float* table, int table_rows,
              const void* q, const void* k, void* q_out, void* k_out, int adjoint, void* stream) {
  const int st = check_rope(rope);
  if (st != LLSA_OK) return st;
  if (B < 1 || H < 1 || N < 1 || D < 1) return LLSA_ERR_INVALID_ARG;
  if (dtype != LLSA_F32 && dtype != LLSA_BF16) return LLSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return LLSA_ERR_UNSUPPORTED;
  if ((long long)H * 2 > 0x7fffffffLL || (long long)B * H > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
  if (rope->rot_dim > D) return LLSA_ERR_INVALID_ARG;
  if (table == nullptr || q == nullptr || q_out == nullptr || (k == nullptr) != (k_out == nullptr))
    return LLSA_ERR_INVALID_ARG;
  if (table_rows != N && (long long)table_rows != (long long)B * N) return LLSA_ERR_INVALID_ARG;
  if (!aligned(table, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16))
    return LLSA_ERR_INVALID_ARG;
  const size_t bytes = (size_t)B * H * N * D * (dtype == LLSA_BF16 ? 2 : 4);
  const int nt = k != nullptr ? 2 : 1;
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  if (!outputs_apart(in, nt, out, nt, bytes)) return LLSA_ERR_INVALID_ARG;
  for (int t = 0; t < nt; ++t)
    if (spans_meet({out[t], bytes}, table_span(rope, table, table_rows))) return LLSA_ERR_INVALID_ARG;
  RopeParams p = rope_params(rope, B, H, N, D, table, table_rows);
  for (int t = 0; t < nt; ++t) {
    p.x[t] = in[t];
    p.y[t] = out[t];
  }
  p.ntensor = nt;
  p.sign = adjoint != 0 ? -1.f : 1.f;
  return launch_status(launch_rope(p, dtype, (cudaStream_t)stream));
}

int llsa_rope_pool(const llsa_desc* desc, const llsa_rope_desc* rope, const float* table, int table_rows,
                   const void* q, const void* k, const void* v, void* q_out, void* k_out, const llsa_pyramid* out,
                   void* stream) {
  int st = check_desc(desc);
  if (st == LLSA_OK) st = check_rope(rope);
  if (st != LLSA_OK) return st;
  if (rope->rot_dim > desc->D) return LLSA_ERR_INVALID_ARG;
  if (table == nullptr || q == nullptr || k == nullptr || v == nullptr || q_out == nullptr || k_out == nullptr ||
      out == nullptr)
    return LLSA_ERR_INVALID_ARG;
  if (table_rows != desc->N && (long long)table_rows != (long long)desc->B * desc->N) return LLSA_ERR_INVALID_ARG;
  const void* all[6] = {table, q, k, v, q_out, k_out};
  for (const void* ptr : all)
    if (!aligned(ptr, 16)) return LLSA_ERR_INVALID_ARG;
  for (int l = 1; l <= desc->L; ++l) {
    if (out->q[l] == nullptr || out->k[l] == nullptr) return LLSA_ERR_INVALID_ARG;
    if (l >= 2 && out->v[l] == nullptr) return LLSA_ERR_INVALID_ARG;
    if (!aligned(out->q[l], 16) || !aligned(out->k[l], 16)) return LLSA_ERR_INVALID_ARG;
  }
  const size_t bytes = (size_t)desc->B * desc->H * desc->N * desc->D * (desc->dtype == LLSA_BF16 ? 2 : 4);
  const void* in[3] = {q, k, v};
  void* rot[2] = {q_out, k_out};
  if (!outputs_apart(in, 3, rot, 2, bytes)) return LLSA_ERR_INVALID_ARG;
  // the pyramid apart from itself, the tensors and the table, the rotated tensors from the table
  Span spans[3 * LLSA_MAX_LEVELS + 6];
  int n = 0;
  size_t level = (size_t)desc->B * desc->H * desc->N * desc->D * sizeof(float);
  for (int l = 1; l <= desc->L; ++l) {
    level /= kBlock;
    spans[n++] = {out->q[l], level};
    spans[n++] = {out->k[l], level};
    if (l >= 2) spans[n++] = {out->v[l], level};
  }
  const int levels = n;
  const Span tab = table_span(rope, table, table_rows);
  spans[n++] = tab;
  for (const void* ptr : {q, k, v, (const void*)q_out, (const void*)k_out}) spans[n++] = {ptr, bytes};
  if (!spans_apart(spans, n, levels)) return LLSA_ERR_INVALID_ARG;
  for (const void* ptr : rot)
    if (spans_meet({ptr, bytes}, tab)) return LLSA_ERR_INVALID_ARG;
  RopeParams p = rope_params(rope, desc->B, desc->H, desc->N, desc->D, table, table_rows);
  PoolParams o;
  memset(&o, 0, sizeof(o));
  for (int t = 0; t < 3; ++t) p.x[t] = in[t];
  for (int t = 0; t < 2; ++t) p.y[t] = rot[t];
  p.ntensor = 2;
  for (int l = 1; l <= desc->L; ++l) {
    o.lvl[0][l] = out->q[l];
    o.lvl[1][l] = out->k[l];
    o.lvl[2][l] = l >= 2 ? out->v[l] : nullptr;
  }
  o.BH = desc->B * desc->H;
  o.N = desc->N;
  o.D = desc->D;
  o.L = desc->L;
  const cudaStream_t s = (cudaStream_t)stream;
  if (rope_pool_fused(rope->rot_dim, p.interleaved != 0, desc->dtype))
    return launch_status(launch_rope_pool(p, o, desc->dtype, s));
  // pairs that straddle the 16-byte chunks: the two calls one after the other
  const cudaError_t e = launch_rope(p, desc->dtype, s);
  if (e != cudaSuccess) return LLSA_ERR_LAUNCH;
  o.x[0] = q_out;
  o.x[1] = k_out;
  o.x[2] = v;
  return launch_status(launch_pool(o, desc->dtype, s));
}

size_t llsa_cross_fwd_workspace_bytes(const llsa_cross_desc* desc) {
  return check_cross(desc) == LLSA_OK ? cross_fwd_ws(desc).total : 0;
}

size_t llsa_cross_bwd_workspace_bytes(const llsa_cross_desc* desc) {
  return check_cross(desc) == LLSA_OK ? cross_bwd_ws(desc).total : 0;
}

int llsa_cross_attn_fwd(const llsa_cross_desc* desc, const void* q, const void* k, const void* v,
                        const int32_t* kv_len, const uint8_t* key_mask, void* o, void* o_res, float* lse, void* ws,
                        size_t ws_bytes, int32_t* dev_status, void* stream) {
  int st = check_cross(desc);
  if (st != LLSA_OK) return st;
  if (q == nullptr || o == nullptr || lse == nullptr) return LLSA_ERR_INVALID_ARG;
  if (desc->S > 0 && (k == nullptr || v == nullptr)) return LLSA_ERR_INVALID_ARG;
  const void* ptrs[5] = {q, k, v, o, o_res};
  for (const void* ptr : ptrs)
    if (!aligned(ptr, 16)) return LLSA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(kv_len, 4)) return LLSA_ERR_INVALID_ARG;
  const CrossWs w = cross_fwd_ws(desc);
  st = check_ws(ws, ws_bytes, w.total);
  if (st != LLSA_OK) return st;
  const size_t e = desc->dtype == LLSA_BF16 ? 2 : 4, rows = (size_t)desc->B * desc->H * desc->N;
  const size_t qb = rows * desc->D * e, kb = (size_t)desc->B * desc->Hkv * desc->S * desc->D * e;
  const Span spans[] = {{o, qb}, {desc->dtype == LLSA_BF16 ? o_res : nullptr, qb}, {lse, rows * 4}, {ws, w.total},
                        {q, qb}, {k, kb}, {v, kb}, {kv_len, (size_t)desc->B * 4}, {key_mask, (size_t)desc->B * desc->S}};
  if (!spans_apart(spans, 9, 4)) return LLSA_ERR_INVALID_ARG;
  CrossParams p = cross_params(desc, q, k, v, kv_len, key_mask, dev_status, w.plan);
  p.o = o;
  p.o_res = desc->dtype == LLSA_BF16 ? o_res : nullptr;
  p.lse = lse;
  char* base = static_cast<char*>(ws);
  if (p.nks > 1) {
    p.part_o = reinterpret_cast<float*>(base + w.a);
    p.part_ml = reinterpret_cast<float2*>(base + w.b);
  }
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t err;
  if (desc->dtype == LLSA_BF16) {
    CUtensorMap qo[2], kv[2];
    const void* const rows_of[2] = {q, o};
    st = make_query_maps(qo, desc, rows_of, 2, 128);
    if (st == LLSA_OK) st = make_key_maps(kv, desc, k, v, q, desc->D == 64 ? 64 : 128);
    if (st != LLSA_OK) return st;
    const CUtensorMap maps[4] = {qo[0], kv[0], kv[1], qo[1]};
    err = launch_cross_fwd_tc(p, maps, s);
  } else {
    err = launch_cross_fwd_simt(p, s);
  }
  if (err == cudaSuccess && p.nks > 1) err = launch_cross_combine(p, desc->dtype, s);
  return launch_status(err);
}

int llsa_cross_attn_bwd(const llsa_cross_desc* desc, const void* q, const void* k, const void* v,
                        const int32_t* kv_len, const uint8_t* key_mask, const void* o, const void* o_res,
                        const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                        int32_t* dev_status, void* stream) {
  int st = check_cross(desc);
  if (st != LLSA_OK) return st;
  if (q == nullptr || o == nullptr || lse == nullptr || dout == nullptr || dq == nullptr) return LLSA_ERR_INVALID_ARG;
  if (desc->S > 0 && (k == nullptr || v == nullptr || dk == nullptr || dv == nullptr)) return LLSA_ERR_INVALID_ARG;
  const void* ptrs[9] = {q, k, v, o, o_res, dout, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!aligned(ptr, 16)) return LLSA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(kv_len, 4)) return LLSA_ERR_INVALID_ARG;
  // the second pass forms lse / sm_scale, which must not pass fp32
  if (desc->dtype == LLSA_BF16 && desc->sm_scale > 0.f && desc->sm_scale < 0x1p-120f) return LLSA_ERR_UNSUPPORTED;
  const CrossWs w = cross_bwd_ws(desc);
  st = check_ws(ws, ws_bytes, w.total);
  if (st != LLSA_OK) return st;
  const size_t rows = (size_t)desc->B * desc->H * desc->N, keys = (size_t)desc->B * desc->Hkv * desc->S;
  const size_t item = desc->dtype == LLSA_BF16 ? 2 : 4, qb = rows * desc->D * item, kb = keys * desc->D * item;
  const Span spans[] = {{dq, qb}, {dk, kb}, {dv, kb}, {ws, w.total}, {q, qb}, {k, kb}, {v, kb}, {o, qb},
                        {desc->dtype == LLSA_BF16 ? o_res : nullptr, qb}, {lse, rows * 4}, {dout, qb},
                        {kv_len, (size_t)desc->B * 4}, {key_mask, (size_t)desc->B * desc->S}};
  if (!spans_apart(spans, 13, 4)) return LLSA_ERR_INVALID_ARG;
  CrossParams p = cross_params(desc, q, k, v, kv_len, key_mask, dev_status, w.plan);
  p.o_in = o;
  p.lse_in = lse;
  p.dout = dout;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  char* base = static_cast<char*>(ws);
  if (desc->dtype == LLSA_BF16) {
    p.delta = reinterpret_cast<float*>(base + w.delta);
    p.alone = reinterpret_cast<int32_t*>(base + w.alone);
  }
  if (p.nks > 1) {
    p.part_dq = reinterpret_cast<float*>(base + w.a);
    p.part_dqb = reinterpret_cast<float*>(base + w.a2);
    p.part_s = reinterpret_cast<float4*>(base + w.s);
  }
  if (p.nz > 1) {
    p.part_dk = reinterpret_cast<float*>(base + w.b);
    p.part_dv = reinterpret_cast<float*>(base + w.c);
  }
  const cudaStream_t s = (cudaStream_t)stream;
  if (desc->dtype == LLSA_BF16) {
    CUtensorMap q128[3], q64[2], kv128[2], kv64[2];
    const void* const rows_of[3] = {q, dout, dq};
    st = make_query_maps(q128, desc, rows_of, 3, 128);
    if (st == LLSA_OK) st = make_query_maps(q64, desc, rows_of, 2, 64);
    if (st == LLSA_OK) st = make_key_maps(kv128, desc, k, v, q, 128);
    if (st == LLSA_OK) st = make_key_maps(kv64, desc, k, v, q, 64);
    if (st != LLSA_OK) return st;
    return launch_status(launch_cross_bwd_tc(p, q128, kv64, kv128, q64, s));
  }
  return launch_status(launch_cross_bwd_simt(p, s));
}

}  // extern "C"
