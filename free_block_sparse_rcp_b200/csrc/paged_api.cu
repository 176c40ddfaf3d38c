// C ABI of the rotary positions and the paged K/V cache: argument checks, workspace layout and
// the launches of each call.
#include <math.h>
#include <stdio.h>

#include "kernels.h"
#include "paged.cuh"

using namespace spr;

namespace {

sparsepr_status fail(sparsepr_status s, const char* msg) {
  set_last_error(msg);
  return s;
}
sparsepr_status failv(sparsepr_status s, const char* msg, long long v) {
  char buf[256];
  snprintf(buf, sizeof(buf), "%s (got %lld)", msg, v);
  set_last_error(buf);
  return s;
}
sparsepr_status fail_cuda(cudaError_t e, const char* where) {
  char buf[256];
  snprintf(buf, sizeof(buf), "CUDA error in %s: %s", where, cudaGetErrorString(e));
  set_last_error(buf);
  return SPARSEPR_ECUDA;
}

#define SPR_CHECK(expr)                          \
  do {                                           \
    sparsepr_status s_ = (expr);                 \
    if (s_ != SPARSEPR_OK) return s_;            \
  } while (0)
#define SPR_NONNULL(ptr)                                                                  \
  do {                                                                                    \
    if (!(ptr)) return fail(SPARSEPR_EINVAL, "required pointer " #ptr " is NULL");        \
  } while (0)
#define SPR_ALIGNED(ptr, n)                                                               \
  do {                                                                                    \
    SPR_NONNULL(ptr);                                                                     \
    if ((uintptr_t)(ptr) & ((n) - 1u)) return fail(SPARSEPR_EINVAL, "tensor " #ptr " is not " #n "-byte aligned"); \
  } while (0)

constexpr long long kMaxInt = 0x7fffffffll;

// ---------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------
// the fields that sparsepr_cache_append reads too
sparsepr_status check_rotation(const sparsepr_rope_params* p) {
  if (!p) return fail(SPARSEPR_EINVAL, "rope params pointer is NULL");
  if (p->rot_dim < 2 || p->rot_dim > p->d || p->rot_dim % 2)
    return failv(SPARSEPR_EINVAL, "rot_dim must be even and in [2, d]", p->rot_dim);
  if (p->layout != 0 && p->layout != 1) return failv(SPARSEPR_EINVAL, "layout must be 0 or 1", p->layout);
  if (p->n_axes < 1 || p->n_axes > 3) return failv(SPARSEPR_EINVAL, "n_axes must be in [1, 3]", p->n_axes);
  long long sum = 0;
  for (int i = 0; i < p->n_axes; ++i) {
    if (p->axis_dim[i] < 2 || p->axis_dim[i] % 2)
      return failv(SPARSEPR_EINVAL, "axis_dim must be even and >= 2", p->axis_dim[i]);
    sum += p->axis_dim[i];
  }
  if (sum != p->rot_dim) return failv(SPARSEPR_EINVAL, "axis_dim must sum to rot_dim", sum);
  if (p->scaling < 0 || p->scaling > 3) return failv(SPARSEPR_EINVAL, "scaling must be in [0, 3]", p->scaling);
  if (!(p->theta > 0.0) || !isfinite(p->theta)) return fail(SPARSEPR_EINVAL, "theta must be > 0");
  if (!(p->factor > 0.0) || !isfinite(p->factor)) return fail(SPARSEPR_EINVAL, "factor must be > 0");
  if (p->scaling == 3) {
    if (p->orig_len < 1) return failv(SPARSEPR_EINVAL, "orig_len must be >= 1 with scaling 3", p->orig_len);
    if (!(p->beta_slow > 0.0) || !(p->beta_fast > p->beta_slow) || !isfinite(p->beta_fast))
      return fail(SPARSEPR_EINVAL, "scaling 3 needs beta_fast > beta_slow > 0");
    if (!(p->theta > 1.0)) return fail(SPARSEPR_EINVAL, "scaling 3 needs theta > 1");
  }
  if (!isfinite(p->magnitude) || p->magnitude < 0.0) return fail(SPARSEPR_EINVAL, "magnitude must be >= 0");
  return SPARSEPR_OK;
}

bool all_zero(const long long* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] != 0) return false;
  return true;
}

// Output strides: distinct elements of a dimension longer than one must not share an address.
sparsepr_status check_rope(const sparsepr_rope_params* p) {
  if (!p) return fail(SPARSEPR_EINVAL, "rope params pointer is NULL");
  if (p->B < 1 || p->H < 1 || p->N < 0 || p->H2 < 0) return fail(SPARSEPR_EINVAL, "B and H must be >= 1, N and H2 >= 0");
  if (p->d < 2 || p->d > 512) return failv(SPARSEPR_EINVAL, "head dim d must be in [2, 512]", p->d);
  if (p->dtype < SPARSEPR_BF16 || p->dtype > SPARSEPR_FP32) return failv(SPARSEPR_EINVAL, "unknown dtype", p->dtype);
  if (p->pos_batched != 0 && p->pos_batched != 1) return failv(SPARSEPR_EINVAL, "pos_batched must be 0 or 1", p->pos_batched);
  if ((long long)p->B * p->N > kMaxInt) return fail(SPARSEPR_EUNSUPPORTED, "B*N too large");
  if ((long long)p->H + p->H2 > 65535) return fail(SPARSEPR_EUNSUPPORTED, "more than 65535 heads");
  SPR_CHECK(check_rotation(p));
  for (int t = 0; t < 2; ++t) {
    const long long* y = t ? p->y2_stride : p->y_stride;
    const int n[3] = {p->B, t ? p->H2 : p->H, p->N};
    if ((t && p->H2 == 0) || all_zero(y, 3)) continue;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && y[i] == 0) return fail(SPARSEPR_EINVAL, "an output stride is 0");
  }
  return SPARSEPR_OK;
}

double rope_magnitude(const sparsepr_rope_params& p) {
  if (p.magnitude > 0.0) return p.magnitude;
  return p.scaling == 3 && p.factor > 1.0 ? 0.1 * log(p.factor) + 1.0 : 1.0;
}

void rope_strides(const sparsepr_rope_params& p, int heads, const long long* s, long long* out) {
  if (all_zero(s, 3)) {
    out[0] = (long long)heads * p.N * p.d;
    out[1] = (long long)p.N * p.d;
    out[2] = p.d;
  } else {
    for (int i = 0; i < 3; ++i) out[i] = s[i];
  }
}

sparsepr_status run_rope(const sparsepr_rope_params* p, const void* x, const int* pos, const double* freq, void* y,
                         const void* x2, void* y2, bool backward, void* stream) {
  set_launch_count(0);
  SPR_CHECK(check_rope(p));
  if (p->N == 0) return SPARSEPR_OK;
  const int es = p->dtype == SPARSEPR_FP32 ? 4 : 2;
  RopeArgs a{};
  a.x[0] = x; a.y[0] = y; a.x[1] = x2; a.y[1] = y2;
  a.H[0] = p->H; a.H[1] = p->H2;
  a.B = p->B; a.N = p->N; a.d = p->d; a.rot = p->rot_dim; a.layout = p->layout; a.n_axes = p->n_axes;
  for (int i = 0; i < 3; ++i) a.axis_pairs[i] = i < p->n_axes ? p->axis_dim[i] / 2 : 0;
  a.pos_batched = p->pos_batched; a.dtype = p->dtype;
  a.mag = (float)rope_magnitude(*p);
  a.sign = backward ? -1.f : 1.f;
  SPR_NONNULL(pos);
  SPR_NONNULL(freq);
  a.pos = pos; a.freq = freq;
  a.vec = p->d * es % 16 == 0;
  for (int t = 0; t < (p->H2 ? 2 : 1); ++t) {
    if (!a.x[t] || !a.y[t]) return fail(SPARSEPR_EINVAL, t ? "the second tensor is NULL" : "the tensor is NULL");
    rope_strides(*p, a.H[t], t ? p->x2_stride : p->x_stride, a.xs[t]);
    rope_strides(*p, a.H[t], t ? p->y2_stride : p->y_stride, a.ys[t]);
    if (((uintptr_t)a.x[t] | (uintptr_t)a.y[t]) & (es - 1)) return fail(SPARSEPR_EINVAL, "a tensor is not aligned to its elements");
    if (a.x[t] == a.y[t])
      for (int i = 0; i < 3; ++i)
        if (a.xs[t][i] != a.ys[t][i]) return fail(SPARSEPR_EINVAL, "in place needs equal strides");
    if (((uintptr_t)a.x[t] | (uintptr_t)a.y[t]) & 15u) a.vec = false;
    for (int i = 0; i < 3; ++i)
      if (a.xs[t][i] * es % 16 || a.ys[t][i] * es % 16) a.vec = false;
  }
  const cudaError_t e = launch_rope(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "launch_rope");
  set_launch_count(1);
  return SPARSEPR_OK;
}

// ---------------------------------------------------------------------------
// Paged cache
// ---------------------------------------------------------------------------
sparsepr_status check_cache(const sparsepr_cache_params* p) {
  if (!p) return fail(SPARSEPR_EINVAL, "params pointer is NULL");
  if (p->B < 1 || p->B > 65536) return failv(SPARSEPR_EINVAL, "B must be in [1, 65536]", p->B);
  if (p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv) return fail(SPARSEPR_EINVAL, "Hkv must divide Hq (both >= 1)");
  if (p->Hq > 4096) return failv(SPARSEPR_EUNSUPPORTED, "more than 4096 query heads", p->Hq);
  if (p->d != 64 && p->d != 128) return failv(SPARSEPR_EUNSUPPORTED, "head dim d must be 64 or 128", p->d);
  if (p->dtype != SPARSEPR_BF16 && p->dtype != SPARSEPR_FP16)
    return failv(SPARSEPR_EUNSUPPORTED, "the cache holds bf16 or fp16", p->dtype);
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128)
    return failv(SPARSEPR_EUNSUPPORTED, "page must be 16, 32, 64 or 128", p->page);
  if (p->n_pages < 1 || p->max_pages < 1) return fail(SPARSEPR_EINVAL, "n_pages and max_pages must be >= 1");
  if ((long long)p->max_pages * p->page > (1ll << 30)) return fail(SPARSEPR_EUNSUPPORTED, "max_pages * page above 2^30");
  if ((long long)p->n_pages * p->Hkv * p->page > kMaxInt) return fail(SPARSEPR_EUNSUPPORTED, "page pool above 2^31 rows");
  if (p->T < 0 || (long long)p->T * p->Hq > kMaxInt) return fail(SPARSEPR_EINVAL, "T must be >= 0 and T * Hq below 2^31");
  if (p->max_chunk < 1) return failv(SPARSEPR_EINVAL, "max_chunk must be >= 1", p->max_chunk);
  if (p->frame < 0) return failv(SPARSEPR_EINVAL, "frame must be >= 0", p->frame);
  if (!(p->scale >= 0.f) || !isfinite(p->scale)) return fail(SPARSEPR_EINVAL, "scale must be >= 0");
  if (p->n_select < 0) return failv(SPARSEPR_EINVAL, "n_select must be >= 0", p->n_select);
  if (p->n_select > 0) {
    if (p->q_block < 1) return failv(SPARSEPR_EINVAL, "q_block must be >= 1 with a selection", p->q_block);
    if (p->n_sink < 0 || p->n_recent < 0 || (long long)p->n_sink + p->n_recent > p->n_select)
      return fail(SPARSEPR_EINVAL, "n_sink and n_recent must be >= 0 and fit in n_select");
    if ((long long)p->n_select * p->page > (1ll << 30)) return fail(SPARSEPR_EUNSUPPORTED, "n_select * page above 2^30");
  }
  const long long* st[4] = {p->q_stride, p->o_stride, p->k_stride, p->v_stride};
  for (int i = 0; i < 4; ++i)
    if (st[i][0] % 8 || st[i][1] % 8) return fail(SPARSEPR_EINVAL, "token and head strides must be multiples of 8 elements");
  const int n[2] = {p->T, p->Hq};
  if (!all_zero(p->o_stride, 2))
    for (int i = 0; i < 2; ++i)
      if (n[i] > 1 && p->o_stride[i] == 0) return fail(SPARSEPR_EINVAL, "an output stride is 0");
  return SPARSEPR_OK;
}

void strides2(const long long* s, int heads, int d, long long& t, long long& h) {
  if (s[0] == 0 && s[1] == 0) {
    t = (long long)heads * d;
    h = d;
  } else {
    t = s[0];
    h = s[1];
  }
}

PagedPlan plan_of(const sparsepr_cache_params& p, bool sel) {
  return paged_plan(p.B, p.Hq, p.Hkv, p.page, p.max_pages, p.T, p.max_chunk, p.q_block, p.n_select, sel);
}

int select_units(const sparsepr_cache_params& p) {
  const long long u = ((long long)p.T + (p.q_block - 1ll) * p.B) / p.q_block;   // sum of ceil(n / q_block)
  return (int)(u < p.T ? u : p.T);
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
  size_t part_lse, part_o, plan, plan_seq, plan_item, plan_pre, scores, bounds, keys, qbar, info, total;
};
Layout layout_of(const sparsepr_cache_params& p) {
  Layout L{};
  size_t o = 256;   // error word
  auto take = [&](size_t bytes) { const size_t at = o; o = al256(o + bytes); return at; };
  // partial results: the pieces of cut items (rows kernel), or two pieces per CTA (tile kernel)
  size_t rows = 0, items = 0;
  for (int sel = 0; sel <= (p.n_select > 0 ? 1 : 0); ++sel) {
    const PagedPlan pl = plan_of(p, sel != 0);
    size_t r = 2ull * kPlanCtas * kPagedTileRows;
    if (pl.rows && pl.kind == paged::kUnits) r = pl.S > 1 ? (size_t)pl.items * p.Hkv * pl.S * 16 * pl.mt : 0;
    if (pl.rows && pl.kind == paged::kWhole) r = (size_t)pl.S * 16 * pl.mt;
    rows = r > rows ? r : rows;
    if (!pl.rows && (size_t)pl.items > items) items = pl.items;
  }
  L.part_lse = take(rows * 4);
  L.part_o = take(rows * p.d * 4);
  L.plan = take(items ? tiles_plan_head_bytes() : 0);
  L.plan_seq = take(items ? (p.B + 1ull) * 4 : 0);
  L.plan_item = take(items * 4);
  L.plan_pre = take(items * p.Hkv * 8);
  // selection: scores of split lists, of units scored together and of lists too long for shared memory,
  // and the latter's 64-bit keys (a batch of lists at a time)
  size_t scores = 0, bounds = 0, keys = 0, qbar = 0, info = 0;
  if (p.n_select > 0) {
    const size_t lists = (size_t)select_units(p) * p.Hkv;
    const SelectPlan sp = select_plan(select_units(p), p.Hkv, p.max_pages, p.B);
    const size_t held = sp.group ? lists : (size_t)sp.bu * sp.bh;
    if (sp.splits > 1 || sp.keys_global || sp.group) scores = held * p.max_pages * 4;
    bounds = held * sp.splits * 4;
    if (sp.keys_global) keys = (size_t)sp.bv * sp.bh * p.max_pages * 8;
    if (sp.group) {
      qbar = lists * p.d * 8;
      info = (size_t)select_units(p) * 8;
    }
  }
  L.scores = take(scores);
  L.bounds = take(bounds);
  L.keys = take(keys);
  L.qbar = take(qbar);
  L.info = take(info);
  L.total = o;
  return L;
}

sparsepr_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return fail(SPARSEPR_EINVAL, "workspace is NULL");
  if ((uintptr_t)ws & 255u) return fail(SPARSEPR_EWORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return failv(SPARSEPR_EWORKSPACE, "workspace too small (bytes needed)", (long long)need);
  return SPARSEPR_OK;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

}  // namespace

extern "C" {

sparsepr_status sparsepr_rope_validate(const sparsepr_rope_params* p) { return check_rope(p); }

sparsepr_status sparsepr_rope_frequencies(const sparsepr_rope_params* p, double* freq_host) {
  if (!p) return fail(SPARSEPR_EINVAL, "rope params pointer is NULL");
  SPR_CHECK(check_rotation(p));
  SPR_NONNULL(freq_host);
  const double two_pi = 6.283185307179586476925286766559;
  int at = 0;
  for (int ax = 0; ax < p->n_axes; ++ax) {
    const int dim = p->axis_dim[ax];
    double base = p->theta;
    if (p->scaling == 2 && dim > 2) base *= pow(p->factor, dim / (dim - 2.0));
    // scaling 3: the pairs that turn beta_fast and beta_slow times within orig_len.  The ramp may end
    // behind the last pair (dim / 2 - 1), which then keeps a share of its frequency: with theta 10,000
    // the slowest pair still turns once within 54,000 positions or more.
    double lo = 0.0, hi = 0.0;
    if (p->scaling == 3) {
      auto pair_of = [&](double turns) { return dim * log(p->orig_len / (turns * two_pi)) / (2.0 * log(p->theta)); };
      lo = fmax(floor(pair_of(p->beta_fast)), 0.0);
      hi = fmin(ceil(pair_of(p->beta_slow)), dim - 1.0);
    }
    for (int j = 0; j < dim / 2; ++j) {
      double w = pow(base, -2.0 * j / dim);
      if (p->scaling == 1) w /= p->factor;
      if (p->scaling == 3) {
        const double ramp = fmin(fmax((j - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
        w = w * (1.0 - ramp) + w / p->factor * ramp;
      }
      freq_host[at++] = w / two_pi;
    }
  }
  return SPARSEPR_OK;
}

sparsepr_status sparsepr_rope(const sparsepr_rope_params* p, const void* x, const int* pos, const double* freq, void* y,
                              const void* x2, void* y2, void* stream) {
  return run_rope(p, x, pos, freq, y, x2, y2, false, stream);
}

sparsepr_status sparsepr_rope_backward(const sparsepr_rope_params* p, const void* dy, const int* pos,
                                       const double* freq, void* dx, const void* dy2, void* dx2, void* stream) {
  return run_rope(p, dy, pos, freq, dx, dy2, dx2, true, stream);
}

sparsepr_status sparsepr_cache_validate(const sparsepr_cache_params* p) { return check_cache(p); }

size_t sparsepr_paged_workspace_bytes(const sparsepr_cache_params* p) {
  if (check_cache(p) != SPARSEPR_OK) return 0;
  return layout_of(*p).total;
}

sparsepr_status sparsepr_cache_append(const sparsepr_cache_params* p, const void* K, const void* V, const int* q_start,
                                      const int* kv_len, const int* page_table, void* k_pages, void* v_pages,
                                      void* k_mean, const sparsepr_rope_params* rope, const int* pos,
                                      const double* rope_freq, void* workspace, size_t ws_bytes, void* stream) {
  set_launch_count(0);
  SPR_CHECK(check_cache(p));
  AppendArgs a{};
  if (rope) {
    if (rope->d != p->d) return failv(SPARSEPR_EINVAL, "rope d differs from the cache's", rope->d);
    SPR_CHECK(check_rotation(rope));
    SPR_NONNULL(pos);
    SPR_NONNULL(rope_freq);
    a.pos = pos; a.freq = rope_freq;
    a.rot = rope->rot_dim; a.layout = rope->layout; a.n_axes = rope->n_axes;
    for (int i = 0; i < 3; ++i) a.axis_pairs[i] = i < rope->n_axes ? rope->axis_dim[i] / 2 : 0;
    a.mag = (float)rope_magnitude(*rope);
  }
  SPR_CHECK(check_ws(workspace, ws_bytes, 256));
  if (p->T == 0) return SPARSEPR_OK;
  SPR_ALIGNED(K, 16); SPR_ALIGNED(V, 16); SPR_NONNULL(q_start); SPR_NONNULL(kv_len); SPR_NONNULL(page_table);
  SPR_ALIGNED(k_pages, 16); SPR_ALIGNED(v_pages, 16); SPR_ALIGNED(k_mean, 16);
  a.K = K; a.V = V; a.q_start = q_start; a.kv_len = kv_len; a.table = page_table;
  a.kp = k_pages; a.vp = v_pages; a.km = k_mean;
  a.err = at<int>(workspace, 0);
  a.B = p->B; a.Hkv = p->Hkv; a.d = p->d; a.dtype = p->dtype; a.page = p->page; a.n_pages = p->n_pages;
  a.max_pages = p->max_pages; a.T = p->T; a.max_chunk = p->max_chunk;
  strides2(p->k_stride, p->Hkv, p->d, a.kst, a.ksh);
  strides2(p->v_stride, p->Hkv, p->d, a.vst, a.vsh);
  const cudaError_t e = launch_cache_append(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "launch_cache_append");
  set_launch_count(2);
  return SPARSEPR_OK;
}

int sparsepr_select_units(const sparsepr_cache_params* p) {
  if (check_cache(p) != SPARSEPR_OK || p->n_select < 1) return -1;
  return select_units(*p);
}

sparsepr_status sparsepr_page_select(const sparsepr_cache_params* p, const void* Q, const int* q_start,
                                     const int* kv_len, const int* page_table, const void* k_mean, int* sel,
                                     int* sel_count, void* workspace, size_t ws_bytes, void* stream) {
  set_launch_count(0);
  SPR_CHECK(check_cache(p));
  if (p->n_select < 1) return failv(SPARSEPR_EINVAL, "n_select must be >= 1 for a selection", p->n_select);
  const Layout L = layout_of(*p);
  SPR_CHECK(check_ws(workspace, ws_bytes, L.total));
  if (p->T == 0) return SPARSEPR_OK;
  SPR_ALIGNED(Q, 16); SPR_NONNULL(q_start); SPR_NONNULL(kv_len); SPR_NONNULL(page_table); SPR_ALIGNED(k_mean, 16);
  SPR_NONNULL(sel); SPR_NONNULL(sel_count);
  if (p->Hkv > 65535) return failv(SPARSEPR_EUNSUPPORTED, "more than 65535 key/value heads", p->Hkv);
  SelectArgs a{};
  a.p.Q = Q; a.p.q_start = q_start; a.p.kv_len = kv_len; a.p.table = page_table;
  a.p.err = at<int>(workspace, 0);
  a.p.B = p->B; a.p.Hq = p->Hq; a.p.Hkv = p->Hkv; a.p.G = p->Hq / p->Hkv; a.p.page = p->page; a.p.n_pages = p->n_pages;
  a.p.max_pages = p->max_pages; a.p.T = p->T; a.p.max_chunk = p->max_chunk; a.p.frame = p->frame;
  a.p.q_block = p->q_block; a.p.n_select = p->n_select;
  strides2(p->q_stride, p->Hq, p->d, a.p.qst, a.p.qsh);
  a.km = k_mean;
  a.sel = sel; a.cnt = sel_count;
  a.scores = at<float>(workspace, L.scores);
  a.bounds = at<float>(workspace, L.bounds);
  a.keys = at<unsigned long long>(workspace, L.keys);
  a.n_sink = p->n_sink; a.n_recent = p->n_recent;
  a.units = select_units(*p);
  const SelectPlan sp = select_plan(a.units, p->Hkv, p->max_pages, p->B);
  a.splits = sp.splits;
  a.keys_global = sp.keys_global;
  a.group = sp.group;
  a.qbar = at<double>(workspace, L.qbar);
  a.info = at<int2>(workspace, L.info);
  int launches = 0;
  const cudaError_t e = launch_page_select(a, sp, p->d, p->dtype, &launches, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "launch_page_select");
  set_launch_count(launches);
  return SPARSEPR_OK;
}

sparsepr_status sparsepr_paged_attention(const sparsepr_cache_params* p, const void* Q, const int* q_start,
                                         const int* kv_len, const int* page_table, const void* k_pages,
                                         const void* v_pages, const int* sel, const int* sel_count, void* O, float* lse,
                                         void* workspace, size_t ws_bytes, void* stream) {
  set_launch_count(0);
  SPR_CHECK(check_cache(p));
  if ((sel == nullptr) != (sel_count == nullptr)) return fail(SPARSEPR_EINVAL, "sel and sel_count come together");
  if (sel && p->n_select < 1) return failv(SPARSEPR_EINVAL, "a selection needs n_select >= 1", p->n_select);
  const Layout L = layout_of(*p);
  SPR_CHECK(check_ws(workspace, ws_bytes, L.total));
  if (p->T == 0) return SPARSEPR_OK;
  SPR_ALIGNED(Q, 16); SPR_NONNULL(q_start); SPR_NONNULL(kv_len); SPR_NONNULL(page_table);
  SPR_ALIGNED(k_pages, 16); SPR_ALIGNED(v_pages, 16); SPR_ALIGNED(O, 16);
  const PagedPlan pl = plan_of(*p, sel != nullptr);
  paged::Args a{};
  a.Q = Q; a.q_start = q_start; a.kv_len = kv_len; a.table = page_table; a.sel = sel; a.sel_cnt = sel_count;
  a.O = O; a.lse = lse;
  a.part_lse = at<float>(workspace, L.part_lse);
  a.part_o = at<float>(workspace, L.part_o);
  a.plan = at<char>(workspace, L.plan);
  a.plan_seq = at<int>(workspace, L.plan_seq);
  a.plan_item = at<int>(workspace, L.plan_item);
  a.plan_pre = at<long long>(workspace, L.plan_pre);
  a.err = at<int>(workspace, 0);
  a.B = p->B; a.Hq = p->Hq; a.Hkv = p->Hkv; a.G = p->Hq / p->Hkv; a.page = p->page; a.n_pages = p->n_pages;
  a.max_pages = p->max_pages; a.T = p->T; a.max_chunk = p->max_chunk; a.frame = p->frame;
  a.q_block = p->q_block > 0 ? p->q_block : 1;
  a.n_select = p->n_select;
  a.ppu = pl.ppu; a.items = pl.items; a.S = pl.S; a.min_split = pl.min_split;
  a.scale_log2 = (p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->d)) * 1.4426950408889634f;
  strides2(p->q_stride, p->Hq, p->d, a.qst, a.qsh);
  strides2(p->o_stride, p->Hq, p->d, a.ost, a.osh);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = pl.rows ? launch_paged_rows(a, pl, p->d, p->dtype, k_pages, v_pages, st)
                          : launch_paged_tiles(a, pl, p->d, p->dtype, k_pages, v_pages, st);
  if (e != cudaSuccess) return fail_cuda(e, "launch_paged_attention");
  if (pl.rows && pl.S > 1) {
    e = launch_paged_combine(a, pl, p->d, p->dtype, st);
    if (e != cudaSuccess) return fail_cuda(e, "launch_paged_combine");
  }
  set_launch_count(!pl.rows ? 3 : (pl.S > 1 ? 2 : 1));
  return SPARSEPR_OK;
}

int sparsepr_paged_error(const void* workspace, void* stream) {
  if (!workspace) return -1;
  int h = 0;
  cudaStream_t st = (cudaStream_t)stream;
  if (cudaMemcpyAsync(&h, workspace, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess) return -1;
  if (cudaStreamSynchronize(st) != cudaSuccess) return -1;
  return h;
}

sparsepr_status sparsepr_paged_clear_error(void* workspace, void* stream) {
  SPR_NONNULL(workspace);
  const cudaError_t e = cudaMemsetAsync(workspace, 0, 4, (cudaStream_t)stream);
  return e == cudaSuccess ? SPARSEPR_OK : fail_cuda(e, "cudaMemsetAsync");
}

}  // extern "C"
