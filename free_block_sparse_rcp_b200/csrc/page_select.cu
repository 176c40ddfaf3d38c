// Page selection: for every unit (q_block consecutive new tokens of a sequence) and key/value
// head, the pages whose mean key scores best against the unit's mean query.
//
//   score(j) = qbar . kbar_j,   qbar = mean of the unit's query rows over tokens and the query
//   heads of the key/value head; the first n_sink and last n_recent visible pages are kept and
//   the best scores fill the list up to n_select, ties to the lowest page.
//
// The list is decided by comparisons, so the scores are summed in 64 bits: in 32 bits the order
// of the sum would decide between pages closer than 2^-24, and with a thousand pages the pair
// at the border is that close in about one list of 10^4.
// A 16-bit element becomes a double without a conversion instruction (those run at a quarter of
// the double multiply-add rate): its exponent and mantissa are shifted into the double's
// fields, which gives x 2^-kBias exactly (subnormals included), and the other factor, qbar,
// carries 2^kBias.  The range holds: |qbar| <= 65504 for fp16 (2^16 2^1008 = 2^1024 is not
// reached) and 2^128 2^896 = 2^1024 likewise for finite bf16 means.
//
// Work: the means are read once per unit (bytes: 1 / page of the keys'), 2 d operations per
// page; the queries once.  One block per (unit, head), or several that share its pages when
// there are few units; the selection then runs as a second kernel over the stored scores.
#include "paged.cuh"

namespace spr {
namespace {

constexpr int kSelThreads = 256;
constexpr int kSelBins = 2048;
constexpr int kSelSmemPages = 8192;   // scores kept in shared memory up to this many pages (64 KB)

template <typename T>
struct Wide;   // exponent field offset of the shifted 16-bit element
template <>
struct Wide<__nv_bfloat16> {
  static constexpr int shift = 13, bias = 896;       // 1023 - 127
  static constexpr uint32_t inf = 0x7f80u;
};
template <>
struct Wide<__half> {
  static constexpr int shift = 10, bias = 1008;      // 1023 - 15
  static constexpr uint32_t inf = 0x7c00u;
};
// x 2^-bias of a finite 16-bit element
template <typename T>
__device__ __forceinline__ double wide(uint32_t e) {
  return __hiloint2double((int)(((e & 0x7fffu) << Wide<T>::shift) | ((e & 0x8000u) << 16)), 0);
}
template <typename T>
__device__ __forceinline__ bool not_finite(uint32_t w) {   // either half of a packed pair
  return (w & Wide<T>::inf) == Wide<T>::inf || ((w >> 16) & Wide<T>::inf) == Wide<T>::inf;
}
__device__ __forceinline__ double pow2(int e) { return __hiloint2double((1023 + e) << 20, 0); }   // |e| <= 1022

// Order of scores as unsigned integers (larger score, larger key); NaN is the lowest.
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (!(x == x)) return 0ull;
  const long long b = __double_as_longlong(x + 0.0);   // -0 becomes +0
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

struct UnitInfo {
  int b, len, ntok, tok0, vis;   // tok0: packed row of the unit's first token; vis: visible pages
};

__device__ __forceinline__ bool unit_of(const SelectArgs& a, int idx, int* sm, UnitInfo& u) {
  const int2 it = paged::find_item<paged::kUnits, kSelThreads>(a.q_start, a.B, a.T, idx, 1, 1, a.q_block, 1, sm);
  if (it.x < 0) return false;
  u.b = it.x;
  const int q0 = min(max(a.q_start[it.x], 0), a.T);
  const int n = max(0, min(a.q_start[it.x + 1], a.T) - q0);
  const int lenr = a.kv_len[it.x];
  u.len = min(max(lenr, 0), a.max_pages * a.page);
  if (lenr != u.len && threadIdx.x == 0) set_error(a.err, DERR_INDEX);
  const int t0 = it.y * a.q_block;     // < n
  u.ntok = min(a.q_block, n - t0);
  u.tok0 = q0 + t0;
  const int end = paged::visible_end(u.len - n + t0 + u.ntok - 1, a.frame, u.len);
  u.vis = (end + a.page - 1) / a.page;
  return true;
}

// Writes the list of one (unit, head) from its order keys (all threads of the block).
__device__ void select_list(const unsigned long long* keys, int vis, int n_sink, int n_recent, int K, int* out, int* cnt,
                            int* hist /* [kSelBins] */) {
  __shared__ unsigned long long s_lo, s_hi;
  __shared__ int s_warp[kSelThreads / 32], s_tie[kSelThreads / 32], s_bin, s_above, s_inbin;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int f0 = min(n_sink, vis), f1 = max(f0, vis - n_recent);   // free pages [f0, f1)
  const int nfree = f1 - f0;
  const int total = min(K, vis);
  int want = total - (vis - nfree);        // free pages to take (>= 0: kept pages fit the list)
  // every key above `hi` is taken and none below `lo`; `want` of those in [lo, hi] are.  The
  // range is narrowed to one of 2048 equal parts per round until all of it or one value is
  // wanted: at most six rounds for 64 bits.
  unsigned long long lo = 0ull, hi = ~0ull;
  bool all = want >= nfree;
  if (!all && want > 0) {
    if (tid == 0) { s_lo = ~0ull; s_hi = 0ull; }
    __syncthreads();
    unsigned long long mn = ~0ull, mx = 0ull;
    for (int j = f0 + tid; j < f1; j += kSelThreads) {
      const unsigned long long k = keys[j];
      mn = k < mn ? k : mn;
      mx = k > mx ? k : mx;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long p = __shfl_xor_sync(0xffffffffu, mn, o), q = __shfl_xor_sync(0xffffffffu, mx, o);
      mn = p < mn ? p : mn;
      mx = q > mx ? q : mx;
    }
    if (lane == 0) {
      atomicMin(&s_lo, mn);
      atomicMax(&s_hi, mx);
    }
    __syncthreads();
    lo = s_lo;
    hi = s_hi;
    while (lo < hi) {
      const unsigned long long span = hi - lo;
      const int bits = 64 - __clzll((long long)span);
      const int sh = bits > 11 ? bits - 11 : 0;
      for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j0 = f0; j0 < f1; j0 += kSelThreads) {
        const int j = j0 + tid;
        int bin = -1;
        if (j < f1) {
          const unsigned long long k = keys[j];
          if (k >= lo && k <= hi) bin = (int)((k - lo) >> sh);
        }
        const unsigned same = __match_any_sync(0xffffffffu, bin);
        if (bin >= 0 && lane == __ffs(same) - 1) atomicAdd(&hist[bin], __popc(same));
      }
      __syncthreads();
      // thread t owns bins 8 t' .. 8 t' + 7 from the top (t' = 255 - t)
      constexpr int PER = kSelBins / kSelThreads;
      const int top = kSelBins - 1 - tid * PER;
      int mine = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) mine += hist[top - i];
      int inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) s_warp[warp] = inc;
      __syncthreads();
      int above = inc - mine;
      for (int w = 0; w < warp; ++w) above += s_warp[w];
      if (above < want && want <= above + mine) {
        for (int i = 0; i < PER; ++i) {
          const int c = hist[top - i];
          if (want <= above + c) {
            s_bin = top - i;
            s_above = above;
            s_inbin = c;
            break;
          }
          above += c;
        }
      }
      __syncthreads();
      want -= s_above;
      const unsigned long long nlo = lo + ((unsigned long long)s_bin << sh);
      const unsigned long long width = (1ull << sh) - 1ull;
      lo = nlo;
      hi = hi - nlo < width ? hi : nlo + width;
      const bool whole = want == s_inbin;
      __syncthreads();
      if (whole) {       // the whole bin is wanted: nothing in [lo, hi] is left out
        all = true;
        break;
      }
    }
  }
  // ascending order: pages in steps of the block, positions by a scan
  int base = 0, ties = 0;
  const bool none = want <= 0 && !all;
  for (int j0 = 0; j0 < vis; j0 += kSelThreads) {
    const int j = j0 + tid;
    bool take = false, tie = false;
    if (j < vis) {
      if (j < f0 || j >= f1) {
        take = true;
      } else if (!none) {
        const unsigned long long k = keys[j];
        take = k > hi || (all && k >= lo);
        tie = !all && k >= lo && k <= hi;      // equal keys: the first `want` pages
      }
    }
    const unsigned mt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) s_tie[warp] = __popc(mt);
    __syncthreads();
    int tb = ties;
    for (int w = 0; w < warp; ++w) tb += s_tie[w];
    if (tie && tb + __popc(mt & ((1u << lane) - 1u)) < want) take = true;
    for (int w = 0; w < kSelThreads / 32; ++w) ties += s_tie[w];
    const unsigned m = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_warp[warp] = __popc(m);
    __syncthreads();
    int at = base;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    at += __popc(m & ((1u << lane) - 1u));
    if (take && at < total) out[at] = j;
    for (int w = 0; w < kSelThreads / 32; ++w) base += s_warp[w];
    __syncthreads();
  }
  for (int i = total + tid; i < K; i += kSelThreads) out[i] = -1;
  if (tid == 0) *cnt = total;
}

// grid (units x splits, Hkv).  Scores of the split's share of the pages; with one split the
// block goes on to the list.
template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads) k_page_score(SelectArgs a) {
  extern __shared__ __align__(16) unsigned char sm_sel[];
  __shared__ int sm_find[kSelThreads / 32 + 2];
  __shared__ double s_q[D];
  __shared__ double s_red[kSelThreads / (D / 8)][D + 1];
  const int tid = threadIdx.x, h = blockIdx.y;
  const int unit = blockIdx.x / a.splits, split = blockIdx.x - unit * a.splits;
  UnitInfo u;
  if (!unit_of(a, unit, sm_find, u)) return;
  const int G = a.Hq / a.Hkv;
  constexpr int CH = D / 8;             // 16-byte chunks of a row
  constexpr int RG = kSelThreads / CH;
  // mean query, in the scaled domain until the last step
  {
    const int c = tid % CH, g0 = tid / CH;
    double s[8] = {0., 0., 0., 0., 0., 0., 0., 0.};
    bool bad = false;
    const int rows = u.ntok * G;
    constexpr int UQ = 8;               // rows in flight
    for (int r = g0; r < rows; r += UQ * RG) {
      uint4 w[UQ];
#pragma unroll
      for (int k = 0; k < UQ; ++k) {
        const int rr = r + k * RG;
        w[k] = make_uint4(0, 0, 0, 0);
        if (rr >= rows) continue;
        const int t = rr / G, gh = rr - t * G;
        w[k] = *reinterpret_cast<const uint4*>((const T*)a.Q + (u.tok0 + t) * a.qst + (long long)(h * G + gh) * a.qsh + c * 8);
      }
#pragma unroll
      for (int k = 0; k < UQ; ++k) {
        const uint32_t p[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bad |= not_finite<T>(p[i]);
          s[2 * i] += wide<T>(p[i]);
          s[2 * i + 1] += wide<T>(p[i] >> 16);
        }
      }
    }
    // a NaN or an infinity in a query row: every score of the unit is NaN
    const double poison = bad ? __longlong_as_double(0x7ff8000000000000ll) : 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s_red[g0][c * 8 + i] = s[i] + poison;
    __syncthreads();
    if (tid < D) {
      double t = 0.;
      for (int g = 0; g < RG; ++g) t += s_red[g][tid];
      // undo the shift of the sum (2^bias) and put 2^bias of the means' shift on qbar
      t = t * pow2(Wide<T>::bias) / (double)((long long)u.ntok * G);
      s_q[tid] = t * pow2(Wide<T>::bias);
    }
    __syncthreads();
  }
  unsigned long long* keys = a.keys_global ? a.keys + ((size_t)unit * a.Hkv + h) * a.max_pages
                                           : reinterpret_cast<unsigned long long*>(sm_sel + kSelBins * 4);
  // eight lanes per page, D / 8 columns each
  constexpr int CPL = D / 8;
  const int sub = tid & 7;
  double q[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) q[i] = s_q[(i / 8) * 64 + sub * 8 + (i & 7)];
  const int p0 = (int)((long long)u.vis * split / a.splits), p1 = (int)((long long)u.vis * (split + 1) / a.splits);
  constexpr int PPB = kSelThreads / 8, UN = 4;   // pages of the block per step, steps in flight
  const int* table = a.table + (size_t)u.b * a.max_pages;
  // ids are loaded two rounds ahead of their scores, means one round
  auto ids = [&](int j0, int* id) {
#pragma unroll
    for (int s = 0; s < UN; ++s) {
      const int j = j0 + s * PPB + (tid >> 3);
      id[s] = j < p1 ? table[j] : -2;
    }
  };
  auto means = [&](const int* id, uint4 (*w)[CPL / 8]) {
#pragma unroll
    for (int s = 0; s < UN; ++s) {
      if (id[s] < 0 || id[s] >= a.n_pages) continue;
      const T* row = (const T*)a.km + ((size_t)id[s] * a.Hkv + h) * D;
#pragma unroll
      for (int c = 0; c < CPL / 8; ++c) w[s][c] = *reinterpret_cast<const uint4*>(row + c * 64 + sub * 8);
    }
  };
  int id0[UN], id1[UN];
  uint4 w[UN][CPL / 8];
  ids(p0, id0);
  ids(p0 + PPB * UN, id1);
  means(id0, w);
  for (int j0 = p0; j0 < p1; j0 += PPB * UN) {
    int id2[UN];
    uint4 wn[UN][CPL / 8];
    ids(j0 + 2 * PPB * UN, id2);
    means(id1, wn);
#pragma unroll
    for (int s = 0; s < UN; ++s) {
      const int j = j0 + s * PPB + (tid >> 3);
      const bool ok = id0[s] >= 0 && id0[s] < a.n_pages;
      double x = 0.;
      bool bad = !ok;
      if (ok) {
#pragma unroll
        for (int c = 0; c < CPL / 8; ++c) {
          const uint32_t p[4] = {w[s][c].x, w[s][c].y, w[s][c].z, w[s][c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bad |= not_finite<T>(p[i]);
            x = fma(wide<T>(p[i]), q[c * 8 + 2 * i], x);
            x = fma(wide<T>(p[i] >> 16), q[c * 8 + 2 * i + 1], x);
          }
        }
      } else if (id0[s] != -2 && sub == 0) {
        set_error(a.err, DERR_INDEX);
      }
      if (bad) x = __longlong_as_double(0x7ff8000000000000ll);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (j < p1 && sub == 0) keys[j] = order_key(x);
    }
#pragma unroll
    for (int s = 0; s < UN; ++s) {
      id0[s] = id1[s];
      id1[s] = id2[s];
#pragma unroll
      for (int c = 0; c < CPL / 8; ++c) w[s][c] = wn[s][c];
    }
  }
  if (a.splits > 1) return;
  __syncthreads();
  const size_t at = (size_t)unit * a.Hkv + h;
  select_list(keys, u.vis, a.n_sink, a.n_recent, a.n_select, a.sel + at * a.n_select, a.cnt + at,
              reinterpret_cast<int*>(sm_sel));
}

// grid (units, Hkv): the lists from stored scores (moved to shared memory when they fit)
__global__ void __launch_bounds__(kSelThreads) k_page_pick(SelectArgs a) {
  extern __shared__ __align__(16) unsigned char sm_sel[];
  __shared__ int sm_find[kSelThreads / 32 + 2];
  const int unit = blockIdx.x, h = blockIdx.y;
  UnitInfo u;
  if (!unit_of(a, unit, sm_find, u)) return;
  const size_t at = (size_t)unit * a.Hkv + h;
  const unsigned long long* keys = a.keys + at * a.max_pages;
  if (u.vis <= kSelSmemPages) {
    unsigned long long* mine = reinterpret_cast<unsigned long long*>(sm_sel + kSelBins * 4);
    for (int j = threadIdx.x; j < u.vis; j += kSelThreads) mine[j] = keys[j];
    __syncthreads();
    keys = mine;
  }
  select_list(keys, u.vis, a.n_sink, a.n_recent, a.n_select, a.sel + at * a.n_select, a.cnt + at,
              reinterpret_cast<int*>(sm_sel));
}

template <typename T, int D>
cudaError_t launch_select_t(const SelectArgs& a, int* launches, cudaStream_t st) {
  const int pages = a.max_pages < kSelSmemPages ? a.max_pages : kSelSmemPages;
  const size_t sm = kSelBins * 4 + (size_t)pages * 8;
  const size_t sm1 = a.splits > 1 ? 0 : (a.keys_global ? kSelBins * 4 : sm);
  cudaError_t e = cudaFuncSetAttribute(k_page_score<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(kSelBins * 4 + kSelSmemPages * 8));
  if (e != cudaSuccess) return e;
  k_page_score<T, D><<<dim3((unsigned)a.units * a.splits, a.Hkv), kSelThreads, sm1, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  *launches = 1;
  if (a.splits > 1) {
    e = cudaFuncSetAttribute(k_page_pick, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kSelBins * 4 + kSelSmemPages * 8));
    if (e != cudaSuccess) return e;
    k_page_pick<<<dim3((unsigned)a.units, a.Hkv), kSelThreads, sm, st>>>(a);
    *launches = 2;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_select_d(const SelectArgs& a, int* launches, cudaStream_t st) {
  return a.d == 64 ? launch_select_t<T, 64>(a, launches, st) : launch_select_t<T, 128>(a, launches, st);
}

}  // namespace

// Splits of a unit's pages: enough blocks for two per SM, at least 128 pages each (four steps
// of a block).
SelectPlan select_plan(int units, int Hkv, int max_pages) {
  SelectPlan p{1, max_pages > kSelSmemPages};
  const long long blocks = (long long)units * Hkv;
  if (blocks > 0 && blocks < 148) {
    long long s = 296 / blocks;
    const long long most = ceil_div(max_pages, 128);
    s = s < most ? s : most;
    p.splits = s < 1 ? 1 : (int)s;
  }
  if (p.splits > 1) p.keys_global = true;
  return p;
}

cudaError_t launch_page_select(const SelectArgs& a, int* launches, cudaStream_t st) {
  return a.dtype == SPARSEPR_FP16 ? launch_select_d<__half>(a, launches, st)
                                  : launch_select_d<__nv_bfloat16>(a, launches, st);
}

}  // namespace spr
