// Page selection: for every unit (q_block consecutive new tokens of a sequence) and key/value
// head, the pages whose mean key scores best against the unit's mean query.
//
//   score(j) = qbar . kbar_j,   qbar = mean of the unit's query rows over tokens and the query
//   heads of the key/value head; the first n_sink and last n_recent visible pages are kept and
//   the best scores fill the list up to n_select, ties to the lowest page.
//
// The list is decided by comparisons, so it is the one of scores summed in 64 bits: in 32 bits
// the order of the sum would decide between pages closer than 2^-24, and with a thousand pages
// the pair at the border is that close in about one list of 10^4.  The scores are made in 32
// bits all the same, with a bound on their error: every score s is off by at most
// eps = 2^-19 max_j sum |qbar||kbar_j| (16 products in a lane's chain, 3 sums across lanes, the
// rounding of qbar: 20 steps of 2^-24, and 32 are counted).  With t the n-th best score in 32
// bits, a page above t + 2 eps is in the list and one below t - 2 eps is not, whatever the
// errors; only the pages between (mostly the n-th itself) are scored again in 64 bits.  All in 64
// bits cost 8 integer instructions per element to widen the 16-bit means and took 40 us for 256
// lists of up to 1,024 pages.
//
// Work: the means are read once per unit, or once per four units scored together (1 / page of the
// keys' bytes each time), 4 d operations per unit and page; the queries once.  One block per (unit, head), or several that share its pages when there are
// few units; the selection then runs as a second kernel over the stored scores, which finds its unit
// and mean query while the scores are made (5 units of a 475-token call over 36,000 keys, with their
// attention: 34.5 us, 39.6 without).
// Several units of one sequence read the same means: with four or more of them per sequence their
// mean queries come from a kernel of their own, and a block scores four units with each mean that it
// reads.  One list per block reads its head's means from L2 for itself (256 lists of 1,024 pages: 64 MB
// at 6 TB/s, 11 of 25 us, and half the instructions per score took the same time).  With the
// attention over the lists: 2,048 tokens in units of 64, 8 heads, 1,024 pages 188 -> 180 us; 2,083
// in units of 16, 4 heads, 1,140 pages 120 -> 100 us; 2,113 in units of 128, 4 heads, 1,530 pages
// 65 -> 58 us; fewer than 64 lists leave the GPU empty in three kernels instead of one.
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace spr {
namespace {

using paged::unpack2;

constexpr int kSelThreads = 512;
constexpr int kSelBins = 2048;
constexpr int kSelSmemPages = 8192;   // scores and keys in shared memory up to this many pages (96 KB)
constexpr int kSelExact = 64;         // pages scored again in one step
constexpr int kSelGroup = 4;          // units that k_group_score scores together
constexpr double kSelTiny = 7.8886090522101181e-31;   // 2^-100

// largest exponent field of a packed pair's halves, as a bit pattern: >= kInf: not finite
template <typename T>
struct InfBits;
template <>
struct InfBits<__nv_bfloat16> {
  static constexpr uint32_t v = 0x7f80u;
};
template <>
struct InfBits<__half> {
  static constexpr uint32_t v = 0x7c00u;
};
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
template <typename T>
__device__ __forceinline__ bool finite2(uint32_t m) { return (m & 0xffffu) < InfBits<T>::v && (m >> 16) < InfBits<T>::v; }

// Order of scores as unsigned integers (larger score, larger key; keys of numbers are above 0).
__device__ __forceinline__ uint32_t order32(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);         // -0 becomes +0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order64(double x) {
  const long long b = __double_as_longlong(x + 0.0);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

// eps of the file's head from max_j sum |qbar||kbar_j| (2^-140: products below fp32's range)
__device__ __forceinline__ float error_bound(float e) { return fmaf(e, 1.9073486328125e-6f, 7.2e-43f); }

struct UnitInfo {
  int b, len, ntok, tok0, vis;   // tok0: packed row of the unit's first token; vis: visible pages
};

template <int NT>
__device__ __forceinline__ bool unit_of(const SelectArgs& a, int idx, int* sm, UnitInfo& u) {
  const paged::Found f = paged::find_item<paged::kUnits, NT>(a.p, idx, 1, 1, sm);
  if (f.b < 0) return false;
  const paged::Seq s = paged::make_seq(a.p, f.b, f.lo, f.hi, f.len);
  if (s.bad && threadIdx.x == 0) set_error(a.p.err, DERR_INDEX);
  u.b = f.b;
  u.len = s.len;
  const int t0 = f.rank * a.p.q_block;     // < n
  u.ntok = min(a.p.q_block, s.n - t0);
  u.tok0 = s.q0 + t0;
  const int end = paged::visible_end(s.len - s.n + t0 + u.ntok - 1, a.p.frame, s.len);
  u.vis = (end + a.p.page - 1) / a.p.page;
  return true;
}

// Exclusive scan over the block (all threads), total in `total`.
__device__ __forceinline__ int sel_scan(int v, int* sm /* [kSelThreads / 32] */, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sm[warp] = inc;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) base += sm[w];
    sum += sm[w];
  }
  total = sum;
  __syncthreads();
  return base + inc - v;
}

struct PickShared {
  int scan[kSelThreads / 32], bin, above, inbin, nfound;
  unsigned long long lo, hi;
  int list[kSelExact];
  unsigned long long exact[kSelExact];   // also the last candidates of nth_key
  int in[kSelExact];
};

// The n-th largest key of keys[f0 .. f1) (1 <= n <= f1 - f0): the range [lo, hi] that holds it is
// narrowed to one of 2048 equal parts per round, until one value or at most 64 keys are left,
// which are ranked against each other.  want: n; on return how many keys of that value are among
// the n.
template <typename K>
__device__ K nth_key(const K* keys, int f0, int f1, int& want, int* hist, PickShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) { sh.lo = ~0ull; sh.hi = 0ull; }
  __syncthreads();
  K mn = ~(K)0, mx = 0;
  for (int j = f0 + tid; j < f1; j += kSelThreads) {
    const K k = keys[j];
    mn = k < mn ? k : mn;
    mx = k > mx ? k : mx;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const K p = __shfl_xor_sync(0xffffffffu, mn, o), q = __shfl_xor_sync(0xffffffffu, mx, o);
    mn = p < mn ? p : mn;
    mx = q > mx ? q : mx;
  }
  if (lane == 0) {
    atomicMin(&sh.lo, (unsigned long long)mn);
    atomicMax(&sh.hi, (unsigned long long)mx);
  }
  __syncthreads();
  K lo = (K)sh.lo, hi = (K)sh.hi;
  constexpr int PER = kSelBins / kSelThreads;
  while (lo < hi) {
    const unsigned long long span = (unsigned long long)hi - (unsigned long long)lo;
    const int bits = 64 - __clzll((long long)span);
    const int s = bits > 11 ? bits - 11 : 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) hist[tid + i * kSelThreads] = 0;
    __syncthreads();
    for (int j = f0 + tid; j < f1; j += kSelThreads) {
      const K k = keys[j];
      if (k >= lo && k <= hi) atomicAdd(&hist[(int)((k - lo) >> s)], 1);
    }
    if (tid == 0) sh.nfound = 0;
    __syncthreads();
    // thread t owns PER bins, from the top
    const int top = kSelBins - 1 - tid * PER;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += hist[top - i];
    int sum;
    int above = sel_scan(mine, sh.scan, sum);
    if (above < want && want <= above + mine) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = hist[top - i];
        if (above < want && want <= above + c) {
          sh.bin = top - i;
          sh.above = above;
          sh.inbin = c;
        }
        above += c;
      }
    }
    __syncthreads();
    want -= sh.above;
    lo = lo + ((K)sh.bin << s);
    const K width = (K)(((unsigned long long)1 << s) - 1ull);
    hi = hi - lo < width ? hi : lo + width;
    const int left = sh.inbin;
    __syncthreads();
    if (left <= kSelExact) {
      for (int j = f0 + tid; j < f1; j += kSelThreads) {
        const K k = keys[j];
        if (k >= lo && k <= hi) sh.exact[atomicAdd(&sh.nfound, 1)] = (unsigned long long)k;
      }
      __syncthreads();
      if (tid < left) {
        const unsigned long long k = sh.exact[tid];
        int above = 0, same = 0;
        for (int m = 0; m < left; ++m) {
          above += sh.exact[m] > k;
          same += sh.exact[m] == k;
        }
        if (above < want && want <= above + same) {     // all threads with this key write the same
          sh.lo = k;
          sh.above = above;
        }
      }
      __syncthreads();
      want -= sh.above;
      lo = (K)sh.lo;
      __syncthreads();
      break;
    }
  }
  return lo;
}

// Score of page j in 64 bits by eight lanes (sub: lane of the eight); 0 for a page without one.
template <typename T, int D>
__device__ __forceinline__ unsigned long long exact_key(const SelectArgs& a, const UnitInfo& u, int h, int j,
                                                        const double* q, int sub) {
  const int pid = j >= 0 ? a.p.table[(size_t)u.b * a.p.max_pages + j] : -1;
  const bool ok = pid >= 0 && pid < a.p.n_pages;
  const T* row = (const T*)a.km + ((size_t)(ok ? pid : 0) * a.p.Hkv + h) * D;
  double x = 0.;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + c * 64 + sub * 8);
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(p[i]);
      x = fma((double)f.x, q[c * 64 + sub * 8 + 2 * i], x);
      x = fma((double)f.y, q[c * 64 + sub * 8 + 2 * i + 1], x);
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return ok && x == x ? order64(x) : 0ull;
}

// Writes the list of one (unit, head) from its 32-bit scores' keys (0: no score) and their error
// bound (all threads of the block).  keys64: room for a 64-bit key per page.
template <typename T, int D>
__device__ void pick_list(const SelectArgs& a, const UnitInfo& u, int h, const uint32_t* keys, float eps, const double* q,
                          unsigned long long* keys64, int* hist, int* out, int* cnt) {
  __shared__ PickShared sh;
  const int tid = threadIdx.x;
  const int vis = u.vis, K = a.p.n_select;
  const int f0 = min(a.n_sink, vis), f1 = max(f0, vis - a.n_recent);   // free pages [f0, f1)
  const int nfree = f1 - f0, total = min(K, vis);
  const int want = total - (vis - nfree);        // free pages to take (>= 0: kept pages fit the list)
  const int per = (vis + kSelThreads - 1) / kSelThreads;
  const int j0 = min(vis, tid * per), j1 = min(vis, j0 + per);      // this thread's run of pages
  // in: key above `above`; undecided: [below, above]; take_all: all of those are in
  uint32_t above = 0xffffffffu, below = 0u;
  bool take_all = want >= nfree, exact = false;
  int need = 0;                                  // undecided pages to take
  int mine = 0;                                  // undecided pages of this thread's run
  int first = 0, nund = 0;                       // their rank in the block, their number
  if (!take_all && want > 0) {
    int left = want;
    const uint32_t t = nth_key<uint32_t>(keys, f0, f1, left, hist, sh);
    if (t == 0u) {
      above = below = 0u;                        // pages without a score are needed: the lowest ones
    } else {
      const float v = value32(t);
      // an infinite score or bound leaves every page with a score undecided
      const float up = v + 2.01f * eps, dn = v - 2.01f * eps;
      above = up == up && fabsf(up) < INFINITY ? order32(up) : 0xffffffffu;
      below = dn == dn && fabsf(dn) < INFINITY ? order32(dn) : 1u;
    }
    int nin = 0;
    for (int j = max(j0, f0); j < min(j1, f1); ++j) {
      const uint32_t k = keys[j];
      nin += k > above;
      mine += k <= above && k >= below;
    }
    int sum;
    sel_scan(nin, sh.scan, sum);
    need = want - sum;
    first = sel_scan(mine, sh.scan, nund);
    if (need == nund) {
      take_all = true;
    } else if (t == 0u) {
      // by index
    } else if (nund <= kSelExact) {
      exact = true;
      int at = first;
      for (int j = max(j0, f0); j < min(j1, f1) && mine > 0; ++j)
        if (keys[j] <= above && keys[j] >= below) sh.list[at++] = j;
      __syncthreads();
      const int i = tid >> 3;
      const unsigned long long k = exact_key<T, D>(a, u, h, i < nund ? sh.list[i] : -1, q, tid & 7);
      if ((tid & 7) == 0) sh.exact[i] = k;
      __syncthreads();
      if (tid < nund) {
        int rank = 0;
        for (int m = 0; m < nund; ++m) rank += sh.exact[m] > sh.exact[tid] || (sh.exact[m] == sh.exact[tid] && m < tid);
        sh.in[tid] = rank < need;
      }
      __syncthreads();
    } else {
      // many undecided pages: their 64-bit keys, and the need-th of them
      for (int jj = f0; jj < f1; jj += kSelThreads / 8) {
        const int j = jj + (tid >> 3);
        const bool und = j < f1 && keys[j] <= above && keys[j] >= below;
        const unsigned long long k = exact_key<T, D>(a, u, h, und ? j : -1, q, tid & 7);
        if (j < f1 && (tid & 7) == 0) keys64[j] = und ? (k > 0ull ? k : 1ull) : 0ull;
      }
      __syncthreads();
      int ties = need;
      const unsigned long long t64 = nth_key<unsigned long long>(keys64, f0, f1, ties, hist, sh);
      // from here on the keys say in (2), tied (1) or out (0)
      int m = 0;
      for (int j = max(j0, f0); j < min(j1, f1); ++j) {
        const unsigned long long k = keys64[j];
        const int c = keys[j] > above ? 2 : (k > t64 ? 2 : (k == t64 ? 1 : 0));
        m += c == 1;
        keys64[j] = c;
      }
      first = sel_scan(m, sh.scan, nund);
      need = ties;
    }
  }
  const bool by64 = !take_all && want > 0 && !exact && !(above == 0u && below == 0u);
  auto walk = [&](auto emit) {
    int und = first;
    for (int j = j0; j < j1; ++j) {
      bool in;
      if (j < f0 || j >= f1) {
        in = true;
      } else if (want <= 0) {
        in = false;
      } else if (by64) {
        const int c = (int)keys64[j];
        in = c == 2 || (c == 1 && und++ < need);
      } else {
        const uint32_t k = keys[j];
        in = k > above || (take_all && k >= below);
        if (!in && !take_all && k >= below) {
          in = exact ? sh.in[und] != 0 : und < need;
          ++und;
        }
      }
      if (in) emit(j);
    }
  };
  int count = 0, sum;
  walk([&](int) { ++count; });
  int at = sel_scan(count, sh.scan, sum);
  walk([&](int j) { out[at++] = j; });
  for (int i = total + tid; i < K; i += kSelThreads) out[i] = -1;
  if (tid == 0) *cnt = total;
}

// The unit's mean query in 64 bits (NaN throughout if a query element is not finite).
template <typename T, int D, int NT>
__device__ void mean_query(const SelectArgs& a, const UnitInfo& u, int h, double* q /* [D] */,
                           double (*red)[D + 1] /* [NT / (D / 8)] */) {
  constexpr int CH = D / 8, RG = NT / CH, UQ = 4;   // chunks of a row, rows per pass, passes in flight
  const int tid = threadIdx.x, c = tid % CH, g0 = tid / CH, G = a.p.G, rows = u.ntok * G;
  if (g0 < rows) {
    double s[8] = {0., 0., 0., 0., 0., 0., 0., 0.};
    for (int r = g0; r < rows; r += UQ * RG) {
      uint4 w[UQ];
#pragma unroll
      for (int k = 0; k < UQ; ++k) {
        const int rr = r + k * RG;
        w[k] = make_uint4(0, 0, 0, 0);
        if (rr >= rows) continue;
        const int t = rr / G, gh = rr - t * G;
        w[k] = *reinterpret_cast<const uint4*>((const T*)a.p.Q + (u.tok0 + t) * a.p.qst +
                                               (long long)(h * G + gh) * a.p.qsh + c * 8);
      }
#pragma unroll
      for (int k = 0; k < UQ; ++k) {
        const uint32_t p[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<T>(p[i]);
          s[2 * i] += (double)f.x;
          s[2 * i + 1] += (double)f.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) red[g0][c * 8 + i] = s[i];
  }
  __syncthreads();
  bool bad = false;
  if (tid < D) {
    double t = 0.;
    const int groups = min(RG, rows);
    for (int g = 0; g < groups; ++g) t += red[g][tid];
    q[tid] = t / (double)rows;
    bad = !(fabs(t) < INFINITY);       // an infinity or a NaN; sums of finite elements stay far below
  }
  if (__syncthreads_or(bad) && tid < D) q[tid] = __longlong_as_double(0x7ff8000000000000ll);
  __syncthreads();
}

// grid (units x splits, heads) of a batch.  Scores of the split's share of the pages; with one split
// the block goes on to the list, unless that is too long for shared memory.
template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads, 2) k_page_score(SelectArgs a) {
  extern __shared__ __align__(16) unsigned char sm_sel[];
  __shared__ int sm_find[kSelThreads / 32 + 8];
  __shared__ double s_q[D];
  __shared__ float s_eps[kSelThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");     // k_page_pick may get ready
  const int tid = threadIdx.x, h = a.h0 + blockIdx.y;
  const int nth = blockIdx.x / a.splits, unit = a.u0 + nth, split = blockIdx.x - nth * a.splits;
  UnitInfo u;
  if (!unit_of<kSelThreads>(a, unit, sm_find, u)) return;
  int* hist = reinterpret_cast<int*>(sm_sel);
  // the reduction of the mean query and, later, the keys share the space behind the bins
  unsigned char* rest = sm_sel + kSelBins * 4;
  mean_query<T, D, kSelThreads>(a, u, h, s_q, reinterpret_cast<double(*)[D + 1]>(rest));
  const size_t list = (size_t)unit * a.p.Hkv + h, slot = (size_t)nth * a.nh + blockIdx.y;
  const bool stored = a.splits > 1 || a.keys_global;
  uint32_t* keys = stored ? reinterpret_cast<uint32_t*>(a.scores) + slot * a.p.max_pages
                          : reinterpret_cast<uint32_t*>(rest);
  // eight lanes per page, D / 8 columns each
  constexpr int CPL = D / 8;
  const int sub = tid & 7;
  float q[CPL];
  // elements near the end of fp32's range lose their relative accuracy: then every score is
  // decided in 64 bits
  bool nan = false, tiny = false;
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const double v = s_q[(i / 8) * 64 + sub * 8 + (i & 7)];
    q[i] = (float)v;
    nan |= !(v == v);
    tiny |= v != 0. && fabs(v) < kSelTiny;
  }
  nan = __any_sync(0xffffffffu, nan);
  tiny = __any_sync(0xffffffffu, tiny);
  const int p0 = (int)((long long)u.vis * split / a.splits), p1 = (int)((long long)u.vis * (split + 1) / a.splits);
  constexpr int PPB = kSelThreads / 8, UN = 4;   // pages of the block per step, steps in flight
  const int* table = a.p.table + (size_t)u.b * a.p.max_pages;
  float eps = tiny ? INFINITY : 0.f;
  int id[UN];
#pragma unroll
  for (int s = 0; s < UN; ++s) id[s] = p0 + s * PPB + (tid >> 3) < p1 ? table[p0 + s * PPB + (tid >> 3)] : -1;
  for (int j0 = p0; j0 < p1; j0 += PPB * UN) {
    uint4 w[UN][CPL / 8];
    bool ok[UN];
#pragma unroll
    for (int s = 0; s < UN; ++s) {
      ok[s] = id[s] >= 0 && id[s] < a.p.n_pages;
      if (!ok[s] && j0 + s * PPB + (tid >> 3) < p1 && sub == 0) set_error(a.p.err, DERR_INDEX);
      const T* row = (const T*)a.km + ((size_t)(ok[s] ? id[s] : 0) * a.p.Hkv + h) * D;
#pragma unroll
      for (int c = 0; c < CPL / 8; ++c) w[s][c] = *reinterpret_cast<const uint4*>(row + c * 64 + sub * 8);
    }
    // the next step's ids
#pragma unroll
    for (int s = 0; s < UN; ++s) {
      const int j = j0 + (UN + s) * PPB + (tid >> 3);
      id[s] = j < p1 ? table[j] : -1;
    }
#pragma unroll
    for (int s = 0; s < UN; ++s) {
      const int j = j0 + s * PPB + (tid >> 3);
      float x = 0.f, e = 0.f;
      uint32_t m = 0u;
#pragma unroll
      for (int c = 0; c < CPL / 8; ++c) {
        const uint32_t p[4] = {w[s][c].x, w[s][c].y, w[s][c].z, w[s][c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<T>(p[i]);
          m = max_abs2(m, p[i]);
          x = fmaf(f.x, q[c * 8 + 2 * i], x);
          x = fmaf(f.y, q[c * 8 + 2 * i + 1], x);
          e = fmaf(fabsf(f.x), fabsf(q[c * 8 + 2 * i]), e);
          e = fmaf(fabsf(f.y), fabsf(q[c * 8 + 2 * i + 1]), e);
        }
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        e += __shfl_xor_sync(0xffffffffu, e, o);
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
      if (j < p1) {
        const bool scored = ok[s] && !nan && finite2<T>(m);
        if (scored) eps = fmaxf(eps, fabsf(x) < INFINITY ? e : INFINITY);
        // a finite page whose score overflows 32 bits is decided in 64 (the bound is infinite)
        if (sub == 0) keys[j] = !scored ? 0u : (fabsf(x) < INFINITY ? order32(x) : 1u);
      }
    }
  }
  eps = warp_max(eps);
  if ((tid & 31) == 0) s_eps[tid >> 5] = eps;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) eps = fmaxf(eps, s_eps[w]);
  if (stored) {
    if (tid == 0) a.bounds[slot * a.splits + split] = eps;
    return;
  }
  pick_list<T, D>(a, u, h, keys, error_bound(eps), s_q,
                  reinterpret_cast<unsigned long long*>(rest + (((size_t)a.p.max_pages * 4 + 15) & ~(size_t)15)), hist,
                  a.sel + list * a.p.n_select, a.cnt + list);
}

// ---------------------------------------------------------------------------
// Several units of a sequence: k_unit_mean (mean queries), k_group_score (each page's mean serves four
// units), k_page_pick.
// ---------------------------------------------------------------------------
constexpr int kGroupThreads = 256;

// grid (units, Hkv)
template <typename T, int D>
__global__ void __launch_bounds__(kGroupThreads) k_unit_mean(SelectArgs a) {
  __shared__ double red[kGroupThreads / (D / 8)][D + 1];
  __shared__ int sm_find[kGroupThreads / 32 + 8];
  __shared__ double s_q[D];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int unit = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  UnitInfo u;
  const bool any = unit_of<kGroupThreads>(a, unit, sm_find, u);
  if (h == 0 && tid == 0) a.info[unit] = any ? make_int2(u.b, u.vis) : make_int2(-1, 0);
  if (!any) return;
  mean_query<T, D, kGroupThreads>(a, u, h, s_q, red);
  if (tid < D) a.qbar[((size_t)unit * a.p.Hkv + h) * D + tid] = s_q[tid];
}

// grid (groups of four units x splits, Hkv): the scores of the split's share of the pages.  The units
// of a group that belong to one sequence are scored together.
template <typename T, int D>
__global__ void __launch_bounds__(kGroupThreads, 2) k_group_score(SelectArgs a) {
  constexpr int U = kSelGroup, CPL = D / 8, NP = CPL / 2;     // columns of a lane, as pairs
  constexpr int PPB = kGroupThreads / 8, UN = 4;              // pages of the block per step, steps in flight
  __shared__ uint64_t s_q2[NP][U][8];
  __shared__ double s_qq[U];
  __shared__ int s_nan[U], s_wide[U];
  __shared__ int2 s_info[U];
  __shared__ float s_kk[kGroupThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = tid & 7, h = blockIdx.y;
  const int group = blockIdx.x / a.splits, split = blockIdx.x - group * a.splits, u0 = group * U;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");     // the mean queries are complete
  if (warp < U) {
    const int unit = u0 + warp;
    const int2 info = unit < a.units ? a.info[unit] : make_int2(-1, 0);
    double qq = 0.;
    bool nan = false, tiny = false;
    for (int i = lane; i < D / 2; i += 32) {      // pair i: columns 2 i, 2 i + 1
      double2 v = make_double2(0., 0.);
      if (info.x >= 0) v = *reinterpret_cast<const double2*>(a.qbar + ((size_t)unit * a.p.Hkv + h) * D + 2 * i);
      const int c = i / 32, l = (i & 31) >> 2, p = i & 3;     // column 2 i = 64 c + 8 l + 2 p
      s_q2[c * 4 + p][warp][l] = tc::f2pack((float)v.x, (float)v.y);
      qq = fma(v.x, v.x, fma(v.y, v.y, qq));
      nan |= !(v.x == v.x) || !(v.y == v.y);
      tiny |= (v.x != 0. && fabs(v.x) < kSelTiny) || (v.y != 0. && fabs(v.y) < kSelTiny);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) qq += __shfl_xor_sync(0xffffffffu, qq, o);
    nan = __any_sync(0xffffffffu, nan);
    tiny = __any_sync(0xffffffffu, tiny);
    if (lane == 0) {
      s_info[warp] = info;
      s_qq[warp] = qq;
      s_nan[warp] = nan;
      s_wide[warp] = tiny;
    }
  }
  __syncthreads();
  // this lane's results: page sub / 2 of the step's four, units 2 (sub & 1) and the next
  const int mp = sub >> 1, mu = 2 * (sub & 1);
  for (int r0 = 0; r0 < U;) {
    const int b = s_info[r0].x;
    int r1 = r0, vis = 0;
    for (; r1 < U && s_info[r1].x == b; ++r1) vis = max(vis, s_info[r1].y);
    if (b < 0) {
      r0 = r1;
      continue;
    }
    const int p0 = (int)((long long)vis * split / a.splits), p1 = (int)((long long)vis * (split + 1) / a.splits);
    const int* table = a.p.table + (size_t)b * a.p.max_pages;
    bool mine[2], nanu[2];
    int visu[2];
    uint32_t* keys[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = mu + k;
      mine[k] = u >= r0 && u < r1;
      nanu[k] = s_nan[u] != 0;
      visu[k] = s_info[u].y;
      keys[k] = reinterpret_cast<uint32_t*>(a.scores) + ((size_t)(u0 + u) * a.p.Hkv + h) * a.p.max_pages;
    }
    bool wide[2] = {false, false}, wide_all = false;
    float kk = 0.f;                  // largest sum of squares of this lane's columns of a page
    int id[UN];
#pragma unroll
    for (int s = 0; s < UN; ++s) id[s] = p0 + s * PPB + (tid >> 3) < p1 ? table[p0 + s * PPB + (tid >> 3)] : -1;
    for (int j0 = p0; j0 < p1; j0 += PPB * UN) {
      uint4 w[UN][CPL / 8];
      bool ok[UN];
#pragma unroll
      for (int s = 0; s < UN; ++s) {
        ok[s] = id[s] >= 0 && id[s] < a.p.n_pages;
        if (!ok[s] && j0 + s * PPB + (tid >> 3) < p1 && sub == 0) set_error(a.p.err, DERR_INDEX);
        const T* row = (const T*)a.km + ((size_t)(ok[s] ? id[s] : 0) * a.p.Hkv + h) * D;
#pragma unroll
        for (int c = 0; c < CPL / 8; ++c) w[s][c] = *reinterpret_cast<const uint4*>(row + c * 64 + sub * 8);
      }
      // the next step's ids
#pragma unroll
      for (int s = 0; s < UN; ++s) {
        const int j = j0 + (UN + s) * PPB + (tid >> 3);
        id[s] = j < p1 ? table[j] : -1;
      }
      uint64_t x2[UN][U], k2[UN];
#pragma unroll
      for (int s = 0; s < UN; ++s) {
        k2[s] = 0ull;
#pragma unroll
        for (int u = 0; u < U; ++u) x2[s][u] = 0ull;
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint64_t q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = s_q2[i][u][sub];
#pragma unroll
        for (int s = 0; s < UN; ++s) {
          const uint4 v = w[s][i >> 2];
          const float2 f = unpack2<T>((i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w);
          const uint64_t f2 = tc::f2pack(f.x, f.y);
          k2[s] = tc::ffma2(f2, f2, k2[s]);
#pragma unroll
          for (int u = 0; u < U; ++u) x2[s][u] = tc::ffma2(f2, q[u], x2[s][u]);
        }
      }
      // sums over the eight lanes, each lane left with two of the sixteen
      float v[UN * U];
#pragma unroll
      for (int s = 0; s < UN; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x0, x1;
          tc::f2unpack(x2[s][u], x0, x1);
          v[s * U + u] = x0 + x1;
        }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        const bool hi = (sub & o) != 0;
#pragma unroll
        for (int i = 0; i < 2 * o; ++i) {
          const float send = hi ? v[i] : v[i + 2 * o], keep = hi ? v[i + 2 * o] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
      bool odd = false;                // something that is not finite among these pages
      bool okm = false;
#pragma unroll
      for (int s = 0; s < UN; ++s) {
        float k0, k1;
        tc::f2unpack(k2[s], k0, k1);
        const float ks = k0 + k1;
        if (ok[s]) {
          if (ks < INFINITY) kk = fmaxf(kk, ks);
          else odd = true;
        }
        if (s == mp) okm = ok[s];
      }
      bool over[2], fin = true;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        over[k] = !(fabsf(v[k]) < INFINITY);
        odd |= over[k] && okm && mine[k] && !nanu[k];
      }
      // An infinity or a NaN among the means shows in the score or in the sum of squares; only then
      // are the elements looked at, since a finite page's sums may overflow 32 bits.
      if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
        for (int s = 0; s < UN; ++s) {
          uint32_t m = 0u;
#pragma unroll
          for (int c = 0; c < CPL / 8; ++c) {
            const uint32_t p[4] = {w[s][c].x, w[s][c].y, w[s][c].z, w[s][c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max_abs2(m, p[i]);
          }
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
          const bool f = finite2<T>(m);
          float k0, k1;
          tc::f2unpack(k2[s], k0, k1);
          if (ok[s] && f && !(k0 + k1 < INFINITY)) wide_all = true;
          if (s == mp) fin = f;
        }
      }
      const int j = j0 + mp * PPB + (tid >> 3);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!mine[k] || j >= p1 || j >= visu[k]) continue;
        const bool scored = okm && fin && !nanu[k];
        // a finite page whose score overflows is decided in 64 bits, and all others with it
        wide[k] |= scored && over[k];
        keys[k][j] = !scored ? 0u : (over[k] ? 1u : order32(v[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (wide[k]) s_wide[mu + k] = 1;
    if (wide_all)
      for (int u = r0; u < r1; ++u) s_wide[u] = 1;
#pragma unroll
    for (int o = 16; o > 4; o >>= 1) kk = fmaxf(kk, __shfl_xor_sync(0xffffffffu, kk, o));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) kk += __shfl_xor_sync(0xffffffffu, kk, o);
    if (lane == 0) s_kk[warp] = kk;
    __syncthreads();
    if (tid >= r0 && tid < r1) {
      float most = 0.f;
      for (int w = 0; w < kGroupThreads / 32; ++w) most = fmaxf(most, s_kk[w]);
      const float eps = (float)sqrt(s_qq[tid] * ((double)most + 7.2e-43));     // products below fp32's range: 2^-140
      a.bounds[((size_t)(u0 + tid) * a.p.Hkv + h) * a.splits + split] = s_wide[tid] || !(eps < INFINITY) ? INFINITY : eps;
    }
    __syncthreads();
    r0 = r1;
  }
}

// grid (units, heads) of a batch: the lists from stored scores (GROUP: those of k_group_score)
template <typename T, int D, bool GROUP>
__global__ void __launch_bounds__(kSelThreads) k_page_pick(SelectArgs a) {
  extern __shared__ __align__(16) unsigned char sm_sel[];
  __shared__ int sm_find[kSelThreads / 32 + 8];
  __shared__ double s_q[D];
  const int unit = a.v0 + blockIdx.x, h = a.h0 + blockIdx.y;
  UnitInfo u;
  int* hist = reinterpret_cast<int*>(sm_sel);
  unsigned char* rest = sm_sel + kSelBins * 4;
  if (GROUP) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");     // the scores are complete
    const int2 info = a.info[unit];
    if (info.x < 0) return;
    u.b = info.x;
    u.vis = info.y;
    if (threadIdx.x < D) s_q[threadIdx.x] = a.qbar[((size_t)unit * a.p.Hkv + h) * D + threadIdx.x];
  } else {
    const bool any = unit_of<kSelThreads>(a, unit, sm_find, u);
    if (any) mean_query<T, D, kSelThreads>(a, u, h, s_q, reinterpret_cast<double(*)[D + 1]>(rest));
    asm volatile("griddepcontrol.wait;\n" ::: "memory");     // the scores are complete
    if (!any) return;
  }
  const size_t list = (size_t)unit * a.p.Hkv + h, held = GROUP ? list : (size_t)(unit - a.u0) * a.nh + blockIdx.y;
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(a.scores) + held * a.p.max_pages;
  unsigned long long* keys64 = a.keys + ((size_t)blockIdx.x * a.nh + blockIdx.y) * a.p.max_pages;
  if (!a.keys_global) {
    uint32_t* mine = reinterpret_cast<uint32_t*>(rest);
    for (int j = threadIdx.x; j < u.vis; j += kSelThreads) mine[j] = keys[j];
    keys = mine;
    keys64 = reinterpret_cast<unsigned long long*>(rest + (((size_t)a.p.max_pages * 4 + 15) & ~(size_t)15));
  }
  float eps = 0.f;
  for (int s = 0; s < a.splits; ++s) eps = fmaxf(eps, a.bounds[held * a.splits + s]);
  __syncthreads();
  pick_list<T, D>(a, u, h, keys, error_bound(eps), s_q, keys64, hist, a.sel + list * a.p.n_select, a.cnt + list);
}

template <typename T, int D>
cudaError_t launch_select_t(SelectArgs a, const SelectPlan& sp, int* launches, cudaStream_t st) {
  const size_t red = (size_t)(kSelThreads / (D / 8)) * (D + 1) * 8;
  const size_t keys = (((size_t)a.p.max_pages * 4 + 15) & ~(size_t)15) + (size_t)a.p.max_pages * 8;
  const bool stored = a.splits > 1 || a.keys_global;
  const size_t all = kSelBins * 4 + (a.keys_global || keys < red ? red : keys), score = kSelBins * 4 + (stored ? red : all - kSelBins * 4);
  cudaError_t e;
  *launches = 0;
  a.nh = sp.bh;
  if (a.group) {
    k_unit_mean<T, D><<<dim3((unsigned)a.units, a.p.Hkv), kGroupThreads, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const unsigned groups = (unsigned)((a.units - 1) / kSelGroup + 1);
    if ((e = launch_early(k_group_score<T, D>, dim3(groups * a.splits, a.p.Hkv), kGroupThreads, 0, st, a)) != cudaSuccess) return e;
    *launches = 2;
    e = cudaFuncSetAttribute(k_page_pick<T, D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)all);
  } else {
    e = cudaFuncSetAttribute(k_page_score<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)score);
    if (e == cudaSuccess && stored)
      e = cudaFuncSetAttribute(k_page_pick<T, D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)all);
  }
  if (e != cudaSuccess) return e;
  auto upto = [](int all, int at, int step) { return (unsigned)(all - at < step ? all - at : step); };
  for (a.h0 = 0; a.h0 < a.p.Hkv; a.h0 += sp.bh)
    for (a.u0 = 0; a.u0 < a.units; a.u0 += sp.bu) {
      const unsigned nu = upto(a.units, a.u0, sp.bu), nh = upto(a.p.Hkv, a.h0, sp.bh);
      if (!a.group) {
        k_page_score<T, D><<<dim3(nu * a.splits, nh), kSelThreads, score, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        ++*launches;
        if (!stored) continue;
      }
      for (a.v0 = a.u0; a.v0 < a.u0 + (int)nu; a.v0 += sp.bv) {
        const dim3 grid(upto(a.u0 + (int)nu, a.v0, sp.bv), nh);
        e = a.group ? launch_early(k_page_pick<T, D, true>, grid, kSelThreads, all, st, a)
                    : launch_early(k_page_pick<T, D, false>, grid, kSelThreads, all, st, a);
        if (e != cudaSuccess) return e;
        ++*launches;
      }
    }
  return cudaSuccess;
}

template <typename T>
cudaError_t launch_select_d(const SelectArgs& a, const SelectPlan& sp, int d, int* launches, cudaStream_t st) {
  return d == 64 ? launch_select_t<T, 64>(a, sp, launches, st) : launch_select_t<T, 128>(a, sp, launches, st);
}

}  // namespace

// Splits of a unit's (or group's) pages: enough blocks for two per SM, at least 256 pages each.
// Lists too long for shared memory keep their scores and 64-bit keys in the workspace, in batches of as
// many lists as kSelWork holds of each, one at least (2,048 units of 8 heads over 16,384 pages: 0.54
// instead of 3.3 GB, 15.6 instead of 15.0 ms).
SelectPlan select_plan(int units, int Hkv, int max_pages, int B) {
  SelectPlan p{1, max_pages > kSelSmemPages, false, units, units, Hkv};
  long long blocks = (long long)units * Hkv;
  // groups of mostly one sequence, and scores that a workspace may hold (4 bytes per list and page)
  p.group = units >= kSelGroup * (long long)B && blocks >= 64 && blocks * max_pages <= kSelWork / 4;
  if (p.keys_global) {
    auto fit = [&](int bytes, long long lists) -> int {     // of `lists`, at least one
      const long long n = kSelWork / ((long long)bytes * max_pages);
      return (int)(n < 1 ? 1 : (n < lists ? n : lists));
    };
    if (fit(8, blocks) < blocks) {
      p.bh = fit(8, Hkv);
      p.bv = fit(8, blocks) / p.bh;
      if (!p.group) p.bu = fit(4, blocks) / p.bh;
      p.bu = p.bu < units ? p.bu : units;
    }
  }
  if (p.group) {
    const long long groups = ceil_div64(units, kSelGroup) * (long long)Hkv, most = ceil_div(max_pages, 256);
    const long long s = 296 / groups < most ? 296 / groups : most;
    p.splits = s < 1 ? 1 : (int)s;
    return p;
  }
  blocks = (long long)p.bu * p.bh;
  if (blocks > 0 && blocks < 148) {
    long long s = 296 / blocks;
    const long long most = ceil_div(max_pages, 256);
    s = s < most ? s : most;
    p.splits = s < 1 ? 1 : (int)s;
  }
  return p;
}

cudaError_t launch_page_select(const SelectArgs& a, const SelectPlan& sp, int d, int dtype, int* launches, cudaStream_t st) {
  return dtype == SPARSEPR_FP16 ? launch_select_d<__half>(a, sp, d, launches, st)
                                : launch_select_d<__nv_bfloat16>(a, sp, d, launches, st);
}

}  // namespace spr
