// Rotary positions, and the cache append that rotates keys on their way into the pages.
//
// Pair (x_a, x_b) of a row turns by t = 2 pi pos f (f in turns per position):
//   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_a sin t + x_b cos t);
// the gradient is the same with -t.  Both kernels move every row once and are bound by
// memory, so a thread keeps the sines and cosines of its pairs in registers, where they serve
// the heads of the token.
// Measured: 32,760 tokens x 80 heads of d 128, bf16 (1.34 GB) 212 us, 6.3 TB/s, a copy's rate; 2 x
// 5,003 tokens x 40 heads, fp32, half of d turned (410 MB) 79 us, 5.2 TB/s; 64 single tokens
// 3.8 us, the latency of one launch with a 64-bit product and a sine.
// The turn count pos f is formed and reduced to [-1/2, 1/2] in 64 bits: in 32 bits the
// angle of position 10^5 would be off by 2^-24 10^5 = 6e-3.
#include <type_traits>

#include "paged.cuh"

namespace spr {
namespace {

using paged::as_f32;
using paged::from_f32;
using paged::pack2;
using paged::unpack2;

// cos and sin of 2 pi turns; the fp32 form corrects for the rounding of the reduced angle
template <bool FINE>
__device__ __forceinline__ float2 turn(double turns) {
  const double r = turns - rint(turns);
  const float hi = (float)r;
  float s, c;
  sincospif(2.f * hi, &s, &c);
  if (FINE) {
    const float lo = 6.28318530717958648f * (float)(r - (double)hi);
    const float c0 = c;
    c = fmaf(-lo, s, c);
    s = fmaf(lo, c0, s);
  }
  return make_float2(c, s);
}

struct Axes {
  int n, pairs[3];
  __device__ __forceinline__ int of(int pair) const {
    return pair < pairs[0] || n == 1 ? 0 : (pair < pairs[0] + pairs[1] || n == 2 ? 1 : 2);
  }
};

// 16 bytes as floats
template <typename T>
struct Vec {
  static constexpr int E = 16 / sizeof(T);
  static __device__ __forceinline__ void load(const T* p, uint4& w) { w = *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint32_t u[4];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  // the first n pairs from v, the others as they are in w (bits: an infinity in one of them must not
  // meet the 0 sine of its partner)
  static __device__ __forceinline__ uint4 pack_pairs(const float* v, const uint4& w, int n) {
    const uint4 p = pack(v);
    if constexpr (sizeof(T) == 4)
      return make_uint4(p.x, p.y, n > 1 ? p.z : w.z, n > 1 ? p.w : w.w);       // n >= 1
    else
      return make_uint4(p.x, n > 1 ? p.y : w.y, n > 2 ? p.z : w.z, n > 3 ? p.w : w.w);
  }
};

// How a row is divided among threads.
//   kInter: one 16-byte chunk, holding whole pairs
//   kMixed: kInter with a rotation that ends inside a chunk, whose other pairs are copied (the loaded words
//           have to be kept for them: 1.3 us of 213 us on 32,760 tokens x 80 heads that need it nowhere)
//   kHalf:  chunk c of the first half with chunk c of the second, then the copied chunks
//   kPair:  one pair, one copied element or (wide) one 16-byte chunk past the rotated part, for
//           rotations that 16-byte chunks do not fit: 2 x 16 heads of 4,000 bf16 rows of d 128, of
//           which 22 elements turn, take 20 us, 39 us with the copied elements one by one
enum RopeMode { kInter = 0, kHalf = 1, kPair = 2, kMixed = 3 };
constexpr bool inter(int mode) { return mode == kInter || mode == kMixed; }

template <typename T, int MODE>
struct RowUnits {
  static constexpr int E = Vec<T>::E;
  // pairs a unit turns, at most
  static constexpr int P = inter(MODE) ? E / 2 : (MODE == kHalf ? E : 1);
  // kPair: first element of the copied chunks
  static __host__ __device__ int tail(int d, int rot, bool wide) { return wide ? (rot + E - 1) / E * E : d; }
  static __host__ __device__ int count(int d, int rot, bool wide = false) {
    if (inter(MODE)) return d / E;
    if (MODE == kHalf) return rot / 2 / E + (d - rot) / E;
    const int t = tail(d, rot, wide);
    return rot / 2 + (t - rot) + (d - t) / E;
  }
};

constexpr int kRopeThreads = 256;

// Thread = one unit of one token; it walks the heads blockIdx.y, blockIdx.y + gridDim.y, ...
template <typename T, int MODE>
__global__ void __launch_bounds__(kRopeThreads) k_rope(RopeArgs a, long long units) {
  using U = RowUnits<T, MODE>;
  constexpr int E = U::E, P = U::P;
  const long long gid = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const int upr = U::count(a.d, a.rot, a.vec);
  if (gid >= units) return;
  const long long row = gid / upr;
  const int u = (int)(gid - row * upr);
  const int b = (int)(row / a.N), n = (int)(row - (long long)b * a.N);
  const int half = a.rot / 2;
  // first element, partner element (kHalf, kPair) and whether the unit turns
  int e0, e1 = 0, p0;
  bool turns, wide = false;       // wide: a chunk of kPair
  if (inter(MODE)) {
    e0 = u * E;
    p0 = e0 / 2;
    turns = p0 < half;
  } else if (MODE == kHalf) {
    turns = u < half / E;
    e0 = turns ? u * E : a.rot + (u - half / E) * E;
    e1 = e0 + half;
    p0 = e0;
  } else {
    turns = u < half;
    p0 = u;
    e0 = !turns ? a.rot + (u - half) : (a.layout == 0 ? u : 2 * u);
    e1 = a.layout == 0 ? e0 + half : e0 + 1;
    const int tail = U::tail(a.d, a.rot, a.vec);
    if (!turns && e0 >= tail) {
      wide = true;
      e0 = tail + (e0 - tail) * E;
    }
    if (!turns) e1 = e0;
  }
  float c[P], s[P];
  if (turns) {
    const Axes ax{a.n_axes, {a.axis_pairs[0], a.axis_pairs[1], a.axis_pairs[2]}};
    const long long stride = a.pos_batched ? (long long)a.B * a.N : a.N;
    const int* pos = a.pos + (a.pos_batched ? row : n);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = p0 + i;
      if (p < half) {
        const float2 cs = turn<sizeof(T) == 4>((double)pos[ax.of(p) * stride] * a.freq[p]);
        c[i] = cs.x * a.mag;
        s[i] = cs.y * (a.mag * a.sign);
      } else {   // kMixed: pairs that pack_pairs copies
        c[i] = 1.f;
        s[i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if (a.H[t] == 0) continue;
    const T* x = (const T*)a.x[t] + b * a.xs[t][0] + n * a.xs[t][2];
    T* y = (T*)a.y[t] + b * a.ys[t][0] + n * a.ys[t][2];
    const long long xh = a.xs[t][1], yh = a.ys[t][1];
    // heads of the two tensors are dealt round robin as one sequence
    const int gy = gridDim.y, first = t == 0 ? (int)blockIdx.y
                                             : (int)(((long long)blockIdx.y - a.H[0] % gy + gy) % gy);
    auto one = [&](int h, const uint4& wa, const uint4& wb) {
      float va[E], vb[E];
      if (inter(MODE)) {
        uint4 out = wa;
        if (turns) {
          Vec<T>::unpack(wa, va);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float p = va[2 * i], q = va[2 * i + 1];
            va[2 * i] = p * c[i] - q * s[i];
            va[2 * i + 1] = p * s[i] + q * c[i];
          }
          out = MODE == kMixed ? Vec<T>::pack_pairs(va, wa, half - p0) : Vec<T>::pack(va);
        }
        *reinterpret_cast<uint4*>(y + h * yh + e0) = out;
      } else if (MODE == kHalf) {
        if (!turns) {
          *reinterpret_cast<uint4*>(y + h * yh + e0) = wa;
          return;
        }
        Vec<T>::unpack(wa, va);
        Vec<T>::unpack(wb, vb);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float p = va[i], q = vb[i];
          va[i] = p * c[i] - q * s[i];
          vb[i] = p * s[i] + q * c[i];
        }
        *reinterpret_cast<uint4*>(y + h * yh + e0) = Vec<T>::pack(va);
        *reinterpret_cast<uint4*>(y + h * yh + e1) = Vec<T>::pack(vb);
      }
    };
    constexpr int UN = 4;   // heads in flight
    if (MODE == kPair) {
      for (int h0 = first; h0 < a.H[t]; h0 += UN * gy) {
        if (wide) {
          uint4 w[UN];
#pragma unroll
          for (int i = 0; i < UN; ++i)
            if (h0 + i * gy < a.H[t]) Vec<T>::load(x + (h0 + i * gy) * xh + e0, w[i]);
#pragma unroll
          for (int i = 0; i < UN; ++i)
            if (h0 + i * gy < a.H[t]) *reinterpret_cast<uint4*>(y + (h0 + i * gy) * yh + e0) = w[i];
          continue;
        }
        T p[UN], q[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i)
          if (h0 + i * gy < a.H[t]) {
            p[i] = x[(h0 + i * gy) * xh + e0];
            q[i] = x[(h0 + i * gy) * xh + e1];
          }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
          if (h0 + i * gy >= a.H[t]) continue;
          T* o = y + (h0 + i * gy) * yh;
          if (turns) {
            const float f = as_f32(p[i]), g = as_f32(q[i]);
            o[e0] = from_f32<T>(f * c[0] - g * s[0]);
            o[e1] = from_f32<T>(f * s[0] + g * c[0]);
          } else {
            o[e0] = p[i];
          }
        }
      }
      continue;
    }
    auto batch = [&](int h0, auto whole) {
      uint4 wa[UN], wb[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int h = h0 + i * gy;
        if (!decltype(whole)::value && h >= a.H[t]) continue;
        Vec<T>::load(x + h * xh + e0, wa[i]);
        if (MODE == kHalf && turns) Vec<T>::load(x + h * xh + e1, wb[i]);
      }
#pragma unroll
      for (int i = 0; i < UN; ++i)
        if (decltype(whole)::value || h0 + i * gy < a.H[t]) one(h0 + i * gy, wa[i], wb[i]);
    };
    int h = first;
    for (; h + (UN - 1) * gy < a.H[t]; h += UN * gy) batch(h, std::true_type{});
    if (h < a.H[t]) batch(h, std::false_type{});
  }
}

template <typename T, int MODE>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t st) {
  const long long units = (long long)a.B * a.N * RowUnits<T, MODE>::count(a.d, a.rot, a.vec);
  const long long blocks = ceil_div64(units, kRopeThreads);
  const int heads = a.H[0] + a.H[1];
  // Heads are dealt to enough blocks to fill the GPU once (148 SMs x 4 blocks), and for large calls
  // to seven rounds of it, so that the last round is a small share, as long as a thread keeps 16
  // heads for its angles: 32,760 tokens x 80 heads take 207 us in 3 shares, 215 us in one; 10,006
  // fp32 rows x 40 heads 70 us in 2 shares, 97 us in 3 and 140 us in 10.
  const long long once = ceil_div64(592, blocks), rounds = ceil_div64(4440, blocks), keep = heads / 16;
  long long hs = once < heads ? once : heads;
  const long long more = rounds < keep ? rounds : keep;
  if (more > hs) hs = more;
  k_rope<T, MODE><<<dim3((unsigned)blocks, (unsigned)hs), kRopeThreads, 0, st>>>(a, units);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rope_m(const RopeArgs& a, cudaStream_t st) {
  constexpr int E = Vec<T>::E;
  if (a.vec && a.layout == 1) return a.rot % E ? launch_rope_t<T, kMixed>(a, st) : launch_rope_t<T, kInter>(a, st);
  if (a.vec && (a.rot / 2) % E == 0) return launch_rope_t<T, kHalf>(a, st);
  return launch_rope_t<T, kPair>(a, st);
}

// ---------------------------------------------------------------------------
// Cache append
// ---------------------------------------------------------------------------
// Two kernels.  k_cache_rows moves the new rows of K (rotated) and V to their slots, a thread per
// unit of a token as in k_rope, so that a token's angles serve its heads from registers.
// k_page_means then takes the mean key of every touched page over its rows in use; the page's
// new rows come from L2.  Its sum over rows has a fixed order (row r belongs to row group
// r mod RG, the groups are added in order), so the mean depends on the page's contents alone.
// Both together in one block per page had to hold a page's angles in shared memory and its blocks
// waited for one another's latencies: 38 us for 4 x 1,024 tokens of 16 heads (d 128) on pages of
// 128, against 18.9 us for the two and the 10 us that the 67 MB need; what is left is the latency of
// two short kernels (angle, load, store; then table, rows, mean).  One token of each of 64
// sequences takes 6.8 us.

// Sequence that holds packed row t (-1: none), by the whole warp: 32 probes a step.  v: this lane's
// first probe, first_probe().
__device__ __forceinline__ int first_probe(const int* __restrict__ q_start, int B, int lane) {
  const int i = lane * ((B + 31) >> 5);
  return i < B ? q_start[i] : 0;
}
__device__ __forceinline__ int find_seq(const int* __restrict__ q_start, int B, int t, int lane, int v) {
  int lo = 0, n = B;            // the last b in [lo, lo + n) with q_start[b] <= t
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lane * step;
    const bool le = i < n && (n == B ? v : q_start[lo + i]) <= t;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    const int at = cnt > 0 ? (cnt - 1) * step : 0;
    lo += at;
    n = min(step, n - at);
  }
  return q_start[lo] <= t && t < q_start[lo + 1] ? lo : -1;
}

// Whether the sequence with these entries is appended: its rows lie within the call's and between the
// first and the last offset, its new tokens within max_chunk, its length within the table.  Otherwise nothing of it is written: rows moved to the
// slots of a length cut to the table would replace the last keys of a full cache, and the page means
// count on the pages that a chunk of max_chunk can touch.
__device__ __forceinline__ bool usable(const AppendArgs& a, int row0, int row1, int lo, int hi, int len) {
  return lo >= max(row0, 0) && hi >= lo && hi <= min(row1, a.T) && hi - lo <= a.max_chunk && len >= 0 &&
         len <= a.max_pages * a.page;
}

template <typename T, int MODE, bool ROPE>
__global__ void __launch_bounds__(kRopeThreads) k_cache_rows(AppendArgs a) {
  using U = RowUnits<T, MODE>;
  constexpr int E = U::E, P = U::P, UN = 2;   // heads of a batch; one batch is loaded ahead
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int d = a.d, page = a.page, rot = ROPE ? a.rot : 0, half = rot / 2;
  const int upr = U::count(d, rot, true);      // the cache's rows are whole chunks
  const long long gid = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const int row = (int)min(gid / upr, (long long)a.T);       // a.T: past the last row
  const int u = (int)(gid - (long long)row * upr);
  int e0, e1 = 0, p0;
  bool turns = false, wide = false;
  if (inter(MODE)) {
    e0 = u * E;
    p0 = e0 / 2;
    turns = ROPE && p0 < half;
  } else if (MODE == kHalf) {
    turns = u < half / E;
    e0 = turns ? u * E : rot + (u - half / E) * E;
    e1 = e0 + half;
    p0 = e0;
  } else {
    turns = u < half;
    p0 = u;
    e0 = !turns ? rot + (u - half) : (a.layout == 0 ? u : 2 * u);
    e1 = a.layout == 0 ? e0 + half : e0 + 1;
    const int tail = U::tail(d, rot, true);
    if (!turns && e0 >= tail) {
      wide = true;
      e0 = tail + (e0 - tail) * E;
    }
  }
  // value chunks of the unit: u and u + upr, as far as the row has them (upr is at least half of
  // its chunks)
  constexpr int VE = Vec<T>::E;
  const int f0 = u * VE < d ? u * VE : -1, f1 = (u + upr) * VE < d ? (u + upr) * VE : -1;
  // rows of no sequence are not read: a call may be padded with rows that its buffers do not hold.  The
  // offsets that say so come with the search's first probes (loaded before those they cost 0.4 us).
  const int probe = first_probe(a.q_start, a.B, lane), row1 = a.q_start[a.B], row0 = __shfl_sync(0xffffffffu, probe, 0);
  const bool live = row < a.T && row >= row0 && row < row1;
  const T* K = (const T*)a.K + (live ? row * a.kst : 0);
  const T* V = (const T*)a.V + (live ? row * a.vst : 0);
  const int gy = gridDim.y;
  struct Batch {
    uint4 ka[UN], kb[UN], va[UN], vb[UN];
  };
  auto load = [&](Batch& w, int h0) {
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int h = h0 + i * gy;
      if (!live || h >= a.Hkv) continue;
      if (MODE != kPair) Vec<T>::load(K + h * a.ksh + e0, w.ka[i]);
      if (MODE == kHalf && turns) Vec<T>::load(K + h * a.ksh + e1, w.kb[i]);
      if (f0 >= 0) Vec<T>::load(V + h * a.vsh + f0, w.va[i]);
      if (f1 >= 0) Vec<T>::load(V + h * a.vsh + f1, w.vb[i]);
    }
  };
  Batch cur;
  load(cur, blockIdx.y);       // in flight while the slot and the angles are found
  // the sequences of the warp's rows: one search, then steps
  int b = -1;
  {
    const int first = __shfl_sync(0xffffffffu, row, 0), last = min(__shfl_sync(0xffffffffu, row, 31), a.T - 1);
    if (first < a.T) {
      b = find_seq(a.q_start, a.B, first, lane, probe);
      if (b >= 0 && a.q_start[b + 1] <= last)        // the warp's rows leave the first one's sequence
        while (b < a.B && row >= a.q_start[b + 1]) ++b;
      if (b < 0)                                     // rows that belong to no sequence, or broken offsets
        for (int r = first; r <= last; ++r) {
          const int f = find_seq(a.q_start, a.B, r, lane, probe);
          if (r == row) b = f;
        }
    }
  }
  if (!live || b < 0 || b >= a.B || row < a.q_start[b]) return;
  const int qs = a.q_start[b], qe = a.q_start[b + 1], len = a.kv_len[b], n = qe - qs;
  if (!usable(a, row0, row1, qs, qe, len)) {
    if (u == 0 && row == max(qs, 0) && blockIdx.y == 0) set_error(a.err, DERR_INDEX);
    return;
  }
  const int slot = len - n + (row - qs);
  if (slot < 0 || slot >= len) return;
  const int j = slot / page;
  const int pid = a.table[(size_t)b * a.max_pages + j];
  if (pid < 0 || pid >= a.n_pages) {
    if (u == 0) set_error(a.err, DERR_INDEX);
    return;
  }
  const size_t dst = ((size_t)pid * a.Hkv * page + (slot - j * page)) * d;
  const size_t hstep = (size_t)page * d;
  float c[P], s[P];
  if (ROPE && turns) {
    const Axes ax{a.n_axes, {a.axis_pairs[0], a.axis_pairs[1], a.axis_pairs[2]}};
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = p0 + i;
      c[i] = 1.f;
      s[i] = 0.f;
      if (p < half) {
        const float2 cs = turn<false>((double)a.pos[(size_t)ax.of(p) * a.T + row] * a.freq[p]);
        c[i] = cs.x * a.mag;
        s[i] = cs.y * a.mag;
      }
    }
  }
  T* kp = (T*)a.kp + dst;
  T* vp = (T*)a.vp + dst;
  for (int h0 = blockIdx.y; h0 < a.Hkv; h0 += UN * gy) {
    Batch nxt;
    load(nxt, h0 + UN * gy);
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int h = h0 + i * gy;
      if (h >= a.Hkv) continue;
      if (MODE == kPair) {
        if (wide) {
          *reinterpret_cast<uint4*>(kp + h * hstep + e0) = *reinterpret_cast<const uint4*>(K + h * a.ksh + e0);
        } else if (!turns) {
          kp[h * hstep + e0] = K[h * a.ksh + e0];
        } else {
          const float p = as_f32(K[h * a.ksh + e0]), q = as_f32(K[h * a.ksh + e1]);
          kp[h * hstep + e0] = from_f32<T>(p * c[0] - q * s[0]);
          kp[h * hstep + e1] = from_f32<T>(p * s[0] + q * c[0]);
        }
      } else {
        if (ROPE && turns) {
          float va[E], vb[E];
          Vec<T>::unpack(cur.ka[i], va);
          if (inter(MODE)) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
              const float p = va[2 * k], q = va[2 * k + 1];
              va[2 * k] = p * c[k] - q * s[k];
              va[2 * k + 1] = p * s[k] + q * c[k];
            }
          } else {
            Vec<T>::unpack(cur.kb[i], vb);
#pragma unroll
            for (int k = 0; k < P; ++k) {
              const float p = va[k], q = vb[k];
              va[k] = p * c[k] - q * s[k];
              vb[k] = p * s[k] + q * c[k];
            }
            *reinterpret_cast<uint4*>(kp + h * hstep + e1) = Vec<T>::pack(vb);
          }
          cur.ka[i] = MODE == kMixed ? Vec<T>::pack_pairs(va, cur.ka[i], half - p0) : Vec<T>::pack(va);
        }
        *reinterpret_cast<uint4*>(kp + h * hstep + e0) = cur.ka[i];
      }
      if (f0 >= 0) *reinterpret_cast<uint4*>(vp + h * hstep + f0) = cur.va[i];
      if (f1 >= 0) *reinterpret_cast<uint4*>(vp + h * hstep + f1) = cur.vb[i];
    }
    cur = nxt;
  }
}

constexpr int kMeanThreads = 128;
// The sums are kept 2^-7 of their size (exactly; a page has at most 128 rows), so that bf16 keys near
// fp32's largest value have a mean.
constexpr float kMeanScale = 1.f / 128.f;

// grid (page slots that the call can touch, Hkv): tp slots per sequence, or (tp = 0) slots counted
// sequence by sequence.
template <typename T, int D>
__global__ void __launch_bounds__(kMeanThreads) k_page_means(AppendArgs a, int tp) {
  constexpr int E = 8, CH = D / E, RG = kMeanThreads / CH, UN = 8;
  __shared__ float red[RG][D];
  __shared__ int sm_find[kMeanThreads / 32 + 2];
  const int tid = threadIdx.x, page = a.page, row0 = a.q_start[0], row1 = a.q_start[a.B];
  // sequence b and its touched page: pages floor((len - n) / page) .. floor((len - 1) / page)
  auto pages_of = [&](int b) -> int {
    const int lo = a.q_start[b], hi = a.q_start[b + 1], len = a.kv_len[b], n = hi - lo;
    if (n <= 0 || len == 0 || !usable(a, row0, row1, lo, hi, len)) return 0;
    return (len - 1) / page - max(len - n, 0) / page + 1;
  };
  int b, jt;
  if (tp > 0) {
    b = blockIdx.x / tp;
    jt = blockIdx.x - b * tp;
  } else {
    const int lane = tid & 31, warp = tid >> 5;
    const int run = (a.B + kMeanThreads - 1) / kMeanThreads;
    const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
    unsigned mine = 0;
    for (int i = b0; i < b1; ++i) mine = paged::add_sat(mine, (unsigned)pages_of(i));
    mine = min(mine, 0x7fffffffu);
    unsigned inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc = paged::add_sat(inc, v);
    }
    if (lane == 31) sm_find[warp] = (int)inc;
    __syncthreads();
    unsigned at = inc - mine;      // beyond every index once the sum has stopped
    for (int w = 0; w < warp; ++w) at = paged::add_sat(at, (unsigned)sm_find[w]);
    __syncthreads();
    if (tid == 0) sm_find[0] = -1;
    __syncthreads();
    const unsigned x = blockIdx.x;
    if (x >= at && x - at < mine) {
      for (int i = b0; i < b1; ++i) {
        const unsigned c = (unsigned)pages_of(i);
        if (x - at < c) {
          sm_find[0] = i;
          sm_find[1] = (int)(x - at);
          break;
        }
        at += c;
      }
    }
    __syncthreads();
    b = sm_find[0];
    jt = sm_find[1];
    if (b < 0) {
      asm volatile("griddepcontrol.wait;\n" ::: "memory");
      return;
    }
  }
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], n = q1 - q0, len = a.kv_len[b];
  const int j = max(len - n, 0) / page + jt, base = j * page, h = blockIdx.y;
  const bool used = n > 0 && usable(a, row0, row1, q0, q1, len) && base < len;
  const int pid = used ? a.table[(size_t)b * a.max_pages + j] : -1;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");     // the rows are in their slots
  if (pid < 0 || pid >= a.n_pages) return;        // recorded by k_cache_rows
  const int rows = min(len - base, page);
  const T* kp = (const T*)a.kp + ((size_t)pid * a.Hkv + h) * page * D;
  const int c = tid % CH, rg = tid / CH;
  float acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0.f;
  for (int r = rg; r < rows; r += UN * RG) {
    uint4 w[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i)
      if (r + i * RG < rows) Vec<T>::load(kp + (size_t)(r + i * RG) * D + c * E, w[i]);
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      if (r + i * RG >= rows) continue;
      float v[E];
      Vec<T>::unpack(w[i], v);
#pragma unroll
      for (int k = 0; k < E; ++k) acc[k] = fmaf(v[k], kMeanScale, acc[k]);
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) red[rg][c * E + i] = acc[i];
  __syncthreads();
  if (tid < D) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < RG; ++g) s += red[g][tid];
    ((T*)a.km)[((size_t)pid * a.Hkv + h) * D + tid] = from_f32<T>(s / (float)rows * (1.f / kMeanScale));
  }
}

template <typename T>
cudaError_t launch_means(const AppendArgs& a, cudaStream_t st) {
  // Page slots: every sequence touches at most ceil((n - 1) / page) + 1 pages.  With the longest
  // chunk's number for each sequence a block finds its page without counting the others' (the
  // shortest way for single tokens); unequal chunks would leave most of those slots empty, and
  // are counted.
  const long long counted = (long long)a.T / a.page + 2ll * a.B;
  long long tp = ceil_div64((long long)a.max_chunk - 1, a.page) + 1;
  if (tp > a.max_pages) tp = a.max_pages;
  long long slots = tp * a.B;
  if (slots > 2 * counted) {
    tp = 0;
    slots = counted < a.T ? counted : a.T;
  }
  const dim3 grid((unsigned)slots, a.Hkv);
  return a.d == 64 ? launch_early(k_page_means<T, 64>, grid, kMeanThreads, 0, st, a, (int)tp)
                   : launch_early(k_page_means<T, 128>, grid, kMeanThreads, 0, st, a, (int)tp);
}

template <typename T, int MODE, bool ROPE>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t st) {
  const long long units = (long long)a.T * RowUnits<T, MODE>::count(a.d, ROPE ? a.rot : 0, true);
  const long long blocks = ceil_div64(units, kRopeThreads);
  // Heads are dealt to 256 blocks: 4 x 1,024 tokens of 16 heads take 19.0 us that way (8 heads per
  // thread), 21.3 us with 128 and 25.4 us with 1,024, where the angles serve two heads only.
  long long hs = ceil_div64(256, blocks);
  hs = hs < a.Hkv ? hs : a.Hkv;
  k_cache_rows<T, MODE, ROPE><<<dim3((unsigned)blocks, (unsigned)hs), kRopeThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_means<T>(a, st);
}

template <typename T>
cudaError_t launch_append_m(const AppendArgs& a, cudaStream_t st) {
  if (!a.pos) return launch_append_t<T, kInter, false>(a, st);
  if (a.layout == 1) return a.rot % Vec<T>::E ? launch_append_t<T, kMixed, true>(a, st) : launch_append_t<T, kInter, true>(a, st);
  if ((a.rot / 2) % Vec<T>::E == 0) return launch_append_t<T, kHalf, true>(a, st);
  return launch_append_t<T, kPair, true>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.dtype == SPARSEPR_FP32) return launch_rope_m<float>(a, st);
  return a.dtype == SPARSEPR_FP16 ? launch_rope_m<__half>(a, st) : launch_rope_m<__nv_bfloat16>(a, st);
}

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  return a.dtype == SPARSEPR_FP16 ? launch_append_m<__half>(a, st) : launch_append_m<__nv_bfloat16>(a, st);
}

}  // namespace spr
