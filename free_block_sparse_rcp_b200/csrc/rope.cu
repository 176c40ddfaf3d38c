// Rotary positions, and the cache append that rotates keys on their way into the pages.
//
// Pair (x_a, x_b) of a row turns by t = 2 pi pos f (f in turns per position):
//   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_a sin t + x_b cos t);
// the gradient is the same with -t.  Both kernels move every row once and are bound by
// memory, so a thread keeps the sines and cosines of its pairs in registers (rope: they
// serve every head of the token) or shared memory (append: every head of the page).
// The turn count pos f is formed and reduced to [-1/2, 1/2] in 64 bits: in 32 bits the
// angle of position 10^5 would be off by 2^-24 10^5 = 6e-3.
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
};

// How a row is divided among threads.
//   kInter: one 16-byte chunk, holding whole pairs (pairs past rot/2 turn by 0)
//   kHalf:  chunk c of the first half with chunk c of the second, then the copied chunks
//   kPair:  one pair (or one copied element), for rows that 16-byte chunks do not fit
enum RopeMode { kInter = 0, kHalf = 1, kPair = 2 };

template <typename T, int MODE>
struct RowUnits {
  static constexpr int E = Vec<T>::E;
  // pairs a unit turns, at most
  static constexpr int P = MODE == kInter ? E / 2 : (MODE == kHalf ? E : 1);
  static __host__ __device__ int count(int d, int rot) {
    if (MODE == kInter) return d / E;
    if (MODE == kHalf) return rot / 2 / E + (d - rot) / E;
    return rot / 2 + (d - rot);
  }
};

constexpr int kRopeThreads = 256;

// Thread = one unit of one token; it walks the heads blockIdx.y, blockIdx.y + gridDim.y, ...
template <typename T, int MODE>
__global__ void __launch_bounds__(kRopeThreads) k_rope(RopeArgs a, long long units) {
  using U = RowUnits<T, MODE>;
  constexpr int E = U::E, P = U::P;
  const long long gid = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const int upr = U::count(a.d, a.rot);
  if (gid >= units) return;
  const long long row = gid / upr;
  const int u = (int)(gid - row * upr);
  const int b = (int)(row / a.N), n = (int)(row - (long long)b * a.N);
  const int half = a.rot / 2;
  // first element, partner element (kHalf, kPair) and whether the unit turns
  int e0, e1 = 0, p0;
  bool turns;
  if (MODE == kInter) {
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
      } else {   // kInter: copied pairs of a chunk that the rotation ends in
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
      if (MODE == kInter) {
        uint4 out = wa;
        if (turns) {
          Vec<T>::unpack(wa, va);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float p = va[2 * i], q = va[2 * i + 1];
            va[2 * i] = p * c[i] - q * s[i];
            va[2 * i + 1] = p * s[i] + q * c[i];
          }
          out = Vec<T>::pack(va);
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
    if (MODE == kPair) {
      for (int h = first; h < a.H[t]; h += gy) {
        if (!turns) {
          y[h * yh + e0] = x[h * xh + e0];
          continue;
        }
        const float p = as_f32(x[h * xh + e0]), q = as_f32(x[h * xh + e1]);
        y[h * yh + e0] = from_f32<T>(p * c[0] - q * s[0]);
        y[h * yh + e1] = from_f32<T>(p * s[0] + q * c[0]);
      }
      continue;
    }
    constexpr int UN = MODE == kInter ? 4 : 2;   // heads in flight
    int h = first;
    for (; h + (UN - 1) * gy < a.H[t]; h += UN * gy) {
      uint4 wa[UN], wb[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        Vec<T>::load(x + (h + i * gy) * xh + e0, wa[i]);
        if (MODE == kHalf && turns) Vec<T>::load(x + (h + i * gy) * xh + e1, wb[i]);
      }
#pragma unroll
      for (int i = 0; i < UN; ++i) one(h + i * gy, wa[i], wb[i]);
    }
    for (; h < a.H[t]; h += gy) {
      uint4 wa, wb = make_uint4(0, 0, 0, 0);
      Vec<T>::load(x + h * xh + e0, wa);
      if (MODE == kHalf && turns) Vec<T>::load(x + h * xh + e1, wb);
      one(h, wa, wb);
    }
  }
}

template <typename T, int MODE>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t st) {
  const long long units = (long long)a.B * a.N * RowUnits<T, MODE>::count(a.d, a.rot);
  const long long blocks = ceil_div64(units, kRopeThreads);
  const int heads = a.H[0] + a.H[1];
  // Heads are dealt to enough blocks for eight rounds of the GPU's resident blocks (148 SMs x
  // 8): few tokens get one head per block, and many tokens a last round that is a small share.
  long long hs = ceil_div64(8 * 148 * 8, blocks);
  hs = hs < heads ? hs : heads;
  k_rope<T, MODE><<<dim3((unsigned)blocks, (unsigned)hs), kRopeThreads, 0, st>>>(a, units);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rope_m(const RopeArgs& a, cudaStream_t st) {
  constexpr int E = Vec<T>::E;
  if (a.vec && a.layout == 1) return launch_rope_t<T, kInter>(a, st);
  if (a.vec && (a.rot / 2) % E == 0) return launch_rope_t<T, kHalf>(a, st);
  return launch_rope_t<T, kPair>(a, st);
}

// ---------------------------------------------------------------------------
// Cache append
// ---------------------------------------------------------------------------
// grid (page slots that the call can touch, head groups), one block = one touched page of one
// sequence and hpb heads: new rows of K (rotated) and V go to their slots, and the page's mean
// key is taken over all its rows in use.  The sum over rows has a fixed order (row r belongs
// to row group r mod RG, the groups are added in order), so the mean depends on the page's
// contents alone.
constexpr int kAppThreads = 256;

template <typename T, int MODE, bool ROPE>
__global__ void __launch_bounds__(kAppThreads) k_cache_append(AppendArgs a, int hpb) {
  using U = RowUnits<T, MODE>;
  constexpr int E = U::E, P = U::P;
  constexpr int NC = MODE == kHalf ? 2 * E : (MODE == kInter ? E : 2);   // columns of a unit
  extern __shared__ __align__(16) unsigned char sm_app[];
  __shared__ int sm_find[kAppThreads / 32 + 4];
  const int tid = threadIdx.x;
  const int d = a.d, page = a.page, rot = ROPE ? a.rot : 0, half = rot / 2;
  // sequence b and its touched page: pages floor((len - n) / page) .. floor((len - 1) / page)
  const int2 it = [&]() {
    const int lane = tid & 31, warp = tid >> 5;
    const int run = (a.B + kAppThreads - 1) / kAppThreads;
    const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
    auto count = [&](int b) -> int {
      const int lo = min(max(a.q_start[b], 0), a.T);
      const int n = max(0, min(a.q_start[b + 1], a.T) - lo);
      const int len = min(max(a.kv_len[b], 0), a.max_pages * page);
      if (n == 0 || len == 0) return 0;
      return (len - 1) / page - max(len - n, 0) / page + 1;
    };
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += count(b);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sm_find[warp] = inc;
    if (tid == 0) sm_find[kAppThreads / 32] = -1;
    __syncthreads();
    int at = inc - mine;
    for (int w = 0; w < warp; ++w) at += sm_find[w];
    const int idx = blockIdx.x;
    if (idx >= at && idx < at + mine) {
      for (int b = b0; b < b1; ++b) {
        const int c = count(b);
        if (idx < at + c) {
          sm_find[kAppThreads / 32] = b;
          sm_find[kAppThreads / 32 + 1] = idx - at;
          break;
        }
        at += c;
      }
    }
    __syncthreads();
    return make_int2(sm_find[kAppThreads / 32], sm_find[kAppThreads / 32 + 1]);
  }();
  if (it.x < 0) return;
  const int b = it.x;
  const int qs = a.q_start[b], qe = a.q_start[b + 1], lenr = a.kv_len[b];
  const int q0 = min(max(qs, 0), a.T), n = max(0, min(qe, a.T) - q0);
  const int len = min(max(lenr, 0), a.max_pages * page);
  if (tid == 0 && blockIdx.y == 0 && (qs < 0 || qe > a.T || len != lenr)) set_error(a.err, DERR_INDEX);
  const int s0 = max(len - n, 0);                 // first new slot
  const int j = s0 / page + it.y;                 // page of the sequence
  const int pid = a.table[(size_t)b * a.max_pages + j];
  if (pid < 0 || pid >= a.n_pages) {
    if (tid == 0) set_error(a.err, DERR_INDEX);
    return;
  }
  const int base = j * page;
  const int r0 = max(s0, base) - base, r1 = min(len, base + page) - base;   // new rows of the page
  const int tok = q0 + (base + r0) - (len - n);    // packed row of page row r0
  // cos and sin of every (new row, pair)
  float2* tab = reinterpret_cast<float2*>(sm_app);
  if (ROPE) {
    const Axes ax{a.n_axes, {a.axis_pairs[0], a.axis_pairs[1], a.axis_pairs[2]}};
    for (int e = tid; e < (r1 - r0) * half; e += kAppThreads) {
      const int r = e / half, p = e - r * half;
      const float2 cs = turn<false>((double)a.pos[(size_t)ax.of(p) * a.T + tok + r] * a.freq[p]);
      tab[e] = make_float2(cs.x * a.mag, cs.y * a.mag);
    }
    __syncthreads();
  }
  const int upr = U::count(d, rot);
  const int RG = kAppThreads / upr;                // rows in flight
  const int rg = tid / upr, u = tid - rg * upr;
  const bool on = rg < RG;
  int e0, e1 = 0, p0 = 0;
  bool turns = false;
  if (MODE == kInter) {
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
  }
  float* red = reinterpret_cast<float*>(sm_app + (ROPE ? (size_t)page * half * 8 : 0));   // [RG][d]
  for (int h = blockIdx.y * hpb; h < min(a.Hkv, (int)(blockIdx.y + 1) * hpb); ++h) {
    T* kp = (T*)a.kp + ((size_t)pid * a.Hkv + h) * page * d;
    T* vp = (T*)a.vp + ((size_t)pid * a.Hkv + h) * page * d;
    const T* K = (const T*)a.K + tok * a.kst + h * a.ksh;
    const T* V = (const T*)a.V + tok * a.vst + h * a.vsh;
    float acc[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) acc[i] = 0.f;
    if (on) {
      for (int r = rg; r < r1; r += RG) {
        const bool fresh = r >= r0;
        const T* src = fresh ? K + (r - r0) * a.kst : kp + (size_t)r * d;
        const float2* cs = tab + (size_t)(r - r0) * half + p0;
        if (MODE == kPair) {
          float va = as_f32(src[e0]), vb = turns ? as_f32(src[e1]) : 0.f;
          if (fresh) {
            if (turns) {
              const float2 t = *cs;
              const float p = va, q = vb;
              va = as_f32(from_f32<T>(p * t.x - q * t.y));
              vb = as_f32(from_f32<T>(p * t.y + q * t.x));
              kp[(size_t)r * d + e1] = from_f32<T>(vb);
            }
            kp[(size_t)r * d + e0] = from_f32<T>(va);
          }
          acc[0] += va;
          acc[1] += vb;
        } else {
          uint4 wa, wb = make_uint4(0, 0, 0, 0);
          float va[E], vb[E];
          Vec<T>::load(src + e0, wa);
          if (MODE == kHalf && turns) Vec<T>::load(src + e1, wb);
          Vec<T>::unpack(wa, va);
          Vec<T>::unpack(wb, vb);
          if (fresh) {
            if (turns) {
              if (MODE == kInter) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                  const float2 t = p0 + i < half ? cs[i] : make_float2(1.f, 0.f);
                  const float p = va[2 * i], q = va[2 * i + 1];
                  va[2 * i] = p * t.x - q * t.y;
                  va[2 * i + 1] = p * t.y + q * t.x;
                }
              } else {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                  const float2 t = cs[i];
                  const float p = va[i], q = vb[i];
                  va[i] = p * t.x - q * t.y;
                  vb[i] = p * t.y + q * t.x;
                }
                wb = Vec<T>::pack(vb);
                Vec<T>::unpack(wb, vb);
                *reinterpret_cast<uint4*>(kp + (size_t)r * d + e1) = wb;
              }
              wa = Vec<T>::pack(va);
              Vec<T>::unpack(wa, va);   // the mean is of the stored keys
            }
            *reinterpret_cast<uint4*>(kp + (size_t)r * d + e0) = wa;
          }
#pragma unroll
          for (int i = 0; i < E; ++i) acc[i] += va[i];
          if (MODE == kHalf) {
#pragma unroll
            for (int i = 0; i < E; ++i) acc[E + i] += vb[i];
          }
        }
      }
      // column sums of this row group
      float* row = red + (size_t)rg * d;
      if (MODE == kPair) {
        row[e0] = acc[0];
        if (turns) row[e1] = acc[1];
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) row[e0 + i] = acc[i];
        if (MODE == kHalf && turns) {
#pragma unroll
          for (int i = 0; i < E; ++i) row[e1 + i] = acc[E + i];
        }
      }
    }
    // V rows
    const int cpr = d / E;
    for (int e = tid; e < (r1 - r0) * cpr; e += kAppThreads) {
      const int r = e / cpr, c = e - r * cpr;
      *reinterpret_cast<uint4*>(vp + (size_t)(r0 + r) * d + c * E) =
          *reinterpret_cast<const uint4*>(V + r * a.vst + c * E);
    }
    __syncthreads();
    if (tid < d) {
      float s = 0.f;
      for (int g = 0; g < RG; ++g) s += red[(size_t)g * d + tid];
      ((T*)a.km)[((size_t)pid * a.Hkv + h) * d + tid] = from_f32<T>(s / (float)r1);
    }
    __syncthreads();
  }
}

template <typename T, int MODE, bool ROPE>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t st) {
  const int half = ROPE ? a.rot / 2 : 0;
  const int rg = kAppThreads / RowUnits<T, MODE>::count(a.d, ROPE ? a.rot : 0);
  const size_t sm = (size_t)a.page * half * 8 + (size_t)rg * a.d * 4;
  auto kern = k_cache_append<T, MODE, ROPE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  // every sequence touches at most ceil((n - 1) / page) + 1 pages; at least two blocks per SM,
  // then as many heads per block as that leaves, to share the angles
  long long slots = (long long)a.T / a.page + 2ll * a.B;
  slots = slots < a.T ? slots : a.T;
  int hpb = (int)(slots * a.Hkv / (2 * 148));
  hpb = hpb < 1 ? 1 : (hpb > a.Hkv ? a.Hkv : hpb);
  kern<<<dim3((unsigned)slots, ceil_div(a.Hkv, hpb)), kAppThreads, sm, st>>>(a, hpb);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_append_m(const AppendArgs& a, cudaStream_t st) {
  if (!a.pos) return launch_append_t<T, kInter, false>(a, st);
  if (a.layout == 1) return launch_append_t<T, kInter, true>(a, st);
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
