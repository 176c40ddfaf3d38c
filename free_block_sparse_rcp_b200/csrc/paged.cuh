// Shared pieces of the paged-cache kernels: element types, the call's arguments, and the
// mapping of work items to sequences.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace spr {

constexpr int kPagedTileRows = 256;   // query rows of an item of the tile kernel
constexpr int kPagedRowsBN = 64;      // keys of a tile of the rows kernel
constexpr int kPagedTileBN = 128;     // keys of a chunk of the tile kernel
constexpr int kPlanCtas = 148;        // CTAs of the tile kernel

namespace paged {

// ---------------------------------------------------------------------------
// 16-bit element types (packed pairs in 32-bit words, low half first)
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);   // round to nearest even
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <typename T>
__device__ __forceinline__ float as_f32(T x);
template <>
__device__ __forceinline__ float as_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float as_f32<__half>(__half x) { return __half2float(x); }

// The probabilities enter the second product as 16-bit values, which is what the matrix
// instructions take beside 16-bit values; their sum is of the 32-bit ones.  Each is off by half a step
// at most: outputs are 2.0 to 2.3e-3 (relative norm) from 64 bits in bf16, 1.7e-3 by the output's own
// rounding alone, and 2.5 to 2.9e-4 in fp16, 2.1e-4 alone.  fp16 has no room below
// 2^-24, so they are kept 2^kShift higher there (at most 2^15 with the sum bound below);
// a key 2^-31 below the row's largest then still counts.  bf16 has fp32's range.
template <typename T>
struct ProbShift;
template <>
struct ProbShift<__nv_bfloat16> {
  static constexpr float v = 0.f;
};
template <>
struct ProbShift<__half> {
  static constexpr float v = 7.f;
};

// Largest sum of a thread's probabilities of a step against an earlier maximum, before the sums are
// rescaled: below fp16's largest value, and for bf16 far enough from fp32's that sums with values
// of 10^30 hold.
template <typename T>
struct ProbBound;
template <>
struct ProbBound<__nv_bfloat16> {
  static constexpr float v = 1048576.f;   // 2^20
};
template <>
struct ProbBound<__half> {
  static constexpr float v = 32768.f;                  // 2^15
};

// ---------------------------------------------------------------------------
// Arguments of the attention kernels
// ---------------------------------------------------------------------------
struct Args {
  const void* Q;
  const int* q_start;
  const int* kv_len;
  const int* table;
  const int* sel;        // NULL: the whole cache
  const int* sel_cnt;
  void* O;
  float* lse;
  float* part_o;         // rows kernel [slot][16 mt][d], tile kernel [2 kPlanCtas][d / 4][256][4]
  float* part_lse;
  void* plan;            // tile kernel: PlanHead
  int* plan_seq;         // [B + 1] first item of each sequence
  int* plan_item;        // [items] sequence of each item
  long long* plan_pre;   // [items Hkv] inclusive prefix of the entries' chunks
  int* err;
  int B, Hq, Hkv, G, page, n_pages, max_pages, T, max_chunk, frame;
  int q_block, n_select;
  int ppu;               // row parts per unit (rows kernel, whole sequences: at most, per sequence)
  int items;             // upper bound of the (sequence, unit, part) items of a head
  int S, min_split;      // rows kernel: pieces to aim for (whole sequences) or pieces of a list at most;
                         // fewest tiles of a piece
  float scale_log2;
  long long qst, qsh, ost, osh;
};

// One sequence's token range and cache length, with whatever the caller's arrays hold
// brought into bounds (bad: something had to be).
struct Seq {
  int b, q0, n, len;
  bool bad;
};

__device__ __forceinline__ Seq make_seq(const Args& a, int b, int lo, int hi, int len) {
  Seq s;
  s.b = b;
  const int cap = a.max_pages * a.page;
  s.q0 = min(max(lo, 0), a.T);
  s.n = max(0, min(hi, a.T) - s.q0);
  s.len = min(max(len, 0), cap);
  s.bad = lo < 0 || hi > a.T || hi < lo || len != s.len || s.n > a.max_chunk;
  return s;
}
__device__ __forceinline__ Seq load_seq(const Args& a, int b) {
  return make_seq(a, b, a.q_start[b], a.q_start[b + 1], a.kv_len[b]);
}

// Items of a sequence with n new tokens.  Kinds: kWhole one item per sequence, kRows
// ceil(n G / rows) parts of the whole sequence, kUnits ceil(n / q_block) units of ppu parts.
enum ItemKind { kWhole = 0, kRows = 1, kUnits = 2 };

template <int KIND>
__device__ __forceinline__ int item_count(int n, int G, int rows, int q_block, int ppu) {
  if (KIND == kWhole) return 1;
  if (KIND == kRows) return (int)(((long long)n * G + rows - 1) / rows);
  return (int)(((long long)n + q_block - 1) / q_block) * ppu;
}

// Sums of counts that stop at 2^32 - 1: offsets out of order can promise more items than there are
// rows, and a sum that wrapped would send a block to an item that its sequence does not have.
__device__ __forceinline__ unsigned add_sat(unsigned a, unsigned b) {
  const unsigned s = a + b;
  return s < a ? 0xffffffffu : s;
}

// Sequence and rank of item `idx` (counted sequence by sequence), with the sequence's raw entries;
// every thread of the block calls it, all get the result; b = -1 past the last item.  Each thread
// takes a run of sequences, their counts are scanned, and the run that holds idx is walked by its
// thread.
struct Found {
  int b, rank, lo, hi, len;
};
template <int KIND, int NT>
__device__ __forceinline__ Found find_item(const Args& a, int idx, int rows, int ppu, int* sm /* [NT / 32 + 8] */) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (KIND == kWhole) {
    if (idx >= a.B) return Found{-1, 0, 0, 0, 0};
    return Found{idx, 0, a.q_start[idx], a.q_start[idx + 1], a.kv_len[idx]};
  }
  const int run = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
  auto items = [&](int lo, int hi) -> int {
    lo = min(max(lo, 0), a.T);
    return item_count<KIND>(max(0, min(hi, a.T) - lo), a.G, rows, a.q_block, ppu);
  };
  unsigned mine = 0;
  int len0 = 0, lo0 = 0, hi0 = 0;
  for (int b = b0; b < b1; ++b) {
    lo0 = a.q_start[b];
    hi0 = a.q_start[b + 1];
    len0 = a.kv_len[b];
    mine = add_sat(mine, (unsigned)items(lo0, hi0));
  }
  mine = min(mine, 0x7fffffffu);
  unsigned inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = add_sat(inc, v);
  }
  if (lane == 31) sm[warp] = (int)inc;
  if (tid == 0) sm[NT / 32] = -1;
  __syncthreads();
  unsigned at = inc - mine;        // beyond every idx once the sum has stopped
#pragma unroll
  for (int w = 0; w < NT / 32; ++w)
    if (w < warp) at = add_sat(at, (unsigned)sm[w]);
  const unsigned x = (unsigned)idx;
  if (x >= at && x - at < mine) {
    int b = b0;
    for (; b + 1 < b1; ++b) {
      const unsigned c = (unsigned)items(a.q_start[b], a.q_start[b + 1]);
      if (x - at < c) break;
      at += c;
    }
    if (b + 1 < b1) {
      lo0 = a.q_start[b];
      hi0 = a.q_start[b + 1];
      len0 = a.kv_len[b];
    }
    sm[NT / 32] = b;
    sm[NT / 32 + 1] = (int)(x - at);
    sm[NT / 32 + 2] = lo0;
    sm[NT / 32 + 3] = hi0;
    sm[NT / 32 + 4] = len0;
  }
  __syncthreads();
  const int* f = sm + NT / 32;
  return Found{f[0], f[1], f[2], f[3], f[4]};
}

// Keys [0, end) that a token at position pos may see.
__device__ __forceinline__ int visible_end(int pos, int frame, int len) {
  if (frame == 0) return len;
  if (pos < 0) return 0;
  const long long e = ((long long)(pos / frame) + 1) * frame;
  return e < len ? (int)e : len;
}

// The keys of an item form a stream: the cache in order, or the pages of its list in order.
// Everything a token may see is a prefix of that stream, because pages ascend; its length
// for the visible range [0, end):
__device__ __forceinline__ int stream_limit(int end, const int* __restrict__ list, int cnt, int page,
                                           int* entries = nullptr) {
  if (!list) return end;
  int lo = 0, hi = cnt;            // entries whose page starts below `end`: mostly all
  if (cnt > 0 && (long long)list[cnt - 1] * page < end) lo = cnt;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((long long)list[mid] * page < end) lo = mid + 1; else hi = mid;
  }
  if (entries) *entries = lo;
  if (lo == 0) return 0;
  const long long in = (long long)end - (long long)list[lo - 1] * page;
  return (lo - 1) * page + (int)(in < 0 ? 0 : in < page ? in : page);
}

// Splits of an item whose stream has `tiles` tiles (at least min_split each): split s of ns takes
// [tiles s / ns, tiles (s + 1) / ns).
__device__ __forceinline__ int split_count(int tiles, int S, int min_split) {
  const int n = tiles / min_split;
  return n < 1 ? 1 : (n < S ? n : S);
}
__device__ __forceinline__ int split_at(int tiles, int s, int ns) { return (int)((long long)tiles * s / ns); }

}  // namespace paged

// A launch that may begin while the kernel before it in the stream ends.  The kernel waits for that
// one's results itself (griddepcontrol.wait, in every block and on every path).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int threads, size_t sm, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = sm;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
struct RopeArgs {
  const void* x[2];
  void* y[2];
  long long xs[2][3], ys[2][3];   // batch, head, token strides (elements)
  int B, N, H[2], d, rot, layout, n_axes, axis_pairs[3], pos_batched, dtype;
  float mag, sign;
  const int* pos;
  const double* freq;
  bool vec;                       // 16-byte accesses allowed
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st);

struct AppendArgs {
  const void* K;
  const void* V;
  const int* q_start;
  const int* kv_len;
  const int* table;
  void* kp;
  void* vp;
  void* km;
  const int* pos;                 // NULL: no rotation
  const double* freq;
  int* err;
  int B, Hkv, d, dtype, page, n_pages, max_pages, T, max_chunk;
  int rot, layout, n_axes, axis_pairs[3];
  float mag;
  long long kst, ksh, vst, vsh;
};
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st);

struct SelectArgs {
  paged::Args p;                  // Q, q_start, kv_len, table, err, sizes, strides
  const void* km;
  int* sel;
  int* cnt;
  // A batch of lists: units u0 .. u0 + bu - 1 (scores) or v0 .. (keys), heads h0 .. h0 + nh - 1
  int u0, v0, h0, nh;
  float* scores;                  // [unit - u0][h - h0][max_pages] (group: [units][Hkv][max_pages]) and
  float* bounds;                  // [unit - u0][h - h0][splits] (group: [units][Hkv][splits]), used with
                                  // splits > 1, `keys_global` or `group`
  unsigned long long* keys;       // [unit - v0][h - h0][max_pages], used when `keys_global`
  double* qbar;                   // [units][Hkv][d] and
  int2* info;                     // [units] sequence and visible pages, used when `group`
  int n_sink, n_recent, units, splits;
  bool keys_global, group;
};
struct SelectPlan {
  int splits;
  bool keys_global;
  bool group;       // four units' scores together
  int bu, bv, bh;   // units and heads whose scores (bu x bh) and keys (bv x bh) are kept at once: all,
                    // unless they would need more than kSelWork bytes
};
constexpr long long kSelWork = 1ll << 28;
SelectPlan select_plan(int units, int Hkv, int max_pages, int B);
cudaError_t launch_page_select(const SelectArgs& a, const SelectPlan& sp, int d, int dtype, int* launches, cudaStream_t st);

// rows kernel: items of at most 16 * mt query rows on mma.sync; tile kernel: 256-row items on
// tcgen05; combine: the join of split items.
struct PagedPlan {
  bool rows;        // rows kernel, else tile kernel
  int mt;           // 16-row tiles of the rows kernel
  int kind;         // paged::ItemKind
  int ppu, items, S, min_split;
};
PagedPlan paged_plan(int B, int Hq, int Hkv, int page, int max_pages, int T, int max_chunk, int q_block, int n_select,
                     bool sel);
cudaError_t launch_paged_rows(const paged::Args& a, const PagedPlan& pl, int d, int dtype, const void* kp,
                              const void* vp, cudaStream_t st);
cudaError_t launch_paged_tiles(const paged::Args& a, const PagedPlan& pl, int d, int dtype, const void* kp,
                               const void* vp, cudaStream_t st);
cudaError_t launch_paged_combine(const paged::Args& a, const PagedPlan& pl, int d, int dtype, cudaStream_t st);
size_t tiles_plan_head_bytes();

}  // namespace spr
