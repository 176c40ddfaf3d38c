// Attention of a chunk of new tokens over the paged cache on the 5th-generation tensor cores.
//
// An item is up to 256 query rows (tokens x the query heads of one key/value head) that share
// one stream of keys: the pages of their sequence, or of their unit's list, in order.  Two
// 128-row tiles use every 128-key chunk that reaches shared memory, so the tensor cores work on
// one tile while the other's softmax runs.
//   warps 0-7, 8-15  softmax and epilogue of tile 0 and 1: two threads per query row r = TMEM lane r,
//                    each with 32 of every 64 keys (a single warp per scheduler and tile stalls on
//                    its own exponentials: 13 cycles per element against 8.4 with two)
//   warp 16          TMA: boxes of min(page, 128) rows of the pages of a chunk, into rings of K and V
//   warp 17          issues the MMAs
//   warps 18-19      walk the CTA's work list and load the query rows
// TMEM (512 columns): S, O and P of both tiles, P as packed 16-bit pairs and the second product's A
// operand.  With d = 128, S and O take all columns and P overlays the first 64 columns of its S, so
// the next S waits for P V.  With d = 64 P has columns of its own: the next S starts as soon as the
// softmax has read the last one, and its latency hides behind the second half's exponentials.
// Everything a row may see is a prefix of the stream, so the mask is one comparison with the
// row's limit in the chunks that straddle one.  Value rows of the last chunk past the item's
// last visible key are zeroed in shared memory before their MMA: a page's unused slots may hold
// NaN, and 0 NaN would reach every row.
//
// Work: one CTA per SM (it takes all of TMEM), and 148 of them would leave up to half of a last
// round idle.  k_tiles_plan therefore counts every entry's chunks (an entry is an item of one
// key/value head) and gives each CTA the same number: whole entries in rounds, next to each other
// in item order so that CTAs that run together share keys in L2, as long as the longest entry
// allows it, and then a run of the chunks of the remaining entries, cut wherever the CTA's share
// ends.  The pieces of a cut entry are joined by k_tiles_join.
//
// Bounds.  d = 128: a chunk of both tiles takes 1.65 us, and long calls run into the power limit besides:
// 4,680 tokens x 40 heads over 32,760 keys take 2.65 to 2.71 ms from one GPU to another, 1,130 to 1,105
// TFLOP/s, the last 1,024-token frame of 4 x 16 heads over 16,384 keys 545 to 562 us, 1,010 to 980
// TFLOP/s (457 us in a single launch, before the clock falls).  d = 64: half the products, as many exponentials: a chunk of both tiles takes 1.45 us, and
// the unit that computes exponentials 1.18 us of it; six ragged chunks (87 GFLOP) take 173 us.
// Measured without gain: keys in double-buffered halves (N = 64 products take as long as N = 128: 2.0
// us per chunk), a quarter or half of the exponentials as polynomials in the FMA units, P handed
// over warp by warp, pieces of two chunks.
#include <cuda.h>

#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace spr {
namespace paged {

using namespace spr::tc;

constexpr int BM = 128, TPC = 2, BN = kPagedTileBN;
constexpr int PROD_WARP = 16, MMA_WARP = 17, LOAD_WARP = 18, NTT = 640;
constexpr int NSOFT = 256;             // softmax threads of a tile
constexpr uint32_t kCols = 512;

// What the roles of a CTA need to know about a piece of work.
struct Seg {
  int b, q0, n, len;      // sequence
  int tok0, row0, nrows;  // first token of the unit, first row within it, rows
  int h, cnt;             // key/value head, entries of the list
  int c0, nch, nch0;      // first chunk, chunks, chunks of tile 0
  int total;              // keys of the stream
  int slot;               // partial result, -1: the whole entry
  int bad, last;          // inputs out of range; no more work after this one (nrows = 0)
  const int* list;
};

// K and V chunks in shared memory: as many as fit with d = 128, five of each with d = 64
template <int D>
struct Ring {
  static constexpr int K = D == 64 ? 5 : 3, V = D == 64 ? 5 : 2;
};
constexpr int kMaxRing = 5;

struct TileBars {
  uint64_t q, qfree, kfull[kMaxRing], kempty[kMaxRing], vfull[kMaxRing], vempty[kMaxRing], vtail, s_full[TPC], p_full[TPC][2], pv_half[TPC],
      pv_done[TPC], s_free[TPC], o_done[TPC], o_free[TPC], seg_full[2], seg_free[2], mma_done;
};

template <int D>
struct TileLayout {
  static constexpr uint32_t kTile = (uint32_t)D * 128 * 2;
  static constexpr uint32_t oQ = 0;
  static constexpr uint32_t oK = oQ + TPC * kTile;
  static constexpr uint32_t oV = oK + Ring<D>::K * kTile;
  static constexpr uint32_t oBar = oV + Ring<D>::V * kTile;
  static constexpr uint32_t oSeg = oBar + 384;
  static constexpr uint32_t oInt = oSeg + 256;
  static constexpr uint32_t oEx = oInt + 64;                 // [tile][half][row] exchange of the row's threads
  static constexpr uint32_t kBytes = oEx + TPC * 2 * BM * 4;
};
static_assert(sizeof(TileBars) <= 384 && 2 * sizeof(Seg) <= 256, "barrier and segment blocks");

// Taking up an entry (its rows, the first softmax, the epilogue) costs about as much as two chunks:
// an entry's cost begins with that many.
constexpr int kEntryCost = 2;

// ---------------------------------------------------------------------------
// The plan (one block).  Entries e = h n_items + r, item n_items - 1 - r: the last parts of a
// causal sequence see the most keys and come first.
// ---------------------------------------------------------------------------
struct PlanHead {
  int nc, rounds, n_items, pad;   // CTAs with work; rounds of whole entries
  long long bound[kPlanCtas + 1]; // shares of the chunks behind the rounds
};

template <bool SEL>
__device__ __forceinline__ bool item_rows(const Args& a, const Seq& s, int rank, int& tok0, int& row0, int& nrows,
                                          int& last_tok) {
  if (SEL) {
    const int u = rank / a.ppu, part = rank - u * a.ppu;
    tok0 = u * a.q_block;
    const int ntok = min(a.q_block, s.n - tok0);
    row0 = part * kPagedTileRows;
    nrows = (int)min((long long)kPagedTileRows, (long long)ntok * a.G - row0);
  } else {
    tok0 = 0;
    row0 = rank * kPagedTileRows;
    nrows = (int)min((long long)kPagedTileRows, (long long)s.n * a.G - row0);
  }
  last_tok = tok0 + (row0 + nrows - 1) / a.G;
  return nrows > 0;
}

constexpr int kPlanThreads = 1024;

template <typename V>
__device__ __forceinline__ V block_scan(V v, V* sm, V& total) {   // exclusive, all threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sm[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    V w = sm[lane];
    V i2 = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V u = __shfl_up_sync(0xffffffffu, i2, o);
      if (lane >= o) i2 += u;
    }
    sm[32 + lane] = i2 - w;
    if (lane == 31) sm[64] = i2;
  }
  __syncthreads();
  const V r = sm[32 + warp] + inc - v;
  total = sm[64];
  __syncthreads();
  return r;
}

template <bool SEL>
__global__ void __launch_bounds__(kPlanThreads) k_tiles_plan(Args a) {
  __shared__ long long sm[65];
  __shared__ int s_max;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  PlanHead* ph = reinterpret_cast<PlanHead*>(a.plan);
  int* seq_first = a.plan_seq;          // [B + 1]
  int* item_seq = a.plan_item;          // [items]
  long long* pre = a.plan_pre;          // [items Hkv] inclusive prefix of the chunks
  if (tid == 0) s_max = 0;
  // items of every sequence
  int n_items;
  {
    const int run = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
    auto count = [&](int b) -> int {
      const int lo = min(max(a.q_start[b], 0), a.T);
      return item_count<SEL ? kUnits : kRows>(max(0, min(a.q_start[b + 1], a.T) - lo), a.G, kPagedTileRows, a.q_block,
                                              a.ppu);
    };
    long long mine = 0, total;
    for (int b = b0; b < b1; ++b) mine += count(b);
    long long at = block_scan(mine, sm, total);
    // q_start out of order could promise more than the packed rows hold
    const int cap = a.items;
    n_items = (int)(total < cap ? total : cap);
    for (int b = b0; b < b1; ++b) {
      const int c = count(b);
      seq_first[b] = (int)min(at, (long long)n_items);
      for (int i = 0; i < c && at + i < n_items; ++i) item_seq[at + i] = b;
      at += c;
    }
    if (tid == 0) seq_first[a.B] = n_items;
  }
  __syncthreads();
  // chunks of every entry
  const long long N = (long long)n_items * a.Hkv;
  const long long run = (N + kPlanThreads - 1) / kPlanThreads;
  const long long e0 = min(N, tid * run), e1 = min(N, e0 + run);
  auto cost = [&](long long e) -> int {
    const int h = (int)(e / n_items), item = n_items - 1 - (int)(e - (long long)h * n_items);
    const int b = item_seq[item], rank = item - seq_first[b];
    const Seq s = load_seq(a, b);
    int tok0, row0, nrows, last;
    if (!item_rows<SEL>(a, s, rank, tok0, row0, nrows, last)) return 0;
    int keys = visible_end(s.len - s.n + last, a.frame, s.len);
    if (SEL) {      // at most the list's pages
      const int c = min(max(a.sel_cnt[(size_t)(item / a.ppu) * a.Hkv + h], 0), a.n_select);
      keys = min(c * a.page, keys);
    }
    return kEntryCost + (keys + BN - 1) / BN;
  };
  long long mine = 0, W;
  int mx = 0;
  for (long long e = e0; e < e1; ++e) {
    const int c = cost(e);
    pre[e] = c;
    mine += c;
    mx = max(mx, c);
  }
  long long at = block_scan(mine, sm, W);
  for (long long e = e0; e < e1; ++e) {
    at += pre[e];
    pre[e] = at;
  }
  atomicMax(&s_max, mx);
  __syncthreads();
  // shares: at least min_split chunks per CTA
  long long ncl = (W + a.min_split - 1) / a.min_split;
  const int nc = (int)(ncl < 1 ? 1 : (ncl < kPlanCtas ? ncl : kPlanCtas));
  const int M = max(1, s_max);
  const long long r1 = N / nc, r2 = W / nc / M;
  const int rounds = (int)(r1 < r2 ? r1 : r2);
  long long whole = 0, all;
  if (tid < nc) {
    for (int w = 0; w < rounds; ++w) {
      const long long e = (long long)w * nc + tid;
      whole += pre[e] - (e ? pre[e - 1] : 0);
    }
  }
  const long long done = block_scan(whole, sm, all);
  // CTA c's cut: c shares less what the rounds give to the CTAs before it.  Cuts never descend,
  // since a share holds `rounds` of the longest entry.
  if (tid <= nc) ph->bound[tid] = (W / nc) * tid + (W % nc) * tid / nc - (tid < nc ? done : all);
  if (tid == 0) {
    ph->nc = nc;
    ph->rounds = rounds;
    ph->n_items = n_items;
  }
}

// First entry at or behind `first` whose inclusive prefix exceeds x.
__device__ __forceinline__ long long find_entry(const long long* __restrict__ pre, long long first, long long N, long long x) {
  long long lo = first, hi = N;
  while (lo < hi) {
    const long long mid = (lo + hi) >> 1;
    if (pre[mid] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Entry e, [x0, x1) of its `cost`.
template <bool SEL>
__device__ __forceinline__ void make_seg(const Args& a, long long e, int n_items, int x0, int x1, int cost, int cta, Seg& g) {
  g.h = (int)(e / n_items);
  const int item = n_items - 1 - (int)(e - (long long)g.h * n_items);
  const int b = a.plan_item[item], rank = item - a.plan_seq[b];
  const Seq s = load_seq(a, b);
  g.b = b; g.q0 = s.q0; g.n = s.n; g.len = s.len;
  g.bad = s.bad ? 1 : 0;
  g.list = nullptr;
  g.cnt = 0;
  g.last = 0;
  int last_tok;
  item_rows<SEL>(a, s, rank, g.tok0, g.row0, g.nrows, last_tok);
  if (SEL) {
    const size_t at = (size_t)(item / a.ppu) * a.Hkv + g.h;
    g.list = a.sel + at * a.n_select;
    const int c = a.sel_cnt[at];
    g.cnt = min(max(c, 0), a.n_select);
    const int ul = g.tok0 + min(a.q_block, s.n - g.tok0) - 1;     // the unit's last token sees every page of the list
    const int end = visible_end(s.len - s.n + ul, a.frame, s.len);
    int seen = g.cnt;
    // (more keys than there are: a page twice, perhaps behind the chunks that the plan counted)
    if (stream_limit(end, g.list, g.cnt, a.page, &seen) > end || c != g.cnt || seen != g.cnt) g.bad = 1;
  }
  auto limit_of = [&](int r) -> int {
    return stream_limit(visible_end(s.len - s.n + g.tok0 + (g.row0 + r) / a.G, a.frame, s.len), g.list, g.cnt, a.page);
  };
  g.total = limit_of(g.nrows - 1);
  const int chunks = (g.total + BN - 1) / BN;
  g.slot = x0 == 0 && x1 == cost ? -1 : (x0 > 0 ? 2 * cta : 2 * cta + 1);
  g.c0 = min(max(x0 - kEntryCost, 0), chunks);
  g.nch = min(max(x1 - kEntryCost, 0), chunks) - g.c0;
  // tile 0 stops at its own last row's limit
  g.nch0 = g.nrows <= BM ? g.nch : min(g.nch, max(0, (limit_of(BM - 1) + BN - 1) / BN - g.c0));
}

// TMEM columns of tile t
template <int D>
struct Tmem {
  static constexpr bool kOwnP = D == 64;
  static __device__ __forceinline__ uint32_t S(int t) { return kOwnP ? 128 * t : 256 * t; }
  static __device__ __forceinline__ uint32_t O(int t) { return kOwnP ? 256 + 64 * t : 256 * t + 128; }
  static __device__ __forceinline__ uint32_t P(int t) { return kOwnP ? 384 + 64 * t : 256 * t; }
};

// Instruction descriptor of kind::f16 for the element type (bits 7-9 and 10-12: 0 fp16, 1 bf16)
template <typename T>
__host__ __device__ constexpr uint32_t idesc_t(int M, int N, bool b_mn) {
  constexpr uint32_t f = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (f << 7) | (f << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

template <typename T, int D, bool SEL>
__global__ void __launch_bounds__(NTT, 1)
    k_paged_tiles(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, Args a) {
  using L = TileLayout<D>;
  constexpr int KST = Ring<D>::K, VST = Ring<D>::V;
  constexpr float SHIFT = ProbShift<T>::v;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = su32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (base & 1023u) {
    if (tid == 0) set_error(a.err, DERR_INDEX);
    return;
  }
  TileBars* bars = reinterpret_cast<TileBars*>(smem + L::oBar);
  Seg* segs = reinterpret_cast<Seg*>(smem + L::oSeg);
  int* ints = reinterpret_cast<int*>(smem + L::oInt);   // [0] tmem base, [1] abort, [2..3] bad pages of a segment
  volatile int* abort_flag = ints + 1;
  volatile int* bad_page = ints + 2;
  if (tid < 2) prefetch_tmap(tid ? &tmv : &tmk);
  if (tid == 0) {
    ints[1] = ints[2] = ints[3] = 0;
    mbar_init(su32(&bars->q), 64);
    mbar_init(su32(&bars->qfree), 1);
    for (int i = 0; i < KST; ++i) {
      mbar_init(su32(&bars->kfull[i]), 1);
      mbar_init(su32(&bars->kempty[i]), 1);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(su32(&bars->vfull[i]), 1);
      mbar_init(su32(&bars->vempty[i]), 1);
    }
    mbar_init(su32(&bars->vtail), 1);
    for (int t = 0; t < TPC; ++t) {
      mbar_init(su32(&bars->s_full[t]), 1);
      mbar_init(su32(&bars->p_full[t][0]), NSOFT);
      mbar_init(su32(&bars->p_full[t][1]), NSOFT);
      mbar_init(su32(&bars->pv_half[t]), 1);
      mbar_init(su32(&bars->pv_done[t]), 1);
      mbar_init(su32(&bars->s_free[t]), NSOFT);
      mbar_init(su32(&bars->o_done[t]), 1);
      mbar_init(su32(&bars->o_free[t]), NSOFT);
      mbar_init(su32(&bars->seg_full[t]), 1);
      mbar_init(su32(&bars->seg_free[t]), 2 * NSOFT + 3 * 32);   // softmax threads, TMA, MMA and the second load warp
    }
    mbar_init(su32(&bars->mma_done), 1);
    fence_barrier_init();
  }
  if (warp == MMA_WARP) {
    tc_alloc(su32(&ints[0]), kCols);
    tc_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, (uint32_t)ints[0], 0);   // known to be uniform: see below
  const uint32_t sQ = base + L::oQ, sK = base + L::oK, sV = base + L::oV;
  auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
    return bounded_wait(su32(&bar), parity, abort_flag, a.err);
  };
  auto waits = [&](uint64_t& bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
  // segment i of this CTA, as published by the first load warp
  auto get_seg = [&](int i, Seg& g) -> bool {
    if (!waits(bars->seg_full[i & 1], (i >> 1) & 1)) return false;
    g = segs[i & 1];
    return g.last == 0;
  };
  auto free_seg = [&](int i) { mbar_arrive(su32(&bars->seg_free[i & 1])); };

  if (warp >= LOAD_WARP) {
    // ---------------- work list and query rows ----------------
    asm volatile("griddepcontrol.wait;\n" ::: "memory");     // the plan is complete
    const PlanHead* ph = reinterpret_cast<const PlanHead*>(a.plan);
    const int nc = ph->nc, rounds = ph->rounds, n_items = ph->n_items, cta = blockIdx.x;
    const long long N = (long long)n_items * a.Hkv, first = (long long)rounds * nc;
    const long long off = first > 0 ? a.plan_pre[first - 1] : 0;
    long long x = cta < nc ? ph->bound[cta] + off : 0, xe = cta < nc ? ph->bound[cta + 1] + off : 0;
    long long e = 0;
    int round = 0;
    bool placed = false;
    const int lt = tid - LOAD_WARP * 32;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      Seg g;
      if (warp == LOAD_WARP) {
        bool more = false;
        for (; cta < nc && round < rounds && !more; ++round) {
          const long long w = (long long)round * nc + cta;
          const int c = (int)(a.plan_pre[w] - (w ? a.plan_pre[w - 1] : 0));
          if (c == 0) continue;           // an entry without rows
          make_seg<SEL>(a, w, n_items, 0, c, c, cta, g);
          more = true;
        }
        if (!more && x < xe) {
          if (!placed) e = find_entry(a.plan_pre, first, N, x);
          placed = true;
          long long hi = a.plan_pre[e], lo = e > 0 ? a.plan_pre[e - 1] : 0;
          while (hi <= x) {             // entries without rows
            ++e;
            lo = hi;
            hi = a.plan_pre[e];
          }
          const long long end = hi < xe ? hi : xe;
          make_seg<SEL>(a, e, n_items, (int)(x - lo), (int)(end - lo), (int)(hi - lo), cta, g);
          x = end;
          more = true;
        }
        ok = i < 2 || waits(bars->seg_free[i & 1], ((i >> 1) - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          if (!more) {
            g.last = 1;
          } else if (g.bad) {
            set_error(a.err, DERR_INDEX);
          }
          bad_page[i & 1] = 0;
          segs[i & 1] = g;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(su32(&bars->seg_full[i & 1]));
        if (!more) break;
      } else {
        if (!get_seg(i, g)) break;
        free_seg(i);
      }
      // query rows of both tiles, 16 bytes at a time (rows past the item are zero)
      ok = i == 0 || waits(bars->qfree, (i - 1) & 1);
      if (!ok) break;
      // thread: chunk lt % (D / 8) of rows lt / (D / 8), + RS, ...; token and head advance with them
      const int rows = g.nrows > BM ? 2 * BM : BM;
      constexpr int CH = D / 8, RS = 64 / CH;
      const int c = lt % CH, dt = RS / a.G, dh = RS - dt * a.G;
      const int v0 = g.row0 + lt / CH;
      int tr = v0 / a.G, gh = v0 - tr * a.G;
      const T* qb = (const T*)a.Q + (long long)(g.q0 + g.tok0) * a.qst + (long long)g.h * a.G * a.qsh + c * 8;
#pragma unroll 8
      for (int r = lt / CH; r < rows; r += RS) {
        const bool in = r < g.nrows;
        cp_async16(sQ + (r >> 7) * L::kTile + tile_off(r & 127, c, 128),
                   in ? qb + (long long)tr * a.qst + (long long)gh * a.qsh : (const T*)a.Q, in);
        tr += dt;
        gh += dh;
        if (gh >= a.G) {
          gh -= a.G;
          ++tr;
        }
      }
      cp_async_wait_all();
      fence_proxy_async();
      mbar_arrive(su32(&bars->q));
    }
  } else if (warp == PROD_WARP) {
    // ---------------- TMA ----------------
    const int box = a.page, boxes = BN / box;             // page <= 128 = BN
    const int jobs = boxes * (D / 64);                    // column halves of the boxes, <= 16
    const int bx = lane / (D / 64), half = lane % (D / 64);
    bool ok = true;
    int kc = 0, vc = 0, tails = 0;                        // chunks and tails so far
    Seg g;
    for (int i = 0; ok && get_seg(i, g); ++i) {
      auto fetch = [&](int c) -> int {                    // page of this lane's box of chunk c
        const long long p = (long long)c * BN + bx * box;
        if (lane >= jobs || c >= g.c0 + g.nch || p >= g.total) return -2;
        int j = (int)(p / box);
        if (SEL) {
          const int k = j;
          j = g.list[k];
          if (j < 0 || (long long)j * box >= g.len || (k > 0 && g.list[k - 1] >= j)) return -1;
        }
        const int pid = a.table[(size_t)g.b * a.max_pages + j];
        return pid >= 0 && pid < a.n_pages ? pid : -1;
      };
      int pid = fetch(g.c0);
      for (int j = 0; j < g.nch; ++j, ++kc, ++vc) {
        const int ks = kc % KST, vs = vc % VST;
        const int next = fetch(g.c0 + j + 1);
        if (pid == -1) {        // the rows become NaN; a page that exists is loaded instead
          bad_page[i & 1] = 1;
          set_error(a.err, DERR_INDEX);
          pid = 0;
        }
        __syncwarp();
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, pid >= 0)) * box * 128;
        const uint32_t off = half * 16384 + bx * box * 128;
        const int y = (pid * a.Hkv + g.h) * box;
        ok = kc < KST || waits(bars->kempty[ks], ((kc / KST) - 1) & 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(su32(&bars->kfull[ks]), bytes);
        __syncwarp();
        if (pid >= 0) tma_load_2d(sK + ks * L::kTile + off, &tmk, 64 * half, y, su32(&bars->kfull[ks]));
        const bool tail = (g.c0 + j + 1) * (long long)BN > g.total;
        uint64_t* vbar = tail ? &bars->vtail : &bars->vfull[vs];
        ok = vc < VST || waits(bars->vempty[vs], ((vc / VST) - 1) & 1);
        if (!ok) {
          if (lane == 0) drain_wait(su32(&bars->kfull[ks]), (kc / KST) & 1);
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(su32(vbar), bytes);
        __syncwarp();
        if (pid >= 0) tma_load_2d(sV + vs * L::kTile + off, &tmv, 64 * half, y, su32(vbar));
        if (tail) {
          // zero the value rows past the last visible key, then hand the stage over
          ok = waits(bars->vtail, tails & 1);
          if (!ok) {
            if (lane == 0) {
              drain_wait(su32(&bars->vtail), tails & 1);
              drain_wait(su32(&bars->kfull[ks]), (kc / KST) & 1);
            }
            break;
          }
          ++tails;
          const int first = g.total - (g.c0 + j) * BN;
          const uint32_t v = sV + vs * L::kTile;
          for (int z = lane; z < (BN - first) * (D / 8); z += 32) {
            const int r = first + z / (D / 8), c = z % (D / 8);
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(v + tile_off(r, c, BN)), "r"(0) : "memory");
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(su32(&bars->vfull[vs]));
        }
        pid = next;
      }
      free_seg(i);
    }
    if (!ok && lane == 0) {   // a wait ran out: let the loads in flight land
      for (int i = kc > KST ? kc - KST : 0; i < kc; ++i) drain_wait(su32(&bars->kfull[i % KST]), (i / KST) & 1);
      for (int i = vc > VST ? vc - VST : 0; i < vc; ++i) drain_wait(su32(&bars->vfull[i % VST]), (i / VST) & 1);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ---------------- MMA issuer (the whole warp, converged) ----------------
    constexpr uint32_t IDS = idesc_t<T>(128, BN, false);
    constexpr uint32_t IDO = idesc_t<T>(128, D, true);
    const uint32_t lead = elect_one();
    bool ok = true;
    int kc = 0;                       // chunks of the earlier segments
    int tc0 = 0, tc1 = 0;             // chunks of each tile so far
    int use0 = 0, use1 = 0;           // segments with chunks of each tile so far
    Seg g;
    for (int i = 0; ok && get_seg(i, g); ++i) {
      // Broadcast, so that the compiler knows the counts to be the same in all lanes: descriptors
      // derived from them then stay in uniform registers.
      const int nch = __shfl_sync(0xffffffffu, g.nch, 0), nch0 = __shfl_sync(0xffffffffu, g.nch0, 0);
      const int ntile = __shfl_sync(0xffffffffu, g.nrows > BM ? 2 : 1, 0);
      const int cn0 = nch0, cn1 = ntile > 1 ? nch : 0;
      __syncwarp();
      free_seg(i);
      ok = waits(bars->q, i & 1);
      if (!ok) break;
      tc_fence_after();
      auto count = [&](int t) -> int { return t == 0 ? cn0 : cn1; };
      auto first_user = [&](int j) -> int { return j < nch0 ? 0 : 1; };
      // S_t = Q_t K_j^T; the last tile releases K_j
      auto issue_s = [&](int t, int j) -> bool {
        const int ks = (kc + j) % KST;
        if (t == first_user(j)) {
          if (!waits(bars->kfull[ks], ((kc + j) / KST) & 1)) return false;
          tc_fence_after();
        }
        const uint64_t kd = sdesc(sK + ks * L::kTile, 16, 1024), qd = sdesc(sQ + t * L::kTile, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
          tc_mma_lead(lead, tmem + Tmem<D>::S(t), qd + off, kd + off, IDS, k > 0 ? 1u : 0u);
        }
        tc_commit_lead(lead, su32(&bars->s_full[t]));
        if (t == ntile - 1) {
          tc_commit_lead(lead, su32(&bars->kempty[ks]));
          if (j + 1 == nch) tc_commit_lead(lead, su32(&bars->qfree));   // the last use of the query rows
        }
        return true;
      };
      // half hh of O_t += P_t V_j, P from TMEM; the last tile's second half releases V_j
      auto issue_pv = [&](int t, int j, int hh) -> bool {
        const int vs = (kc + j) % VST;
        const uint64_t vd = sdesc(sV + vs * L::kTile, 16384, 1024);
        const int tc = t == 0 ? tc0 : tc1, use = t == 0 ? use0 : use1;
        if (!waits(bars->p_full[t][hh], (tc + j) & 1)) return false;
        if (hh == 0) {
          if (t == first_user(j) && !waits(bars->vfull[vs], ((kc + j) / VST) & 1)) return false;
          // the previous segment's sums have been read
          if (j == 0 && use > 0 && !waits(bars->o_free[t], (use - 1) & 1)) return false;
        }
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_ts_lead(lead, tmem + Tmem<D>::O(t), tmem + Tmem<D>::P(t) + (4 * hh + k) * 8, vd + (4 * hh + k) * 128, IDO,
                         (j > 0 || hh > 0 || k > 0) ? 1u : 0u);
        tc_commit_lead(lead, su32(hh == 0 ? &bars->pv_half[t] : &bars->pv_done[t]));
        if (hh == 1) {
          if (t == ntile - 1) tc_commit_lead(lead, su32(&bars->vempty[vs]));
          if (j + 1 == count(t)) tc_commit_lead(lead, su32(&bars->o_done[t]));
        }
        return true;
      };
      if (nch == 0) tc_commit_lead(lead, su32(&bars->qfree));
      for (int t = 0; ok && t < ntile; ++t)
        if (count(t) > 0) ok = issue_s(t, 0);
      for (int j = 0; ok && j < nch; ++j) {
        for (int t = 0; ok && t < ntile; ++t) {
          if (j >= count(t)) continue;
          const bool more = j + 1 < count(t);
          ok = issue_pv(t, j, 0);
          if (Tmem<D>::kOwnP && ok && more) {
            ok = waits(bars->s_free[t], ((t == 0 ? tc0 : tc1) + j) & 1);
            tc_fence_after();
            ok = ok && issue_s(t, j + 1);
          }
          ok = ok && issue_pv(t, j, 1);
          if (!Tmem<D>::kOwnP && ok && more) ok = issue_s(t, j + 1);
        }
      }
      kc += nch;
      tc0 += cn0;
      tc1 += cn1;
      use0 += cn0 > 0 ? 1 : 0;
      use1 += cn1 > 0 ? 1 : 0;
    }
    tc_commit_lead(lead, su32(&bars->mma_done));   // every MMA completes before the TMEM is released
    if (!waits(bars->mma_done, 0) && lane == 0) drain_wait(su32(&bars->mma_done), 0);
    __syncwarp();
  } else {
    // ---------------- softmax + epilogue ----------------
    const int t = warp >> 3, hv = (warp >> 2) & 1;     // tile; which 32 of every 64 keys
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + Tmem<D>::S(t) + lane_off, tO = tmem + Tmem<D>::O(t) + lane_off,
                   tP = tmem + Tmem<D>::P(t) + lane_off;
    const int row = t * BM + r;
    const int pair = 1 + t * 4 + (warp & 3);           // named barrier of the two warps of these rows
    float* mine = reinterpret_cast<float*>(smem + L::oEx) + (t * 2 + hv) * BM + r;
    const float* other = reinterpret_cast<const float*>(smem + L::oEx) + (t * 2 + (hv ^ 1)) * BM + r;
    const bool wide_rows = (((uintptr_t)a.O | (uintptr_t)(a.ost * 2) | (uintptr_t)(a.osh * 2)) & 31) == 0;
    bool ok = true, out = false;      // out: left by a vote
    int tc = 0, use = 0;              // chunks and segments of this tile so far
    Seg g;
    for (int i = 0; ok && get_seg(i, g); ++i) {
      const int ntile = g.nrows > BM ? 2 : 1;
      const bool in = row < g.nrows;
      const int nct = t < ntile ? (t == 0 ? g.nch0 : g.nch) : 0;
      if (t >= ntile) {
        free_seg(i);
        continue;
      }
      int lim = g.total;
      if (in && a.frame != 0)
        lim = min(g.total, stream_limit(visible_end(g.len - g.n + g.tok0 + (g.row0 + row) / a.G, a.frame, g.len), g.list,
                                        g.cnt, a.page));
      float m_used = -INFINITY, l = 0.f;     // m_used: the same in both threads of a row
      const uint64_t sc2 = f2pack(a.scale_log2, a.scale_log2);
      // 32 columns of S to probabilities against the running maximum, and their sums in rs2
      auto probs = [&](auto masked, const uint32_t* sr, uint32_t* pk, int left, uint64_t nmu2, uint64_t& rs2) {
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float s0 = __uint_as_float(sr[c]), s1 = __uint_as_float(sr[c + 1]);
          if constexpr (decltype(masked)::value) {
            if (c >= left) s0 = -INFINITY;
            if (c + 1 >= left) s1 = -INFINITY;
          }
          float x0, x1;
          f2unpack(ffma2(f2pack(s0, s1), sc2, nmu2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          rs2 = fadd2(rs2, f2pack(p0, p1));
          pk[c >> 1] = pack2<T>(p0, p1);
        }
      };
      // half hh of chunk j against its own maximum (both threads of the rows): O is rescaled first,
      // half its columns by each
      auto redo = [&](int j, int hh, int left, const uint32_t* sr, uint32_t* pk) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c < left) mx = fmaxf(mx, __uint_as_float(sr[c]));
        *mine = mx;
        named_sync(pair, 64);
        mx = fmaxf(mx, *other);
        const float m_new = fmaxf(m_used, mx * a.scale_log2);
        float alpha = 1.f;
        if (m_new > m_used) {
          alpha = (m_used == -INFINITY) ? 0.f : ex2(m_used - m_new);
          m_used = m_new;
        }
        // the products of the earlier chunks are complete (they were before S_t,j with d = 128, and
        // have been waited for with d = 64); those of this chunk's first half are waited for
        if (hh == 1) ok = ok && waits(bars->pv_half[t], (tc + j) & 1);
        if (j > 0 || hh == 1) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {       // 16 columns
            uint32_t o[16];
            tc_ld16(tO + hv * (D / 2) + c * 16, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc_st16(tO + hv * (D / 2) + c * 16, o);
          }
        }
        l *= alpha;
        const float mu = (m_used == -INFINITY) ? 0.f : m_used - SHIFT;
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float p0 = c < left ? ex2(__uint_as_float(sr[c]) * a.scale_log2 - mu) : 0.f;
          const float p1 = c + 1 < left ? ex2(__uint_as_float(sr[c + 1]) * a.scale_log2 - mu) : 0.f;
          l += p0 + p1;
          pk[c >> 1] = pack2<T>(p0, p1);
        }
        // P goes where the other thread's half of S may lie
        named_sync(pair, 64);
      };
      for (int j = 0; j < nct; ++j) {
        ok = ok && waits(bars->s_full[t], (tc + j) & 1);
        // both warps of the rows take the same way out: after a timeout they may see different
        // answers, and one that has left its loop votes against the other below
        if (!bar_and(pair, 64, ok)) {
          out = true;
          break;
        }
        tc_fence_after();
        const int valid = lim - (g.c0 + j) * BN - 32 * hv;
        const bool full = __all_sync(0xffffffffu, valid >= 96);
        // one speculative pass of each half against the running maximum, kept while the row sums
        // of both threads stay in range
        auto chunk = [&](auto masked) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int left = valid - 64 * hh;
            uint32_t sr[32], pk[16];
            tc_ld32(tS + 64 * hh + 32 * hv, sr);
            if (Tmem<D>::kOwnP && hh == 1) {      // S has been read
              tc_fence_before();
              mbar_arrive(su32(&bars->s_free[t]));
            }
            const float nm = SHIFT - m_used;
            const uint64_t nmu2 = f2pack(nm, nm);
            uint64_t rs2 = 0ull;
            probs(masked, sr, pk, left, nmu2, rs2);
            float r0, r1;
            f2unpack(rs2, r0, r1);
            const bool keep = m_used != -INFINITY && r0 + r1 <= ProbBound<T>::v;
            if (Tmem<D>::kOwnP && hh == 0 && tc + j > 0)      // P_j-1 has been used
              ok = ok && waits(bars->pv_done[t], (tc + j - 1) & 1);
            // also: both have read their half of S, which P may overlay
            if (bar_and(pair, 64, keep)) l += r0 + r1;
            else redo(j, hh, left, sr, pk);
            tc_st16(tP + 32 * hh + 16 * hv, pk);
            tc_fence_before();
            mbar_arrive(su32(&bars->p_full[t][hh]));
          }
        };
        if (full) chunk(std::false_type{});
        else chunk(std::true_type{});
      }
      if (out) break;
      if (nct > 0) {
        ok = ok && waits(bars->o_done[t], use & 1);
        tc_fence_after();
        // the row's sum over both threads (the exchange slots are free: their last use was read
        // before the chunk's barrier)
        *mine = ok ? l : __int_as_float(0x7fffffff);
        named_sync(pair, 64);
        l = hv ? *other + *mine : *mine + *other;
      }
      const bool poison = g.bad != 0 || bad_page[i & 1] != 0 || !(l == l);
      const float inv = poison ? __int_as_float(0x7fffffff) : (l > 0.f ? 1.f / l : 0.f);
      const float z = poison ? __int_as_float(0x7fffffff)
                             : (l > 0.f ? (m_used - SHIFT + log2f(l)) * 0.69314718055994531f : -INFINITY);
      const int tr = (g.row0 + row) / a.G, gh = g.row0 + row - tr * a.G;
      const long long qrow = in ? g.q0 + g.tok0 + tr : 0;
      const int qh = g.h * a.G + (in ? gh : 0);
      T* orow = (T*)a.O + qrow * a.ost + (long long)qh * a.osh;
      const size_t prow = (size_t)(g.slot < 0 ? 0 : g.slot) * kPagedTileRows + row;
      // pieces are kept as [slot][d / 4][256 rows] groups of four, so that a warp's rows are adjacent
      float4* prt = reinterpret_cast<float4*>(a.part_o) + (size_t)(g.slot < 0 ? 0 : g.slot) * (D / 4) * kPagedTileRows + row;
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        const int c = hv * (D / 64) + cc;      // 32 columns
        uint32_t o[32];
        if (nct > 0 && ok) {
          tc_ld32(tO + c * 32, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (cc == D / 64 - 1 && nct > 0) {       // the sums have been read: the next segment may start its own
          tc_fence_before();
          mbar_arrive(su32(&bars->o_free[t]));
        }
        if (in) {
          if (g.slot >= 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              prt[(c * 8 + e / 4) * kPagedTileRows] =
                  make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                              __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
          } else {
            // a lane's row is its own: 32 bytes per store fill whole sectors where the rows allow it
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                w[k] = pack2<T>(__uint_as_float(o[16 * e + 2 * k]) * inv, __uint_as_float(o[16 * e + 2 * k + 1]) * inv);
              T* dst = orow + c * 32 + e * 16;
              if (wide_rows) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                             "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                             : "memory");
              } else {
                reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
      }
      if (in && hv == 0) {
        if (g.slot >= 0) a.part_lse[prow] = z;
        else if (a.lse) a.lse[qrow * a.Hq + qh] = z;
      }
      if (nct > 0) named_sync(pair, 64);      // the sums have been read before the next segment's maxima
      tc += nct;
      use += nct > 0 ? 1 : 0;
      free_seg(i);
    }
    if (!out) bar_and(pair, 64, false);
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tc_dealloc(tmem, kCols);
}

// ---------------------------------------------------------------------------
// Join of the entries that were cut: block (c, part) takes the entry that CTA c's share begins
// inside of, if it is the first cut in that entry.  The piece of the CTA in which the entry
// begins is in its second slot, later pieces in their CTAs' first.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256, kJoinParts = 8;

template <typename T, int D, bool SEL>
__global__ void __launch_bounds__(kJoinThreads) k_tiles_join(Args a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const PlanHead* ph = reinterpret_cast<const PlanHead*>(a.plan);
  const int nc = ph->nc, n_items = ph->n_items, c1 = blockIdx.x + 1;
  if (c1 >= nc) return;
  const long long N = (long long)n_items * a.Hkv, first = (long long)ph->rounds * nc;
  const long long off = first > 0 ? a.plan_pre[first - 1] : 0;
  const long long x = ph->bound[c1] + off;
  if (ph->bound[c1] == ph->bound[nc]) return;         // nothing behind this cut
  if (ph->bound[c1 - 1] == ph->bound[c1]) return;     // an earlier block has this cut
  const long long e = find_entry(a.plan_pre, first, N, x);
  const long long lo = e > 0 ? a.plan_pre[e - 1] : 0, hi = a.plan_pre[e];
  if (lo == x) return;                                 // the share begins with the entry
  if (ph->bound[c1 - 1] + off > lo) return;            // cut before: an earlier block's
  const int h = (int)(e / n_items), item = n_items - 1 - (int)(e - (long long)h * n_items);
  const int b = a.plan_item[item];
  const Seq s = load_seq(a, b);
  int tok0, row0, nrows, last;
  if (!item_rows<SEL>(a, s, item - a.plan_seq[b], tok0, row0, nrows, last)) return;
  // CTAs c1 - 1 .. cl have pieces (those with an empty share have none)
  int cl = c1;
  while (cl + 1 < nc && ph->bound[cl + 1] + off < hi) ++cl;
  // a lane per row, a warp per D / 8 columns
  static_assert(kPagedTileRows / kJoinParts == 32 && kJoinThreads == 256, "one row per lane, eight column groups");
  constexpr int CG = D / 32;       // groups of four columns per thread
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), cg = (threadIdx.x >> 5) * CG;
  if (r >= nrows) return;
  auto slot = [&](int c) -> size_t { return c == c1 - 1 ? 2 * c + 1 : 2 * c; };
  float mx = -INFINITY, den = 0.f;
  bool nan = false;
  float4 acc[CG];
#pragma unroll
  for (int i = 0; i < CG; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c1 - 1; c <= cl; ++c) {
    if (ph->bound[c] == ph->bound[c + 1]) continue;
    const float z = a.part_lse[slot(c) * kPagedTileRows + r];
    const float4* po = reinterpret_cast<const float4*>(a.part_o) + (slot(c) * (D / 4) + cg) * kPagedTileRows + r;
    float4 v[CG];
#pragma unroll
    for (int i = 0; i < CG; ++i) v[i] = po[i * kPagedTileRows];
    nan |= !(z == z);
    const float mn = fmaxf(mx, z), mu = mn == -INFINITY ? 0.f : mn;
    const float f = expf(mx - mu), w = expf(z - mu);     // 0 for -infinity
    mx = mn;
    den = den * f + w;
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      acc[i].x = acc[i].x * f + w * v[i].x;
      acc[i].y = acc[i].y * f + w * v[i].y;
      acc[i].z = acc[i].z * f + w * v[i].z;
      acc[i].w = acc[i].w * f + w * v[i].w;
    }
  }
  nan |= !(den == den);
  const float inv = nan ? __int_as_float(0x7fffffff) : (den > 0.f ? 1.f / den : 0.f);
  const int tr = (row0 + r) / a.G, qh = h * a.G + (row0 + r - tr * a.G);
  const long long qrow = s.q0 + tok0 + tr;
  T* op = (T*)a.O + qrow * a.ost + (long long)qh * a.osh + cg * 4;
#pragma unroll
  for (int i = 0; i < CG; i += 2)
    *reinterpret_cast<uint4*>(op + i * 4) =
        make_uint4(pack2<T>(acc[i].x * inv, acc[i].y * inv), pack2<T>(acc[i].z * inv, acc[i].w * inv),
                   pack2<T>(acc[i + 1].x * inv, acc[i + 1].y * inv), pack2<T>(acc[i + 1].z * inv, acc[i + 1].w * inv));
  if (cg == 0 && a.lse)
    a.lse[qrow * a.Hq + qh] = nan ? __int_as_float(0x7fffffff) : (den > 0.f ? mx + logf(den) : -INFINITY);
}

}  // namespace paged

namespace {

template <typename T, int D, bool SEL>
cudaError_t tiles_t(const paged::Args& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  auto kern = paged::k_paged_tiles<T, D, SEL>;
  // at most one CTA per SM: the kernel takes all 512 TMEM columns
  const size_t need = paged::TileLayout<D>::kBytes, sm = need < 120 * 1024 ? 120 * 1024 : need;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  paged::k_tiles_plan<SEL><<<1, paged::kPlanThreads, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_early(kern, dim3(kPlanCtas), paged::NTT, sm, st, tk, tv, a)) != cudaSuccess) return e;
  return launch_early(paged::k_tiles_join<T, D, SEL>, dim3(kPlanCtas - 1, paged::kJoinParts), paged::kJoinThreads, 0, st, a);
}
template <typename T, int D>
cudaError_t tiles_d(const paged::Args& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  return a.sel ? tiles_t<T, D, true>(a, tk, tv, st) : tiles_t<T, D, false>(a, tk, tv, st);
}

}  // namespace

size_t tiles_plan_head_bytes() { return sizeof(paged::PlanHead); }

cudaError_t launch_paged_tiles(const paged::Args& a, const PagedPlan&, int d, int dtype, const void* kp, const void* vp,
                               cudaStream_t st) {
  CUtensorMap tk{}, tv{};
  const unsigned long long rows = (unsigned long long)a.n_pages * a.Hkv * a.page;
  cudaError_t e;
  if ((e = make_tmap_bf16_rows(&tk, kp, rows, d, a.page)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16_rows(&tv, vp, rows, d, a.page)) != cudaSuccess) return e;
  if (dtype == SPARSEPR_FP16) return d == 64 ? tiles_d<__half, 64>(a, tk, tv, st) : tiles_d<__half, 128>(a, tk, tv, st);
  return d == 64 ? tiles_d<__nv_bfloat16, 64>(a, tk, tv, st) : tiles_d<__nv_bfloat16, 128>(a, tk, tv, st);
}

}  // namespace spr
