// Attention of few query rows over the paged cache (single tokens, short chunks), and the join
// of split items.
//
// An item is the new tokens of one sequence (or of one unit with its page list) and the query
// heads of one key/value head, or 32 rows of them in a small call: at most 32 rows, which share one
// stream of keys.  The work is
// reading that stream: 4 d bytes per key for 4 d rows operations, so the kernel is built to
// keep memory busy and uses the small warp-wide matrix product (16 x 8 x 16); a 128-row
// tensor-core tile would be mostly padding here.
//   producer warp   TMA boxes of min(page, 64) rows, 64 keys of K and V per stage
//   4 MT warps      warp (mt, slice) takes 16 query rows and 16 of the stage's 64 keys, keeps
//                   its own running maximum, sum and O in registers; the four slices are joined
//                   at the end through shared memory
// Whole sequences are cut into pieces of about equal length, so that all of them together fill the
// GPU once whatever the lengths (find_piece); page lists, which are equally long, into a fixed
// number.  A piece of a cut item writes its normalised O and lse in fp32, and k_paged_combine joins
// them.
//
// Measured: one token of each of 48 sequences of 500 to 32,000 keys, 8 heads of d 128 (3.2 GB)
// 480 to 494 us, 6.5 TB/s, a copy's rate; 256 lists of 64 pages of 64 keys (537 MB) 96 us, 5.6 TB/s in
// one round of CTAs; one sequence of 4,097 keys 9.6 us, the latency of two launches and of the
// chain table, keys, values, parts.
#include <cuda.h>

#include "kernels.h"
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace spr {
namespace paged {

using namespace spr::tc;

constexpr int BNR = kPagedRowsBN;

template <int D>
struct RowsCfg {
  static constexpr int ST = D == 128 ? 3 : 6;                  // stages: two CTAs per SM
  static constexpr uint32_t kTile = (uint32_t)BNR * D * 2;     // bytes of K (or V) of a stage
  static constexpr uint32_t kBytes = ST * 2 * kTile;
};

template <typename T>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// What an item reads, computed alike by the attention and the join.
struct Item {
  Seq s;
  int h;                   // key/value head
  int tok0;                // first token of the sequence (or of its unit)
  int row0, nrows;         // this item's rows among those of the sequence (unit)
  const int* list;         // page list (NULL: the whole cache)
  int cnt, total;          // list entries; keys of the stream
  int ns, part, slot;      // pieces of the item, this piece, first piece's slot of partial results
  bool bad;
};

// Pieces of whole sequences.  Sequence b has parts_b items of R rows per head, each of t_b tiles of
// keys (at most).  Of `target` pieces each gets floor(target t_b / sum t parts Hkv), at least one and
// none of fewer than min_split of t_b's tiles: no more than target pieces are of cut items, which is
// what the partial results have slots for, and pieces are about equally long however unequal the
// sequences are.  Every block computes this from
// q_start and kv_len.  By piece (JOIN false): the idx-th piece; by item (JOIN true): the idx-th cut
// item.  ns = 0: there is none.
struct Piece {
  int b, h, rows, part, ns, slot, lo, hi, len;     // rows: which of the sequence's items
};
template <int NT, bool JOIN>
__device__ __forceinline__ Piece find_piece(const Args& a, int idx, int R, int* sm /* [3 NT / 32 + 8] */) {
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
  int parts = 1;
  auto tiles_of = [&](int b, int& lo, int& hi, int& len) -> int {    // -1: no new tokens
    lo = a.q_start[b];
    hi = a.q_start[b + 1];
    len = a.kv_len[b];
    const Seq s = make_seq(a, b, lo, hi, len);
    if (s.n <= 0) return -1;
    // (more tokens than max_chunk: an error, and not more items than were counted on)
    if (a.ppu > 1) parts = (int)min((long long)a.ppu, ((long long)s.n * a.G + R - 1) / R);
    return (visible_end(s.len - 1, a.frame, s.len) + BNR - 1) / BNR;
  };
  int lo = 0, hi = 0, len = 0, t = -1;
  if (a.B == 1) {        // nothing to count
    t = tiles_of(0, lo, hi, len);
    int ns = t < 0 ? 0 : max(1, min(t / a.min_split, a.S / a.Hkv / parts));
    if (JOIN && ns <= 1) ns = 0;
    if (idx >= (long long)a.Hkv * parts * (JOIN ? 1 : ns)) ns = 0;
    const int item = ns == 0 ? 0 : (JOIN ? idx : idx / ns), h = parts == 1 ? item : item / parts;
    return Piece{0, h, item - h * parts, ns == 0 || JOIN ? 0 : idx - item * ns, ns, item * ns, lo, hi, len};
  }
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    t = tiles_of(b, lo, hi, len);
    mine += (long long)max(t, 0) * parts;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  long long* sums = reinterpret_cast<long long*>(sm);
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) total += sums[w];
  total *= a.Hkv;
  auto pieces_of = [&](int t) -> int {
    if (t < 2 * a.min_split) return t < 0 ? 0 : 1;
    const long long n = (long long)t * a.S / total;
    return n < 1 ? 1 : (int)(n < t / a.min_split ? n : t / a.min_split);
  };
  __syncthreads();
  // pieces, and pieces (by piece) or number (JOIN) of cut sequences before this thread's run
  int np = 0, nc = 0;
  for (int b = b0; b < b1; ++b) {
    if (run > 1) t = tiles_of(b, lo, hi, len);
    const int ns = pieces_of(t);
    np += parts * (JOIN ? (ns > 1) : ns);
    nc += ns > 1 ? parts * ns : 0;
  }
  int ip = np, ic = nc;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, ip, o), v = __shfl_up_sync(0xffffffffu, ic, o);
    if (lane >= o) {
      ip += u;
      ic += v;
    }
  }
  int* wp = sm;
  int* wc = sm + NW;
  int* f = sm + 2 * NW;
  if (lane == 31) {
    wp[warp] = ip;
    wc[warp] = ic;
  }
  if (tid == 0) f[1] = 0;
  __syncthreads();
  int ap = ip - np, ac = ic - nc;
#pragma unroll
  for (int w = 0; w < NW; ++w)
    if (w < warp) {
      ap += wp[w];
      ac += wc[w];
    }
  const long long at = (long long)idx;
  if (at >= (long long)ap * a.Hkv && at < (long long)(ap + np) * a.Hkv) {
    for (int b = b0; b < b1; ++b) {
      if (run > 1) t = tiles_of(b, lo, hi, len);
      const int ns = pieces_of(t);
      const int c = parts * (JOIN ? (ns > 1) : ns);
      if (at < (long long)(ap + c) * a.Hkv) {
        f[0] = b;
        f[1] = ns;
        f[2] = (int)(at - (long long)ap * a.Hkv);
        f[3] = ac * a.Hkv;
        f[4] = lo;
        f[5] = hi;
        f[6] = len;
        f[7] = parts;
        break;
      }
      ap += c;
      ac += ns > 1 ? parts * ns : 0;
    }
  }
  __syncthreads();
  Piece p;
  p.b = f[0];
  p.ns = f[1];
  if (p.ns == 0) return p;
  const int item = JOIN ? f[2] : f[2] / p.ns;
  parts = f[7];
  p.h = parts == 1 ? item : item / parts;
  p.rows = item - p.h * parts;
  p.part = JOIN ? 0 : f[2] - item * p.ns;
  p.slot = f[3] + item * p.ns;
  p.lo = f[4];
  p.hi = f[5];
  p.len = f[6];
  return p;
}

// kWhole: block x is a piece (or, JOIN, a cut item); kUnits: block (x, y, z) is piece z of item x (a
// unit, or R of its rows) and head y.  False: nothing to do.
template <int KIND, int NT, bool JOIN>
__device__ __forceinline__ bool load_item(const Args& a, int R, int* sm /* [3 NT / 32 + 8] */, Item& it) {
  it.list = nullptr;
  it.cnt = 0;
  if (KIND == kWhole) {
    const Piece p = find_piece<NT, JOIN>(a, blockIdx.x, R, sm);
    if (p.ns == 0) return false;
    it.s = make_seq(a, p.b, p.lo, p.hi, p.len);
    it.bad = it.s.bad;
    it.h = p.h;
    it.tok0 = 0;
    it.row0 = p.rows * R;
    it.nrows = (int)min((long long)R, (long long)it.s.n * a.G - it.row0);
    it.ns = p.ns;
    it.part = p.part;
    it.slot = p.slot;
    it.total = visible_end(it.s.len - it.s.n + (it.row0 + it.nrows - 1) / a.G, a.frame, it.s.len);
    return true;
  }
  const Found f = find_item<KIND, NT>(a, blockIdx.x, 0, a.ppu, sm);
  if (f.b < 0) return false;
  it.s = make_seq(a, f.b, f.lo, f.hi, f.len);
  it.bad = it.s.bad;
  it.h = blockIdx.y;
  const int unit = a.ppu == 1 ? f.rank : f.rank / a.ppu;
  it.tok0 = unit * a.q_block;
  it.row0 = (f.rank - unit * a.ppu) * R;
  const int ntok = min(a.q_block, it.s.n - it.tok0);
  it.nrows = (int)min((long long)R, (long long)ntok * a.G - it.row0);
  const size_t at = (size_t)(a.ppu == 1 ? blockIdx.x : blockIdx.x / a.ppu) * a.Hkv + it.h;
  it.list = a.sel + at * a.n_select;
  const int c = a.sel_cnt[at];
  it.cnt = min(max(c, 0), a.n_select);
  it.bad |= c != it.cnt;
  if (it.nrows <= 0) return false;
  const int end = visible_end(it.s.len - it.s.n + it.tok0 + ntok - 1, a.frame, it.s.len);
  int seen = it.cnt;
  it.total = stream_limit(end, it.list, it.cnt, a.page, &seen);
  // the unit's last token sees every page of its list, and no page is there twice
  it.bad |= seen != it.cnt || it.total > end;
  const int last = it.tok0 + (it.row0 + it.nrows - 1) / a.G;       // of these rows
  if (a.ppu > 1 && a.frame != 0)
    it.total = min(it.total, stream_limit(visible_end(it.s.len - it.s.n + last, a.frame, it.s.len), it.list, it.cnt, a.page));
  it.ns = split_count((it.total + BNR - 1) / BNR, a.S, a.min_split);
  it.part = JOIN ? 0 : blockIdx.z;
  it.slot = (int)(((size_t)blockIdx.x * a.Hkv + it.h) * a.S);
  return JOIN ? it.ns > 1 : it.part < it.ns;
}

// Page of stream row p (a multiple of the box height), checked: -1 if it may not be read.
__device__ __forceinline__ int stream_page(const Args& a, const Item& it, int p) {
  int j = p / a.page;
  if (it.list) {
    const int k = j;
    j = it.list[k];
    // lists ascend strictly and stay within the sequence
    if (j < 0 || (long long)j * a.page >= it.s.len || (k > 0 && it.list[k - 1] >= j)) return -1;
  }
  const int pid = a.table[(size_t)it.s.b * a.max_pages + j];
  return pid >= 0 && pid < a.n_pages ? pid : -1;
}

template <typename T, int D, int MT, int KIND>
__global__ void __launch_bounds__(128 * MT + 32) k_paged_rows(const __grid_constant__ CUtensorMap tmk,
                                                              const __grid_constant__ CUtensorMap tmv, Args a) {
  using C = RowsCfg<D>;
  constexpr int NT = 128 * MT + 32, NW = 4 * MT, ST = C::ST;
  constexpr float SHIFT = ProbShift<T>::v;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint64_t s_full[ST], s_empty[ST];
  __shared__ __align__(8) int s_find[3 * NT / 32 + 8];
  __shared__ int s_abort, s_bad;
  __shared__ float s_m[MT][4][16], s_l[MT][4][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = su32(smem);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");     // the join may get ready
  if (tid < 2) prefetch_tmap(tid ? &tmv : &tmk);
  if (base & 1023u) {
    if (tid == 0) set_error(a.err, DERR_INDEX);
    return;
  }
  Item it;
  if (!load_item<KIND, NT, false>(a, 16 * MT, s_find, it)) return;
  const int tiles = (it.total + BNR - 1) / BNR, ns = it.ns, h = it.h;
  const int t0 = split_at(tiles, it.part, ns), t1 = split_at(tiles, it.part + 1, ns);
  if (tid == 0) {
    s_abort = 0;
    s_bad = it.bad ? 1 : 0;
    if (it.bad) set_error(a.err, DERR_INDEX);
    for (int i = 0; i < ST; ++i) {
      mbar_init(su32(&s_full[i]), 1);
      mbar_init(su32(&s_empty[i]), NW);
    }
    fence_barrier_init();
  }
  __syncthreads();
  const int nrows = it.nrows;

  if (warp == NW) {
    // ---------------- producer ----------------
    const int box = min(a.page, BNR), boxes = BNR / box;          // boxes of a tile
    const int jobs = boxes * (D / 64) * 2;                        // box x column half x {K, V}; <= 16
    const int bx = lane / (D / 64 * 2), rest = lane % (D / 64 * 2), half = rest >> 1, isv = rest & 1;
    bool ok = true;
    int pid = 0, issued = 0;
    auto fetch = [&](int t) -> int {
      const int p = t * BNR + bx * box;
      return lane < jobs && t < t1 && p < it.total ? stream_page(a, it, p) : -2;
    };
    pid = fetch(t0);
    for (int t = t0; t < t1; ++t) {
      const int i = t - t0, st = i % ST;
      const int next = fetch(t + 1);
      if (lane == 0) ok = i < ST || bounded_wait(su32(&s_empty[st]), ((i / ST) - 1) & 1, &s_abort, a.err);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (pid == -1) {           // the rows become NaN; the load is replaced by a page that exists
        s_bad = 1;
        set_error(a.err, DERR_INDEX);
        pid = 0;
      }
      __syncwarp();
      const unsigned go = __ballot_sync(0xffffffffu, pid >= 0);
      if (lane == 0) mbar_arrive_expect_tx(su32(&s_full[st]), (uint32_t)__popc(go) * box * 128);
      __syncwarp();
      if (pid >= 0) {
        const int sub = (t * BNR + bx * box) % a.page;
        const uint32_t dst = base + st * 2 * C::kTile + isv * C::kTile + half * (BNR * 128) + bx * box * 128;
        tma_load_2d(dst, isv ? &tmv : &tmk, 64 * half, (pid * a.Hkv + h) * a.page + sub, su32(&s_full[st]));
      }
      pid = next;
      issued = i + 1;
    }
    // a wait that ran out: let the loads in flight land before the block ends
    if (!ok && lane == 0)
      for (int i = issued > ST ? issued - ST : 0; i < issued; ++i) drain_wait(su32(&s_full[i % ST]), (i / ST) & 1);
    __syncwarp();
  } else {
    // ---------------- 16 rows x 16-key slices ----------------
    if (KIND == kUnits && a.ppu > 1)
      // these rows may end before a wrong entry, which is read as it comes otherwise: the list is
      // the unit's, and so is its error
      for (int k = tid; k < it.cnt; k += 128 * MT)
        if (it.list[k] <= (k > 0 ? it.list[k - 1] : -1)) {
          s_bad = 1;
          set_error(a.err, DERR_INDEX);
        }
    const int mt = warp >> 2, sl = warp & 3;
    const int g = lane >> 2, q2 = (lane & 3) * 2;
    uint32_t qf[D / 16][4];
    int lim[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = mt * 16 + g + 8 * r;
      const bool in = row < nrows;
      const int tok = in ? (it.row0 + row) / a.G : 0, gh = in ? it.row0 + row - tok * a.G : 0;
      const T* qp = (const T*)a.Q + (long long)(it.s.q0 + it.tok0 + tok) * a.qst + (long long)(h * a.G + gh) * a.qsh;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][r] = in ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + q2) : 0u;
        qf[k][2 + r] = in ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + 8 + q2) : 0u;
      }
      lim[r] = it.total;
      if (in && a.frame != 0) {
        const int e = visible_end(it.s.len - it.s.n + it.tok0 + tok, a.frame, it.s.len);
        lim[r] = min(it.total, stream_limit(e, it.list, it.cnt, a.page));
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool ok = true;
    // K fragments: matrices (keys 0-7, k 0-7), (keys 0-7, k 8-15), (keys 8-15, k 0-7), (keys 8-15, k 8-15)
    const int kr = sl * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, kc = (lane >> 3) & 1;
    // V fragments: matrices (keys 0-7, n 0-7), (keys 8-15, n 0-7), (keys 0-7, n 8-15), (keys 8-15, n 8-15)
    const int vr = sl * 16 + (lane & 15), vc = lane >> 4;
    for (int t = t0; t < t1; ++t) {
      const int i = t - t0, st = i % ST;
      ok = __all_sync(0xffffffffu, bounded_wait(su32(&s_full[st]), (i / ST) & 1, &s_abort, a.err));
      if (!ok) break;
      const uint32_t sk = base + st * 2 * C::kTile, sv = sk + C::kTile;
      // even and odd steps of d in sums of their own: half the chain of dependent products
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      float so[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm4(b, sk + tile_off(kr, 2 * k + kc, BNR));
        mma16816<T>(k & 1 ? so[0] : s[0], qf[k], b[0], b[1]);
        mma16816<T>(k & 1 ? so[1] : s[1], qf[k], b[2], b[3]);
      }
      const int k0 = t * BNR + sl * 16;     // stream row of the slice's first key
      const bool edge = __any_sync(0xffffffffu, k0 + 16 > min(lim[0], lim[1]));
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = (s[n][e] + so[n][e]) * a.scale_log2;
          if (edge && k0 + n * 8 + q2 + (e & 1) >= lim[e >> 1]) x = -INFINITY;
          s[n][e] = x;
          mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
      bool moved = false;
      float mu[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        moved |= mx[r] > m[r];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float mn = fmaxf(m[r], mx[r]);
          const float al = m[r] == -INFINITY ? 0.f : ex2(m[r] - mn);
          m[r] = mn;
          l[r] *= al;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][2 * r] *= al;
            o[n][2 * r + 1] *= al;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) mu[r] = m[r] == -INFINITY ? 0.f : m[r] - SHIFT;
      uint32_t pf[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = ex2(s[n][2 * r] - mu[r]), p1 = ex2(s[n][2 * r + 1] - mu[r]);
          l[r] += p0 + p1;
          pf[2 * n + r] = pack2<T>(p0, p1);
        }
      const bool tail = k0 + 16 > it.total;   // value rows past the stream may hold anything
      uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
      if (tail) {
        const int left = it.total - k0 - q2;   // this thread's keys q2, q2 + 1, q2 + 8, q2 + 9
        keep0 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
        keep1 = (left > 8 ? 0xffffu : 0u) | (left > 9 ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldsm4t(b, sv + tile_off(vr, 2 * n + vc, BNR));
        if (tail) {
          b[0] &= keep0;
          b[1] &= keep1;
          b[2] &= keep0;
          b[3] &= keep1;
        }
        mma16816<T>(o[2 * n], pf, b[0], b[1]);
        mma16816<T>(o[2 * n + 1], pf, b[2], b[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(su32(&s_empty[st]));
    }
    // ---------------- join of the four slices ----------------
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if ((lane & 3) == 0) {
        s_m[mt][sl][g + 8 * r] = m[r];
        s_l[mt][sl][g + 8 * r] = l[r];
      }
    }
    named_sync(1 + mt, 128);
    float ms[2], ls[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_m[mt][w][g + 8 * r]);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float mw = s_m[mt][w][g + 8 * r];
        if (mw != -INFINITY) ll += s_l[mt][w][g + 8 * r] * ex2(mw - mm);
      }
      ms[r] = mm;
      ls[r] = ll;
      const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - mm);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][2 * r] *= f;
        o[n][2 * r + 1] *= f;
      }
    }
    // every stage has landed and been read by all warps of all row tiles: the buffers are free
    // (a row tile uses 4 x 16 x D x 4 bytes); each warp adds a quarter of the columns
    named_sync(15, 128 * MT);
    float4* buf = reinterpret_cast<float4*>(smem) + (size_t)mt * 4 * (D / 8) * 32;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) buf[((size_t)sl * (D / 8) + n) * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
    named_sync(1 + mt, 128);
    const bool poison = !ok || s_bad != 0 || s_abort != 0;
    float4 acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 v = buf[((size_t)w * (D / 8) + sl * (D / 32) + i) * 32 + lane];
        acc[i].x += v.x;
        acc[i].y += v.y;
        acc[i].z += v.z;
        acc[i].w += v.w;
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = mt * 16 + g + 8 * r;
      if (row >= nrows) continue;
      float inv = ls[r] > 0.f ? 1.f / ls[r] : 0.f;
      float z = ls[r] > 0.f ? (ms[r] - SHIFT + log2f(ls[r])) * 0.69314718055994531f : -INFINITY;
      if (!(ls[r] == ls[r]) || poison) inv = z = __int_as_float(0x7fffffff);
      const int tok = (it.row0 + row) / a.G, gh = it.row0 + row - tok * a.G;
      const long long qrow = it.s.q0 + it.tok0 + tok;
      const int qh = h * a.G + gh;
      const size_t prow = (size_t)(it.slot + it.part) * (16 * MT) + row;      // [slot][16 MT rows]
      T* op = (T*)a.O + qrow * a.ost + (long long)qh * a.osh;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int col = (sl * (D / 32) + i) * 8 + q2;
        const float x = (r ? acc[i].z : acc[i].x) * inv, y = (r ? acc[i].w : acc[i].y) * inv;
        if (ns > 1) *reinterpret_cast<float2*>(a.part_o + prow * D + col) = make_float2(x, y);
        else *reinterpret_cast<uint32_t*>(op + col) = pack2<T>(x, y);
      }
      if (sl == 0 && (lane & 3) == 0) {
        if (ns > 1) a.part_lse[prow] = z;
        else if (a.lse) a.lse[qrow * a.Hq + qh] = z;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Join of cut items: a block per cut item (kWhole) or per unit and head (kUnits), rows of the item
// dealt to the block's warps.
//   O = sum_s exp(lse_s - lse) O_s,  lse = ln sum_s exp(lse_s)
// ---------------------------------------------------------------------------
constexpr int kCombThreads = 256;

template <typename T, int D, int KIND>
__global__ void __launch_bounds__(kCombThreads) k_paged_combine(Args a, int max_rows) {
  __shared__ __align__(8) int s_find[3 * kCombThreads / 32 + 8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Item it;
  const bool any = load_item<KIND, kCombThreads, true>(a, max_rows, s_find, it);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");     // the parts are complete
  if (!any) return;
  const int nrows = it.nrows, ns = it.ns, h = it.h;
  for (int r = warp; r < nrows; r += kCombThreads / 32) {
    const int tok = (it.row0 + r) / a.G, qh = h * a.G + (it.row0 + r - tok * a.G);
    const size_t qrow = (size_t)it.s.q0 + it.tok0 + tok, prow = (size_t)it.slot * max_rows + r, step = max_rows;
    const float* po = a.part_o + prow * D + lane * (D / 32);
    constexpr int UN = 16;              // parts in flight; the first ones beside their lse
    float v[UN][D / 32];
    auto load = [&](int s0) {
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        if (s0 + i >= ns) continue;
        const float* p = po + (size_t)(s0 + i) * step * D;
        if constexpr (D == 128) {
          const float4 f = *reinterpret_cast<const float4*>(p);
          v[i][0] = f.x;
          v[i][1] = f.y;
          v[i][2] = f.z;
          v[i][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(p);
          v[i][0] = f.x;
          v[i][1] = f.y;
        }
      }
    };
    load(0);
    // the largest lse of all parts; the weights and their sum come with the parts
    float mx = -INFINITY;
    bool nan = false;
    for (int s = lane; s < ns; s += 32) {
      const float z = a.part_lse[prow + s * step];
      nan |= !(z == z);
      mx = fmaxf(mx, z);
    }
    mx = warp_max(mx);
    nan = __any_sync(0xffffffffu, nan);
    const float mu = mx == -INFINITY ? 0.f : mx;
    float den = 0.f;
    float acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
    for (int s0 = 0; s0 < ns; s0 += UN) {
      if (s0 > 0) load(s0);
      const float w = lane < UN && s0 + lane < ns ? expf(a.part_lse[prow + (s0 + lane) * step] - mu) : 0.f;
      den += warp_sum(w);
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const float ws = __shfl_sync(0xffffffffu, w, i);
        if (s0 + i >= ns) continue;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) acc[k] += ws * v[i][k];
      }
    }
    nan |= !(den == den);
    const float inv = nan ? __int_as_float(0x7fffffff) : (den > 0.f ? 1.f / den : 0.f);
    T* op = (T*)a.O + (long long)qrow * a.ost + (long long)qh * a.osh + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; i += 2)
      *reinterpret_cast<uint32_t*>(op + i) = pack2<T>(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0 && a.lse) a.lse[qrow * a.Hq + qh] = nan ? __int_as_float(0x7fffffff) : (den > 0.f ? mu + logf(den) : -INFINITY);
  }
}

}  // namespace paged

namespace {

template <typename T, int D, int MT, int KIND>
cudaError_t rows_t(const paged::Args& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  auto kern = paged::k_paged_rows<T, D, MT, KIND>;
  const size_t sm = paged::RowsCfg<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  // kWhole: at most S pieces of cut items and one of every other, and none of fewer than min_split
  // tiles of the longest possible stream
  const long long items = (long long)a.items * a.Hkv, tiles = ceil_div64((long long)a.max_pages * a.page, paged::BNR);
  long long pieces = a.B == 1 ? (items > a.S ? items : a.S) : items + a.S;
  const long long most = items * (tiles / a.min_split > 1 ? tiles / a.min_split : 1);
  pieces = pieces < most ? pieces : most;
  const dim3 grid = KIND == paged::kWhole ? dim3((unsigned)pieces) : dim3(a.items, a.Hkv, a.S);
  kern<<<grid, 128 * MT + 32, sm, st>>>(tk, tv, a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t rows_d(const paged::Args& a, const PagedPlan& pl, const CUtensorMap& tk, const CUtensorMap& tv,
                   cudaStream_t st) {
  if (pl.kind == paged::kUnits)
    return pl.mt == 1 ? rows_t<T, D, 1, paged::kUnits>(a, tk, tv, st) : rows_t<T, D, 2, paged::kUnits>(a, tk, tv, st);
  return pl.mt == 1 ? rows_t<T, D, 1, paged::kWhole>(a, tk, tv, st) : rows_t<T, D, 2, paged::kWhole>(a, tk, tv, st);
}

template <typename T, int D>
cudaError_t combine_t(const paged::Args& a, const PagedPlan& pl, cudaStream_t st) {
  const int rows = 16 * pl.mt;
  // fewer than S items are cut (kWhole)
  const long long items = (long long)a.items * a.Hkv;
  const dim3 grid = pl.kind == paged::kUnits ? dim3(a.items, a.Hkv) : dim3((unsigned)(items < a.S ? items : a.S));
  if (pl.kind == paged::kUnits) return launch_early(paged::k_paged_combine<T, D, paged::kUnits>, grid, paged::kCombThreads, 0, st, a, rows);
  return launch_early(paged::k_paged_combine<T, D, paged::kWhole>, grid, paged::kCombThreads, 0, st, a, rows);
}

}  // namespace

// Rows: the unit's (or the longest sequence's) tokens times the heads that share a key/value head.  Up
// to 32 are one item of the rows kernel, whatever the work: 32 rows of d 128 take 29 us there against
// 39 us in the 256-row tensor tiles (2 x 8 heads of 8,192 keys), 69 against 71 us (8 x 8 heads) and
// 113 against 113 us (16 x 8 heads).  More rows are cut into items of 32 as long as the call is small:
// the tiles' plan, their first chunks and their join take 20 us of latency, which the rows kernel
// does not have, and their rate counts beyond that.  By pairs of query row and key (as many as the
// pages and lists could hold), rows against tiles: 49 tokens x 2 heads, 383 keys (4 10^4) 10.8
// against 20.1 us; 70 x 8, 2,112 keys (10^6) 17.6 against 32.0; 978 x 8, 848 keys (7 10^6) 32.6
// against 33.4; 889 x 4, 6,904 keys (2 10^7) 88 against 39.  Lists, with their selection: 35 x 32, 5
// pages of 128 (7 10^5) 28 against 38 us; 577 x 2, 64 of 32 (2 10^6) 42 against 43; 180 x 32, 33 of 16
// (3 10^6) 63 against 57.
PagedPlan paged_plan(int B, int Hq, int Hkv, int page, int max_pages, int T, int max_chunk, int q_block, int n_select,
                     bool sel) {
  PagedPlan p{};
  const long long G = Hq / Hkv;
  const int most_new = max_chunk < T ? max_chunk : T;
  const long long tok = sel && q_block < most_new ? q_block : most_new;
  const long long rows = tok * G;
  const long long pairs = (long long)T * Hq * ((sel ? n_select : max_pages) * (long long)page);
  p.rows = rows <= 32 || pairs <= (sel ? 2000000 : 5000000);
  p.mt = rows <= 16 ? 1 : 2;
  p.ppu = 1;
  const long long units = sel ? ((long long)T + (q_block - 1ll) * B) / q_block : B;   // sum of ceil(n / q_block)
  long long items = units < T || !sel ? units : T;
  if (p.rows) {
    p.kind = sel ? paged::kUnits : paged::kWhole;
    if (rows > 32) {
      p.ppu = (int)ceil_div64(rows, 32);
      // kWhole: sum of ceil(n G / 32), at most ppu each
      const long long all = sel ? items * p.ppu : ((long long)T * G + 31ll * B) / 32, most = items * p.ppu;
      items = all < most ? all : most;
    }
  } else if (sel) {
    p.kind = paged::kUnits;
    p.ppu = (int)ceil_div64(rows, kPagedTileRows);
    items *= p.ppu;
  } else {
    p.kind = paged::kRows;
    items = ((long long)T * G + (kPagedTileRows - 1ll) * B) / kPagedTileRows;   // sum of ceil(n G / 256)
    const long long most = (long long)T * G;
    items = items < most ? items : most;
  }
  p.items = (int)items;
  p.min_split = 4;
  p.S = 1;
  if (!p.rows) return p;
  const int once = p.mt == 1 ? 296 : 148;       // resident CTAs: two per SM, or one of 32 rows
  if (!sel) {
    // One round when the items alone do not fill the GPU, whatever their lengths (16 x 8 heads of
    // 8,192 keys: 88 us, 91 us with two rounds, 97 us with four).  More items than that make a
    // last round of uncut ones, which four rounds of pieces keep short (48 sequences of 500 to
    // 32,000 keys: 494 us against 568 us; 64 equal ones of 8,192: 320 us against 304 us); of 32 rows
    // two rounds do (32 x 8 heads of 1,024 keys: 45 us, 64 us with four).
    p.S = items * Hkv < once ? once : (p.mt == 1 ? 4 : 2) * once;
    return p;
  }
  // lists are equally long: one round of CTAs (256 lists of 64 pages of 64 keys with their selection
  // take 126 us uncut, 96 of them here, and 145 us in four pieces)
  const long long most = ceil_div64((long long)max_pages * page, kPagedRowsBN) / p.min_split;
  long long S = items * Hkv > 0 ? once / (items * Hkv) : 1;
  S = S < most ? S : most;
  S = S < 64 ? S : 64;
  p.S = S < 1 ? 1 : (int)S;
  return p;
}

cudaError_t launch_paged_rows(const paged::Args& a, const PagedPlan& pl, int d, int dtype, const void* kp,
                              const void* vp, cudaStream_t st) {
  CUtensorMap tk{}, tv{};
  const unsigned long long rows = (unsigned long long)a.n_pages * a.Hkv * a.page;
  const int box = a.page < kPagedRowsBN ? a.page : kPagedRowsBN;
  cudaError_t e;
  if ((e = make_tmap_bf16_rows(&tk, kp, rows, d, box)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16_rows(&tv, vp, rows, d, box)) != cudaSuccess) return e;
  if (dtype == SPARSEPR_FP16) return d == 64 ? rows_d<__half, 64>(a, pl, tk, tv, st) : rows_d<__half, 128>(a, pl, tk, tv, st);
  return d == 64 ? rows_d<__nv_bfloat16, 64>(a, pl, tk, tv, st) : rows_d<__nv_bfloat16, 128>(a, pl, tk, tv, st);
}

cudaError_t launch_paged_combine(const paged::Args& a, const PagedPlan& pl, int d, int dtype, cudaStream_t st) {
  if (dtype == SPARSEPR_FP16) return d == 64 ? combine_t<__half, 64>(a, pl, st) : combine_t<__half, 128>(a, pl, st);
  return d == 64 ? combine_t<__nv_bfloat16, 64>(a, pl, st) : combine_t<__nv_bfloat16, 128>(a, pl, st);
}

}  // namespace spr
