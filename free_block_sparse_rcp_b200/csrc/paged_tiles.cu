// Attention of a chunk of new tokens over the paged cache on the 5th-generation tensor cores.
//
// An item is up to 256 query rows (tokens x the query heads of one key/value head) that share
// one stream of keys: the pages of their sequence, or of their unit's list, in order.  Two
// 128-row tiles use every 128-key chunk that reaches shared memory, so the tensor cores work on
// one tile while the other's softmax runs.
//   warps 0-3, 4-7   softmax and epilogue of tile 0 and 1: thread r owns query row r = TMEM lane r
//   warp 8           TMA: boxes of min(page, 128) rows of the pages of a chunk (K ring of 3, V
//                    ring of 2)
//   warp 9           issues the MMAs
// TMEM (512 columns): tile t holds S at 256 t and O at 256 t + 128; P overlays the first 64
// columns of S as packed 16-bit pairs and is the second product's A operand.
// Everything a row may see is a prefix of the stream, so the mask is one comparison with the
// row's limit in the chunks that straddle one.  Value rows of the last chunk past the item's
// last visible key are zeroed in shared memory before their MMA: a page's unused slots may hold
// NaN, and 0 NaN would reach every row.
// With splits (grid z) an item's chunks are divided and k_paged_combine joins the parts.
#include <cuda.h>

#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace spr {
namespace paged {

using namespace spr::tc;

constexpr int BM = 128, TPC = 2, BN = kPagedTileBN, KST = 3, VST = 2;
constexpr int NSOFT = 256, PROD_WARP = 8, MMA_WARP = 9, NTT = 320;
constexpr uint32_t kCols = 512;

struct TileBars {
  uint64_t q, kfull[KST], kempty[KST], vfull[VST], vempty[VST], vtail, s_full[TPC], p_full[TPC][2], pv_half[TPC],
      o_done[TPC], mma_done;
};

template <int D>
struct TileLayout {
  static constexpr uint32_t kTile = (uint32_t)D * 128 * 2;
  static constexpr uint32_t oQ = 0;
  static constexpr uint32_t oK = oQ + TPC * kTile;
  static constexpr uint32_t oV = oK + KST * kTile;
  static constexpr uint32_t oBar = oV + VST * kTile;
  static constexpr uint32_t oInt = oBar + 256;
  static constexpr uint32_t kBytes = oInt + 256;
};
static_assert(sizeof(TileBars) <= 256, "barrier block");

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
  constexpr float SHIFT = ProbShift<T>::v;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = su32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (base & 1023u) {
    if (tid == 0) set_error(a.err, DERR_INDEX);
    return;
  }
  TileBars* bars = reinterpret_cast<TileBars*>(smem + L::oBar);
  // [0] tmem base, [1] abort, [2] bad input, [4..] scratch of the item search
  int* ints = reinterpret_cast<int*>(smem + L::oInt);
  volatile int* abort_flag = ints + 1;
  volatile int* bad_flag = ints + 2;

  // ---------------- the item ----------------
  // the last parts of a causal sequence see the most keys: items are taken from the back
  const int idx = a.items - 1 - (int)blockIdx.x, h = blockIdx.y;
  Seq s;
  int row0, nrows, tok0 = 0, cnt = 0;
  const int* list = nullptr;
  bool bad;
  if (SEL) {
    const int2 f = find_item<kUnits, NTT>(a.q_start, a.B, a.T, idx, a.G, 0, a.q_block, a.ppu, ints + 4);
    if (f.x < 0) return;
    s = load_seq(a, f.x);
    bad = s.bad;
    const int u = f.y / a.ppu, part = f.y - u * a.ppu;
    tok0 = u * a.q_block;
    row0 = part * kPagedTileRows;
    nrows = min(kPagedTileRows, min(a.q_block, s.n - tok0) * a.G - row0);
    if (nrows <= 0) return;
    const size_t at = (size_t)(idx / a.ppu) * a.Hkv + h;
    list = a.sel + at * a.n_select;
    const int c = a.sel_cnt[at];
    cnt = min(max(c, 0), a.n_select);
    const int last = tok0 + min(a.q_block, s.n - tok0) - 1;     // sees every page of the list
    int seen = cnt;
    stream_limit(visible_end(s.len - s.n + last, a.frame, s.len), list, cnt, a.page, &seen);
    bad |= c != cnt || seen != cnt;
  } else {
    const int2 f = find_item<kRows, NTT>(a.q_start, a.B, a.T, idx, a.G, kPagedTileRows, 1, 1, ints + 4);
    if (f.x < 0) return;
    s = load_seq(a, f.x);
    bad = s.bad;
    row0 = f.y * kPagedTileRows;
    nrows = (int)min((long long)kPagedTileRows, (long long)s.n * a.G - row0);
  }
  // stream limit of row r of the item
  auto limit_of = [&](int r) -> int {
    const int tok = tok0 + (row0 + r) / a.G;
    return stream_limit(visible_end(s.len - s.n + tok, a.frame, s.len), list, cnt, a.page);
  };
  const int total = limit_of(nrows - 1);
  const int ntile = nrows > BM ? 2 : 1;
  const int chunks = (total + BN - 1) / BN;
  const int ns = split_count(chunks, a.S, a.min_split);
  if ((int)blockIdx.z >= ns) return;
  const int c0 = split_at(chunks, blockIdx.z, ns), c1 = split_at(chunks, blockIdx.z + 1, ns);
  const int nch = c1 - c0;
  // tile 0 stops at its own last row's limit
  const int nch0 = ntile == 1 ? nch : min(nch, max(0, (limit_of(BM - 1) + BN - 1) / BN - c0));

  if (tid == 0) {
    ints[1] = 0;
    ints[2] = bad ? 1 : 0;
    if (bad) set_error(a.err, DERR_INDEX);
    mbar_init(su32(&bars->q), NSOFT);
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
      mbar_init(su32(&bars->p_full[t][0]), 128);
      mbar_init(su32(&bars->p_full[t][1]), 128);
      mbar_init(su32(&bars->pv_half[t]), 1);
      mbar_init(su32(&bars->o_done[t]), 1);
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
  const uint32_t tmem = (uint32_t)ints[0];
  const uint32_t sQ = base + L::oQ, sK = base + L::oK, sV = base + L::oV;
  auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
    return bounded_wait(su32(&bar), parity, abort_flag, a.err);
  };

  if (warp == PROD_WARP) {
    // ---------------- TMA ----------------
    const int box = a.page, boxes = BN / box;             // page <= 128 = BN
    const int jobs = boxes * (D / 64);                    // column halves of the boxes, <= 16
    const int bx = lane / (D / 64), half = lane % (D / 64);
    auto fetch = [&](int c) -> int {                      // page of this lane's box of chunk c
      const long long p = (long long)c * BN + bx * box;
      if (lane >= jobs || c >= c1 || p >= total) return -2;
      int j = (int)(p / box);
      if (SEL) {
        const int k = j;
        j = list[k];
        if (j < 0 || (long long)j * box >= s.len || (k > 0 && list[k - 1] >= j)) return -1;
      }
      const int pid = a.table[(size_t)s.b * a.max_pages + j];
      return pid >= 0 && pid < a.n_pages ? pid : -1;
    };
    bool ok = true;
    int pid = fetch(c0), kis = 0, vis = 0;
    for (int j = 0; j < nch; ++j) {
      const int ks = j % KST, vs = j % VST;
      const int next = fetch(c0 + j + 1);
      if (pid == -1) {        // the rows become NaN; a page that exists is loaded instead
        *bad_flag = 1;
        set_error(a.err, DERR_INDEX);
        pid = 0;
      }
      __syncwarp();
      const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, pid >= 0)) * box * 128;
      const uint32_t off = half * 16384 + bx * box * 128;
      const int y = (pid * a.Hkv + h) * box;
      if (lane == 0) {
        ok = j < KST || wait(bars->kempty[ks], ((j / KST) - 1) & 1);
        if (ok) mbar_arrive_expect_tx(su32(&bars->kfull[ks]), bytes);
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (pid >= 0) tma_load_2d(sK + ks * L::kTile + off, &tmk, 64 * half, y, su32(&bars->kfull[ks]));
      kis = j + 1;
      const bool tail = (c0 + j + 1) * (long long)BN > total;
      uint64_t* vbar = tail ? &bars->vtail : &bars->vfull[vs];
      if (lane == 0) {
        ok = j < VST || wait(bars->vempty[vs], ((j / VST) - 1) & 1);
        if (ok) mbar_arrive_expect_tx(su32(vbar), bytes);
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (pid >= 0) tma_load_2d(sV + vs * L::kTile + off, &tmv, 64 * half, y, su32(vbar));
      if (!tail) {
        vis = j + 1;
      } else {
        // zero the value rows past the last visible key, then hand the stage over
        ok = __all_sync(0xffffffffu, wait(bars->vtail, 0));
        if (!ok) {
          if (lane == 0) drain_wait(su32(&bars->vtail), 0);
          __syncwarp();
          break;
        }
        const int first = total - (c0 + j) * BN;
        const uint32_t v = sV + vs * L::kTile;
        for (int e = lane; e < (BN - first) * (D / 8); e += 32) {
          const int r = first + e / (D / 8), c = e % (D / 8);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(v + tile_off(r, c, BN)), "r"(0) : "memory");
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(su32(&bars->vfull[vs]));
      }
      pid = next;
    }
    if (!ok && lane == 0) {   // a wait ran out: let the loads in flight land
      for (int i = kis > KST ? kis - KST : 0; i < kis; ++i) drain_wait(su32(&bars->kfull[i % KST]), (i / KST) & 1);
      for (int i = vis > VST ? vis - VST : 0; i < vis; ++i) drain_wait(su32(&bars->vfull[i % VST]), (i / VST) & 1);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ---------------- MMA issuer (the whole warp, converged) ----------------
    constexpr uint32_t IDS = idesc_t<T>(128, BN, false);
    constexpr uint32_t IDO = idesc_t<T>(128, D, true);
    const uint32_t lead = elect_one();
    auto waits = [&](uint64_t& bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
    bool ok = nch == 0 || waits(bars->q, 0);
    auto count = [&](int t) -> int { return t == 0 ? nch0 : nch; };
    auto first_user = [&](int j) -> int { return j < nch0 ? 0 : 1; };
    // S_t = Q_t K_j^T; the last tile releases K_j
    auto issue_s = [&](int t, int j) -> bool {
      const int ks = j % KST;
      if (t == first_user(j)) {
        if (!waits(bars->kfull[ks], (j / KST) & 1)) return false;
        tc_fence_after();
      }
      const uint64_t kd = sdesc(sK + ks * L::kTile, 16, 1024), qd = sdesc(sQ + t * L::kTile, 16, 1024);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
        tc_mma_lead(lead, tmem + 256 * t, qd + off, kd + off, IDS, k > 0 ? 1u : 0u);
      }
      tc_commit_lead(lead, su32(&bars->s_full[t]));
      if (t == ntile - 1) tc_commit_lead(lead, su32(&bars->kempty[ks]));
      return true;
    };
    // O_t += P_t V_j, P from TMEM, half a chunk at a time; the last tile releases V_j
    auto issue_pv = [&](int t, int j) -> bool {
      const int vs = j % VST;
      const uint64_t vd = sdesc(sV + vs * L::kTile, 16384, 1024);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        if (!waits(bars->p_full[t][hh], j & 1)) return false;
        if (hh == 0 && t == first_user(j) && !waits(bars->vfull[vs], (j / VST) & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 4 * hh; k < 4 * hh + 4; ++k)
          tc_mma_ts_lead(lead, tmem + 256 * t + 128, tmem + 256 * t + k * 8, vd + k * 128, IDO,
                         (j > 0 || k > 0) ? 1u : 0u);
        if (hh == 0) tc_commit_lead(lead, su32(&bars->pv_half[t]));
      }
      if (t == ntile - 1) tc_commit_lead(lead, su32(&bars->vempty[vs]));
      return true;
    };
    for (int t = 0; ok && t < ntile; ++t)
      if (count(t) > 0) ok = issue_s(t, 0);
    bool early0 = false;
    for (int j = 0; ok && j < nch; ++j) {
      for (int t = 0; ok && t < ntile; ++t) {
        if (j >= count(t)) continue;
        ok = issue_pv(t, j);
        if (ok && j + 1 < count(t)) ok = issue_s(t, j + 1);
        if (ok && t == 0 && ntile > 1 && j + 1 == nch0) {   // tile 0 may end before the item
          tc_commit_lead(lead, su32(&bars->o_done[0]));
          early0 = true;
        }
      }
    }
    for (int t = 0; t < ntile; ++t)
      if (!(t == 0 && early0)) tc_commit_lead(lead, su32(&bars->o_done[t]));
    tc_commit_lead(lead, su32(&bars->mma_done));   // every MMA completes before the TMEM is released
    if (!waits(bars->mma_done, 0) && lane == 0) drain_wait(su32(&bars->mma_done), 0);
    __syncwarp();
  } else {
    // ---------------- softmax + epilogue ----------------
    // query rows of both tiles, 16 bytes at a time (rows past the item are zero)
    for (int e = tid; e < ntile * BM * (D / 8); e += NSOFT) {
      const int r = e / (D / 8), c = e % (D / 8);
      const int tr = (row0 + r) / a.G, gh = row0 + r - tr * a.G;
      const bool in = r < nrows;
      const T* qp = (const T*)a.Q + (in ? (long long)(s.q0 + tok0 + tr) * a.qst + (long long)(h * a.G + gh) * a.qsh : 0);
      cp_async16(sQ + (r / BM) * L::kTile + tile_off(r % BM, c, 128), qp + c * 8, in);
    }
    cp_async_wait_all();
    fence_proxy_async();
    mbar_arrive(su32(&bars->q));

    const int t = warp >> 2;
    const int r = tid & (BM - 1);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 256 * t + lane_off, tO = tS + 128;
    const int row = t * BM + r;
    const bool in = row < nrows;
    const int nct = t < ntile ? (t == 0 ? nch0 : nch) : 0;
    const int lim = in ? min(total, limit_of(row)) : total;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    if (t < ntile) {
      const uint64_t sc2 = f2pack(a.scale_log2, a.scale_log2);
      // 32 columns of S to probabilities against the running maximum; returns with the packed
      // row sum in rs2
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
      // half hh of chunk j against its own maximum: O is rescaled first
      auto redo = [&](int j, int hh, int left, uint32_t* pk) {
        uint32_t sr[32];
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tc_ld32(tS + 64 * hh + 32 * q, sr);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (32 * q + c < left) mx = fmaxf(mx, __uint_as_float(sr[c]));
        }
        const float m_new = fmaxf(m_used, mx * a.scale_log2);
        float alpha = 1.f;
        if (m_new > m_used) {
          alpha = (m_used == -INFINITY) ? 0.f : ex2(m_used - m_new);
          m_used = m_new;
        }
        // the products of the earlier chunks completed before S_t,j did; those of this chunk's
        // first half are waited for
        if (hh == 1) ok = ok && __all_sync(0xffffffffu, wait(bars->pv_half[t], j & 1));
        if (j > 0 || hh == 1) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            tc_ld32(tO + c * 32, sr);
#pragma unroll
            for (int e = 0; e < 32; ++e) sr[e] = __float_as_uint(__uint_as_float(sr[e]) * alpha);
            tc_st32(tO + c * 32, sr);
          }
        }
        l *= alpha;
        const float mu = (m_used == -INFINITY) ? 0.f : m_used - SHIFT;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tc_ld32(tS + 64 * hh + 32 * q, sr);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float p0 = 32 * q + c < left ? ex2(__uint_as_float(sr[c]) * a.scale_log2 - mu) : 0.f;
            const float p1 = 32 * q + c + 1 < left ? ex2(__uint_as_float(sr[c + 1]) * a.scale_log2 - mu) : 0.f;
            l += p0 + p1;
            pk[16 * q + (c >> 1)] = pack2<T>(p0, p1);
          }
        }
      };
      for (int j = 0; j < nct; ++j) {
        ok = __all_sync(0xffffffffu, wait(bars->s_full[t], j & 1));
        if (!ok) break;
        tc_fence_after();
        const int valid = lim - (c0 + j) * BN;
        const bool full = __all_sync(0xffffffffu, valid >= BN);
        uint32_t ra[32], rb[32], pk[32];
        tc_ld32_start(tS, ra);
        tc_ld32_start(tS + 32, rb);
        tc_ld32_wait(ra);
        tc_ld32_wait(rb);
        // one speculative pass of each half against the running maximum, kept while the half's
        // row sum stays in range
        auto chunk = [&](auto masked) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int left = valid - 64 * hh;
            const bool spec = __all_sync(0xffffffffu, m_used != -INFINITY);
            const float nm = SHIFT - m_used;
            const uint64_t nmu2 = f2pack(nm, nm);
            uint64_t rs2 = 0ull;
            probs(masked, ra, pk, left, nmu2, rs2);
            if (hh == 0) tc_ld32_start(tS + 64, ra);
            probs(masked, rb, pk + 16, left - 32, nmu2, rs2);
            if (hh == 0) tc_ld32_start(tS + 96, rb);
            float r0, r1;
            f2unpack(rs2, r0, r1);
            const bool keep = spec && r0 + r1 <= ProbBound<T>::v;
            if (hh == 0) {
              tc_ld32_wait(ra);
              tc_ld32_wait(rb);
            }
            if (__all_sync(0xffffffffu, keep)) l += r0 + r1;
            else redo(j, hh, left, pk);
            tc_st32(tS + 32 * hh, pk);
            tc_fence_before();
            mbar_arrive(su32(&bars->p_full[t][hh]));
          }
        };
        if (full) chunk(std::false_type{});
        else chunk(std::true_type{});
      }
      if (ok && nct > 0) ok = __all_sync(0xffffffffu, wait(bars->o_done[t], 0));
      tc_fence_after();
      const bool poison = !ok || *bad_flag != 0 || !(l == l);
      const float inv = poison ? __int_as_float(0x7fffffff) : (l > 0.f ? 1.f / l : 0.f);
      const float z = poison ? __int_as_float(0x7fffffff)
                             : (l > 0.f ? (m_used - SHIFT + log2f(l)) * 0.69314718055994531f : -INFINITY);
      const int tr = (row0 + row) / a.G, gh = row0 + row - tr * a.G;
      const long long qrow = in ? s.q0 + tok0 + tr : 0;
      const int qh = h * a.G + (in ? gh : 0);
      const size_t prow = ((size_t)blockIdx.z * a.T + qrow) * a.Hq + qh;
      T* orow = (T*)a.O + qrow * a.ost + (long long)qh * a.osh;
      float* prt = a.part_o + prow * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (nct > 0 && ok) {
          tc_ld32(tO + c * 32, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (in) {
          if (ns > 1) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(prt + c * 32 + e) =
                  make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                              __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
          } else {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w[e] = pack2<T>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        }
      }
      if (in) {
        if (ns > 1) a.part_lse[prow] = z;
        else if (a.lse) a.lse[qrow * a.Hq + qh] = z;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tc_dealloc(tmem, kCols);
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
  kern<<<dim3(a.items, a.Hkv, a.S), paged::NTT, sm, st>>>(tk, tv, a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t tiles_d(const paged::Args& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  return a.sel ? tiles_t<T, D, true>(a, tk, tv, st) : tiles_t<T, D, false>(a, tk, tv, st);
}

}  // namespace

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
