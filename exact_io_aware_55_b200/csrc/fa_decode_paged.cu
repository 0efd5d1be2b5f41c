// Attention of a few new queries per request over an 8-bit paged KV cache.
//
//   s_j = scale * ks_j * (q . K_j)        K_j, V_j e4m3 codes; ks_j, vs_j the
//   p_j = softmax over the visible keys   scales of key j's page and KV head
//   O   = sum_j p_j * vs_j * V_j,  LSE = ln sum_j exp(s_j)
// Key j of a request is row j % P of page block_table[b][j / P]; keys at or
// past the request's length are never used, whatever their bytes hold.  A row
// without a visible key gives O = 0 and LSE = -inf.
//
// Bound by memory: every code is read once, 2 d bytes per token and KV head.
// The codes therefore go from the pages straight to the tensor cores, as the
// A operand of both products, and are never converted:
//   S^T = K Q^T     keys x rows (M = 128 keys).  A bf16 query is the sum of two
//                   e4m3 values: with the row scaled to |q| < 256, hi rounds to
//                   4 bits and lo = 16 (q - hi) holds the other 4, so hi and lo
//                   are two columns of the B operand and the scores are those
//                   of the bf16 query (elements below 2^-10 of the row's
//                   largest keep 2^-22 of it).
//   O^T += V^T P^T  d x rows (A = V tile, MN-major).  p * vs is rounded to fp16
//                   and split into three e5m2 parts, hi + mid/8 + lo/64, which
//                   is exact: 11 bits in three times 3 plus the signs.  e5m2 has
//                   fp16's exponent range, so a key down to 2^-29 of the largest
//                   keeps its 11 bits.  A and B of one product may differ in
//                   type among the 8-bit floats.
// A page's K scale multiplies its keys' scores; its V scale is added to the
// score's exponent (t = s + log2 vs, P = exp2(t - m)), so that the parts cannot
// overflow whatever the scales are, and l sums exp2(t - m) / vs.
//
// Work.  A unit is (request, KV head, tile of up to R query rows); its keys are
// cut into tiles of 128 (d = 128) or 256 (d = 64) tokens, 32 KB of codes.  The
// lengths are known on the device only, so every CTA adds them up itself and
// takes an equal share of all tiles, a contiguous range that may begin and end
// inside a unit.  A unit that lies within one CTA is written directly; of a
// unit cut between CTAs each CTA leaves its normalised O and LSE in one of its
// two slots of the workspace (one for a piece that does not begin its unit, one
// for a piece that does), the CTA that ends the unit notes who took part, and
// paged_merge_kernel combines them by their log-sum-exp.  No atomics: a call's
// results do not depend on timing.
//
// Warps: 0 page ids and TMA, 1 MMA issuer and TMEM owner, 2 page scales,
// 3 queries, 4-7 and 8-11 softmax (thread = key, each group half of the rows;
// TMEM lane quarter = warp % 4), 12-15 epilogue.  Pages that lie behind the length or outside the cache are not
// loaded; the softmax warps clear the V rows of keys that are not there, since
// p = 0 times a stale NaN code would be NaN.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kPgThreads = 512;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescaleThreshold = 4.0f;   // log2 units
constexpr float kBase = 2048.0f;            // P is scaled by 2^11: at most 2^15, of e5m2's 57344

template <int D, int R>
struct PgShape {
  static constexpr int kSub = (D == 64) ? 2 : 1;              // 128-key sub-tiles per tile
  static constexpr int kTileKeys = 128 * kSub;
  static constexpr int kTileBytes = kTileKeys * D;            // K (or V) codes of one tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kNS = (R == 32) ? 5 : 6;               // ring depth: 160 or 192 KB
  static constexpr int kMaxPages = kTileKeys / 16;
  static constexpr int kQRows = 2 * R;                        // hi, lo
  static constexpr int kQBytes = kQRows * D;
  static constexpr int kPRows = (R == 8) ? 32 : 3 * R;        // hi, mid, lo (and zero rows up to a multiple of 16)
  static constexpr int kPSub = kPRows * 128;                  // P^T of one sub-tile
  static constexpr int kPBytes = kSub * kPSub;
  static constexpr int kKSteps = D / 32;                      // S^T k-steps per sub-tile
  static constexpr int kPvSteps = kTileKeys / 32;             // O^T k-steps per tile
  static constexpr uint32_t kIdS = idesc_e4m3(128, kQRows, false, false);
  static constexpr uint32_t kIdO = idesc_e4m3(D, kPRows, true, false) | (1u << 10);   // B format 1: e5m2
  static constexpr uint32_t kColS = 0;                        // two S^T buffers of kQRows * kSub columns
  static constexpr uint32_t kColO = 2 * kQRows * kSub;        // two O^T buffers of kPRows columns
  static constexpr uint32_t kCols = kColO + 2 * kPRows;
  static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM columns");
};

template <int R, int NS, int PAGES>
struct PgBarriers {
  uint64_t kv_full[NS], kv_empty[NS];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2], pv_done[2];
  uint64_t o_full[2], o_free[2];
  uint64_t stats_full[2];
  alignas(16) float4 page[NS][PAGES];      // per page of a tile: K factor, log2 vs, 1 / vs, share of vs
  alignas(16) float q_factor[2][R];        // power of two that a row of queries was divided by
  alignas(16) float red_max[4][R];         // per-warp tile maxima (log2 units)
  alignas(16) float stat_m[2][R];          // piece's running max
  alignas(16) float stat_l[2][4][R];       // piece's per-warp sums
  long long scan[kPgThreads / 32];
  long long start_base;
  int start_b;
  uint32_t tmem_base;
  uint32_t abort;
};

template <int D, int R>
using PgBar = PgBarriers<R, PgShape<D, R>::kNS, PgShape<D, R>::kMaxPages>;

template <int D, int R>
constexpr size_t pg_smem_bytes() {
  using S = PgShape<D, R>;
  return 1024 + size_t(S::kNS) * S::kStageBytes + 2 * S::kQBytes + 2 * S::kPBytes + sizeof(PgBar<D, R>);
}

// Shared-memory matrix descriptor: rows of D bytes, swizzled over D bytes.
template <int D>
__device__ __forceinline__ uint64_t pg_desc(uint32_t saddr) {
  uint64_t d = sdesc_sw128(saddr, 16, 8 * D);
  if (D == 64) d = (d & ~(uint64_t(7) << 61)) | (uint64_t(4) << 61);   // 64-byte swizzle
  return d;
}
// 16-byte unit `c` of row `row` in that layout, as a byte offset.
template <int D>
__device__ __forceinline__ int pg_unit(int row, int c) {
  return row * D + ((D == 128 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & 3))) << 4);
}

__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// Hardware barrier of the 128 threads of a softmax group, and one that also
// tells whether `x` holds for any of them.
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(static_cast<uint32_t>(x)), "r"(id)
      : "memory");
  return y != 0;
}
// Two warp-uniform waits whose first looks overlap.
__device__ __forceinline__ bool mbar_wait2_warp(uint64_t* x, uint32_t px, uint64_t* y, uint32_t py, const WaitCtx& w,
                                                uint32_t where) {
  const bool a = mbar_try_wait(x, px), b = mbar_try_wait(y, py);
  if (__all_sync(0xffffffffu, a && b)) return true;
  return mbar_wait_warp(x, px, w, where) && mbar_wait_warp(y, py, w, where);
}

// N (4, 8, 16) consecutive TMEM columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[N]) {
  if constexpr (N == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(t) : "memory");
  else if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t) : "memory");
  else
    tmem_ld_x16(t, r);
}
// Two such loads with one wait.
template <int N>
__device__ __forceinline__ void tmem_ld2(uint32_t t, uint32_t t2, uint32_t (&r)[N], uint32_t (&q)[N]) {
  if constexpr (N == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%8];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%4, %5, %6, %7}, [%9];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
                 : "r"(t), "r"(t2) : "memory");
  else if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7])
                 : "r"(t), "r"(t2) : "memory");
  else {
    tmem_ld_x16(t, r);
    tmem_ld_x16(t2, q);
  }
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[N]) {
  if constexpr (N == 4)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]) : "memory");
  else if constexpr (N == 8)
    tmem_st_x8(t, r);
  else
    tmem_st_x16(t, r);
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__device__ __forceinline__ int pg_len(const PagedArgs& a, int b) { return min(max(a.seq_lens[b], 0), a.max_pages * a.page); }

// A piece: tiles [j0, j0 + n) of one unit.
struct Piece {
  int b, unit, len, nt, j0, n;
};
// Walks over a CTA's range of tiles, piece by piece.
template <int TILE>
struct Walk {
  const PagedArgs& a;
  long long g, g1, base;      // next tile, end of the range, first tile of request b
  int b, len, nt;
  __device__ __forceinline__ Walk(const PagedArgs& a_, long long g0, long long g1_, int b0, long long base0)
      : a(a_), g(g0), g1(g1_), base(base0), b(b0), len(0), nt(0) {
    if (g < g1) load();
  }
  __device__ __forceinline__ void load() {
    len = pg_len(a, b);
    nt = (len + TILE - 1) / TILE;
  }
  // Unit and tile of position `at` (>= g of the last call).
  __device__ __forceinline__ void seek(long long at, int& unit, int& j) {
    while (at >= base + static_cast<long long>(nt) * a.units) {
      base += static_cast<long long>(nt) * a.units;
      ++b;
      load();
    }
    const int local = static_cast<int>(at - base);
    unit = local / nt;
    j = local - unit * nt;
  }
  __device__ __forceinline__ bool next(Piece& p) {
    if (g >= g1) return false;
    seek(g, p.unit, p.j0);
    p.b = b;
    p.len = len;
    p.nt = nt;
    p.n = static_cast<int>(min(static_cast<long long>(nt - p.j0), g1 - g));
    g += p.n;
    return true;
  }
};

// Page ids of a CTA's tiles, 32 at a time: lane (u, i) has page i of tile
// t0 + u, with ids of the next batch fetched while this one is used.
template <int TILE>
struct PageBatch {
  const PagedArgs& a;
  Walk<TILE> w;
  long long g0;
  int n, per_tile, tiles, u, i;
  __device__ __forceinline__ PageBatch(const PagedArgs& a_, long long g0_, int n_, int b0, long long base0, int lane)
      : a(a_), w(a_, g0_, g0_ + n_, b0, base0), g0(g0_), n(n_) {
    per_tile = TILE / a.page;
    tiles = 32 / per_tile;
    u = lane / per_tile;
    i = lane - u * per_tile;
  }
  // (page, KV head) row of this lane's page in the batch that starts at tile
  // t0: -1 where the tile has no such page, -2 where the table names none.
  __device__ __forceinline__ long long fetch(int t0) {
    const int t = t0 + u;
    if (t >= n) return -1;
    int unit, j;
    w.seek(g0 + t, unit, j);
    const int lp = j * per_tile + i;
    if (lp * a.page >= w.len) return -1;
    const int id = a.block_table[static_cast<size_t>(w.b) * a.max_pages + lp];
    if (id < 0 || id >= a.num_pages) return -2;
    return static_cast<long long>(id) * a.Hkv + unit / a.row_tiles;
  }
};

template <int D, int R>
__global__ void __launch_bounds__(kPgThreads, 1)
    decode_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const PagedArgs a) {
  using S = PgShape<D, R>;
  constexpr int NS = S::kNS, U = S::kSub, TILE = S::kTileKeys;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;                               // NS x (K tile, V tile)
  uint8_t* sP = sKV + NS * S::kStageBytes;           // 2 x P^T
  uint8_t* sQ = sP + 2 * S::kPBytes;                 // 2 x (hi, lo) queries
  auto* b = reinterpret_cast<PgBar<D, R>*>(sQ + 2 * S::kQBytes);
  const WaitCtx wc{&b->abort, a.status, FA_WAIT_LIMIT_NS};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&b->kv_full[s], 2);
      mbar_init(&b->kv_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->q_full[i], 1);
      mbar_init(&b->q_empty[i], 9);
      mbar_init(&b->s_full[i], 1);
      mbar_init(&b->s_free[i], 8);
      mbar_init(&b->p_full[i], 8);
      mbar_init(&b->pv_done[i], 1);
      mbar_init(&b->o_full[i], 1);
      mbar_init(&b->o_free[i], 4);
      mbar_init(&b->stats_full[i], 8);
    }
    b->abort = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&b->tmem_base, S::kTmemCols);
    tmem_relinquish();
  }
  if (R == 8) {                                      // the zero rows of P^T
    for (int i = threadIdx.x; i < 2 * U * 64; i += kPgThreads)
      *reinterpret_cast<uint4*>(sP + (i >> 6) * S::kPSub + 24 * 128 + (i & 63) * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  // This CTA's share of all tiles, and the request that it begins in.
  const int chunk = (a.B + kPgThreads - 1) / kPgThreads;
  const int c0 = min(a.B, static_cast<int>(threadIdx.x) * chunk), c1 = min(a.B, c0 + chunk);
  long long mine = 0;
  for (int i = c0; i < c1; ++i) mine += (pg_len(a, i) + TILE - 1) / TILE;
  long long upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += y;
  }
  if (lane == 31) b->scan[warp] = upto;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kPgThreads / 32; ++w) {
    if (w < warp) before += b->scan[w];
    total += b->scan[w];
  }
  total *= a.units;
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long g0 = min(total, static_cast<long long>(blockIdx.x) * per), g1 = min(total, g0 + per);
  {
    long long first = (before + upto - mine) * a.units;
    const long long last = (before + upto) * a.units;
    if (g0 < g1 && first <= g0 && g0 < last) {
      int i = c0;
      for (;; ++i) {
        const long long t = static_cast<long long>((pg_len(a, i) + TILE - 1) / TILE) * a.units;
        if (g0 < first + t) break;
        first += t;
      }
      b->start_b = i;
      b->start_base = first;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b->tmem_base;
  const int n_tiles = static_cast<int>(g1 - g0);
  const int b0 = b->start_b;
  const long long base0 = b->start_base;

  if (n_tiles == 0) {
    // nothing but the empty requests below
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    // the cache is streamed once, unless several row tiles read it
    const uint64_t pol = a.row_tiles > 1 ? policy_evict_last() : policy_evict_first();
    PageBatch<TILE> pb(a, g0, n_tiles, b0, base0, lane);
    long long row = pb.fetch(0);
    bool ok = true;
    for (int t0 = 0; t0 < n_tiles && ok; t0 += pb.tiles) {
      const long long next = pb.fetch(t0 + pb.tiles);
      const int m = min(pb.tiles, n_tiles - t0);
      if (row == -2) report_status(a.status, DEVSTATUS_BAD_PAGE, WAIT_PAGED_TABLE);
      const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
      for (int u = 0; u < m; ++u) {
        const int t = t0 + u, s = t % NS;
        if (t >= NS && !mbar_wait_warp(&b->kv_empty[s], ((t / NS) + 1) & 1, wc, WAIT_PAGED_KV_EMPTY)) {
          ok = false;
          break;
        }
        const uint32_t in_tile = pb.per_tile == 32 ? 0xffffffffu : ((1u << pb.per_tile) - 1u) << (u * pb.per_tile);
        mbar_arrive_expect_tx_e(&b->kv_full[s], 2u * D * a.page * __popc(have & in_tile));
        __syncwarp();
        if (pb.u == u && row >= 0) {
          uint8_t* st = sKV + s * S::kStageBytes + pb.i * a.page * D;
          tma_load_3d_hint(st, &tmK, &b->kv_full[s], 0, 0, static_cast<int>(row), pol);
          tma_load_3d_hint(st + S::kTileBytes, &tmV, &b->kv_full[s], 0, 0, static_cast<int>(row), pol);
        }
        __syncwarp();
      }
      row = next;
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    const uint64_t dK = pg_desc<D>(smem_u32(sKV));                              // K tiles, K-major (A)
    const uint64_t dV = pg_desc<D>(smem_u32(sKV + S::kTileBytes));              // V tiles, MN-major (A of O^T)
    const uint64_t dQ = pg_desc<D>(smem_u32(sQ));                               // queries, K-major (B)
    const uint64_t dP = sdesc_sw128(smem_u32(sP), 16, 1024);                    // P^T, K-major (B)
    Walk<TILE> walk(a, g0, g1, b0, base0);
    Piece pc;
    bool ok = true;
    int g = 0, it = 0;
    // O^T(ob) (+)= V^T P^T for the tile with ring index gg.
    auto issue_pv = [&](int gg, int ob, bool first) -> bool {
      const int pb = gg & 1;
      if (first && it >= 2 && !mbar_wait_warp(&b->o_free[ob], ((it >> 1) + 1) & 1, wc, WAIT_PAGED_O_FREE)) return false;
      if (!mbar_wait_warp(&b->p_full[pb], (gg >> 1) & 1, wc, WAIT_PAGED_P)) return false;
      tc_fence_after();
      const int s = gg % NS;
#pragma unroll
      for (int kt = 0; kt < S::kPvSteps; ++kt) {
        const uint64_t va = uint64_t((s * S::kStageBytes + kt * 32 * D) >> 4);
        const uint64_t po = uint64_t((pb * S::kPBytes + (kt >> 2) * S::kPSub + (kt & 3) * 32) >> 4);
        mma_f8_ss_e(tmem + S::kColO + S::kPRows * ob, dV + va, dP + po, S::kIdO, (!first || kt > 0) ? 1u : 0u);
      }
      tc_commit_e(&b->pv_done[pb]);
      tc_commit_e(&b->kv_empty[s]);
      return true;
    };
    for (; ok && walk.next(pc); ++it) {
      const int qb = it & 1, ob = it & 1;
      if (!mbar_wait_warp(&b->q_full[qb], (it >> 1) & 1, wc, WAIT_PAGED_Q)) break;
      for (int j = 0; j < pc.n; ++j, ++g) {
        const int s = g % NS, sb = g & 1;
        if (!mbar_wait_warp(&b->kv_full[s], (g / NS) & 1, wc, WAIT_PAGED_KV) ||
            (g >= 2 && !mbar_wait_warp(&b->s_free[sb], ((g >> 1) + 1) & 1, wc, WAIT_PAGED_S_FREE))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int ks = 0; ks < S::kKSteps; ++ks) {
            const uint64_t ka = uint64_t((s * S::kStageBytes + u * 128 * D + ks * 32) >> 4);
            const uint64_t qo = uint64_t((qb * S::kQBytes + ks * 32) >> 4);
            mma_f8_ss_e(tmem + S::kColS + S::kQRows * (sb * U + u), dK + ka, dQ + qo, S::kIdS, ks > 0 ? 1u : 0u);
          }
        tc_commit_e(&b->s_full[sb]);
        if (j == pc.n - 1) tc_commit_e(&b->q_empty[qb]);
        if (j > 0 && !issue_pv(g - 1, ob, j == 1)) {
          ok = false;
          break;
        }
      }
      if (!ok || !issue_pv(g - 1, ob, pc.n == 1)) break;
      tc_commit_e(&b->o_full[ob]);
    }
  } else if (warp == 2) {
    // --------------------------------------------------------- page scales
    PageBatch<TILE> pb(a, g0, n_tiles, b0, base0, lane);
    long long row = pb.fetch(0);
    float ks = row >= 0 ? a.k_scale[row] : 0.0f, vs = row >= 0 ? a.v_scale[row] : 0.0f;
    bool ok = true;
    for (int t0 = 0; t0 < n_tiles && ok; t0 += pb.tiles) {
      const long long next = pb.fetch(t0 + pb.tiles);
      const int m = min(pb.tiles, n_tiles - t0);
      // vs = 0 or tiny: the exponent takes 2^-60 and P the share vs / 2^-60
      const float v = fmaxf(vs, 8.673617379884035e-19f);
      const float4 f = row >= 0 ? make_float4(ks * a.c_log2, log2f(v), 1.0f / v, vs / v * kBase)
                                : make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
      for (int u = 0; u < m; ++u) {
        const int t = t0 + u, s = t % NS;
        if (t >= NS && !mbar_wait_warp(&b->kv_empty[s], ((t / NS) + 1) & 1, wc, WAIT_PAGED_SC_EMPTY)) {
          ok = false;
          break;
        }
        if (pb.u == u) b->page[s][pb.i] = f;
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->kv_full[s]);
      }
      row = next;
      ks = row >= 0 ? a.k_scale[row] : 0.0f;
      vs = row >= 0 ? a.v_scale[row] : 0.0f;
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------- queries
    constexpr int kWords = D / 64;                   // 32-bit words (two elements) of a row per lane
    Walk<TILE> walk(a, g0, g1, b0, base0);
    Piece pc;
    for (int it = 0; walk.next(pc); ++it) {
      const int qb = it & 1;
      if (it >= 2 && !mbar_wait_warp(&b->q_empty[qb], ((it >> 1) + 1) & 1, wc, WAIT_PAGED_Q_EMPTY)) break;
      const int hk = pc.unit / a.row_tiles;
      const int r0 = (pc.unit - hk * a.row_tiles) * R;
      const uint32_t* q = static_cast<const uint32_t*>(a.q) +
                          (static_cast<size_t>(pc.b) * a.Hkv + hk) * a.rows * (D / 2) + static_cast<size_t>(r0) * (D / 2);
      uint8_t* dst = sQ + qb * S::kQBytes;
#pragma unroll
      for (int rg = 0; rg < R; rg += 8) {
        uint32_t w[8][kWords];
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
          for (int c = 0; c < kWords; ++c)
            w[r][c] = r0 + rg + r < a.rows ? q[static_cast<size_t>(rg + r) * (D / 2) + lane * kWords + c] : 0u;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          uint32_t top = 0;
#pragma unroll
          for (int c = 0; c < kWords; ++c) top = max(top, max(w[r][c] & 0x7fffu, (w[r][c] >> 16) & 0x7fffu));
          top = __reduce_max_sync(0xffffffffu, top);
          // the row times 2^-e has its largest element in [128, 256)
          const int e = min(max(static_cast<int>(top >> 7) - 134, -110), 121);
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          uint32_t hi = 0, lo = 0;
#pragma unroll
          for (int c = 0; c < kWords; ++c) {
            const float x = __uint_as_float(w[r][c] << 16) * inv, y = __uint_as_float(w[r][c] & 0xffff0000u) * inv;
            const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h), __NV_E4M3);
            const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hr));
            const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2((x - hf.x) * 16.0f, (y - hf.y) * 16.0f),
                                                        __NV_SATFINITE, __NV_E4M3);
            hi |= h << (16 * c);
            lo |= l << (16 * c);
          }
          const int byte = lane * kWords * 2;
          const int hr_off = pg_unit<D>(rg + r, byte >> 4) + (byte & 15);
          const int lr_off = pg_unit<D>(R + rg + r, byte >> 4) + (byte & 15);
          if (kWords == 2) {
            *reinterpret_cast<uint32_t*>(dst + hr_off) = hi;
            *reinterpret_cast<uint32_t*>(dst + lr_off) = lo;
          } else {
            *reinterpret_cast<uint16_t*>(dst + hr_off) = static_cast<uint16_t>(hi);
            *reinterpret_cast<uint16_t*>(dst + lr_off) = static_cast<uint16_t>(lo);
          }
          // a row that holds something not finite has no scores
          if (lane == 0)
            b->q_factor[qb][rg + r] = top >= 0x7f80u ? NAN : __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->q_full[qb]);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------- softmax
    // Two groups of four warps; each has half of the rows, for every key.
    constexpr int H = R / 2;
    const int wq = warp & 3;
    const int half = (warp >> 2) - 1;
    const int hr = half * H;                         // this group's first row
    const uint32_t lane_base = tmem + (uint32_t(wq * 32) << 16);
    const int page_shift = 31 - __clz(a.page);
    Walk<TILE> walk(a, g0, g1, b0, base0);
    Piece pc;
    // A warp whose wait ran out goes on without waiting or arriving, so that
    // the group's hardware barriers are still met by all four warps.
    bool ok = true;
    int g = 0, it = 0;
    for (; walk.next(pc); ++it) {
      const int ob = it & 1, qb = it & 1;
      const int row0 = (pc.unit % a.row_tiles) * R + hr;
      float m_used[H], l_t[H];
#pragma unroll
      for (int r = 0; r < H; ++r) {
        m_used[r] = -INFINITY;
        l_t[r] = 0.0f;
      }
      // the queries' factors are this warp's to read from here on
      ok = ok && mbar_wait_warp(&b->q_full[qb], (it >> 1) & 1, wc, WAIT_PAGED_Q);
      for (int j = 0; j < pc.n; ++j, ++g) {
        const int sb = g & 1, st = g % NS;
        ok = ok && mbar_wait2_warp(&b->kv_full[st], (g / NS) & 1, &b->s_full[sb], (g >> 1) & 1, wc, WAIT_PAGED_S);
        tc_fence_after();
        const int tile0 = (pc.j0 + j) * TILE;
        float s[U][H];
        float inv[U], share[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t col = lane_base + S::kColS + S::kQRows * (sb * U + u) + hr;
          uint32_t x[H], y[H];
          tmem_ld2<H>(col, col + R, x, y);
#pragma unroll
          for (int r = 0; r < H; ++r) s[u][r] = fmaf(__uint_as_float(y[r]), 0.0625f, __uint_as_float(x[r]));
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&b->s_free[sb]);
        bool need = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int kt = 128 * u + wq * 32 + lane;
          const float4 f = b->page[st][kt >> page_shift];
          inv[u] = f.z;
          share[u] = f.w;
          const bool there = tile0 + kt < pc.len && f.y != -INFINITY;
#pragma unroll
          for (int r = 0; r < H; r += 4) {
            const float4 qf = *reinterpret_cast<const float4*>(&b->q_factor[qb][hr + r]);
            s[u][r] = there ? fmaf(s[u][r], qf.x * f.x, f.y) : -INFINITY;
            s[u][r + 1] = there ? fmaf(s[u][r + 1], qf.y * f.x, f.y) : -INFINITY;
            s[u][r + 2] = there ? fmaf(s[u][r + 2], qf.z * f.x, f.y) : -INFINITY;
            s[u][r + 3] = there ? fmaf(s[u][r + 3], qf.w * f.x, f.y) : -INFINITY;
          }
          if (!there) {      // stale codes of V must not meet p = 0; each group clears half of the row
            uint8_t* v = sKV + st * S::kStageBytes + S::kTileBytes + kt * D + half * (D / 2);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) *reinterpret_cast<uint4*>(v + c * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        if (a.causal && tile0 + TILE > pc.len - a.Nq + 1) {
          int i = row0 % a.Nq;                       // query of row r
#pragma unroll
          for (int r = 0; r < H; ++r) {
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (tile0 + 128 * u + wq * 32 + lane > pc.len - a.Nq + i) s[u][r] = -INFINITY;
            i = i + 1 == a.Nq ? 0 : i + 1;
          }
        }
        // Does any key of the tile lift a row's maximum by more than the
        // threshold?  One barrier with a vote; the maxima themselves are only
        // exchanged when one does.
#pragma unroll
        for (int r = 0; r < H; ++r)
#pragma unroll
          for (int u = 0; u < U; ++u) need |= s[u][r] > m_used[r] + kRescaleThreshold;
        if (group_any(1 + half, need)) {
#pragma unroll
          for (int r = 0; r < H; ++r) {
            float x = s[0][r];
#pragma unroll
            for (int u = 1; u < U; ++u) x = fmaxf(x, s[u][r]);
            x = redux_max(x);
            if (lane == 0) b->red_max[wq][hr + r] = x;
          }
          group_sync(1 + half);
          float alpha[H];
#pragma unroll
          for (int r = 0; r < H; ++r) {
            const float mt = fmaxf(fmaxf(b->red_max[0][hr + r], b->red_max[1][hr + r]),
                                   fmaxf(b->red_max[2][hr + r], b->red_max[3][hr + r]));
            const float mn = fmaxf(m_used[r], mt);
            alpha[r] = (mn == -INFINITY) ? 1.0f : ex2_approx(m_used[r] - mn);
            m_used[r] = mn;
            l_t[r] *= alpha[r];
          }
          if (j > 0) {   // O^T holds earlier tiles of this piece: rescale it once PV(g-1) is done
            ok = ok && mbar_wait_warp(&b->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, wc, WAIT_PAGED_PV);
            tc_fence_after();
            if (ok) {
#pragma unroll
              for (int part = 0; part < 3; ++part) {
                const uint32_t col = lane_base + S::kColO + S::kPRows * ob + part * R + hr;
                uint32_t o[H];
                tmem_ld<H>(col, o);
#pragma unroll
                for (int r = 0; r < H; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[r]);
                tmem_st<H>(col, o);
              }
              tmem_wait_st();
            }
          }
        }
        // P^T into shared memory: B operand, K-major, rows = parts of the query
        // rows, the sub-tile's 128 keys in one 128-byte swizzled row.  The
        // buffer is free: S(g) was committed behind PV(g - 2), which read it.
        const int pb = g & 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int key = wq * 32 + lane;
          uint8_t* pbase = sP + pb * S::kPBytes + u * S::kPSub + (key & 15) + hr * 128;
          const int unit = key >> 4;
#pragma unroll
          for (int r = 0; r < H; r += 2) {
            const float p0 = (s[u][r] == -INFINITY) ? 0.0f : ex2_approx(s[u][r] - m_used[r]);
            const float p1 = (s[u][r + 1] == -INFINITY) ? 0.0f : ex2_approx(s[u][r + 1] - m_used[r + 1]);
            l_t[r] = fmaf(p0, inv[u], l_t[r]);
            l_t[r + 1] = fmaf(p1, inv[u], l_t[r + 1]);
            // p * vs in fp16, then its three e5m2 parts (e5m2 is fp16's upper
            // byte; adding 0x80 rounds the magnitude to nearest)
            const __half2 h = __floats2half2_rn(p0 * share[u], p1 * share[u]);
            const uint32_t hi = (*reinterpret_cast<const uint32_t*>(&h) + 0x00800080u) & 0xff00ff00u;
            const __half2 d1 = __hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&hi)), __float2half2_rn(8.0f));
            const uint32_t mid = (*reinterpret_cast<const uint32_t*>(&d1) + 0x00800080u) & 0xff00ff00u;
            const __half2 d2 = __hmul2(__hsub2(d1, *reinterpret_cast<const __half2*>(&mid)), __float2half2_rn(8.0f));
            const uint32_t lo = *reinterpret_cast<const uint32_t*>(&d2) + 0x00800080u;
            // hr is 4 or a multiple of 8: row & 7 as the swizzle sees it
            const int x0 = ((H == 4 ? hr : 0) + r) & 7;
            uint8_t* p_even = pbase + r * 128 + ((unit ^ x0) << 4);
            uint8_t* p_odd = pbase + (r + 1) * 128 + ((unit ^ (x0 + 1)) << 4);
            p_even[0] = static_cast<uint8_t>(hi >> 8);
            p_odd[0] = static_cast<uint8_t>(hi >> 24);
            p_even[R * 128] = static_cast<uint8_t>(mid >> 8);
            p_odd[R * 128] = static_cast<uint8_t>(mid >> 24);
            p_even[2 * R * 128] = static_cast<uint8_t>(lo >> 8);
            p_odd[2 * R * 128] = static_cast<uint8_t>(lo >> 24);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&b->p_full[pb]);
      }
      if (ok && lane == 0) mbar_arrive(&b->q_empty[qb]);
      // Piece done: once its last PV has completed (which also orders these
      // writes after the epilogue's read of this stats buffer two pieces ago),
      // publish the running max and the per-warp sums.
      ok = ok && mbar_wait_warp(&b->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, wc, WAIT_PAGED_PV);
#pragma unroll
      for (int r = 0; r < H; ++r) {
        const float l = warp_sum(l_t[r]);
        if (ok && lane == 0) {
          b->stat_l[ob][wq][hr + r] = l;
          if (wq == 0) b->stat_m[ob][hr + r] = m_used[r];
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&b->stats_full[ob]);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int wq = warp & 3;
    const uint32_t lane_base = tmem + (uint32_t(wq * 32) << 16);
    // O^T row (= output column) held by this thread: M = d = 128 uses every
    // lane; M = 64 puts rows 16w..16w+15 in lanes 0-15 of quarter w.
    const int drow = (D == 128) ? wq * 32 + lane : (lane < 16 ? wq * 16 + lane : -1);
    PagedNote note{-1, 0, 0, 0};
    Walk<TILE> walk(a, g0, g1, b0, base0);
    Piece pc;
    for (int it = 0;; ++it) {
      const long long at = walk.g;
      if (!walk.next(pc)) break;
      const int ob = it & 1;
      if (!mbar_wait_warp(&b->o_full[ob], (it >> 1) & 1, wc, WAIT_PAGED_O) ||
          !mbar_wait_warp(&b->stats_full[ob], (it >> 1) & 1, wc, WAIT_PAGED_STATS))
        break;
      tc_fence_after();
      const bool whole = pc.n == pc.nt;
      const int slot = 2 * blockIdx.x + (pc.j0 > 0 ? 0 : 1);
      if (pc.j0 > 0 && pc.j0 + pc.n == pc.nt) note = PagedNote{pc.b, pc.unit, static_cast<int>((at - pc.j0) / per), 0};
      const int hk = pc.unit / a.row_tiles;
      const int row0 = (pc.unit - hk * a.row_tiles) * R;
      const size_t out = (static_cast<size_t>(pc.b) * a.Hkv + hk) * a.rows + row0;
      constexpr int kStep = R == 8 ? 8 : 16;
#pragma unroll
      for (int rg = 0; rg < R; rg += kStep) {
        float o[kStep];
        if constexpr (R == 8) {
          uint32_t x[32];
          tmem_ld_x32(lane_base + S::kColO + S::kPRows * ob, x);
#pragma unroll
          for (int r = 0; r < 8; ++r)
            o[r] = fmaf(__uint_as_float(x[16 + r]), 1.0f / 64.0f,
                        fmaf(__uint_as_float(x[8 + r]), 0.125f, __uint_as_float(x[r])));
        } else {
          uint32_t x[16];
          const uint32_t col = lane_base + S::kColO + S::kPRows * ob + rg;
          tmem_ld_x16(col + 2 * R, x);
#pragma unroll
          for (int r = 0; r < 16; ++r) o[r] = __uint_as_float(x[r]) * (1.0f / 64.0f);
          tmem_ld_x16(col + R, x);
#pragma unroll
          for (int r = 0; r < 16; ++r) o[r] = fmaf(__uint_as_float(x[r]), 0.125f, o[r]);
          tmem_ld_x16(col, x);
#pragma unroll
          for (int r = 0; r < 16; ++r) o[r] += __uint_as_float(x[r]);
        }
        if (drow >= 0) {
#pragma unroll
          for (int k = 0; k < kStep; ++k) {
            const int r = rg + k;
            if (row0 + r < a.rows) {
              const float L = b->stat_l[ob][0][r] + b->stat_l[ob][1][r] + b->stat_l[ob][2][r] + b->stat_l[ob][3][r];
              const float val = L == 0.0f ? 0.0f : o[k] * (1.0f / kBase) / L;
              const float lse = L == 0.0f ? -INFINITY : (b->stat_m[ob][r] + log2f(L)) * kLn2;
              if (whole) {
                static_cast<__nv_bfloat16*>(a.o)[(out + r) * D + drow] = __float2bfloat16_rn(val);
                if (drow == 0) a.lse[out + r] = lse;
              } else {
                a.part_o[(static_cast<size_t>(slot) * R + r) * D + drow] = val;
                if (drow == 0) a.part_lse[slot * R + r] = lse;
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->o_free[ob]);
    }
    if (threadIdx.x == 384) a.notes[blockIdx.x] = note;
  }
  if (n_tiles == 0 && threadIdx.x == 384) a.notes[blockIdx.x] = PagedNote{-1, 0, 0, 0};
  // requests without a token
  if (warp >= 12) {
    const int t = threadIdx.x - 384;
    for (int i = blockIdx.x; i < a.B; i += gridDim.x) {
      if (pg_len(a, i) > 0) continue;
      const size_t rows = static_cast<size_t>(a.Hkv) * a.rows;
      for (size_t c = t; c < rows * (D / 8); c += 128)
        reinterpret_cast<uint4*>(a.o)[i * rows * (D / 8) + c] = make_uint4(0u, 0u, 0u, 0u);
      for (size_t c = t; c < rows; c += 128) a.lse[i * rows + c] = -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// O = sum_s exp(LSE_s - LSE) O_s with LSE = log sum_s exp(LSE_s) over the
// pieces of a unit that CTA `x` ended: its own and those of the CTAs before it
// down to the one that began it.  One block per (CTA, row of the unit);
// thread = (output column, one of kParts interleaved subsets of the pieces).
constexpr int kMergeThreads = 256;

template <int D, int R>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedArgs a) {
  constexpr int kParts = kMergeThreads / D;
  __shared__ float red[kMergeThreads / 32];
  __shared__ float acc_s[kParts][D];
  __shared__ float l_s[kParts];
  const int cta = blockIdx.x, r = blockIdx.y;
  const PagedNote note = a.notes[cta];
  if (note.b < 0) return;
  const int hk = note.unit / a.row_tiles;
  const int row = (note.unit - hk * a.row_tiles) * R + r;
  if (row >= a.rows) return;
  const int ns = cta - note.first + 1;
  const int c = threadIdx.x % D, part = threadIdx.x / D;
  // the first piece is in its CTA's second slot, the others in the first
  auto slot = [&](int s) { return static_cast<size_t>(2 * (note.first + s) + (s == 0 ? 1 : 0)) * R + r; };
  float m = -INFINITY;
  bool bad = false;                                   // NaN must not hide from the maximum
  for (int s = threadIdx.x; s < ns; s += kMergeThreads) {
    const float x = a.part_lse[slot(s)];
    bad |= x != x;
    m = fmaxf(m, x);
  }
  m = redux_max(m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; ++w) m = fmaxf(m, red[w]);
  float L = 0.0f, acc = 0.0f;
  if (m != -INFINITY) {
#pragma unroll 4
    for (int s = part; s < ns; s += kParts) {
      const float wgt = ex2_approx((a.part_lse[slot(s)] - m) * 1.4426950408889634f);
      L += wgt;
      acc = fmaf(wgt, a.part_o[slot(s) * D + c], acc);
    }
  }
  acc_s[part][c] = acc;
  if (c == 0) l_s[part] = L;
  __syncthreads();
  if (part == 0) {
    float at = 0.0f, lt = 0.0f;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      at += acc_s[p][c];
      lt += l_s[p];
    }
    const size_t out = (static_cast<size_t>(note.b) * a.Hkv + hk) * a.rows + row;
    static_cast<__nv_bfloat16*>(a.o)[out * D + c] = __float2bfloat16_rn(bad ? NAN : lt > 0.0f ? at / lt : 0.0f);
    if (c == 0) a.lse[out] = bad ? NAN : lt > 0.0f ? m + log2f(lt) * kLn2 : -INFINITY;
  }
}

template <int D, int R>
cudaError_t launch_paged_t(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas, cudaStream_t stream) {
  constexpr size_t smem = pg_smem_bytes<D, R>();
  static_assert(smem <= 227 * 1024, "shared memory budget");
  auto kern = decode_paged_kernel<D, R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  kern<<<ctas, kPgThreads, smem, stream>>>(tk, tv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  paged_merge_kernel<D, R><<<dim3(ctas, R < a.rows ? R : a.rows), kMergeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int d, int row_tile,
                                int ctas, cudaStream_t stream) {
  if (d == 64)
    return row_tile == 8    ? launch_paged_t<64, 8>(tk, tv, a, ctas, stream)
           : row_tile == 16 ? launch_paged_t<64, 16>(tk, tv, a, ctas, stream)
                            : launch_paged_t<64, 32>(tk, tv, a, ctas, stream);
  return row_tile == 8    ? launch_paged_t<128, 8>(tk, tv, a, ctas, stream)
         : row_tile == 16 ? launch_paged_t<128, 16>(tk, tv, a, ctas, stream)
                          : launch_paged_t<128, 32>(tk, tv, a, ctas, stream);
}

}  // namespace fa
