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
//                   8-bit floats: with the row scaled to |q| < 256, hi rounds to
//                   e4m3's 4 bits and lo is the rest, at most 8 of its last
//                   steps.  Both multiply K, so the scores are those of the bf16
//                   query (elements below 2^-10 of the row's largest, and far
//                   below, keep 2^-21 of it).
//   O^T += V^T P^T  d x rows (A = V tile, MN-major).  p * vs is rounded to fp16
//                   and split into three e5m2 parts, hi + mid/8 + lo/64: 11 bits
//                   in three times 3 plus the signs.  The last step of lo is
//                   2^-22 where the maximum in use is 2^11, so the split is exact
//                   from 2^-23 of that maximum on; below, p * vs is rounded to
//                   multiples of 2^-33 of it and under 2^-34 is gone.  The
//                   maximum in use is at most the largest p * vs of the row, V
//                   scales included: a column in which heavy keys are 0 has of
//                   light ones what this leaves.  A and B of one product may
//                   differ in type among the 8-bit floats.
// A page's K scale multiplies its keys' scores; its V scale goes into the
// exponent (t = s + log2 vs, P = exp2(t - m)), so that the parts cannot overflow
// whatever the scales are, and l sums exp2(t - m) / vs.  t counts from a whole
// number r near the log2 vs of the piece's first page, so that m and with it LSE
// are no larger than the scores; O gets the factor 2^r at the end.
//
// Work.  A unit is (request, KV head, tile of up to R query rows); its keys are
// cut into tiles of 128 (d = 128) or 256 (d = 64) tokens, 32 KB of codes.  The
// lengths are known on the device only, so every CTA adds them up itself and
// takes an equal share of all tiles (a unit counts for two more), a contiguous
// range that may begin and end inside a unit.  A unit that lies within one CTA is
// written directly; of a unit cut between CTAs each CTA leaves its normalised O and LSE in one of its
// two slots of the workspace (one for a piece that does not begin its unit, one
// for a piece that does), and the CTA that is the last to finish a piece of the
// unit combines them by their log-sum-exp, in the order of the pieces, so that
// results do not depend on timing.
//
// Warps: 0 K and V pages, 1 S products and TMEM owner, 2 page scales, queries
// and, with many small pages, V pages, 3 PV products; from 4 on the softmax
// groups of four (thread = key, each group its share of the rows; TMEM lane
// quarter = warp % 4), the last four epilogue.  Pages that lie behind the length
// or outside the cache are not loaded; the softmax warps clear the V rows of keys
// that are not there, since p = 0 times a stale NaN code would be NaN.
//
// Measured, in a CUDA graph, H/Hkv = 4, ragged lengths up to n: B32 Hkv8 n8192
// d128 56 us with pages of 16, 53 with 64 (300 MB, 5.4 and 5.7 TB/s; loads alone
// 49); B8 n131072 125 and 120 us (772 MB, 6.2 and 6.4 TB/s).  32 rows (B48 Hkv8,
// 4 queries of 8 heads, n16384, 965 MB) 199 us, 4.9 TB/s: half of the issue slots
// are used, the softmax warps wait for S, which each loads and needs at once, and
// for one another (under a sustained load at lower clocks 230 us).  What short
// pieces cost is the chain from pages to output, about 10 us from launch to end:
// B1 n1000 12.4 us, of which the launch, lengths, table and first tile are 6.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.4426950408889634f;
// What a piece costs beside its tiles, in tiles (measured: a batch of 256 x 512
// keys took 72 us with 0, 65 with 2).
constexpr int kPieceCost = 2;
constexpr float kRescaleThreshold = 4.0f;   // log2 units
constexpr float kBase = 2048.0f;            // P is scaled by 2^11: at most 2^15, of e5m2's 57344

template <int D, int R>
struct PgShape {
  // Groups of softmax warps: kSplit share a tile's rows, kTurns take the tiles
  // in turn, each with a maximum, a sum and an O of its own.
  static constexpr int kSplit = R / 8;
  static constexpr int kTurns = R == 32 ? 1 : 2;
  static constexpr int kGroups = kSplit * kTurns;
  static constexpr int kRows = R / kSplit;                    // rows of a group
  static constexpr int kEpi = 4 + 4 * kGroups;                // first epilogue warp
  static constexpr int kThreads = 32 * (kEpi + 4);
  static constexpr int kSub = (D == 64) ? 2 : 1;              // 128-key sub-tiles per tile
  static constexpr int kTileKeys = 128 * kSub;
  static constexpr int kTileBytes = kTileKeys * D;            // K (or V) codes of one tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kBufs = 2 * kTurns;                    // of S^T and of the queries
  // Ring depth: a stage is K, V and P of a tile, 32 KB and kPBytes.
  static constexpr int kNS = R == 8 ? 5 : R == 16 ? (D == 128 ? 5 : 4) : (D == 128 ? 4 : 3);
  static constexpr int kMaxPages = kTileKeys / 16;
  // The query's parts are columns of their own for 8 rows (a product has 16
  // columns at least), the low part 16 times itself; from 16 rows on both products
  // go into the same columns, the low part as it is, in e5m2, whose range it needs.
  static constexpr bool kFold = R >= 16;
  static constexpr int kQRows = 2 * R;                        // hi, lo
  static constexpr int kSCols = kFold ? R : 2 * R;
  static constexpr int kQBytes = kQRows * D;
  static constexpr int kPRows = (R == 8) ? 32 : 3 * R;        // hi, mid, lo (and zero rows up to a multiple of 16)
  static constexpr int kPChunk = kTileKeys * 16;              // 16 rows of P^T for every key
  static constexpr int kPBytes = kPRows / 16 * kPChunk;
  static constexpr int kKSteps = D / 32;                      // S^T k-steps per sub-tile
  static constexpr int kPvSteps = kTileKeys / 32;             // O^T k-steps per tile
  static constexpr uint32_t kIdS = idesc_e4m3(128, kSCols, false, false);
  static constexpr uint32_t kIdSLo = kIdS | (1u << 10);       // B format 1: e5m2
  static constexpr uint32_t kIdO = idesc_e4m3(D, kPRows, true, true) | (1u << 10);    // B format 1: e5m2
  static constexpr uint32_t kColS = 0;                        // kBufs S^T buffers of kSCols * kSub columns
  static constexpr uint32_t kColO = kBufs * kSCols * kSub;        // two O^T buffers of kPRows columns per turn
  static constexpr uint32_t kCols = kColO + 2 * kTurns * kPRows;
  static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM columns");
};

// A unit to combine: row tile `unit` of request b, in pieces of CTAs first..last.
struct Merge {
  int b, unit, first, last;
};
// A place among the tiles: tile j of unit `unit` of request b, which has nt.
struct Place {
  int b, unit, j, len, nt;
};

template <int R, int NS, int PAGES, int TURNS, int BUFS>
struct PgBarriers {
  uint64_t kv_full[NS], kv_empty[NS], p_full[NS];
  uint64_t q_full[BUFS], q_empty[BUFS];
  uint64_t s_full[BUFS], s_free[BUFS];
  uint64_t o_full[2], o_free[2];
  uint64_t stats_full[2];
  uint64_t merged;
  alignas(16) float4 page[NS][PAGES];      // per page of a tile: K factor, log2 vs - r, 2^r / vs, 0 if vs is
  float page_ref[BUFS];                    // 2^r of a piece
  float stat_ref[2];
  alignas(16) float q_factor[BUFS][R];        // power of two that a row of queries was divided by
  alignas(16) float red_max[TURNS][4][R];  // per-warp tile maxima (log2 units)
  alignas(16) float stat_m[2][TURNS][R];     // piece's running max
  alignas(16) float stat_l[2][TURNS][4][R];  // piece's per-warp sums
  uint32_t nan_keys[2][128];               // per column of a piece: boundary keys whose V code is NaN
  long long first_tile[2];                 // of this CTA's share and of the next
  int per, start_rest;                     // length of a share; how far into a unit's line it begins
  int n_merge;                             // units that this CTA is the last to have finished a piece of
  Merge merge[2];
  Place start;
  uint32_t tmem_base;
  uint32_t abort;
  uint32_t drained;                        // `abort` of the waits for copies in flight
};

template <int D, int R>
using PgBar = PgBarriers<R, PgShape<D, R>::kNS, PgShape<D, R>::kMaxPages, PgShape<D, R>::kTurns, PgShape<D, R>::kBufs>;

template <int D, int R>
constexpr size_t pg_smem_bytes() {
  using S = PgShape<D, R>;
  return 1024 + size_t(S::kNS) * (S::kStageBytes + S::kPBytes) + S::kBufs * S::kQBytes + sizeof(PgBar<D, R>);
}

// Shared-memory matrix descriptor: rows of D bytes, swizzled over D bytes.
template <int D>
__device__ __forceinline__ uint64_t pg_desc(uint32_t saddr) {
  uint64_t d = sdesc_sw128(saddr, 16, 8 * D);
  if (D == 64) d = (d & ~(uint64_t(7) << 61)) | (uint64_t(4) << 61);   // 64-byte swizzle
  return d;
}
// P^T without swizzle: 8 keys x 16 rows in 128 bytes, a key's 16 rows together;
// 8-key groups follow one another, chunks of 16 rows are `chunk` bytes apart.
__device__ __forceinline__ uint64_t pg_desc_p(uint32_t saddr, uint32_t chunk) {
  return sdesc_sw128(saddr, 128, chunk) & ~(uint64_t(7) << 61);
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
// Other threads' global writes, seen by this one -> visible to its bulk copies.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Bounded waits.  The roles' code shares the SM's instruction cache, so only
// the first look is inline.
__device__ __noinline__ bool pg_wait_slow(uint64_t* bar, uint32_t parity, const WaitCtx& w, uint32_t where) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, w, where));
}
__device__ __forceinline__ bool pg_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w, uint32_t where) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || pg_wait_slow(bar, parity, w, where);
}
// Two and three waits whose first looks overlap.
__device__ __forceinline__ bool pg_wait2(uint64_t* x, uint32_t px, uint64_t* y, uint32_t py, const WaitCtx& w, uint32_t where) {
  const bool a = mbar_try_wait(x, px), b = mbar_try_wait(y, py);
  return __all_sync(0xffffffffu, a && b) || (pg_wait_slow(x, px, w, where) && pg_wait_slow(y, py, w, where));
}
__device__ __forceinline__ bool pg_wait3(uint64_t* x, uint32_t px, uint64_t* y, uint32_t py, uint64_t* z, uint32_t pz,
                                         const WaitCtx& w, uint32_t where) {
  const bool a = mbar_try_wait(x, px), b = mbar_try_wait(y, py), c = mbar_try_wait(z, pz);
  return __all_sync(0xffffffffu, a && b && c) ||
         (pg_wait_slow(x, px, w, where) && pg_wait_slow(y, py, w, where) && pg_wait_slow(z, pz, w, where));
}

// Eight consecutive TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t) : "memory");
}
// Two such loads with one wait.
__device__ __forceinline__ void tmem_ld2(uint32_t t, uint32_t t2, uint32_t (&r)[8], uint32_t (&q)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
               "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7])
               : "r"(t), "r"(t2) : "memory");
}
// Sums over the warp of H = 8 values per lane; lane gets that of value
// lane / 4.  Each step but the last two halves the values: a lane keeps one half
// and hands the other to its partner.
template <int H>
__device__ __forceinline__ float rows_sum(const float (&x)[H], int lane) {
  static_assert(H == 8, "three halvings");
  float y[4], z[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float keep = lane & 16 ? x[4 + k] : x[k], give = lane & 16 ? x[k] : x[4 + k];
    y[k] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float keep = lane & 8 ? y[2 + k] : y[k], give = lane & 8 ? y[k] : y[2 + k];
    z[k] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
  }
  const float keep = lane & 4 ? z[1] : z[0], give = lane & 4 ? z[0] : z[1];
  float w = keep + __shfl_xor_sync(0xffffffffu, give, 4);
  w += __shfl_xor_sync(0xffffffffu, w, 2);
  return w + __shfl_xor_sync(0xffffffffu, w, 1);
}

__device__ __forceinline__ int kv_head(const PagedArgs& a, int unit) { return a.row_tiles == 1 ? unit : unit / a.row_tiles; }

// Two bf16 queries times `inv` (below 256) as two parts each: the value rounded
// to e4m3, and what is left of it, in e5m2 (FOLD) or 16 times in e4m3.
template <bool FOLD>
__device__ __forceinline__ void split_pair(uint32_t q, float inv, uint32_t& hi, uint32_t& lo) {
  const float x = __uint_as_float(q << 16) * inv, y = __uint_as_float(q & 0xffff0000u) * inv;
  hi = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  constexpr float k = FOLD ? 1.0f : 16.0f;
  lo = __nv_cvt_float2_to_fp8x2(make_float2((x - f.x) * k, (y - f.y) * k), __NV_SATFINITE, FOLD ? __NV_E5M2 : __NV_E4M3);
}

__device__ __forceinline__ int pg_len(const PagedArgs& a, int b) { return min(max(a.seq_lens[b], 0), a.max_pages * a.page); }

// Clears the NaN codes (0x7f, 0xff) in part `part` of row `kt` of a V tile and sets
// bit `edge` for their columns; the flags of the piece two before are the
// epilogue's until it frees them.
template <int D, int PARTS>
__device__ __noinline__ bool clear_nan_codes(uint8_t* v, int kt, int part, int edge, uint32_t* nan_keys,
                                             uint64_t* o_free, int it, bool ok, const WaitCtx& wc) {
  uint32_t* row = reinterpret_cast<uint32_t*>(v + kt * D + part * (D / PARTS));
  bool waited = it < 2;
  for (int c = 0; c < D / PARTS / 4; ++c) {
    const uint32_t x = row[c], bad = __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
    if (bad == 0u) continue;
    if (!waited) ok = ok && mbar_wait(o_free, ((it >> 1) + 1) & 1, wc, WAIT_PAGED_O_FREE);
    waited = true;
    row[c] = x & ~bad;
    const int byte = part * (D / PARTS) + c * 4;                       // place in the swizzled row
    const int unit = (byte >> 4) ^ (D == 128 ? kt & 7 : (kt >> 1) & 3);
    for (int k = 0; k < 4; ++k)
      if ((bad >> (8 * k)) & 1u) atomicOr(&nan_keys[unit * 16 + (byte & 15) + k], 1u << edge);
  }
  return ok;
}

// A piece: tiles [j0, j0 + n) of one unit.
struct Piece {
  int b, unit, len, nt, j0, n;
};
// Query rows become two e4m3 parts each, by one warp, eight rows at a time, four
// lanes to a row.  Loading and splitting are apart, so that the next piece's
// rows come in while this one's work goes on.
template <int D>
struct QueryRows {
  static constexpr int kChunks = D / 32;             // 16-byte groups of eight elements per lane
  uint4 w[kChunks];
  // rows first..first + 7 of (b, unit), zeros behind the last row
  template <int R>
  __device__ __forceinline__ void load(const PagedArgs& a, const Piece& pc, int first, int lane) {
    const int hk = kv_head(a, pc.unit);
    const int row = (pc.unit - hk * a.row_tiles) * R + first + (lane >> 2);
    const uint4* q = static_cast<const uint4*>(a.q) +
                     ((static_cast<size_t>(pc.b) * a.Hkv + hk) * a.rows + row) * (D / 8) + (lane & 3) * kChunks;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) w[c] = row < a.rows ? q[c] : make_uint4(0u, 0u, 0u, 0u);
  }
  // as rows first.. (hi) and R + first.. (lo) of the B operand, and the powers
  // of two that the rows were divided by
  template <int R>
  __device__ __forceinline__ void split(uint8_t* dst, float* factor, int first, int lane) const {
    const int r = first + (lane >> 2);
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint32_t x = __vmaxu2(__vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu),
                                  __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu));
      top = max(top, max(x & 0xffffu, x >> 16));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the row times 2^-e has its largest element in [128, 256)
    const int e = min(max(static_cast<int>(top >> 7) - 134, -110), 121);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) split_pair<PgShape<D, R>::kFold>(x[k], inv, hi[k], lo[k]);
      const int place = (lane & 3) * (D / 64) + (c >> 1);
      *reinterpret_cast<uint2*>(dst + pg_unit<D>(r, place) + (c & 1) * 8) =
          make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
      *reinterpret_cast<uint2*>(dst + pg_unit<D>(R + r, place) + (c & 1) * 8) =
          make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
    }
    // a row that holds something not finite has no scores
    if ((lane & 3) == 0) factor[r] = top >= 0x7f80u ? NAN : __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  }
};

// Walks over a CTA's range of tiles; `left` are to come.
template <int TILE>
struct Walk {
  const PagedArgs& a;
  Place p;
  int left;
  __device__ __forceinline__ Walk(const PagedArgs& a_, const Place& start, int n) : a(a_), p(start), left(n) {}
  // Carries tile counts over a unit's end into the next units.
  __device__ __forceinline__ void settle() {
    while (p.j >= p.nt) {
      p.j -= p.nt;
      if (++p.unit == a.units) {
        p.unit = 0;
        do {
          p.len = pg_len(a, ++p.b);
          p.nt = (p.len + TILE - 1) / TILE;
        } while (p.nt == 0);
      }
    }
  }
  __device__ __forceinline__ bool next(Piece& pc) {
    if (left <= 0) return false;
    settle();
    pc.b = p.b;
    pc.unit = p.unit;
    pc.len = p.len;
    pc.nt = p.nt;
    pc.j0 = p.j;
    pc.n = min(p.nt - p.j, left);
    p.j += pc.n;
    left -= pc.n;
    return true;
  }
};

// Page ids of a CTA's tiles, 32 at a time: lane (u, i) has page i of tile u of
// the batch.  The next batch's ids are fetched while this one's are used.
template <int TILE>
struct PageBatch {
  Walk<TILE> w;
  int per_tile, tiles, u, i;
  __device__ __forceinline__ PageBatch(const PagedArgs& a, const Place& start, int n, int lane) : w(a, start, n) {
    const int shift = 31 - __clz(TILE / a.page);
    per_tile = 1 << shift;
    tiles = 32 >> shift;
    u = lane >> shift;
    i = lane & (per_tile - 1);
    w.p.j += u;
    w.left -= u;
  }
  // (page, KV head) row of this lane's page in the next batch: -1 where the
  // tile has no such page, -2 where the table names none of the cache's.
  __device__ __forceinline__ int fetch() {
    const PagedArgs& a = w.a;
    if (w.left <= 0) return -1;
    w.settle();
    const int lp = w.p.j * per_tile + i;
    int row = -1;
    if (lp * a.page < w.p.len) {
      const int id = a.block_table[static_cast<size_t>(w.p.b) * a.max_pages + lp];
      row = id >= 0 && id < a.num_pages ? id * a.Hkv + kv_head(a, w.p.unit) : -2;
    }
    w.p.j += tiles;
    w.left -= tiles;
    return row;
  }
  // Loads the pages of tile `tile` of the batch, whose rows the lanes hold, of one
  // map or of two (the second `apart` bytes behind), and arrives at `bar` with
  // their bytes.  A copy per lane, 67 cycles for each (issued in a loop by the
  // converged warp it took twice that).
  __device__ __forceinline__ void load(const CUtensorMap& map, const CUtensorMap* map2, int apart, int row, int tile,
                                       uint8_t* dst, int d, uint64_t* bar, uint64_t pol) const {
    const int page_bytes = w.a.page * d;
    const uint32_t in_tile = per_tile == 32 ? 0xffffffffu : ((1u << per_tile) - 1u) << (tile * per_tile);
    const int bytes = page_bytes * __popc(__ballot_sync(0xffffffffu, row >= 0) & in_tile);
    mbar_arrive_expect_tx_e(bar, map2 ? 2 * bytes : bytes);
    __syncwarp();
    if (u == tile && row >= 0) {
      tma_load_3d_hint(dst + i * page_bytes, &map, bar, 0, 0, row, pol);
      if (map2) tma_load_3d_hint(dst + apart + i * page_bytes, map2, bar, 0, 0, row, pol);
    }
    __syncwarp();
  }
};

// Marks this CTA's piece of a unit as done and looks whether all of them are,
// by one warp, behind a barrier of the threads that wrote the piece.  A mark is
// the call's nonce, so what the workspace held before is none.  Store, fence,
// load: of the CTAs of a unit at least the last one sees every mark; if several
// do, each combines the unit and writes the same bytes.  Who sees them all
// clears them, for a replay of the call has the same nonce; a CTA that then
// misses one leaves the unit to that one.
__device__ __forceinline__ bool mark_done(unsigned long long* marks, unsigned long long nonce, int own, int first, int last,
                                          int lane) {
  if (lane == 0) {
    __threadfence();
    *static_cast<volatile unsigned long long*>(marks + own) = nonce;
  }
  __syncwarp();
  __threadfence();
  bool all = true;
#pragma unroll 1
  for (int c = first + lane; c <= last; c += 32) {
    unsigned long long x;     // the first piece is in its CTA's second slot, the others in the first
    asm volatile("ld.acquire.gpu.u64 %0, [%1];" : "=l"(x) : "l"(marks + 2 * c + (c == first)) : "memory");
    all = all && x == nonce;
  }
  if (!__all_sync(0xffffffffu, all)) return false;
#pragma unroll 1
  for (int c = first + lane; c <= last; c += 32) *static_cast<volatile unsigned long long*>(marks + 2 * c + (c == first)) = 0;
  return true;
}

// O = sum_s exp(LSE_s - LSE) O_s with LSE = log sum_s exp(LSE_s) over a unit's
// pieces, a warp per row, the pieces in order (the same sum whichever CTA came
// last).  Runs once, when its code is in no cache yet: the pieces come into the
// ring's memory by bulk copies, as many at a time as fit, and are then added in
// short loops.
template <int D, int R>
__device__ __forceinline__ void merge_unit(const PagedArgs& a, const Merge& u, uint8_t* ring, uint64_t* bar, uint32_t& phase,
                                           const WaitCtx& wc) {
  using S = PgShape<D, R>;
  constexpr int kVec = D / 32;                       // columns per lane
  constexpr int kRing = S::kNS * (S::kStageBytes + S::kPBytes);
  constexpr int kLse = kPagedCtas * R * 4;           // every piece's LSE comes first
  constexpr int kBatch = (kRing - kLse) / (R * D * 4);
  static_assert(kBatch >= 8, "pieces at a time");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = kv_head(a, u.unit);
  const int row0 = (u.unit - hk * a.row_tiles) * R;
  const int rows = min(R, a.rows - row0);
  const int ns = u.last - u.first + 1;
  const float* lse_s = reinterpret_cast<const float*>(ring);
  const float* o_s = reinterpret_cast<const float*>(ring + kLse);
  constexpr int kWarps = S::kThreads / 32, kRows = (R + kWarps - 1) / kWarps;
  float m[kRows], L[kRows], acc[kRows][kVec];        // of rows warp, warp + kWarps
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    m[k] = -INFINITY;
    L[k] = 0.0f;
#pragma unroll
    for (int c = 0; c < kVec; ++c) acc[k][c] = 0.0f;
  }
  for (int s0 = 0; s0 < ns; s0 += kBatch) {
    const int n = min(kBatch, ns - s0);
    if (warp == 0) {
      fence_proxy_async_all();
      if (lane == 0) mbar_arrive_expect_tx(bar, n * rows * D * 4 + (s0 == 0 ? ns * R * 4 : 0));
      __syncwarp();
#pragma unroll 1
      for (int s = lane; s < (s0 == 0 ? ns : n); s += 32) {
        // the first piece is in its CTA's second slot, the others in the first
        if (s0 == 0)
          bulk_load(ring + s * (R * 4), a.part_lse + static_cast<size_t>(2 * (u.first + s) + (s == 0)) * R, R * 4, bar);
        if (s < n)
          bulk_load(ring + kLse + s * (R * D * 4),
                    a.part_o + static_cast<size_t>(2 * (u.first + s0 + s) + (s0 + s == 0)) * (R * D), rows * D * 4, bar);
      }
    }
    (void)pg_wait(bar, phase, wc, WAIT_PAGED_MERGE);    // if it runs out, the sums mean nothing
    phase ^= 1u;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = warp + kWarps * k;
      if (r >= rows) break;
      if (s0 == 0)
#pragma unroll 1
        for (int s = 0; s < ns; ++s) m[k] = fmaxf(m[k], lse_s[s * R + r]);
#pragma unroll 1
      for (int s = 0; s < n; ++s) {
        const float x = lse_s[(s0 + s) * R + r];
        const float w = x == -INFINITY ? 0.0f : ex2_approx((x - m[k]) * kLog2e);
        L[k] += w;
        const float* o = o_s + (s * R + r) * D + lane * kVec;
#pragma unroll
        for (int c = 0; c < kVec; ++c) acc[k][c] = fmaf(w, o[c], acc[k][c]);
      }
    }
    __syncthreads();                                 // the ring is read: the next batch or unit may come
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = warp + kWarps * k;
    if (r >= rows) break;
    const float inv = L[k] == 0.0f ? 0.0f : 1.0f / L[k];
    const size_t out = (static_cast<size_t>(u.b) * a.Hkv + hk) * a.rows + row0 + r;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o) + out * D + lane * kVec);
#pragma unroll
    for (int c = 0; c < kVec; c += 2) dst[c / 2] = pack_bf16x2(acc[k][c] * inv, acc[k][c + 1] * inv);
    if (lane == 0) a.lse[out] = L[k] == 0.0f ? -INFINITY : m[k] + log2f(L[k]) * kLn2;
  }
}

// CAUSAL: a boundary between keys that some queries see and others do not.
// SHARED: K and V pages are loaded by a warp each.
template <int D, int R, bool CAUSAL, bool SHARED>
__global__ void __launch_bounds__(PgShape<D, R>::kThreads, 1)
    decode_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const PagedArgs a) {
  using S = PgShape<D, R>;
  constexpr int NS = S::kNS, U = S::kSub, TILE = S::kTileKeys;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;                               // NS x (K tile, V tile)
  uint8_t* sP = sKV + NS * S::kStageBytes;           // NS x P^T
  uint8_t* sQ = sP + NS * S::kPBytes;                 // kBufs x (hi, lo) queries
  auto* b = reinterpret_cast<PgBar<D, R>*>(sQ + S::kBufs * S::kQBytes);
  const WaitCtx wc{&b->abort, a.status, FA_WAIT_LIMIT_NS};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 1) {
    tmem_alloc(&b->tmem_base, S::kTmemCols);
    tmem_relinquish();
  } else if (warp == 2) {
    if (lane < NS) {
      mbar_init(&b->kv_full[lane], 2);
      mbar_init(&b->kv_empty[lane], 1);
      mbar_init(&b->p_full[lane], 4 * S::kSplit);
    }
    fence_mbar_init();
  } else if (warp == 3) {
    if (lane < S::kBufs) {
      mbar_init(&b->q_full[lane], 1);
      mbar_init(&b->q_empty[lane], 1 + 4 * S::kGroups);
      mbar_init(&b->s_full[lane], 1);
      mbar_init(&b->s_free[lane], 4 * S::kSplit);
    }
    if (lane < 2) {
      mbar_init(&b->o_full[lane], 1);
      mbar_init(&b->o_free[lane], 4);
      mbar_init(&b->stats_full[lane], 4 * S::kGroups);
    }
    if (lane == 0) {
      mbar_init(&b->merged, 1);
      b->abort = b->drained = 0u;
    }
    fence_mbar_init();
  } else if (CAUSAL && warp >= S::kEpi) {
    for (int i = threadIdx.x - 32 * S::kEpi; i < 256; i += 128) b->nan_keys[i >> 7][i & 127] = 0u;
  }
  if (R == 8 && warp >= 4 && warp < 8) {             // the zero rows of P^T
    for (int i = threadIdx.x - 128; i < NS * TILE; i += 128)
      *reinterpret_cast<uint2*>(sP + i / TILE * S::kPBytes + S::kPChunk + i % TILE * 16 + 8) = make_uint2(0u, 0u);
    fence_proxy_async_smem();
  }
  // What came before in the stream may have written any of the inputs.
  grid_dependency_wait();
  // This CTA's share of all tiles, and the place where it begins.  The units
  // are laid on one line, each kPieceCost and a step per tile long; a CTA has the
  // tiles in its equal part of the line.  One KV head's tiles, and its length of
  // line, are summed in 32 bits (there are fewer tiles than table entries).
  if (warp == 0) {
    const int chunk = (a.B + 31) >> 5;
    const int c0 = min(a.B, lane * chunk), c1 = min(a.B, c0 + chunk);
    unsigned long long mine = 0;                     // length of line, number of tiles
#pragma unroll 4
    for (int i = c0; i < c1; ++i) {
      const unsigned nt = (pg_len(a, i) + TILE - 1) / TILE;
      mine += (static_cast<unsigned long long>(nt > 0 ? nt + kPieceCost : 0) << 32) + nt;
    }
    unsigned long long upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, m);
      if (lane >= m) upto += y;
    }
    const unsigned long long sums = __shfl_sync(0xffffffffu, upto, 31);
    const long long total = static_cast<long long>(sums >> 32) * a.units;
    const int per = static_cast<int>((static_cast<unsigned long long>(total) + kPagedCtas - 1) / kPagedCtas);
    const long long x0 = static_cast<long long>(blockIdx.x) * per;
    const long long line = static_cast<long long>((upto - mine) >> 32) * a.units;    // where this lane's requests begin
    const long long tiles = static_cast<long long>(static_cast<unsigned>(upto - mine)) * a.units;
    if (lane == 0) {
      b->per = per;
      b->n_merge = 0;
      b->first_tile[0] = b->first_tile[1] = static_cast<long long>(static_cast<unsigned>(sums)) * a.units;
    }
    __syncwarp();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {                    // the first tile of this share and that of the next
      const long long x = x0 + (k == 0 ? 0 : per);
      if (line <= x && x < line + static_cast<long long>(mine >> 32) * a.units) {
        long long at = line, t = tiles;
        int i = c0, len = pg_len(a, c0), nt = (len + TILE - 1) / TILE;
        while (nt == 0 || x >= at + static_cast<long long>(nt + kPieceCost) * a.units) {
          if (nt > 0) at += static_cast<long long>(nt + kPieceCost) * a.units;
          t += static_cast<long long>(nt) * a.units;
          len = pg_len(a, ++i);
          nt = (len + TILE - 1) / TILE;
        }
        const unsigned off = static_cast<unsigned>(x - at), unit = off / static_cast<unsigned>(nt + kPieceCost);
        const int rest = static_cast<int>(off - unit * (nt + kPieceCost));
        const int j = max(rest - kPieceCost, 0);
        b->first_tile[k] = t + static_cast<long long>(unit) * nt + j;
        if (k == 0) {
          b->start = Place{i, static_cast<int>(unit), j, len, nt};
          b->start_rest = rest;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b->tmem_base;
  const Place start = b->start;
  const int per = b->per, n_tiles = static_cast<int>(b->first_tile[1] - b->first_tile[0]);

  // the cache is streamed once, unless several row tiles read it
  const uint64_t pol = a.row_tiles > 1 ? policy_evict_last() : policy_evict_first();
  int loaded = 0;                                    // tiles that this warp has issued copies of
  if (n_tiles == 0) {
    // nothing but the empty requests below
  } else if (warp == 0) {
    // ------------------------------------------- K pages, V pages if few
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    PageBatch<TILE> pb(a, start, n_tiles, lane);
    int row = pb.fetch();
    bool ok = true;
    for (int t0 = 0; t0 < n_tiles && ok; t0 += pb.tiles) {
      const int next = pb.fetch();
      const int m = min(pb.tiles, n_tiles - t0);
      if (row == -2) report_status(a.status, DEVSTATUS_BAD_PAGE, WAIT_PAGED_TABLE);
      for (int u = 0; u < m; ++u) {
        const int t = t0 + u, s = t % NS;
        if (t >= NS && !pg_wait(&b->kv_empty[s], ((t / NS) + 1) & 1, wc, WAIT_PAGED_KV_EMPTY)) {
          ok = false;
          break;
        }
        pb.load(tmK, SHARED ? nullptr : &tmV, S::kTileBytes, row, u, sKV + s * S::kStageBytes, D, &b->kv_full[s], pol);
        loaded = t + 1;
      }
      row = next;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------- S
    const uint64_t dK = pg_desc<D>(smem_u32(sKV));                              // K tiles, K-major (A)
    const uint64_t dQ = pg_desc<D>(smem_u32(sQ));                               // queries, K-major (B)
    Walk<TILE> walk(a, start, n_tiles);
    Piece pc;
    int left = 0;                                    // tiles of the piece
    for (int g = 0, it = -1; g < n_tiles; ++g) {
      const bool begins = left == 0;
      if (begins) {
        walk.next(pc);
        left = pc.n;
        ++it;
      }
      const int s = g % NS, sb = g % S::kBufs, qb = it % S::kBufs;
      uint64_t* q_bar = &b->q_full[qb];
      // before its first use an S buffer is free: look at the K barrier twice
      const bool used = g >= S::kBufs;
      if ((begins && !pg_wait(q_bar, (it / S::kBufs) & 1, wc, WAIT_PAGED_Q)) ||
          !pg_wait2(&b->kv_full[s], (g / NS) & 1, used ? &b->s_free[sb] : &b->kv_full[s],
                    (used ? (g / S::kBufs) + 1 : g / NS) & 1, wc, WAIT_PAGED_KV))
        break;
      tc_fence_after();
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int ks = 0; ks < S::kKSteps; ++ks) {
          const uint64_t ka = uint64_t((s * S::kStageBytes + u * 128 * D + ks * 32) >> 4);
          const uint64_t qo = uint64_t((qb * S::kQBytes + ks * 32) >> 4);
          const uint32_t col = tmem + S::kColS + S::kSCols * (sb * U + u);
          mma_f8_ss_e(col, dK + ka, dQ + qo, S::kIdS, ks > 0 ? 1u : 0u);
          if (S::kFold) mma_f8_ss_e(col, dK + ka, dQ + qo + uint64_t((R * D) >> 4), S::kIdSLo, 1u);
        }
      tc_commit_e(&b->s_full[sb]);
      if (--left == 0) tc_commit_e(&b->q_empty[qb]);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------ PV
    const uint64_t dV = pg_desc<D>(smem_u32(sKV + S::kTileBytes));              // V tiles, MN-major (A)
    const uint64_t dP = pg_desc_p(smem_u32(sP), S::kPChunk);                    // P^T, MN-major (B)
    Walk<TILE> walk(a, start, n_tiles);
    Piece pc;
    int j = 0, n = 0;                                // tile of the piece, its tiles
    for (int g = 0, it = -1; g < n_tiles; ++g, ++j) {
      if (j == n) {
        walk.next(pc);
        n = pc.n;
        j = 0;
        ++it;
      }
      const int s = g % NS, ob = it & 1;
      const bool first = j < S::kTurns;              // into its turn's O
      const uint32_t col_o = tmem + S::kColO + S::kPRows * (S::kTurns * ob + g % S::kTurns);
      if ((j == 0 && it >= 2 && !pg_wait(&b->o_free[ob], ((it >> 1) + 1) & 1, wc, WAIT_PAGED_O_FREE)) ||
          !pg_wait(&b->p_full[s], (g / NS) & 1, wc, WAIT_PAGED_P))
        break;
      tc_fence_after();
#pragma unroll
      for (int kt = 0; kt < S::kPvSteps; ++kt) {
        const uint64_t va = uint64_t((s * S::kStageBytes + kt * 32 * D) >> 4);
        const uint64_t po = uint64_t((s * S::kPBytes + kt * 512) >> 4);
        mma_f8_ss_e(col_o, dV + va, dP + po, S::kIdO, (!first || kt > 0) ? 1u : 0u);
      }
      tc_commit_e(&b->kv_empty[s]);                  // P is read with V, and O has the tile
      if (j + 1 == n) tc_commit_e(&b->o_full[ob]);
    }
  } else if (warp == 2) {
    // ---------------------------- V pages if many, page scales and queries
    PageBatch<TILE> pb(a, start, n_tiles, lane);
    int row = pb.fetch();
    float ks = row >= 0 ? a.k_scale[row] : 0.0f, vs = row >= 0 ? a.v_scale[row] : 0.0f;
    Walk<TILE> walk(a, start, n_tiles);
    Piece pc, coming;
    walk.next(coming);
    QueryRows<D> rows;
    rows.template load<R>(a, coming, 0, lane);
    int it = 0, left = 0;                            // pieces begun, tiles left of the last
    float ref = 0.0f, ref2 = 1.0f;                   // r of the piece, 2^r
    bool ok = true;
    for (int t0 = 0; t0 < n_tiles && ok; t0 += pb.tiles) {
      const int next = pb.fetch();
      const int m = min(pb.tiles, n_tiles - t0);
      const float v = fmaxf(vs, 8.673617379884035e-19f);     // 2^-60; the values of a scale of 0 are cleared
      // a NaN or negative scale shows in the scores (1 / v stays finite: it meets
      // p = 0 of rows that do not see the page)
      const float lv = vs >= 0.0f ? log2f(v) : NAN, iv = 1.0f / v;
      for (int u = 0; u < m; ++u) {
        if (left == 0) {
          pc = coming;
          left = pc.n;
          const int qb = it % S::kBufs;
          if (it >= S::kBufs && !pg_wait(&b->q_empty[qb], ((it / S::kBufs) + 1) & 1, wc, WAIT_PAGED_Q_EMPTY)) {
            ok = false;
            break;
          }
          const float first_lv = __shfl_sync(0xffffffffu, row >= 0 && vs > 0.0f ? lv : 0.0f, u * pb.per_tile);
          ref = fminf(fmaxf(rintf(first_lv), -100.0f), 100.0f);
          ref2 = __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(ref)) << 23);
          if (lane == 0) b->page_ref[qb] = ref2;
#pragma unroll 1
          for (int first = 0;;) {
            rows.template split<R>(sQ + qb * S::kQBytes, b->q_factor[qb], first, lane);
            first += 8;
            if (first == R) break;
            rows.template load<R>(a, pc, first, lane);
          }
          const bool more = walk.next(coming);
          if (more) rows.template load<R>(a, coming, 0, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->q_full[qb]);
          ++it;
        }
        --left;
        const int t = t0 + u, s = t % NS;
        if (t >= NS && !pg_wait(&b->kv_empty[s], ((t / NS) + 1) & 1, wc, WAIT_PAGED_SC_EMPTY)) {
          ok = false;
          break;
        }
        if (pb.u == u)
          b->page[s][pb.i] = row >= 0 ? make_float4(ks * a.c_log2, lv - ref, iv * ref2, vs)
                                      : make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
        __syncwarp();
        if (SHARED) {
          pb.load(tmV, nullptr, 0, row, u, sKV + s * S::kStageBytes + S::kTileBytes, D, &b->kv_full[s], pol);
          loaded = t + 1;
        } else if (lane == 0) {
          mbar_arrive(&b->kv_full[s]);
        }
      }
      row = next;
      ks = row >= 0 ? a.k_scale[row] : 0.0f;
      vs = row >= 0 ? a.v_scale[row] : 0.0f;
    }
  } else if (warp < S::kEpi) {
    // ------------------------------------------------------------- softmax
    // Groups of four warps; each has its share of the rows, and its turns of the tiles.
    constexpr int H = S::kRows;
    const int wq = warp & 3;
    const int group = (warp >> 2) - 1;
    const int part = group % S::kSplit, turn = group / S::kSplit;
    const int hr = part * H;                        // this group's first row
    const uint32_t lane_base = tmem + (uint32_t(wq * 32) << 16);
    const int page_shift = 31 - __clz(a.page);
    Walk<TILE> walk(a, start, n_tiles);
    Piece pc;
    // A warp whose wait ran out goes on without waiting or arriving, so that
    // the group's hardware barriers are still met by all four warps.
    bool ok = true;
    int g = 0, it = 0;
    for (; walk.next(pc); ++it) {
      const int ob = it & 1, qb = it % S::kBufs;
      const int row0 = (a.row_tiles == 1 ? 0 : pc.unit % a.row_tiles) * R + hr;
      // minus the maximum in use, the sum, and the rows that have a maximum
      float nm[H], l_t[H];
      uint32_t have = 0;
#pragma unroll
      for (int r = 0; r < H; ++r) nm[r] = l_t[r] = 0.0f;
      bool began = false;                            // O holds a tile of this piece
      for (int j = 0; j < pc.n; ++j, ++g) {
        if (g % S::kTurns != turn) continue;
        const int sb = g % S::kBufs, st = g % NS;
        // with S come the page factors (kv_full) and the queries' factors (q_full)
        ok = ok && pg_wait3(&b->kv_full[st], (g / NS) & 1, &b->q_full[qb], (it / S::kBufs) & 1, &b->s_full[sb],
                            (g / S::kBufs) & 1, wc, WAIT_PAGED_S);
        tc_fence_after();
        const int tile0 = (pc.j0 + j) * TILE;
        float s[U][H], inv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t col = lane_base + S::kColS + S::kSCols * (sb * U + u) + hr;
          uint32_t x[H], y[H];
          if constexpr (S::kFold) {
            tmem_ld(col, x);
#pragma unroll
            for (int r = 0; r < H; ++r) s[u][r] = __uint_as_float(x[r]);
          } else {
            tmem_ld2(col, col + R, x, y);
#pragma unroll
            for (int r = 0; r < H; ++r) s[u][r] = fmaf(__uint_as_float(y[r]), 0.0625f, __uint_as_float(x[r]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&b->s_free[sb]);
        // s becomes the exponent of P, t - m
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int kt = 128 * u + wq * 32 + lane;
          const float4 f = b->page[st][kt >> page_shift];
          inv[u] = f.z;
          const bool there = tile0 + kt < pc.len && f.y != -INFINITY;
#pragma unroll
          for (int r = 0; r < H; r += 4) {
            const float4 qf = *reinterpret_cast<const float4*>(&b->q_factor[qb][hr + r]);
            const float2 k2 = make_float2(f.x, f.x), v2 = make_float2(f.y, f.y);
            const float2 x = ffma2(make_float2(s[u][r], s[u][r + 1]), fmul2(make_float2(qf.x, qf.y), k2),
                                   fadd2(v2, make_float2(nm[r], nm[r + 1])));
            const float2 y = ffma2(make_float2(s[u][r + 2], s[u][r + 3]), fmul2(make_float2(qf.z, qf.w), k2),
                                   fadd2(v2, make_float2(nm[r + 2], nm[r + 3])));
            s[u][r] = x.x;
            s[u][r + 1] = x.y;
            s[u][r + 2] = y.x;
            s[u][r + 3] = y.y;
          }
          if (!there)        // whatever came of stale codes
#pragma unroll
            for (int r = 0; r < H; ++r) s[u][r] = -INFINITY;
          if (!there || f.w == 0.0f) {   // of V, they must not meet p = 0
            uint8_t* v = sKV + st * S::kStageBytes + S::kTileBytes + kt * D + part * (D / S::kSplit);
#pragma unroll
            for (int c = 0; c < D / S::kSplit / 16; ++c) *reinterpret_cast<uint4*>(v + c * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        if (CAUSAL && tile0 + TILE > pc.len - a.Nq + 1) {
          // V codes that are NaN must not meet p = 0 either: of a key that not
          // every query sees they are cleared here, and noted for the epilogue
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int kt = 128 * u + wq * 32 + lane;
            const int edge = tile0 + kt - (pc.len - a.Nq + 1);
            if (edge >= 0 && tile0 + kt < pc.len)
              ok = clear_nan_codes<D, S::kSplit>(sKV + st * S::kStageBytes + S::kTileBytes, kt, part, edge, b->nan_keys[ob],
                                      &b->o_free[ob], it, ok, wc);
          }
          ok = __all_sync(0xffffffffu, ok);
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
        // threshold, or has a row none yet?  One barrier with a vote; the maxima
        // themselves are only exchanged when one does.
        bool need = have != (1u << H) - 1u;
        float most = -INFINITY;
#pragma unroll
        for (int r = 0; r < H; ++r)
#pragma unroll
          for (int u = 0; u < U; ++u) most = fmaxf(most, s[u][r]);
        need |= most > kRescaleThreshold;
        if (group_any(1 + group, need)) {
#pragma unroll
          for (int r = 0; r < H; r += 4) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = s[0][r + k];
#pragma unroll
              for (int u = 1; u < U; ++u) x[k] = fmaxf(x[k], s[u][r + k]);
              x[k] = redux_max(x[k]);
            }
            if (lane == 0) *reinterpret_cast<float4*>(&b->red_max[turn][wq][hr + r]) = make_float4(x[0], x[1], x[2], x[3]);
          }
          group_sync(1 + group);
          float alpha[H];
#pragma unroll
          for (int r = 0; r < H; r += 4) {
            const float4 x0 = *reinterpret_cast<const float4*>(&b->red_max[turn][0][hr + r]);
            const float4 x1 = *reinterpret_cast<const float4*>(&b->red_max[turn][1][hr + r]);
            const float4 x2 = *reinterpret_cast<const float4*>(&b->red_max[turn][2][hr + r]);
            const float4 x3 = *reinterpret_cast<const float4*>(&b->red_max[turn][3][hr + r]);
            const float x[4] = {fmaxf(fmaxf(x0.x, x1.x), fmaxf(x2.x, x3.x)), fmaxf(fmaxf(x0.y, x1.y), fmaxf(x2.y, x3.y)),
                                fmaxf(fmaxf(x0.z, x1.z), fmaxf(x2.z, x3.z)), fmaxf(fmaxf(x0.w, x1.w), fmaxf(x2.w, x3.w))};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // the first maximum is taken as it is, later ones only rise
              const bool first = !((have >> (r + k)) & 1u);
              const float shift = x[k] == -INFINITY ? 0.0f : first ? x[k] : fmaxf(x[k], 0.0f);
              alpha[r + k] = first ? 1.0f : ex2_approx(-shift);
              nm[r + k] -= shift;
#pragma unroll
              for (int u = 0; u < U; ++u) s[u][r + k] -= shift;
              if (x[k] != -INFINITY) have |= 1u << (r + k);
            }
          }
          if (began) {   // rescale O^T, once the last product into it is done
            ok = ok && pg_wait(&b->kv_empty[(g - S::kTurns) % NS], ((g - S::kTurns) / NS) & 1, wc, WAIT_PAGED_PV);
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < H; ++r) l_t[r] *= alpha[r];
            if (ok) {
#pragma unroll
              for (int k = 0; k < 3; ++k) {
                const uint32_t col = lane_base + S::kColO + S::kPRows * (S::kTurns * ob + turn) + k * R + hr;
                uint32_t o[H];
                tmem_ld(col, o);
#pragma unroll
                for (int r = 0; r < H; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[r]);
                tmem_st_x8(col, o);
              }
              tmem_wait_st();
            }
          }
        }
        // P^T into shared memory: B operand, MN-major, so that a key's eight rows
        // of one part are eight bytes in one place.  The buffer is the stage's: K
        // could only come into it once the tile before had been read, P included.
        began = true;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t hi[H / 2], mid[H / 2], lo[H / 2];
#pragma unroll
          for (int r = 0; r < H; r += 2) {
            const float2 p2 = make_float2(ex2_approx(s[u][r]), ex2_approx(s[u][r + 1]));
            const float2 l2 = ffma2(p2, make_float2(inv[u], inv[u]), make_float2(l_t[r], l_t[r + 1]));
            const float2 b2 = fmul2(p2, make_float2(kBase, kBase));
            l_t[r] = l2.x;
            l_t[r + 1] = l2.y;
            // in fp16, then its three e5m2 parts (e5m2 is fp16's upper
            // byte; adding 0x80 rounds the magnitude to nearest)
            const __half2 h = __floats2half2_rn(b2.x, b2.y);
            hi[r / 2] = (*reinterpret_cast<const uint32_t*>(&h) + 0x00800080u) & 0xff00ff00u;
            const __half2 d1 = __hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&hi[r / 2])), __float2half2_rn(8.0f));
            mid[r / 2] = (*reinterpret_cast<const uint32_t*>(&d1) + 0x00800080u) & 0xff00ff00u;
            const __half2 d2 = __hmul2(__hsub2(d1, *reinterpret_cast<const __half2*>(&mid[r / 2])), __float2half2_rn(8.0f));
            lo[r / 2] = *reinterpret_cast<const uint32_t*>(&d2) + 0x00800080u;
          }
          // the upper bytes of eight rows together
          const uint2 h8 = make_uint2(__byte_perm(hi[0], hi[1], 0x7531), __byte_perm(hi[2], hi[3], 0x7531));
          const uint2 m8 = make_uint2(__byte_perm(mid[0], mid[1], 0x7531), __byte_perm(mid[2], mid[3], 0x7531));
          const uint2 l8 = make_uint2(__byte_perm(lo[0], lo[1], 0x7531), __byte_perm(lo[2], lo[3], 0x7531));
          uint8_t* dst = sP + st * S::kPBytes + (128 * u + wq * 32 + lane) * 16;
          if constexpr (R == 8) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(h8.x, h8.y, m8.x, m8.y);
            *reinterpret_cast<uint2*>(dst + S::kPChunk) = l8;
          } else {
            uint8_t* at = dst + hr / 16 * S::kPChunk + (hr & 8);
            *reinterpret_cast<uint2*>(at) = h8;
            *reinterpret_cast<uint2*>(at + R / 16 * S::kPChunk) = m8;
            *reinterpret_cast<uint2*>(at + R / 8 * S::kPChunk) = l8;
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&b->p_full[st]);
      }
      // Piece done: publish the running max and the per-warp sums, once the
      // epilogue has let go of this buffer two pieces ago.  That every group had
      // left that piece is also why this one, which may have had no tile to wait
      // for in this piece, is not ahead of q_empty's phase.
      if (it >= 2) ok = ok && pg_wait(&b->o_free[ob], ((it >> 1) + 1) & 1, wc, WAIT_PAGED_O_FREE);
      // (by a group that had a tile, and with it waited for the piece's queries)
      if (ok && began && part == 0 && wq == 0 && lane == 0) b->stat_ref[ob] = b->page_ref[qb];
      if (ok && lane == 0) mbar_arrive(&b->q_empty[qb]);
      if (ok) {
        // Without a tile, or without a key that is there, the maximum is -inf and
        // the sum 0; scores that are all NaN leave no maximum either, but a NaN in
        // the sum of whichever warp had them.
        const float l = rows_sum<H>(l_t, lane);      // of row lane / (32 / H)
        if (lane % (32 / H) == 0) b->stat_l[ob][turn][wq][hr + lane / (32 / H)] = l;
        if (wq == 0 && lane == 0) {
#pragma unroll
          for (int r = 0; r < H; ++r) b->stat_m[ob][turn][hr + r] = (have >> r) & 1u ? -nm[r] : -INFINITY;
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
    Walk<TILE> walk(a, start, n_tiles);
    Piece pc;
    int unit_at = -b->start_rest;                    // where the unit's line begins, from this CTA's part on
    bool ok = true;          // as for the softmax warps, for the barrier of cut pieces
    for (int it = 0; walk.next(pc); ++it) {
      const int ob = it & 1;
      ok = ok && pg_wait(&b->stats_full[ob], (it >> 1) & 1, wc, WAIT_PAGED_STATS);
      const bool whole = pc.n == pc.nt;
      const int began = unit_at;                     // tile j of the unit is at began + kPieceCost + j
      if (pc.j0 + pc.n == pc.nt) unit_at += pc.nt + kPieceCost;
      const int slot = 2 * blockIdx.x + (pc.j0 > 0 ? 0 : 1);
      const int hk = kv_head(a, pc.unit);
      const int row0 = (pc.unit - hk * a.row_tiles) * R;
      const int rows = min(R, a.rows - row0);
      const size_t out = (static_cast<size_t>(pc.b) * a.Hkv + hk) * a.rows + row0;
      // lane r has row r's sum, and the factor of each turn's O: a turn without a
      // visible key has none, -1 (its O may never have been written); a factor of 0
      // counts, so that a NaN among the values shows
      float f[S::kTurns];
#pragma unroll
      for (int k = 0; k < S::kTurns; ++k) f[k] = -1.0f;
      if (ok && lane < rows) {
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int k = 0; k < S::kTurns; ++k) M = fmaxf(M, b->stat_m[ob][k][lane]);
#pragma unroll
        for (int k = 0; k < S::kTurns; ++k) {
          const float m = b->stat_m[ob][k][lane];
          const float l = b->stat_l[ob][k][0][lane] + b->stat_l[ob][k][1][lane] + b->stat_l[ob][k][2][lane] + b->stat_l[ob][k][3][lane];
          const float x = m == -INFINITY ? 0.0f : ex2_approx(m - M);
          if (m != -INFINITY || l != 0.0f) f[k] = x;    // without a maximum the sum is 0 or NaN
          L = fmaf(x, l, L);
        }
        const float inv = L == 0.0f ? 0.0f : b->stat_ref[ob] * (1.0f / kBase) / L;
#pragma unroll
        for (int k = 0; k < S::kTurns; ++k)
          if (!(f[k] < 0.0f)) f[k] *= inv;
        if (wq == 0) {
          const float lse = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
          if (whole)
            a.lse[out + lane] = lse;
          else
            a.part_lse[slot * R + lane] = lse;
        }
      }
      ok = ok && pg_wait(&b->o_full[ob], (it >> 1) & 1, wc, WAIT_PAGED_O);
      tc_fence_after();
      const uint32_t bad = CAUSAL && drow >= 0 ? b->nan_keys[ob][drow] : 0u;
      constexpr int kStep = R == 8 ? 8 : 16;
#pragma unroll 1
      for (int rg = 0; rg < R; rg += kStep) {
        float o[kStep];
#pragma unroll
        for (int t = 0; t < S::kTurns; ++t) {
          float v[kStep];
          const uint32_t col = lane_base + S::kColO + S::kPRows * (S::kTurns * ob + t) + rg;
          if constexpr (R == 8) {
            uint32_t x[32];
            tmem_ld_x32(col, x);
#pragma unroll
            for (int r = 0; r < 8; ++r)
              v[r] = fmaf(__uint_as_float(x[16 + r]), 1.0f / 64.0f,
                          fmaf(__uint_as_float(x[8 + r]), 0.125f, __uint_as_float(x[r])));
          } else {
            uint32_t x[16];
            tmem_ld_x16(col + 2 * R, x);
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] = __uint_as_float(x[r]) * (1.0f / 64.0f);
            tmem_ld_x16(col + R, x);
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] = fmaf(__uint_as_float(x[r]), 0.125f, v[r]);
            tmem_ld_x16(col, x);
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] += __uint_as_float(x[r]);
          }
#pragma unroll
          for (int k = 0; k < kStep; ++k) {
            const float w = __shfl_sync(0xffffffffu, f[t], rg + k);
            const float y = w < 0.0f ? 0.0f : v[k] * w;
            o[k] = t == 0 ? y : o[k] + y;
          }
        }
        if (CAUSAL && bad != 0u) {     // query i sees the boundary keys 0..i-1
          int i = (row0 + rg) % a.Nq;
#pragma unroll
          for (int k = 0; k < kStep; ++k) {
            if (bad & ((1u << i) - 1u)) o[k] = NAN;
            i = i + 1 == a.Nq ? 0 : i + 1;
          }
        }
        if (ok && drow >= 0) {
          if (whole) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (out + rg) * D + drow;
#pragma unroll
            for (int k = 0; k < kStep; ++k)
              if (rg + k < rows) dst[k * D] = __float2bfloat16_rn(o[k]);
          } else {
            float* dst = a.part_o + (static_cast<size_t>(slot) * R + rg) * D + drow;
#pragma unroll
            for (int k = 0; k < kStep; ++k)
              if (rg + k < rows) dst[k * D] = o[k];
          }
        }
      }
      if (CAUSAL && bad != 0u) b->nan_keys[ob][drow] = 0u;
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&b->o_free[ob]);
      if (!whole) {
        // the CTAs whose parts of the line its first and last tile are in
        const int to = began + kPieceCost;           // this CTA's part is 0..per - 1
        const int c0 = static_cast<int>(blockIdx.x) - (pc.j0 > 0 ? (per - 1 - to) / per : 0);
        const int c1 = static_cast<int>(blockIdx.x) + (to + pc.nt - 1) / per;
        group_sync(1 + S::kGroups);
        if (ok && warp == S::kEpi && mark_done(a.marks, a.nonce, slot, c0, c1, lane) && lane == 0)
          b->merge[b->n_merge++] = Merge{pc.b, pc.unit, c0, c1};
      }
    }
  }
  // requests without a token
  if (warp >= S::kEpi) {
    const int t = threadIdx.x - 32 * S::kEpi;
    for (int i = blockIdx.x; i < a.B; i += kPagedCtas) {
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
  if (b->abort) {
    // A wait ran out: outputs are undefined, but no copy may outlive the CTA.
    const WaitCtx drain{&b->drained, a.status, 1000000ull};
    for (int t = max(0, loaded - NS); t < loaded; ++t) (void)mbar_wait(&b->kv_full[t % NS], (t / NS) & 1, drain, WAIT_PAGED_KV);
    return;
  }
  uint32_t phase = 0;
  const int n_merge = b->n_merge;
  for (int i = 0; i < n_merge; ++i) merge_unit<D, R>(a, b->merge[i], smem, &b->merged, phase, wc);
}

template <int D, int R, bool CAUSAL, bool SHARED>
cudaError_t launch_paged_v(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, cudaStream_t stream) {
  constexpr size_t smem = pg_smem_bytes<D, R>();
  static_assert(smem <= 227 * 1024, "shared memory budget");
  auto kern = decode_paged_kernel<D, R, CAUSAL, SHARED>;
  static std::atomic<unsigned long long> configured{0};       // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !((configured.load(std::memory_order_acquire) >> dev) & 1u)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    if (dev <= 63) configured.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch_dependent(kern, dim3(kPagedCtas), dim3(PgShape<D, R>::kThreads), smem, stream, tk, tv, a);
}

template <int D, int R>
cudaError_t launch_paged_t(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, cudaStream_t stream) {
  // With more than four pages a tile the copies of K and V together take one warp
  // longer than the tile, so each has a warp of its own (B32 n8192, pages of 16:
  // 60.4 us with one warp, 57.7 with two; pages of 64: 54.3 and 55.5, the second
  // warp has the scales and queries to do). With few tiles a CTA that second
  // warp's start counts for more (B1 n1000: 12.4 and 13.6 us; B7 n5003, eight
  // tiles a CTA: 22.5 and 23.6). How many there are is known here by what the
  // table can hold.
  constexpr int kTile = PgShape<D, R>::kTileKeys;
  const int64_t tiles = int64_t(a.B) * a.Hkv * ((int64_t(a.max_pages) * a.page + kTile - 1) / kTile);
  const bool shared = kTile / a.page > 4 && tiles > 16 * kPagedCtas;
  if (a.causal) return shared ? launch_paged_v<D, R, true, true>(tk, tv, a, stream) : launch_paged_v<D, R, true, false>(tk, tv, a, stream);
  return shared ? launch_paged_v<D, R, false, true>(tk, tv, a, stream) : launch_paged_v<D, R, false, false>(tk, tv, a, stream);
}

}  // namespace

cudaError_t launch_decode_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int d, int row_tile,
                                cudaStream_t stream) {
  if (d == 64)
    return row_tile == 8    ? launch_paged_t<64, 8>(tk, tv, a, stream)
           : row_tile == 16 ? launch_paged_t<64, 16>(tk, tv, a, stream)
                            : launch_paged_t<64, 32>(tk, tv, a, stream);
  return row_tile == 8    ? launch_paged_t<128, 8>(tk, tv, a, stream)
         : row_tile == 16 ? launch_paged_t<128, 16>(tk, tv, a, stream)
                          : launch_paged_t<128, 32>(tk, tv, a, stream);
}

}  // namespace fa
