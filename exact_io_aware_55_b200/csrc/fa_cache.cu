// The 8-bit paged KV cache: writing new tokens into it, and its page tables.
//
// cache_append_kernel.  A page holds PAGE tokens of one KV head as e4m3 codes
// with one scale, value = code * scale.  The tokens that a call writes to one
// page are quantised together:
//   e      = smallest exponent with amax <= 448 * 2^e over the finite new values
//   scale' = max(scale, 2^e), or 2^e where the page starts anew (its first
//            slot is among those written)
//   code   = e4m3(x / scale'), and where the scale grew the codes that stay
//            become e4m3(code * scale / scale').
// Scales are powers of two: a floating code gains nothing from a finer one,
// x / scale' is exact, and so is moving old codes to a larger scale except
// where they fall among the type's subnormals.  A page is written by one group
// of threads that holds all of it, 64 elements per thread (fewer where a page is
// small), in registers: the new values are read once.  Many tokens are bound by
// memory, 3 bytes per element (B4 Hkv8 N8192 d128, 164 MB: 33.8 us among others,
// 4.8 TB/s, 37 alone), and by loads of which each waits for the one before: slot,
// scale, values.  A few tokens are that chain (B64 N1: 4.2 us, most of it the
// launch).
//
// page_tables_kernel.  See the comment there.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kAppendThreads = 256;

// x / scale with inv = 1 / scale rounded: the product, and what is left of x added
// in the same way (one step of refinement, so that a quotient of few bits, a tie of
// the rounding that follows among them, comes out exactly).
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, scale, x), inv, q);
}
// Eight bf16 values times `inv` -> eight e4m3 codes.
__device__ __forceinline__ uint2 quantise8(uint4 x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}
// The same with quotients, for a scale that is no power of two (of a cache filled
// elsewhere); a value that is not finite becomes the type's NaN (the conversion
// alone makes the largest value of an infinity).  A function of its own, so that
// the common path keeps its registers: B4 Hkv8 N8192 d128 33.8 us (pages of 32
// 33.7), inline 34.9 (38.6).
__device__ __noinline__ uint2 quantise8_odd(uint4 x, float scale, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = __nv_cvt_float2_to_fp8x2(make_float2(quotient(__uint_as_float(w[i] << 16), scale, inv),
                                                quotient(__uint_as_float(w[i] & 0xffff0000u), scale, inv)),
                                    __NV_SATFINITE, __NV_E4M3);
    if ((w[i] & 0x7f80u) == 0x7f80u) r[i] = (r[i] & 0xff00u) | 0x7fu;
    if ((w[i] & 0x7f800000u) == 0x7f800000u) r[i] = (r[i] & 0x00ffu) | 0x7f00u;
  }
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Eight e4m3 codes times `ratio` (at most 1).
__device__ __forceinline__ uint2 rescale8(uint2 x, float ratio) {
  uint32_t w[2] = {x.x, x.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> (16 * k)), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      r |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE,
                                                          __NV_E4M3)) << (16 * k);
    }
    w[i] = r;
  }
  return make_uint2(w[0], w[1]);
}

// Largest absolute values of the lower and the upper halves of bf16 pairs, as bits.
__device__ __forceinline__ uint32_t amax2(uint4 x) {
  constexpr uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
}
// Bits of a pair with what is not finite made 0.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0x7fffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0x7fff0000u);
}

// Power of two 2^e with the smallest e in [-60, 60] such that amax <= 448 * 2^e.
__device__ __forceinline__ float scale_for(uint32_t bf16_bits) {
  const int x = static_cast<int>(bf16_bits >> 7) - 127;       // amax = m * 2^x, 448 = 1.75 * 2^8
  int e = x - 8 + ((bf16_bits & 0x7fu) > 0x60u ? 1 : 0);
  e = min(max(e, -60), 60);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// A group of kTpi threads holds a page of one head, K or V, and works alone: it
// takes a window of PAGE tokens of one request, finds the tokens that begin a
// run on a page (none, or one or two as a rule) and writes those pages.  Every
// warp of the group looks at the slots by itself; the group meets only for the
// maximum.
template <int D, int PAGE>
struct AppendShape {
  static constexpr int kTpi = PAGE * D / 64 > 32 ? PAGE * D / 64 : 32;
  static constexpr int kChunks = PAGE * D / 8 / kTpi;  // 16-byte groups of eight elements per thread
  static constexpr int kGroups = kAppendThreads / kTpi;
};

template <int D, int PAGE>
__global__ void __launch_bounds__(kAppendThreads, 4) cache_append_kernel(const AppendArgs a) {
  using S = AppendShape<D, PAGE>;
  constexpr int kTpi = S::kTpi, kChunks = S::kChunks;
  constexpr int kRowChunks = D / 8;
  __shared__ int s_slot[S::kGroups][2 * PAGE];
  __shared__ int s_src[S::kGroups][PAGE];
  __shared__ uint32_t s_max[kAppendThreads / 32];
  const int group = threadIdx.x / kTpi, t = threadIdx.x % kTpi, lane = threadIdx.x & 31;
  auto meet = [&]() {        // the group's threads (ids 1.. of the hardware barriers)
    if constexpr (kTpi == 32)
      __syncwarp();
    else
      asm volatile("barrier.cta.sync %0, %1;" ::"r"(group + 1), "n"(kTpi) : "memory");
  };
  // (request, window, head, K or V), the last fastest: neighbours read the same slots
  const unsigned item = blockIdx.x * S::kGroups + group;
  const bool is_v = item & 1u;
  const unsigned bwh = item >> 1, bw = bwh / static_cast<unsigned>(a.Hkv);
  const int h = static_cast<int>(bwh - bw * a.Hkv);
  const int b = static_cast<int>(bw / static_cast<unsigned>(a.windows));
  const int n0 = static_cast<int>(bw - static_cast<unsigned>(b) * a.windows) * PAGE;
  if (b >= a.B) return;
  grid_dependency_wait();
  const int* slots = a.slots + static_cast<long long>(b) * a.N;
  const int n_slots = static_cast<int>(min(static_cast<long long>(a.num_pages) * PAGE, 0x7fffffffll));
  auto fetch = [&](int n) {
    const int s = n < a.N ? slots[n] : -1;
    return s < n_slots ? s : -1;
  };
  // the window's slots and as many behind it; -1: none
  int* near = s_slot[group];
  int before = n0 > 0 && t == 0 ? fetch(n0 - 1) : -1;
#pragma unroll
  for (int i = t; i < 2 * PAGE; i += kTpi) {
    near[i] = fetch(n0 + i);
    if (i < PAGE && n0 + i < a.N && slots[n0 + i] >= n_slots) report_status(a.status, DEVSTATUS_BAD_PAGE, WAIT_APPEND_SLOT);
  }
  meet();
  if constexpr (kTpi > 32) {
    if (t == 0) s_src[group][0] = before;
    meet();
    before = s_src[group][0];
    meet();
  } else {
    before = __shfl_sync(0xffffffffu, before, 0);
  }
  auto slot_of = [&](int n) { return n - n0 < 2 * PAGE ? near[n - n0] : fetch(n); };   // n >= n0
  const int n1 = min(a.N, n0 + PAGE);
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(is_v ? a.v : a.k) +
                           (static_cast<long long>(b) * a.Hkv + h) * a.N * D;
#pragma unroll 1
  for (int c0 = n0; c0 < n1; c0 += 32) {
    const int mine = c0 + lane;
    const int slot = mine < n1 ? near[mine - n0] : -1;
    const int prev = mine == n0 ? before : mine < n1 ? near[mine - n0 - 1] : -1;
    uint32_t leads = __ballot_sync(0xffffffffu, slot >= 0 && (prev < 0 || prev / PAGE != slot / PAGE));
#pragma unroll 1
    for (; leads != 0; leads &= leads - 1) {
      const int lead = c0 + __ffs(leads) - 1;
      const int first = __shfl_sync(0xffffffffu, slot, __ffs(leads) - 1);
      const int page = first / PAGE, off = first - page * PAGE;
      // tokens in a row on slots in a row, up to the page's end
      int len = 0;
#pragma unroll 1
      for (;; len += 32) {
        const int k = len + lane;
        const uint32_t in = __ballot_sync(0xffffffffu, k < PAGE - off && near[lead - n0 + k] == first + k);
        if (in != 0xffffffffu) {
          len += __ffs(~in) - 1;
          break;
        }
      }
      // a run that goes on upon the page in another order: the later of two
      // tokens of one slot is stored
      const int behind = slot_of(lead + len);
      const bool odd = behind >= 0 && behind / PAGE == page;
      int* src = s_src[group];
      if (odd) {
        for (int i = t; i < PAGE; i += kTpi) src[i] = -1;
        meet();
#pragma unroll 1
        for (int base = lead;; base += 32) {
          const int q = slot_of(base + lane);
          const uint32_t in = __ballot_sync(0xffffffffu, q >= 0 && q / PAGE == page);
          const int n = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
          if (lane < n) atomicMax(&src[q % PAGE], base + lane);
          if (n < 32) break;
        }
        meet();
      }
      const bool fresh = odd ? src[0] >= 0 : off == 0;
      const long long ph = static_cast<long long>(page) * a.Hkv + h;
      float* scale = (is_v ? a.v_scale : a.k_scale) + ph;
      uint8_t* codes = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + ph * (PAGE * D);
      float was = fresh ? 0.0f : *scale;
      uint4 val[kChunks];
      uint32_t put = 0;
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = i * kTpi + t, row = c / kRowChunks;
        const int n = odd ? src[row] : row >= off && row < off + len ? lead + row - off : -1;
        if (n >= 0) put |= 1u << i;
        val[i] = n >= 0 ? *reinterpret_cast<const uint4*>(x + static_cast<long long>(n) * D + (c % kRowChunks) * 8)
                        : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < kChunks; ++i) top = __vmaxu2(top, amax2(val[i]));
      bool strange = __any_sync(0xffffffffu, (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u);
      if (strange) {         // the finite ones alone
        top = 0;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          top = __vmaxu2(top, amax2(make_uint4(finite2(val[i].x), finite2(val[i].y), finite2(val[i].z), finite2(val[i].w))));
      }
      top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
      if constexpr (kTpi > 32) {
        if (lane == 0) s_max[threadIdx.x >> 5] = top;
        meet();
#pragma unroll
        for (int w = 0; w < kTpi / 32; ++w) top = max(top, s_max[group * (kTpi / 32) + w]);
      }
      if (!(was > 0.0f && was <= 3.0e38f)) was = 0.0f;    // no usable scale: nothing of the page is kept
      const float now = fmaxf(was, scale_for(top));
      const float inv = 1.0f / now;
      strange |= (__float_as_uint(now) & 0x7fffffu) != 0u;
      const bool grow = !fresh && now != was;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        uint2* p = reinterpret_cast<uint2*>(codes + (i * kTpi + t) * 8);
        if ((put >> i) & 1u)
          *p = strange ? quantise8_odd(val[i], now, inv) : quantise8(val[i], inv);
        else if (grow)
          *p = was > 0.0f ? rescale8(*p, was * inv) : make_uint2(0u, 0u);
      }
      meet();               // the old scale, the slot map and the maxima are read
      if (t == 0) *scale = now;
    }
  }
}

template <int D, int PAGE>
cudaError_t launch_append_t(AppendArgs a, cudaStream_t stream) {
  a.windows = (a.N + PAGE - 1) / PAGE;
  const long long items = static_cast<long long>(a.B) * a.windows * a.Hkv * 2;
  const long long blocks = (items + AppendShape<D, PAGE>::kGroups - 1) / AppendShape<D, PAGE>::kGroups;
  return launch_dependent(cache_append_kernel<D, PAGE>, dim3(static_cast<unsigned>(blocks)), dim3(kAppendThreads), 0, stream, a);
}

// Page tables of a batch.  Request b holds ceil(ctx / P) pages (or more, where
// the caller keeps their number, see held_pages) and wants to grow by new_lens[b] tokens, or (negative) has finished.  Pages of finished
// requests go in front of the free ones; then requests take pages in order:
// request b is granted when need = 0 or the needs up to and with b still fit.
// Two prefix sums over the batch, taken together in the halves of one 64-bit
// number.  The blocks of one cluster each take them redundantly, kTabThreads
// requests at a time (the lengths are a few kilobytes out of L2), and share the
// writing; the cluster barrier puts the returned pages before their reuse and
// every read of an input before the write of an output that may be the same
// memory.
constexpr int kTabThreads = 1024;
constexpr int kTabCluster = 16;       // B24 N8192: 12.9 us, with 8 (the portable size) 15.1; B1024 N1: 8.3 and 8.5

struct TabRow {
  int ctx, nw, held, start, need;      // nw < 0: no slots
};

// Inclusive prefix sum over the block; `total` gets the sum.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long x, unsigned long long* s_warp,
                                                         unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  unsigned long long w = s_warp[lane];     // every warp scans the warps' sums
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, w, m);
    if (lane >= m) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const unsigned long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  __syncthreads();
  return warp > 0 ? x + before : x;
}

__global__ void __launch_bounds__(kTabThreads) __cluster_dims__(kTabCluster, 1, 1) page_tables_kernel(const TableArgs a) {
  namespace cg = cooperative_groups;
  __shared__ TabRow s_row[kTabThreads];
  __shared__ unsigned long long s_warp[32];
  __shared__ int s_taken;
  const auto cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int warp = (threadIdx.x >> 5) + rank * (kTabThreads / 32), lane = threadIdx.x & 31;   // of the cluster
  constexpr int kWarps = kTabCluster * kTabThreads / 32;
  const int shift = 31 - __clz(a.page), P = a.page;
  const int cap = a.max_pages << shift;
  if (threadIdx.x == 0) s_taken = 0;
  grid_dependency_wait();
  const int head = min(max(*a.free_head, 0), a.n_free);
  const bool once = a.B <= kTabThreads;
  TabRow row;
  bool finished;
  // request b's row before anything is granted; pages that come back in `back`
  auto load = [&](int b, int& back) {
    row = TabRow{0, -1, 0, 0, 0};
    finished = false;
    back = 0;
    if (b >= a.B) return;
    const int nw = a.new_lens[b];
    row.ctx = min(max(a.ctx_lens[b], 0), cap);
    row.held = (row.ctx + P - 1) >> shift;
    if (a.held_pages) row.held = min(max(a.held_pages[b], row.held), a.max_pages);
    finished = nw < 0;
    if (finished) back = row.held;
    if (nw >= 0 && nw <= a.N && nw <= cap - row.ctx) {
      row.nw = nw;
      row.need = max(((row.ctx + nw + P - 1) >> shift) - row.held, 0);
    }
  };
  unsigned long long end = 0, total = 0, carry = 0;
  int back;
  for (int base = 0; base < a.B; base += kTabThreads) {
    load(base + threadIdx.x, back);
    end = block_scan((static_cast<unsigned long long>(back) << 32) | static_cast<unsigned>(row.need), s_warp, total);
    carry += total >> 32;
  }
  const bool fits = carry <= static_cast<unsigned long long>(head);
  if (!fits && warp == 0 && lane == 0) report_status(a.status, DEVSTATUS_BAD_PAGE, WAIT_TABLES_BACK);
  const int low = fits ? head - static_cast<int>(carry) : head;   // else the lists contradict each other: nothing comes back
  if (fits && carry > 0) {
    unsigned start = 0;
    for (int base = 0; base < a.B; base += kTabThreads) {
      if (!once) {
        load(base + threadIdx.x, back);
        end = block_scan(static_cast<unsigned long long>(back) << 32, s_warp, total);
      }
      s_row[threadIdx.x] = TabRow{0, 0, back, static_cast<int>(start + static_cast<unsigned>(end >> 32)) - back, 0};
      const unsigned end_of_batch = start + static_cast<unsigned>(total >> 32);
      __syncthreads();
      // page i of all is the last row's whose pages begin at or before it; four
      // at a time, so that their loads are on their way together
      const int rows = min(kTabThreads, a.B - base);
      constexpr int kAll = kTabCluster * kTabThreads;
#pragma unroll 1
      for (unsigned i0 = start + rank * kTabThreads + threadIdx.x; i0 < end_of_batch; i0 += 4 * kAll) {
        int page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned i = i0 + k * kAll;
          int r = 0;
#pragma unroll
          for (int step = kTabThreads / 2; step > 0; step >>= 1)
            if (r + step < rows && static_cast<unsigned>(s_row[r + step].start) <= i) r += step;
          page[k] = i < end_of_batch ? a.block_table[static_cast<long long>(base + r) * a.max_pages + (i - s_row[r].start)] : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i0 + k * kAll < end_of_batch) a.free_pages[low + (i0 + k * kAll)] = page[k];
      }
      start = end_of_batch;
      __syncthreads();
    }
  }
  cluster.sync();
  const unsigned avail = a.n_free - low;
  unsigned asked = 0;                    // by the requests of the batches before
  for (int base = 0; base < a.B; base += kTabThreads) {
    if (!once) {
      load(base + threadIdx.x, back);
      end = block_scan(static_cast<unsigned>(row.need), s_warp, total);
      // another block may still read the lengths that are about to be overwritten
      cluster.sync();
    }
    const unsigned upto = asked + static_cast<unsigned>(end);
    asked += static_cast<unsigned>(total);
    if (row.need > 0) {
      if (upto > avail) {
        row.nw = -1;
        row.need = 0;
      } else {
        row.start = low + static_cast<int>(upto) - row.need;
        // needs only add up, so the granted ones come first: what they take is the last's sum
        if (asked > avail) atomicMax(&s_taken, static_cast<int>(upto));
      }
    }
    s_row[threadIdx.x] = row;
    const int b = base + threadIdx.x;
    if (b < a.B && rank == 0) {
      a.seq_lens[b] = finished ? 0 : row.ctx + max(row.nw, 0);
      if (a.held_pages) a.held_pages[b] = finished ? 0 : row.held + row.need;
    }
    if (asked <= avail && threadIdx.x == 0) s_taken = static_cast<int>(asked);
    __syncthreads();
    const int rows = min(kTabThreads, a.B - base);
    // Page of new token t (-1: none), and its slot; the first token on a new page
    // enters it in the table.  Apart, so that the loads of several tokens are on
    // their way together.
    auto page_of = [&](const TabRow& w, int r, int t) {
      if (t >= w.nw) return -1;
      const int lp = (w.ctx + t) >> shift;
      return lp < w.held ? a.block_table[static_cast<long long>(base + r) * a.max_pages + lp] : a.free_pages[w.start + lp - w.held];
    };
    auto put = [&](const TabRow& w, int r, int t, int page, long long at) {
      const bool there = t < w.nw;
      const int pos = there ? w.ctx + t : 0, lp = pos >> shift;
      if (there && lp >= w.held && (pos & (P - 1)) == 0) a.block_table[static_cast<long long>(base + r) * a.max_pages + lp] = page;
      a.slots[at] = there && page >= 0 && page < 0x7fffffff / P ? (page << shift) + (pos & (P - 1)) : -1;
      a.positions[at] = pos;
    };
    if (a.N >= 32) {           // a warp takes 32 * kPer tokens of a request
      constexpr int kPer = 8;
      const unsigned parts = (static_cast<unsigned>(a.N) + 32 * kPer - 1) / (32 * kPer);
      const unsigned long long items = static_cast<unsigned long long>(parts) * rows;
      unsigned r = warp / parts, part = warp - r * parts;
#pragma unroll 1
      for (unsigned long long i = warp; i < items; i += kWarps) {
        const TabRow w = s_row[r];
        const long long at = static_cast<long long>(base + r) * a.N;
        const unsigned t0 = part * (32 * kPer) + lane;
        int page[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          page[k] = t0 + 32 * k < static_cast<unsigned>(a.N) ? page_of(w, r, static_cast<int>(t0 + 32 * k)) : -1;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (t0 + 32 * k < static_cast<unsigned>(a.N)) put(w, r, static_cast<int>(t0 + 32 * k), page[k], at + t0 + 32 * k);
        part += kWarps;
        const unsigned over = part / parts;
        r += over;
        part -= over * parts;
      }
    } else {
      const unsigned cells = static_cast<unsigned>(rows) * a.N;
#pragma unroll 1
      for (unsigned i = rank * kTabThreads + threadIdx.x; i < cells; i += kTabCluster * kTabThreads) {
        const unsigned r = i / static_cast<unsigned>(a.N), t = i - r * a.N;
        put(s_row[r], r, t, page_of(s_row[r], r, t), static_cast<long long>(base) * a.N + i);
      }
    }
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) *a.free_head_out = low + s_taken;
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, int d, cudaStream_t stream) {
  if (d == 64) {
    switch (a.page) {
      case 16: return launch_append_t<64, 16>(a, stream);
      case 32: return launch_append_t<64, 32>(a, stream);
      case 64: return launch_append_t<64, 64>(a, stream);
      default: return launch_append_t<64, 128>(a, stream);
    }
  }
  switch (a.page) {
    case 16: return launch_append_t<128, 16>(a, stream);
    case 32: return launch_append_t<128, 32>(a, stream);
    case 64: return launch_append_t<128, 64>(a, stream);
    default: return launch_append_t<128, 128>(a, stream);
  }
}

cudaError_t launch_page_tables(const TableArgs& a, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};       // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !((configured.load(std::memory_order_acquire) >> dev) & 1u)) {
    e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev <= 63) configured.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch_dependent(page_tables_kernel, dim3(kTabCluster), dim3(kTabThreads), 0, stream, a);
}

}  // namespace fa
