// The 8-bit paged KV cache: writing new tokens into it, and its page tables.
//
// cache_append_kernel.  A page holds kPage tokens of one KV head as e4m3 codes
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
// of threads that holds all of it, 64 elements per thread, in registers: the
// new values are read once.
//
// page_tables_kernel.  See the comment there.
//
// Both are bound by memory or, for a few tokens, by the latency of a chain of
// dependent loads.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxWindow = 128;       // tokens whose runs one block looks for

// Eight bf16 values times `inv` -> eight e4m3 codes; a value that is not finite
// becomes the type's NaN.
__device__ __forceinline__ uint2 quantise8(uint4 x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16) * inv, hi = __uint_as_float(w[i] & 0xffff0000u) * inv;
    r[i] = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
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

// Largest absolute value among the finite ones of two packed bf16, as bits.
__device__ __forceinline__ uint32_t amax_bits(uint32_t w) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  return max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u);
}

// Power of two 2^e with the smallest e in [-60, 60] such that amax <= 448 * 2^e.
__device__ __forceinline__ float scale_for(uint32_t bf16_bits) {
  const int x = static_cast<int>(bf16_bits >> 7) - 127;       // amax = m * 2^x, 448 = 1.75 * 2^8
  int e = x - 8 + ((bf16_bits & 0x7fu) > 0x60u ? 1 : 0);
  e = min(max(e, -60), 60);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

template <int D, int PAGE>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a) {
  constexpr int kTpi = PAGE * D / 64;                  // threads that hold a page
  constexpr int kGroups = kAppendThreads / kTpi;
  constexpr int kRowChunks = D / 8;                    // 16-byte groups of a row
  __shared__ int s_lead[kMaxWindow];
  __shared__ int s_count;
  __shared__ int s_src[kGroups][PAGE];
  __shared__ int s_stop[kGroups];
  __shared__ uint32_t s_max[kAppendThreads / 32];
  const int b = blockIdx.x / a.windows;
  const int n0 = (blockIdx.x - b * a.windows) * a.window;
  const int n1 = min(a.N, n0 + a.window);
  const int h0 = blockIdx.y * a.heads_per_block;
  const int nh = min(a.Hkv - h0, a.heads_per_block);
  const int* slots = a.slots + static_cast<long long>(b) * a.N;
  const long long n_slots = static_cast<long long>(a.num_pages) * PAGE;
  auto page_of = [&](int n) -> int {
    const int s = slots[n];
    return s >= 0 && s < n_slots ? s / PAGE : -1;
  };
  if (threadIdx.x == 0) s_count = 0;
  __syncthreads();
  for (int n = n0 + threadIdx.x; n < n1; n += kAppendThreads) {
    const int p = page_of(n);
    if (slots[n] >= n_slots) report_status(a.status, DEVSTATUS_BAD_PAGE, WAIT_APPEND_SLOT);
    if (p >= 0 && (n == 0 || page_of(n - 1) != p)) s_lead[atomicAdd(&s_count, 1)] = n;
  }
  __syncthreads();
  const int group = threadIdx.x / kTpi, lane = threadIdx.x % kTpi;
  const int items = s_count * nh * 2;
  for (int first = 0; first < items; first += kGroups) {
    const int item = first + group;
    const bool active = item < items;
    const int is_v = item & 1;
    const int h = h0 + (active ? (item >> 1) % nh : 0);
    const int lead = active ? s_lead[(item >> 1) / nh] : 0;
    const int page = active ? page_of(lead) : 0;
    // the token that each of the page's slots gets, from the run of tokens that
    // starts at `lead` and stays on the page (the last one where two name a slot)
    for (int i = lane; i < PAGE; i += kTpi) s_src[group][i] = -1;
    if (lane == 0) s_stop[group] = a.N;
    __syncthreads();
    bool more = active;
    for (int base = lead;; base += kTpi) {
      const int n = base + lane;
      const bool mine = more && n < a.N && page_of(n) == page;
      if (more && !mine) atomicMin(&s_stop[group], n);
      __syncthreads();
      const int stop = s_stop[group];
      if (mine && n < stop) atomicMax(&s_src[group][slots[n] % PAGE], n);
      more = more && stop >= base + kTpi && base + kTpi < a.N;
      if (!__syncthreads_or(more)) break;
    }
    const int* src = s_src[group];
    const bool fresh = src[0] >= 0;
    const long long ph = static_cast<long long>(page) * a.Hkv + h;
    float* scale = (is_v ? a.v_scale : a.k_scale) + ph;
    uint8_t* codes = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + ph * (PAGE * D);
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(is_v ? a.v : a.k) +
                             (static_cast<long long>(b) * a.Hkv + h) * a.N * D;
    uint4 val[8];
    uint32_t top = 0;
    float was = 0.0f;
    if (active) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = i * kTpi + lane;
        const int n = src[c / kRowChunks];
        val[i] = n >= 0 ? *reinterpret_cast<const uint4*>(x + static_cast<long long>(n) * D + (c % kRowChunks) * 8)
                        : make_uint4(0u, 0u, 0u, 0u);
      }
      if (!fresh) was = *scale;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = max(max(top, max(amax_bits(val[i].x), amax_bits(val[i].y))), max(amax_bits(val[i].z), amax_bits(val[i].w)));
    }
#pragma unroll
    for (int m = (kTpi < 32 ? kTpi : 32) / 2; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
    if (kTpi > 32) {
      if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
      __syncthreads();
      constexpr int kWarps = kTpi > 32 ? kTpi / 32 : 1;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = max(top, s_max[group * kWarps + w]);
    }
    if (active) {
      if (!(was > 0.0f && was <= 3.0e38f)) was = 0.0f;    // no usable scale: nothing of the page is kept
      const float now = fmaxf(was, scale_for(top));
      const float inv = 1.0f / now;
      const bool grow = !fresh && now != was;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = i * kTpi + lane;
        uint2* p = reinterpret_cast<uint2*>(codes + c * 8);
        if (src[c / kRowChunks] >= 0)
          *p = quantise8(val[i], inv);
        else if (grow)
          *p = was > 0.0f ? rescale8(*p, was * inv) : make_uint2(0u, 0u);
      }
    }
    __syncthreads();      // every thread has read the old scale and the slot map
    if (active && lane == 0) {
      if (!(was > 0.0f)) *scale = scale_for(top);
      else *scale = fmaxf(was, scale_for(top));
    }
  }
}

template <int D, int PAGE>
cudaError_t launch_append_t(AppendArgs a, cudaStream_t stream) {
  constexpr int kGroups = kAppendThreads / (PAGE * D / 64);
  constexpr int kHalf = kGroups > 1 ? kGroups / 2 : 1;
  // a block has about kGroups pages of K and V: of several heads where there is
  // one run of tokens, of several runs where there are many
  a.heads_per_block = a.N <= PAGE ? kHalf : 1;
  a.window = a.N <= PAGE ? a.N : PAGE * kHalf;
  static_assert(PAGE * kHalf <= kMaxWindow, "window list");
  a.windows = (a.N + a.window - 1) / a.window;
  const dim3 grid(static_cast<unsigned>(a.B) * a.windows, (a.Hkv + a.heads_per_block - 1) / a.heads_per_block);
  cache_append_kernel<D, PAGE><<<grid, kAppendThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// Page tables of a batch.  Request b holds ceil(ctx / P) pages and wants to
// grow by new_lens[b] tokens, or (negative) has finished.  Pages of finished
// requests go in front of the free ones; then requests take pages in order:
// request b is granted when need = 0 or the needs up to and with b still fit.
// Two prefix sums over the batch.  The blocks of one cluster each take the
// sums in batches of kTabThreads requests, redundantly (the lengths are a few
// kilobytes out of L2), and share the writing; the cluster barrier puts the
// returned pages before their reuse and every read of an input before the
// write of an output that may be the same memory.
constexpr int kTabThreads = 1024;
constexpr int kTabCluster = 8;

struct TabRow {
  int ctx, nw, held, start, need;      // nw < 0: not granted
};

// Inclusive prefix sum over the block; *total gets the sum.
__device__ __forceinline__ long long block_scan(long long x, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, m);
      if (lane >= m) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  if (warp > 0) x += s_warp[warp - 1];
  *total = s_warp[31];
  __syncthreads();
  return x;
}

__global__ void __launch_bounds__(kTabThreads) __cluster_dims__(kTabCluster, 1, 1) page_tables_kernel(const TableArgs a) {
  namespace cg = cooperative_groups;
  __shared__ TabRow s_row[kTabThreads];
  __shared__ long long s_warp[32];
  const auto cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int P = a.page;
  const long long cap = static_cast<long long>(a.max_pages) * P;
  const int head = min(max(*a.free_head, 0), a.n_free);
  auto ctx_of = [&](int b) { return static_cast<int>(min(static_cast<long long>(max(a.ctx_lens[b], 0)), cap)); };
  // pages that come back, and their places in front of the free ones
  long long back = 0;
  for (int base = 0; base < a.B; base += kTabThreads) {
    const int b = base + threadIdx.x;
    long long total;
    block_scan(b < a.B && a.new_lens[b] < 0 ? (ctx_of(b) + P - 1) / P : 0, s_warp, &total);
    back += total;
  }
  const bool fits = back <= head;            // else the caller's lists contradict each other: nothing comes back
  if (!fits && rank == 0 && threadIdx.x == 0) report_status(a.status, DEVSTATUS_BAD_PAGE, WAIT_TABLES_BACK);
  const int low = fits ? static_cast<int>(head - back) : head;
  if (fits && back > 0) {
    long long carry = 0;
    for (int base = 0; base < a.B; base += kTabThreads) {
      const int b = base + threadIdx.x;
      const int held = b < a.B && a.new_lens[b] < 0 ? (ctx_of(b) + P - 1) / P : 0;
      long long total;
      const long long end = block_scan(held, s_warp, &total) + carry;
      s_row[threadIdx.x] = TabRow{0, 0, held, static_cast<int>(end - held), 0};
      __syncthreads();
      const int rows = min(kTabThreads, a.B - base);
      for (int r = rank * 32 + (threadIdx.x >> 5); r < rows; r += kTabCluster * 32)
        for (int i = threadIdx.x & 31; i < s_row[r].held; i += 32)
          a.free_pages[low + s_row[r].start + i] =
              a.block_table[static_cast<long long>(base + r) * a.max_pages + i];
      carry += total;
      __syncthreads();
    }
  }
  cluster.sync();
  const long long avail = a.n_free - low;
  long long carry = 0;
  int taken = 0;
  for (int base = 0; base < a.B; base += kTabThreads) {
    const int b = base + threadIdx.x;
    TabRow row{0, -1, 0, 0, 0};
    bool finished = false;
    if (b < a.B) {
      const int nw = a.new_lens[b];
      row.ctx = ctx_of(b);
      row.held = (row.ctx + P - 1) / P;
      finished = nw < 0;
      if (nw >= 0 && nw <= a.N && row.ctx + static_cast<long long>(nw) <= cap) {
        row.nw = nw;
        row.need = (row.ctx + nw + P - 1) / P - row.held;
      }
    }
    long long total;
    const long long end = block_scan(row.need, s_warp, &total) + carry;
    if (row.need > 0 && end > avail) {
      row.nw = -1;
      row.need = 0;
    }
    row.start = static_cast<int>(min(end - row.need, static_cast<long long>(a.n_free)));
    carry += total;
    // the needs' sums never fall, so what is granted is the largest sum that fits
    long long granted;
    block_scan(row.need, s_warp, &granted);
    taken += static_cast<int>(granted);
    s_row[threadIdx.x] = row;
    // another block may still read the lengths that are about to be overwritten
    cluster.sync();
    if (b < a.B && rank == 0) a.seq_lens[b] = finished ? 0 : row.ctx + max(row.nw, 0);
    const int rows = min(kTabThreads, a.B - base);
    for (int r = rank * 32 + (threadIdx.x >> 5); r < rows; r += kTabCluster * 32)
      for (int i = threadIdx.x & 31; i < s_row[r].need; i += 32)
        a.block_table[static_cast<long long>(base + r) * a.max_pages + s_row[r].held + i] =
            a.free_pages[low + s_row[r].start + i];
    const long long cells = static_cast<long long>(rows) * a.N;
    for (long long i = rank * kTabThreads + threadIdx.x; i < cells; i += kTabCluster * kTabThreads) {
      const int r = static_cast<int>(i / a.N);
      const int t = static_cast<int>(i - static_cast<long long>(r) * a.N);
      const TabRow w = s_row[r];
      int slot = -1, pos = 0;
      if (t < w.nw) {
        pos = w.ctx + t;
        const int lp = pos / P;
        const int page = lp < w.held ? a.block_table[static_cast<long long>(base + r) * a.max_pages + lp]
                                     : a.free_pages[low + w.start + lp - w.held];
        if (page >= 0 && page < 0x7fffffff / P) slot = page * P + (pos - lp * P);
      }
      const long long at = static_cast<long long>(base) * a.N + i;
      a.slots[at] = slot;
      a.positions[at] = pos;
    }
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) *a.free_head_out = low + taken;
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
  page_tables_kernel<<<kTabCluster, kTabThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
