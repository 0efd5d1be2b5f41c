// Attention of a few new queries per request over an 8-bit paged KV cache.
//
//   s_j = scale * ks_j * (q . K_j)        K_j, V_j e4m3 codes; ks_j, vs_j the
//   p_j = softmax over the visible keys   scales of key j's page and KV head
//   O   = sum_j p_j * vs_j * V_j,  LSE = ln sum_j exp(s_j)
// Key j of a request is row j % P of page block_table[b][j / P]; keys at or
// past the request's length are never used, whatever their bytes hold.  A row
// without a visible key gives O = 0 and LSE = -inf.
//
// One block per (query row, request): its warps take 32 keys at a time, a lane
// per key for the scores and d / 32 columns per lane for the values, each with
// a running maximum and sum, and merge through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float2 e4m3x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) decode_paged_simple(const PagedArgs a) {
  constexpr int kCols = D / 32;
  __shared__ float s_q[D];
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int row = blockIdx.x;                      // head * Nq + query
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = row / a.Nq, i = row - h * a.Nq;
  const int hk = h / (a.H / a.Hkv);
  const size_t out = (static_cast<size_t>(b) * a.H * a.Nq + row);
  for (int c = threadIdx.x; c < D; c += kWarps * 32)
    s_q[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[out * D + c]);
  __syncthreads();
  const int len = static_cast<int>(min(static_cast<long long>(max(a.seq_lens[b], 0)), static_cast<long long>(a.max_pages) * a.page));
  const int end = a.causal ? len - a.Nq + 1 + i : len;
  const int* table = a.block_table + static_cast<size_t>(b) * a.max_pages;
  float m = -INFINITY, l = 0.0f, o[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c] = 0.0f;
  for (int j0 = warp * 32; j0 < end; j0 += kWarps * 32) {
    const int j = j0 + lane;
    float s = -INFINITY, vs = 0.0f;
    long long r = 0;
    if (j < end) {
      const int page = table[j / a.page];
      if (page >= 0 && page < a.num_pages) {
        const size_t ph = static_cast<size_t>(page) * a.Hkv + hk;
        r = static_cast<long long>(ph) * a.page + j % a.page;
        const uint4* kr = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.k_cache) + r * D);
        float acc = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 w = kr[c];
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float2 lo = e4m3x2(x[t]), hi = e4m3x2(x[t] >> 16);
            acc = fmaf(s_q[c * 16 + t * 4], lo.x, acc);
            acc = fmaf(s_q[c * 16 + t * 4 + 1], lo.y, acc);
            acc = fmaf(s_q[c * 16 + t * 4 + 2], hi.x, acc);
            acc = fmaf(s_q[c * 16 + t * 4 + 3], hi.y, acc);
          }
        }
        s = acc * a.k_scale[ph] * a.c_log2;
        vs = a.v_scale[ph];
      } else {
        report_status(a.status, DEVSTATUS_BAD_PAGE, WAIT_PAGED_TABLE);
      }
    }
    float mt = s == s ? s : 0.0f;      // a NaN score must not hide from the maximum: its p is NaN
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
    const float mn = fmaxf(m, mt);
    if (mn == -INFINITY) continue;
    const float alpha = ex2_approx(m - mn);
    const float p = s == -INFINITY ? 0.0f : ex2_approx(s - mn);
    float lt = p;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, x);
    l = l * alpha + lt;
    m = mn;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c] *= alpha;
    const float pv = p * vs;
    const int n = min(32, end - j0);
    for (int t = 0; t < n; ++t) {
      const float w = __shfl_sync(0xffffffffu, pv, t);
      const long long rt = __shfl_sync(0xffffffffu, r, t);
      if (__shfl_sync(0xffffffffu, s, t) == -INFINITY) continue;
      const uint8_t* vr = static_cast<const uint8_t*>(a.v_cache) + rt * D + lane * kCols;
      if (kCols == 4) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(vr);
        const float2 lo = e4m3x2(x), hi = e4m3x2(x >> 16);
        o[0] = fmaf(w, lo.x, o[0]);
        o[1] = fmaf(w, lo.y, o[1]);
        o[kCols - 2] = fmaf(w, hi.x, o[kCols - 2]);
        o[kCols - 1] = fmaf(w, hi.y, o[kCols - 1]);
      } else {
        const float2 lo = e4m3x2(*reinterpret_cast<const uint16_t*>(vr));
        o[0] = fmaf(w, lo.x, o[0]);
        o[1] = fmaf(w, lo.y, o[1]);
      }
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int c = 0; c < kCols; ++c) s_o[warp][lane * kCols + c] = o[c];
  __syncthreads();
  float M = -INFINITY, L = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  if (M != -INFINITY)
    for (int w = 0; w < kWarps; ++w) L += s_l[w] * ex2_approx(s_m[w] - M);
  for (int c = threadIdx.x; c < D; c += kWarps * 32) {
    float x = 0.0f;
    if (M != -INFINITY)
      for (int w = 0; w < kWarps; ++w) x += s_o[w][c] * ex2_approx(s_m[w] - M);
    static_cast<__nv_bfloat16*>(a.o)[out * D + c] = __float2bfloat16_rn(M != -INFINITY ? x / L : 0.0f);
  }
  if (threadIdx.x == 0) a.lse[out] = M != -INFINITY ? (M + lg2_approx(L)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

cudaError_t launch_decode_paged(const PagedArgs& a, int d, cudaStream_t stream) {
  const dim3 grid(a.H * a.Nq, a.B);
  if (d == 64)
    decode_paged_simple<64><<<grid, kWarps * 32, 0, stream>>>(a);
  else
    decode_paged_simple<128><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
