// Rotary positions: each pair (u, w) of a head row is turned by the angle
// position * inv_freq[pair] and multiplied by a common factor,
//   y_u = factor (u cos a - w sin a),   y_w = factor (w cos a + u sin a);
// the transposed rotation (-a) is its gradient.  Pairs are neighbours
// (interleaved) or the two halves of the first rot_dim elements; the rest of
// the row is copied.
//
// Bound by memory: 2 bytes read and 2 written per element, a few operations
// per element beside them.  A thread keeps eight pairs of one token (two
// 16-byte loads per head either way) and walks over up to eight heads, so the
// eight angles are computed once for all of them.  Measured: B1 H32 N32768 d128
// (537 MB) 88 us, 6.1 TB/s; a decode step's B64 H40 N1 (1.3 MB) 4.2 us, a launch's time.
// Angles: positions reach 10^6 and beyond, where an fp32 product has lost every
// digit behind the point, so position * inv_freq is taken in fp64 as turns
// (inv_freq / 2 pi), reduced to [-1/2, 1/2] there, and only the remainder is
// rounded to fp32 (2^-25 turns) for sincospi.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kRopeThreads = 256;

struct Pair8 {
  uint4 u, w;
};

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

__device__ __forceinline__ void turn(float& u, float& w, float c, float s) {
  const float a = u, b = w;
  u = a * c - b * s;
  w = b * c + a * s;
}

template <bool INTERLEAVED>
__device__ __forceinline__ void turn8(Pair8& x, const float (&c)[8], const float (&s)[8]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(&x.u);
  uint32_t* w = reinterpret_cast<uint32_t*>(&x.w);
  if (INTERLEAVED) {        // 16 neighbouring elements: (lo, hi) of each word is a pair
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = bf_lo(u[i]), b = bf_hi(u[i]), e = bf_lo(w[i]), f = bf_hi(w[i]);
      turn(a, b, c[i], s[i]);
      turn(e, f, c[4 + i], s[4 + i]);
      u[i] = bf_pack(a, b);
      w[i] = bf_pack(e, f);
    }
  } else {                  // element i of the first half with element i of the second
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = bf_lo(u[i]), b = bf_lo(w[i]), e = bf_hi(u[i]), f = bf_hi(w[i]);
      turn(a, b, c[2 * i], s[2 * i]);
      turn(e, f, c[2 * i + 1], s[2 * i + 1]);
      u[i] = bf_pack(a, e);
      w[i] = bf_pack(b, f);
    }
  }
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  const int chunks = a.d >> 4;                       // 16 elements of a row per thread
  const long long t = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long token = t / chunks;
  const int chunk = static_cast<int>(t - token * chunks);
  if (token >= static_cast<long long>(a.B) * a.N) return;
  const int b = static_cast<int>(token / a.N);
  const int n = static_cast<int>(token - static_cast<long long>(b) * a.N);
  const int turned = a.rot_dim >> 4;                 // chunks that are turned
  const bool turns = chunk < turned;
  grid_dependency_wait();
  if (!turns && a.in_place) return;
  int ou, ow;                                        // element offsets of the two 8-element groups
  if (INTERLEAVED || !turns) {
    ou = chunk * 16;
    ow = ou + 8;
  } else {
    ou = chunk * 8;
    ow = ou + (a.rot_dim >> 1);
  }
  float c[8], s[8];
  if (turns) {
    const double pos = a.positions ? static_cast<double>(a.positions[token]) : static_cast<double>(n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double x = pos * (a.inv_freq[chunk * 8 + i] * 0.15915494309189533577);   // turns
      const float r = static_cast<float>(x - rint(x));
      sincospif(2.0f * r, &s[i], &c[i]);
      c[i] *= a.factor;
      s[i] *= a.sin_factor;
    }
  }
  const int h0 = blockIdx.y * a.heads_per_thread;
  const int h1 = min(a.H, h0 + a.heads_per_thread);
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + b * a.xs[0] + n * a.xs[2];
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + b * a.ys[0] + n * a.ys[2];
  for (int h = h0; h < h1; ++h) {
    Pair8 v;
    v.u = *reinterpret_cast<const uint4*>(x + h * a.xs[1] + ou);
    v.w = *reinterpret_cast<const uint4*>(x + h * a.xs[1] + ow);
    if (turns) turn8<INTERLEAVED>(v, c, s);
    *reinterpret_cast<uint4*>(y + h * a.ys[1] + ou) = v.u;
    *reinterpret_cast<uint4*>(y + h * a.ys[1] + ow) = v.w;
  }
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, bool interleaved, cudaStream_t stream) {
  const long long threads = static_cast<long long>(a.B) * a.N * (a.d >> 4);
  // More heads per thread share the angles, more threads hide the latency: as many
  // heads, up to 8, as leave 640 threads an SM.  Measured with 1, 2, 4 and 8 heads:
  // B1 H32 N32768 d128 162, 105, 90, 88 us; B3 H16 N1777 d128 18.5, 14.4, 12.4,
  // 14.4 us (85 thousand threads with 8); B64 H40 N1 4.2, 4.2, 6.2, 6.2 us.
  a.heads_per_thread = 8;
  while (a.heads_per_thread > 1 && threads * ((a.H + a.heads_per_thread - 1) / a.heads_per_thread) < 148ll * 640)
    a.heads_per_thread >>= 1;
  const dim3 grid(static_cast<unsigned>((threads + kRopeThreads - 1) / kRopeThreads),
                  static_cast<unsigned>((a.H + a.heads_per_thread - 1) / a.heads_per_thread));
  return launch_dependent(interleaved ? rope_kernel<true> : rope_kernel<false>, grid, dim3(kRopeThreads), 0, stream, a);
}

}  // namespace fa
