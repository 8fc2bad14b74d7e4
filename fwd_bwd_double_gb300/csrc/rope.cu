// Rotary positions with several axes (time, height, width, ...): coordinate pair i of a
// token turns by the angle freq[i] * pos[axis[i]], (u, v) -> (u cos - v sin, u sin + v cos);
// `inverse` turns back, which is the gradient (the map is orthogonal).
//
// Bound by reading and writing each element once (16 bytes per thread and half).  Angles
// are within 2^-32 of a turn (1.5e-9 radians) before they are rounded, at every int32 position
// and for |freq| up to 2^40: freq / 2 pi as a 64-bit fraction of a turn, within 2^-64, times the
// integer position, modulo 2^64, is the fraction of a turn left over (an fp32 product freq * pos
// would lose its low bits in the thousands, a double's quotient its own far out: 2e-6 radians
// at freq 6.9, 3e-3 at 1e4).
// A thread holds the sines of its pairs and applies them to several heads.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rope.h"
#include "tc_common.cuh"

namespace fbd {
namespace {

constexpr int kT = 256;
constexpr int kMaxPairs = 128;

constexpr int kHU = 4;  // heads whose loads are in flight together

constexpr double kInv2PiHead = 0x1.45f306dc9c883p-3, kInv2PiTail = -0x1.6b01ec5417056p-57;  // 1 / 2 pi

// x in units of 2^-64, modulo 2^64 (its whole part drops out), rounded to the nearest: from the bits of
// a double, since floating point in 64 bits is slow (B2 N1001, 12 heads of 128 in float32: 8.0 us, with
// rint and a conversion 8.9).
__device__ __forceinline__ unsigned long long fraction(double x) {
  const long long b = __double_as_longlong(x);
  const unsigned long long m = (b & 0xfffffffffffffll) | 0x10000000000000ll;
  const int up = static_cast<int>(b >> 52 & 0x7ff) - (1075 - 64);
  unsigned long long v = 0;
  if (up >= 0 && up < 64) v = m << up;
  if (up < 0 && up > -64) v = ((m >> (-up - 1)) + 1) >> 1;
  return b < 0 ? 0ull - v : v;
}

// 16 bytes as floats.
__device__ __forceinline__ void widen(const uint4& v, float (&x)[4]) {
  x[0] = tc::f(v.x), x[1] = tc::f(v.y), x[2] = tc::f(v.z), x[3] = tc::f(v.w);
}
__device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) x[2 * u] = tc::bf16_lo(w[u]), x[2 * u + 1] = tc::bf16_hi(w[u]);
}
__device__ __forceinline__ void stv(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void stv(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]),
                                            ptx::pack_bf16(x[4], x[5]), ptx::pack_bf16(x[6], x[7]));
}

template <typename T, bool HALF>
__global__ void __launch_bounds__(kT)
    rope_kernel(const RopeArgs a, const int* __restrict__ pos, const float* __restrict__ freq,
                const int* __restrict__ axis) {
  constexpr int W = 16 / sizeof(T);  // pairs per thread
  __shared__ unsigned long long sT[kMaxPairs];
  __shared__ int sAx[kMaxPairs];
  const int pairs = a.d / 2, per = pairs / W;  // threads per token
  for (int i = threadIdx.x; i < pairs; i += kT) {
    // Turns per step: freq times 1 / 2 pi held as a sum of two doubles (106 bits), the first
    // product's rounding error recovered by fma; the whole turns drop out of each part.
    const double f = static_cast<double>(freq[i]), head = f * kInv2PiHead;
    sT[i] = fraction(head) + fraction(fma(f, kInv2PiTail, fma(f, kInv2PiHead, -head)));
    const int ax = axis[i];
    sAx[i] = ax < a.axes ? ax : -1;
  }
  __syncthreads();
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x;
  const int64_t token = gid / per;
  const int part = static_cast<int>(gid - token * per);
  if (token >= a.B * a.N) return;
  const int64_t b = token / a.N, n = token - b * a.N;
  float cs[W], sn[W];
#pragma unroll
  for (int u = 0; u < W; ++u) {
    const int i = part * W + u, ax = sAx[i];
    cs[u] = 1.f, sn[u] = 0.f;
    if (ax >= 0) {
      const long long p = pos[ax * a.pos_axis + b * a.pos_batch + n];
      const unsigned long long turn = static_cast<unsigned long long>(p) * sT[i];  // mod 2^64: whole turns drop out
      const int frac = static_cast<int>((turn + 0x80000000ull) >> 32);  // to the nearest 2^-32 of a turn
      sincospif(static_cast<float>(frac) * 4.656612873077393e-10f, &sn[u], &cs[u]);
      if (a.inverse) sn[u] = -sn[u];
    }
  }
  const int hb = blockIdx.y * a.per_thread;
  const int he = min(hb + a.per_thread, a.heads);
  const int c0 = HALF ? part * W : 2 * part * W, c1 = HALF ? c0 + pairs : c0 + W;
  for (int h = hb; h < he; h += kHU) {
    // The loads of kHU heads before the first store (the compiler cannot reorder them: y may be x).
    uint4 lo[kHU], hi[kHU];
    T* y[kHU];
#pragma unroll
    for (int k = 0; k < kHU; ++k) {
      if (h + k >= he) break;
      int t = 0, hh = h + k;  // head h + k of all tensors: head hh of tensor t
      while (hh >= a.t[t].heads) hh -= a.t[t].heads, ++t;
      const RopeTensor& z = a.t[t];
      const T* x = static_cast<const T*>(z.x) + b * z.xs[0] + hh * z.xs[1] + n * z.xs[2];
      y[k] = static_cast<T*>(z.y) + b * z.ys[0] + hh * z.ys[1] + n * z.ys[2];
      lo[k] = *reinterpret_cast<const uint4*>(x + c0);
      hi[k] = *reinterpret_cast<const uint4*>(x + c1);
    }
#pragma unroll
    for (int k = 0; k < kHU; ++k) {
      if (h + k >= he) break;
      float p[W], q[W];
      widen(lo[k], p);
      widen(hi[k], q);
      if constexpr (HALF) {
#pragma unroll
        for (int u = 0; u < W; ++u) {
          const float s = p[u], r = q[u];
          p[u] = s * cs[u] - r * sn[u];
          q[u] = s * sn[u] + r * cs[u];
        }
      } else {  // neighbouring pairs: p holds the thread's first W / 2 pairs, q the rest
#pragma unroll
        for (int u = 0; u < W / 2; ++u) {
          float s = p[2 * u], r = p[2 * u + 1];
          p[2 * u] = s * cs[u] - r * sn[u];
          p[2 * u + 1] = s * sn[u] + r * cs[u];
          s = q[2 * u], r = q[2 * u + 1];
          q[2 * u] = s * cs[W / 2 + u] - r * sn[W / 2 + u];
          q[2 * u + 1] = s * sn[W / 2 + u] + r * cs[W / 2 + u];
        }
      }
      stv(y[k] + c0, p);
      stv(y[k] + c1, q);
    }
  }
}

template <typename T>
cudaError_t run(RopeArgs a, bool half, const int* pos, const float* freq, const int* axis, cudaStream_t st) {
  const int64_t threads = a.B * a.N * (a.d / 2 / (16 / static_cast<int>(sizeof(T))));
  // Heads per thread: eight or four (whole groups of loads in flight) where that leaves a wave of
  // threads on 152 SMs, so that the sines, about fifty instructions a pair, are shared (24 heads of
  // 32768 tokens, bf16: 39.0, 36.5, 37.2, 40.0 us at 4, 8, 12, 24 heads).
  const int64_t hp = a.heads * threads / (152 * 2048);
  a.per_thread = hp >= 8 ? 8 : hp >= kHU ? kHU : 1;
  const dim3 grid(static_cast<unsigned>((threads + kT - 1) / kT),
                  static_cast<unsigned>((a.heads + a.per_thread - 1) / a.per_thread));
  if (half)
    rope_kernel<T, true><<<grid, kT, 0, st>>>(a, pos, freq, axis);
  else
    rope_kernel<T, false><<<grid, kT, 0, st>>>(a, pos, freq, axis);
  return cudaGetLastError();
}

}  // namespace

cudaError_t rope(const RopeArgs& a, int dtype, bool half, const int* pos, const float* freq, const int* axis,
                 cudaStream_t st) {
  return dtype == ATTN_BF16 ? run<__nv_bfloat16>(a, half, pos, freq, axis, st) : run<float>(a, half, pos, freq, axis, st);
}

}  // namespace fbd
