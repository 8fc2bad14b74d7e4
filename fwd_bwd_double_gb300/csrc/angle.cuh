// The rotary's angles and 16-byte pieces of a head, shared by the kernels that turn heads (rope.cu,
// headnorm.cu).
//
// Angles are within 2^-32 of a turn (1.5e-9 radians) before they are rounded, at every int32 position
// and for |freq| up to 2^40: freq / 2 pi as a 64-bit fraction of a turn, within 2^-64, times the
// integer position, modulo 2^64, is the fraction of a turn left over (an fp32 product freq * pos
// would lose its low bits in the thousands, a double's quotient its own far out: 2e-6 radians
// at freq 6.9, 3e-3 at 1e4).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"
#include "tc_common.cuh"

namespace fbd {
namespace angle {

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

// Turns per step of a frequency, in units of 2^-64: freq times 1 / 2 pi held as a sum of two doubles
// (106 bits), the first product's rounding error recovered by fma; the whole turns drop out of each part.
__device__ __forceinline__ unsigned long long turns_per_step(float freq) {
  const double f = static_cast<double>(freq), head = f * kInv2PiHead;
  return fraction(head) + fraction(fma(f, kInv2PiTail, fma(f, kInv2PiHead, -head)));
}

// Sine and cosine of `step` turns times an integer position.
__device__ __forceinline__ void sincos_at(long long pos, unsigned long long step, float* sn, float* cs) {
  const unsigned long long turn = static_cast<unsigned long long>(pos) * step;  // mod 2^64: whole turns drop out
  const int frac = static_cast<int>((turn + 0x80000000ull) >> 32);  // to the nearest 2^-32 of a turn
  sincospif(static_cast<float>(frac) * 4.656612873077393e-10f, sn, cs);
}

// 16 bytes as floats, and back.
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

// A thread's two 16-byte pieces p, q of a head, W pairs, turned: HALF: pair u is (p[u], q[u]); else
// neighbouring elements, p holding the thread's first W / 2 pairs, q the rest.
template <bool HALF, int W>
__device__ __forceinline__ void turn(float (&p)[W], float (&q)[W], const float (&cs)[W], const float (&sn)[W]) {
  if constexpr (HALF) {
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const float s = p[u], r = q[u];
      p[u] = s * cs[u] - r * sn[u];
      q[u] = s * sn[u] + r * cs[u];
    }
  } else {
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
}

}  // namespace angle
}  // namespace fbd
