// Rotary positions with several axes (time, height, width, ...): coordinate pair i of a
// token turns by the angle freq[i] * pos[axis[i]], (u, v) -> (u cos - v sin, u sin + v cos);
// `inverse` turns back, which is the gradient (the map is orthogonal).
//
// Bound by reading and writing each element once (16 bytes per thread and half).  The angles are
// angle.cuh's.  A thread holds the sines of its pairs and applies them to several heads.
#include <cuda_bf16.h>

#include "angle.cuh"
#include "rope.h"

namespace fbd {
namespace {

constexpr int kT = 256;
constexpr int kMaxPairs = 128;

constexpr int kHU = 4;  // heads whose loads are in flight together

template <typename T, bool HALF>
__global__ void __launch_bounds__(kT)
    rope_kernel(const RopeArgs a, const int* __restrict__ pos, const float* __restrict__ freq,
                const int* __restrict__ axis) {
  constexpr int W = 16 / sizeof(T);  // pairs per thread
  __shared__ unsigned long long sT[kMaxPairs];
  __shared__ int sAx[kMaxPairs];
  const int pairs = a.d / 2, per = pairs / W;  // threads per token
  for (int i = threadIdx.x; i < pairs; i += kT) {
    sT[i] = angle::turns_per_step(freq[i]);
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
      angle::sincos_at(pos[ax * a.pos_axis + b * a.pos_batch + n], sT[i], &sn[u], &cs[u]);
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
      angle::widen(lo[k], p);
      angle::widen(hi[k], q);
      angle::turn<HALF>(p, q, cs, sn);
      angle::stv(y[k] + c0, p);
      angle::stv(y[k] + c1, q);
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
