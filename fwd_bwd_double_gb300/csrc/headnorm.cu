// RMS norm of each head's vector and its rotary positions in one pass, to [B, heads, N, d] views or
// into the pages of a cache:  z = w x r,  r = (mean x^2 + eps)^(-1/2),  y = R(angle) z,
// and its gradient:  dz = R(-angle) dy,  dw = sum of dz x r,  dx = r (w dz - x r^2 mean(w dz x)).
//
// Bound by reading and writing each element once.  A group of threads (a power of two of them, so
// that a warp holds whole groups; at d = 96 a quarter of them idle) takes a token: a thread holds
// 16 bytes of each half of the head (neighbouring pairs: 32 bytes in a row), so that both
// coordinates of its pairs are its own and the sum of squares is a few shuffles.  The sines of its
// pairs serve all its heads.  Squares, sums and r are fp32; each output is rounded once.
#include <cuda_bf16.h>

#include "angle.cuh"
#include "diff.h"
#include "paged.h"

namespace fbd {
namespace {

constexpr int kT = 256;
constexpr int kMaxPairs = 128;
constexpr int kHU = 4;  // heads whose loads are in flight together

// Threads per token: its pairs in pieces of W, rounded up to a power of two.
__host__ __device__ inline int group_threads(int d, int W) {
  int n = 1;
  while (n * W < d / 2) n *= 2;
  return n;
}

__device__ __forceinline__ float group_sum(float v, int LG) {
  for (int o = LG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 2 W consecutive-per-piece floats of a table in shared memory.
template <int W>
__device__ __forceinline__ void take(const float* s, int c, float (&x)[W]) {
#pragma unroll
  for (int u = 0; u < W; u += 4) *reinterpret_cast<float4*>(x + u) = *reinterpret_cast<const float4*>(s + c + u);
}

// The frequencies' turns per step and their axes (outside 0 .. axes - 1: -1).
__device__ __forceinline__ void angle_tables(const float* freq, const int* axis, int pairs, int axes,
                                             unsigned long long* sT, int* sAx) {
  for (int i = threadIdx.x; i < pairs; i += kT) {
    sT[i] = angle::turns_per_step(freq[i]);
    const int ax = axis[i];
    sAx[i] = ax < axes ? ax : -1;
  }
}

template <typename T, bool HALF, bool APPEND>
__global__ void __launch_bounds__(kT) head_kernel(const HeadArgs a) {
  constexpr int W = 16 / sizeof(T);  // pairs per thread
  __shared__ unsigned long long sT[kMaxPairs];
  __shared__ int sAx[kMaxPairs];
  __shared__ __align__(16) float sW[4][2 * kMaxPairs];
  const int pairs = a.d / 2, per = pairs / W, LG = group_threads(a.d, W);
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x;
  const int64_t tokens = a.B * a.N, token = gid / LG;
  const int part = static_cast<int>(gid) & (LG - 1);
  const bool in = token < tokens && part < per;  // (the others take part in the shuffles)
  const bool packed = APPEND && a.seqs.cu != nullptr;
  const int64_t b = in && !packed ? token / a.N : 0, n = in ? token - b * a.N : 0;
  const int hb = blockIdx.y * a.per_thread;
  const int he = min(hb + a.per_thread, a.heads);
  const int c0 = HALF ? part * W : 2 * part * W, c1 = HALF ? c0 + pairs : c0 + W;
  // kHU heads' loads at a time, the next ones' before these are worked on (y may be x, but no other head's).
  struct Heads {
    uint4 lo[kHU], hi[kHU];
  };
  auto locate = [&](int h, int& t) {  // head h of all tensors: the returned one of tensor t
    t = 0;
    while (h >= a.t[t].heads) h -= a.t[t].heads, ++t;
    return h;
  };
  auto fetch = [&](int h, Heads& z) {
#pragma unroll
    for (int k = 0; k < kHU; ++k) {
      z.lo[k] = z.hi[k] = make_uint4(0, 0, 0, 0);
      if (h + k >= he || !in) continue;
      int t;
      const int hh = locate(h + k, t);
      const T* x = static_cast<const T*>(a.t[t].x) + b * a.t[t].xs[0] + hh * a.t[t].xs[1] + n * a.t[t].xs[2];
      z.lo[k] = *reinterpret_cast<const uint4*>(x + c0);
      z.hi[k] = *reinterpret_cast<const uint4*>(x + c1);
    }
  };
  Heads now, next;
  fetch(hb, now);
  // Behind those loads: the tables, and where the token belongs.
  if (a.freq != nullptr) angle_tables(a.freq, a.axis, pairs, a.axes, sT, sAx);
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (a.t[t].heads > 0 && a.t[t].norm)
      for (int i = threadIdx.x; i < a.d; i += kT) sW[t][i] = a.t[t].w != nullptr ? a.t[t].w[i] : 1.f;
  bool live = in;
  int at = 0, page = -1, slot = 0;  // its position in its sequence and its place in the cache
  if (APPEND && token < tokens) {
    const Seqs& q = a.seqs;
    int s = static_cast<int>(b);
    if (packed) {  // the last sequence that begins at or before this row
      int lo = 0, hi = q.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.cu[mid] <= token) lo = mid; else hi = mid;
      }
      s = lo;
    }
    const Seq z = seq_at(q, s);
    const int64_t t = (packed ? token : token - static_cast<int64_t>(s) * a.N) - z.row0;
    live = live && t >= 0 && t < z.n;  // (a row of no sequence)
    const int64_t p = static_cast<int64_t>(z.start) + t;
    at = static_cast<int>(p);
    if (live && p >= 0 && p < q.cap) {
      const int e = at / q.page;
      page = page_at(q, s, e), slot = at - e * q.page;
    }
  }
  int pos[W];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < W; ++u) {
    const int ax = a.freq != nullptr && live ? sAx[part * W + u] : -1;
    pos[u] = ax < 0 ? 0 : APPEND && a.pos == nullptr ? at : a.pos[ax * a.pos_axis + b * a.pos_batch + n];
  }
  float cs[W], sn[W];
#pragma unroll
  for (int u = 0; u < W; ++u) {
    const int i = part * W + u;
    cs[u] = 1.f, sn[u] = 0.f;
    if (a.freq != nullptr && live && sAx[i] >= 0) angle::sincos_at(pos[u], sT[i], &sn[u], &cs[u]);
  }
  for (int h = hb; h < he; h += kHU) {
    if (h + kHU < he) fetch(h + kHU, next);
#pragma unroll
    for (int k = 0; k < kHU; ++k) {
      if (h + k >= he) break;
      int t;
      const int hh = locate(h + k, t);
      const HeadTensor& z = a.t[t];
      const bool put = live && !(APPEND && z.paged && page < 0);
      T* y = static_cast<T*>(z.y) + hh * z.ys[1] +
             (APPEND && z.paged ? page * z.ys[0] + slot * z.ys[2] : b * z.ys[0] + n * z.ys[2]);
      if (z.norm || z.turn) {
        float p[W], q[W];
        angle::widen(now.lo[k], p);
        angle::widen(now.hi[k], q);
        if (z.norm) {
          float ss = 0.f;
#pragma unroll
          for (int u = 0; u < W; ++u) ss = fmaf(p[u], p[u], fmaf(q[u], q[u], ss));
          const float r = rsqrtf(group_sum(ss, LG) / static_cast<float>(a.d) + a.eps);
          if (part < per) {
            float w0[W], w1[W];
            take(sW[t], c0, w0);
            take(sW[t], c1, w1);
#pragma unroll
            for (int u = 0; u < W; ++u) p[u] *= r * w0[u], q[u] *= r * w1[u];
          }
        }
        if (z.turn) angle::turn<HALF>(p, q, cs, sn);
        if (put) {
          angle::stv(y + c0, p);
          angle::stv(y + c1, q);
        }
      } else if (put) {
        *reinterpret_cast<uint4*>(y + c0) = now.lo[k];
        *reinterpret_cast<uint4*>(y + c1) = now.hi[k];
      }
    }
    now = next;
  }
}

template <typename T, bool HALF>
__global__ void __launch_bounds__(kT) grad_kernel(const HeadGradArgs a) {
  constexpr int W = 16 / sizeof(T);
  __shared__ unsigned long long sT[kMaxPairs];
  __shared__ int sAx[kMaxPairs];
  __shared__ __align__(16) float sW[2 * kMaxPairs];
  __shared__ float sum[kT / 32][2 * kMaxPairs];
  ptx::grid_dependency_launch();
  const int pairs = a.d / 2, per = pairs / W, LG = group_threads(a.d, W);
  int t = 0;
  while (static_cast<int>(blockIdx.y) >= a.first[t + 1]) ++t;
  const HeadGrad& z = a.t[t];
  const int hb = (blockIdx.y - a.first[t]) * a.per, he = min(hb + a.per, z.heads);
  if (a.freq != nullptr) angle_tables(a.freq, a.axis, pairs, a.axes, sT, sAx);
  for (int i = threadIdx.x; i < a.d; i += kT) sW[i] = z.w != nullptr ? z.w[i] : 1.f;
  __syncthreads();
  const int part = threadIdx.x & (LG - 1);
  const int c0 = HALF ? part * W : 2 * part * W, c1 = HALF ? c0 + pairs : c0 + W;
  const bool mine = part < per;
  float w0[W], w1[W], g0[W], g1[W];
#pragma unroll
  for (int u = 0; u < W; ++u) w0[u] = w1[u] = g0[u] = g1[u] = 0.f;
  if (mine) {
    take(sW, c0, w0);
    take(sW, c1, w1);
  }
  const int64_t tokens = a.B * a.N;
  const int step = kT / LG;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * step; base < tokens; base += static_cast<int64_t>(gridDim.x) * step) {
    const int64_t token = base + threadIdx.x / LG;
    const bool live = mine && token < tokens;
    const int64_t b = live ? token / a.N : 0, n = live ? token - b * a.N : 0;
    float cs[W], sn[W];
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const int i = part * W + u, ax = a.freq != nullptr && live ? sAx[i] : -1;
      cs[u] = 1.f, sn[u] = 0.f;
      if (ax >= 0) {
        angle::sincos_at(a.pos[ax * a.pos_axis + b * a.pos_batch + n], sT[i], &sn[u], &cs[u]);
        sn[u] = -sn[u];
      }
    }
    constexpr int U = 2;  // heads whose loads are in flight together
    for (int h = hb; h < he; h += U) {
      uint4 xl[U], xh[U], yl[U], yh[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        xl[k] = xh[k] = yl[k] = yh[k] = make_uint4(0, 0, 0, 0);
        if (h + k >= he || !live) continue;
        const T* x = static_cast<const T*>(z.x) + b * z.xs[0] + (h + k) * z.xs[1] + n * z.xs[2];
        const T* dy = static_cast<const T*>(z.dy) + b * z.dys[0] + (h + k) * z.dys[1] + n * z.dys[2];
        xl[k] = *reinterpret_cast<const uint4*>(x + c0), xh[k] = *reinterpret_cast<const uint4*>(x + c1);
        yl[k] = *reinterpret_cast<const uint4*>(dy + c0), yh[k] = *reinterpret_cast<const uint4*>(dy + c1);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (h + k >= he) break;
        float p[W], q[W], f[W], e[W];
        angle::widen(xl[k], p);
        angle::widen(xh[k], q);
        angle::widen(yl[k], f);
        angle::widen(yh[k], e);
        angle::turn<HALF>(f, e, cs, sn);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int u = 0; u < W; ++u) {
          ss = fmaf(p[u], p[u], fmaf(q[u], q[u], ss));
          dot = fmaf(w0[u] * f[u], p[u], fmaf(w1[u] * e[u], q[u], dot));
        }
        ss = group_sum(ss, LG), dot = group_sum(dot, LG);
        const float inv = 1.f / static_cast<float>(a.d), r = rsqrtf(ss * inv + a.eps);
        if (!live) continue;
        const float m = dot * inv * r * r;
#pragma unroll
        for (int u = 0; u < W; ++u) {
          g0[u] = fmaf(f[u], p[u] * r, g0[u]);
          g1[u] = fmaf(e[u], q[u] * r, g1[u]);
          p[u] = r * fmaf(-p[u], m, w0[u] * f[u]);
          q[u] = r * fmaf(-q[u], m, w1[u] * e[u]);
        }
        T* dx = static_cast<T*>(z.dx) + b * z.dxs[0] + (h + k) * z.dxs[1] + n * z.dxs[2];
        angle::stv(dx + c0, p);
        angle::stv(dx + c1, q);
      }
    }
  }
  if (z.dw == nullptr) return;
  // This block's share of dw: over the groups of a warp, then over the warps.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int u = 0; u < W; ++u)
    for (int o = LG; o < 32; o <<= 1) {
      g0[u] += __shfl_xor_sync(0xffffffffu, g0[u], o);
      g1[u] += __shfl_xor_sync(0xffffffffu, g1[u], o);
    }
  if (lane < per) {
#pragma unroll
    for (int u = 0; u < W; ++u) sum[warp][c0 + u] = g0[u], sum[warp][c1 + u] = g1[u];
  }
  __syncthreads();
  float* out = a.ws + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.d;
  for (int i = threadIdx.x; i < a.d; i += kT) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) v += sum[w][i];
    out[i] = v;
  }
}

// dw of a tensor: its blocks' shares, in a fixed order.
__global__ void __launch_bounds__(1024) weight_kernel(const HeadGradArgs a) {
  __shared__ float part[1024];
  ptx::grid_dependency_wait();
  const int t = blockIdx.x, d = a.d, groups = 1024 / d;
  const HeadGrad& z = a.t[t];
  if (z.dw == nullptr) return;
  const int64_t from = static_cast<int64_t>(a.first[t]) * a.cols, to = static_cast<int64_t>(a.first[t + 1]) * a.cols;
  const int g = threadIdx.x / d, c = threadIdx.x - g * d;
  float v = 0.f;
  if (g < groups) {
#pragma unroll 4
    for (int64_t s = from + g; s < to; s += groups) v += a.ws[s * d + c];
  }
  part[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < d) {
    for (int k = 1; k < groups; ++k) v += part[k * d + threadIdx.x];
    z.dw[threadIdx.x] = v;
  }
}

template <typename T, bool APPEND>
cudaError_t run(HeadArgs a, bool half, cudaStream_t st) {
  const int64_t threads = a.B * a.N * group_threads(a.d, 16 / static_cast<int>(sizeof(T)));
  // Heads per thread: eight or four (whole groups of loads in flight) where that leaves a wave of
  // threads on 152 SMs, so that the sines are shared.
  const int64_t hp = a.heads * threads / (152 * 2048);
  a.per_thread = hp >= 8 ? 8 : hp >= kHU ? kHU : 1;
  const dim3 grid(static_cast<unsigned>((threads + kT - 1) / kT),
                  static_cast<unsigned>((a.heads + a.per_thread - 1) / a.per_thread));
  if (half)
    head_kernel<T, true, APPEND><<<grid, kT, 0, st>>>(a);
  else
    head_kernel<T, false, APPEND><<<grid, kT, 0, st>>>(a);
  return cudaGetLastError();
}

struct GradPlan {
  int per, rows, cols;
};
GradPlan grad_plan(int64_t B, int64_t N, int64_t d, int dtype, const int64_t* heads, int count) {
  const int W = dtype == ATTN_BF16 ? 8 : 4, step = kT / group_threads(static_cast<int>(d), W);
  const int64_t groups = (B * N + step - 1) / step;  // block columns that have work
  int64_t all = 0;
  for (int t = 0; t < count; ++t) all += heads[t];
  GradPlan p;
  const int64_t hp = all * groups * kT / (152 * 2048);
  p.per = hp >= 8 ? 8 : hp >= 4 ? 4 : 1;
  p.rows = 0;
  for (int t = 0; t < count; ++t) p.rows += static_cast<int>((heads[t] + p.per - 1) / p.per);
  const int64_t want = p.rows > 0 ? (152 * 8 + p.rows - 1) / p.rows : 1;
  p.cols = static_cast<int>(groups < want ? groups : want);
  return p;
}

}  // namespace

cudaError_t head_norm(const HeadArgs& a, int dtype, bool half, bool append, cudaStream_t st) {
  if (append)
    return dtype == ATTN_BF16 ? run<__nv_bfloat16, true>(a, half, st) : run<float, true>(a, half, st);
  return dtype == ATTN_BF16 ? run<__nv_bfloat16, false>(a, half, st) : run<float, false>(a, half, st);
}

size_t head_norm_bwd_bytes(int64_t B, int64_t N, int64_t d, int dtype, const int64_t* heads, int count) {
  const GradPlan p = grad_plan(B, N, d, dtype, heads, count);
  return static_cast<size_t>(p.rows) * p.cols * d * sizeof(float);
}

cudaError_t head_norm_bwd(const HeadGradArgs& args, int dtype, bool half, cudaStream_t st) {
  HeadGradArgs a = args;
  int64_t heads[4] = {0, 0, 0, 0};
  bool dw = false;
  for (int t = 0; t < a.count; ++t) heads[t] = a.t[t].heads, dw = dw || a.t[t].dw != nullptr;
  const GradPlan p = grad_plan(a.B, a.N, a.d, dtype, heads, a.count);
  a.per = p.per, a.cols = p.cols, a.first[0] = 0;
  for (int t = 0; t < a.count; ++t) a.first[t + 1] = a.first[t] + static_cast<int>((heads[t] + p.per - 1) / p.per);
  const dim3 grid(static_cast<unsigned>(p.cols), static_cast<unsigned>(p.rows));
  if (dtype == ATTN_BF16) {
    if (half) grad_kernel<__nv_bfloat16, true><<<grid, kT, 0, st>>>(a);
    else grad_kernel<__nv_bfloat16, false><<<grid, kT, 0, st>>>(a);
  } else {
    if (half) grad_kernel<float, true><<<grid, kT, 0, st>>>(a);
    else grad_kernel<float, false><<<grid, kT, 0, st>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dw) return e;
  return launch_behind(weight_kernel, a.count, 1024, 0, st, a);
}

}  // namespace fbd
