// Differential attention of one new token over a key/value cache.
//
//   o_m = sum_j softmax_j(s q_m.k_mj) v_j over the keys lo <= j < len of the sequence,
//   O = o_1 - lam o_2;  a sequence with no key gives 0.
// Bound by reading the cache once: the g query heads that share a key/value head are
// handled together, both maps against the same V rows.  The keys of a sequence are split
// over `nsplit` CTAs, each leaving (max, sum, unnormalised o) per row and map, which a
// second launch joins; with one split the result is written at once.
#include <cuda_bf16.h>

#include "diff.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace fbd {
namespace {

constexpr int BK = 32;    // keys per tile: one per lane
constexpr int RMAX = 8;   // query heads handled together
constexpr int kT = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct Plan {
  int rows, chunks, nsplit;  // query heads per CTA; CTAs per key/value head for the group; splits of the keys
};
Plan make_plan(const Problem& p) {
  Plan q;
  q.rows = p.group < RMAX ? p.group : RMAX;
  q.chunks = (p.group + q.rows - 1) / q.rows;
  // about four CTAs for each of the 152 SMs, a split no shorter than eight tiles
  const int64_t base = p.BHkv * q.chunks;
  const int64_t want = base > 0 ? (4 * 152 + base - 1) / base : 1;
  const int64_t most = (p.N + 8 * BK - 1) / (8 * BK);
  const int64_t n = want < most ? want : most;
  q.nsplit = static_cast<int>(n < 1 ? 1 : n > 256 ? 256 : n);
  return q;
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(tc::bf16_lo(v.x), tc::bf16_hi(v.x), tc::bf16_lo(v.y), tc::bf16_hi(v.y));
}
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

__device__ __forceinline__ void key_range(const int* lens, int b, int64_t cap, int64_t win, int64_t& lo, int64_t& n) {
  int64_t len = lens[b];
  len = len < 0 ? 0 : (len > cap ? cap : len);
  lo = win > 0 && len > win ? len - win : 0;
  n = len - lo;
}

// ws: per (b, h, map, split) 2d + 2 floats: o, max (scaled, in powers of two), sum.
template <int D, typename T>
__global__ void __launch_bounds__(kT)
    decode_kernel(const T* __restrict__ Q, const T* __restrict__ K, const T* __restrict__ V,
                  const float* __restrict__ lam, const int* __restrict__ lens, T* __restrict__ O,
                  float* __restrict__ ws, int64_t cap, int H, int G, int rows, int nsplit, int64_t win, float c) {
  constexpr int DV = 2 * D, PD = D + 4, PV = DV;
  constexpr int VC = DV / 64;  // a thread's columns: (t & 63) + 64 v of map t >> 6
  __shared__ __align__(16) float sQ[2 * RMAX * D], sK[2 * BK * PD], sV[BK * PV], sP[2 * RMAX * BK];
  __shared__ float sA[2 * RMAX], sM[2 * RMAX], sL[2 * RMAX];
  const int split = blockIdx.x % nsplit, Hkv = H / G, chunks = (G + rows - 1) / rows;
  const int unit = blockIdx.x / nsplit;  // (b, key/value head, chunk of its query heads)
  const int r0 = unit % chunks * rows, n = unit / chunks % Hkv, b = unit / chunks / Hkv;
  const int R = min(rows, G - r0);
  const int64_t kvh = static_cast<int64_t>(b) * Hkv + n;
  const int64_t h0 = static_cast<int64_t>(b) * H + n * G + r0;  // first query head
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t lo, cnt;
  key_range(lens, b, cap, win, lo, cnt);
  const int64_t per = ((cnt + nsplit - 1) / nsplit + BK - 1) / BK * BK;
  const int64_t kb = lo + split * per, ke = min(lo + cnt, kb + per);
  for (int u = threadIdx.x; u < 2 * R * D / 4; u += kT) {
    const int row = u * 4 / D, cc = u * 4 % D;  // row = 2 r + m, the order of the slices
    const float4 q = ld4(Q + (2 * h0 + row) * D + cc);
    *reinterpret_cast<float4*>(sQ + row * D + cc) = make_float4(q.x * c, q.y * c, q.z * c, q.w * c);
  }
  if (threadIdx.x < 2 * RMAX) sM[threadIdx.x] = -INFINITY, sL[threadIdx.x] = 0.f;
  float acc[RMAX][VC];
#pragma unroll
  for (int r = 0; r < RMAX; ++r)
#pragma unroll
    for (int v = 0; v < VC; ++v) acc[r][v] = 0.f;
  const int pm = threadIdx.x >> 6, pc = threadIdx.x & 63;
  for (int64_t k0 = kb; k0 < ke; k0 += BK) {
    __syncthreads();
    // keys past the end are never read: zeros there (a cache row not yet written may hold anything)
    for (int u = threadIdx.x; u < 2 * BK * D / 4; u += kT) {
      const int m = u / (BK * D / 4), w = u % (BK * D / 4), r = w / (D / 4), cc = w % (D / 4) * 4;
      const float4 x = k0 + r < ke ? ld4(K + ((2 * kvh + m) * cap + k0 + r) * D + cc) : make_float4(0, 0, 0, 0);
      *reinterpret_cast<float4*>(sK + (m * BK + r) * PD + cc) = x;
    }
    for (int u = threadIdx.x; u < BK * DV / 4; u += kT) {
      const int r = u / (DV / 4), cc = u % (DV / 4) * 4;
      const float4 x = k0 + r < ke ? ld4(V + (kvh * cap + k0 + r) * DV + cc) : make_float4(0, 0, 0, 0);
      *reinterpret_cast<float4*>(sV + r * PV + cc) = x;
    }
    __syncthreads();
    // warp w: map w & 1, rows w >> 1, + 2, ...; lane = key
    for (int r = warp >> 1; r < R; r += 2) {
      const int row = 2 * r + (warp & 1);
      const float* kr = sK + ((warp & 1) * BK + lane) * PD;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < D; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(kr + k), q = *reinterpret_cast<const float4*>(sQ + row * D + k);
        s = fmaf(x.x, q.x, fmaf(x.y, q.y, fmaf(x.z, q.z, fmaf(x.w, q.w, s))));
      }
      if (k0 + lane >= ke) s = -INFINITY;
      float t = s;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
      const float mo = sM[row], mn = fmaxf(mo, t);
      const float sub = mn == -INFINITY ? 0.f : mn;
      const float p = ptx::ex2(s - sub);
      float z = p;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
      sP[row * BK + lane] = p;
      __syncwarp();
      if (lane == 0) {
        const float a = ptx::ex2(mo - sub);
        sA[row] = a, sM[row] = mn, sL[row] = sL[row] * a + z;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RMAX; ++r) {
      if (r >= R) break;
      const float a = sA[2 * r + pm];
#pragma unroll
      for (int v = 0; v < VC; ++v) acc[r][v] *= a;
    }
#pragma unroll 4
    for (int k = 0; k < BK; ++k) {
      float x[VC];
#pragma unroll
      for (int v = 0; v < VC; ++v) x[v] = sV[k * PV + pc + 64 * v];
#pragma unroll
      for (int r = 0; r < RMAX; ++r) {
        if (r >= R) break;
        const float p = sP[(2 * r + pm) * BK + k];
#pragma unroll
        for (int v = 0; v < VC; ++v) acc[r][v] = fmaf(p, x[v], acc[r][v]);
      }
    }
  }
  __syncthreads();
  if (nsplit > 1) {
#pragma unroll
    for (int r = 0; r < RMAX; ++r)
      if (r < R) {
        float* w = ws + (((h0 + r) * 2 + pm) * nsplit + split) * (DV + 2);
#pragma unroll
        for (int v = 0; v < VC; ++v) w[pc + 64 * v] = acc[r][v];
        if (pc == 0) w[DV] = sM[2 * r + pm], w[DV + 1] = sL[2 * r + pm];
      }
    return;
  }
  // one split: map 2's rows through shared memory (the tiles are done), then the difference
  float* x2 = sK;  // [R][DV]
  static_assert(RMAX * DV <= 2 * BK * PD, "exchange fits");
#pragma unroll
  for (int r = 0; r < RMAX; ++r)
    if (r < R) {
      const float l = sL[2 * r + pm], inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int v = 0; v < VC; ++v) {
        acc[r][v] *= inv;
        if (pm == 1) x2[r * DV + pc + 64 * v] = acc[r][v];
      }
    }
  __syncthreads();
  if (pm == 0) {
#pragma unroll
    for (int r = 0; r < RMAX; ++r)
      if (r < R) {
        const float lm = lam[n * G + r0 + r];
#pragma unroll
        for (int v = 0; v < VC; ++v)
          st1(O + (h0 + r) * DV + pc + 64 * v, acc[r][v] - lm * x2[r * DV + pc + 64 * v]);
      }
  }
}

// One block per (b, h), one thread per column: the splits of both maps joined.
template <int DV, typename T>
__global__ void __launch_bounds__(DV)
    join_kernel(const float* __restrict__ ws, const float* __restrict__ lam, T* __restrict__ O, int H, int nsplit) {
  const int64_t bh = blockIdx.x;
  float o[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float* w = ws + (bh * 2 + m) * nsplit * (DV + 2);
    float mx = -INFINITY;
    for (int s = 0; s < nsplit; ++s) mx = fmaxf(mx, w[s * (DV + 2) + DV]);
    float l = 0.f, a = 0.f;
    if (mx != -INFINITY)
      for (int s = 0; s < nsplit; ++s) {
        const float* x = w + s * (DV + 2);
        const float f = ptx::ex2(x[DV] - mx);
        l = fmaf(f, x[DV + 1], l);
        a = fmaf(f, x[threadIdx.x], a);
      }
    o[m] = l > 0.f ? a / l : 0.f;
  }
  st1(O + bh * DV + threadIdx.x, o[0] - lam[bh % H] * o[1]);
}

template <int D, typename T>
cudaError_t run(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, const int* lens,
                void* O, float* ws, cudaStream_t st) {
  const Plan q = make_plan(p);
  decode_kernel<D, T><<<static_cast<unsigned>(p.BHkv * q.chunks * q.nsplit), kT, 0, st>>>(
      static_cast<const T*>(Q), static_cast<const T*>(K), static_cast<const T*>(V), lam, lens, static_cast<T*>(O), ws,
      p.N, static_cast<int>(p.H), p.group, q.rows, q.nsplit, p.window, p.scale * kLog2e);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || q.nsplit == 1) return e;
  join_kernel<2 * D, T><<<static_cast<unsigned>(p.BH), 2 * D, 0, st>>>(ws, lam, static_cast<T*>(O),
                                                                      static_cast<int>(p.H), q.nsplit);
  return cudaGetLastError();
}

}  // namespace

size_t diff_decode_bytes(const Problem& p) {
  const Plan q = make_plan(p);
  return q.nsplit == 1 ? 0 : static_cast<size_t>(p.BH) * 2 * q.nsplit * (2 * p.d + 2) * sizeof(float);
}

cudaError_t diff_decode(const Problem& p, const void* Q, const void* K, const void* V, const float* lam,
                        const int* lens, void* O, void* ws, cudaStream_t st) {
  float* w = static_cast<float*>(ws);
  if (p.dtype == ATTN_BF16)
    return p.d == 32 ? run<32, __nv_bfloat16>(p, Q, K, V, lam, lens, O, w, st)
                     : run<64, __nv_bfloat16>(p, Q, K, V, lam, lens, O, w, st);
  return p.d == 32 ? run<32, float>(p, Q, K, V, lam, lens, O, w, st)
                   : run<64, float>(p, Q, K, V, lam, lens, O, w, st);
}

}  // namespace fbd
