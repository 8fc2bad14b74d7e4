// Differential attention forward and backward on CUDA cores in fp32 (float32 inputs).
//
//   A_m = softmax(s Q_m K_m^T + mask), O = (A_1 - lam A_2) V,
// one block of 32 query rows per CTA, both maps' running maxima and sums kept per row
// while 32-key tiles stream through shared memory; V's tile serves both maps.  The
// backward recomputes P from the stored log-sum-exps in two passes over the same tiles:
// with dP = dO V^T, D_2 = dO.O_2, D_1 = dO.O + lam D_2 and w = (1, -lam)
//   dS_m = w_m P_m (dP - D_m),  dQ_m = s dS_m K_m,  dK_m = s dS_m^T Q_m,
//   dV = (P_1 - lam P_2)^T dO,  dlam = -sum P_2 dP.
// One kernel does both passes: it holds 32 rows of one side (queries, or keys) and
// streams 32 rows of the other, and forms the score tiles [held x streamed]; every
// output is written once and summed in a fixed order.
//
// Each of the 128 threads owns 4 held rows: 4 x 2 elements of a score tile, and
// 4 x (width / 16) columns of an accumulator, so that a k-step of four does 32 to 64
// multiply-adds on 6 to 8 16-byte shared-memory reads.  The streamed tiles come by
// asynchronous copies into two buffers, the next one while this one is used; two (backward) or
// three CTAs share an SM.  (Blocks of 64 rows without the second buffer: 667 against 372 us
// for the backward of B1 H6 N1000 d64.)
#include "diff.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace fbd {
namespace {

constexpr int BQ = 32;   // held rows
constexpr int BK = 32;   // streamed rows
constexpr int kT = 128;  // threads: 8 (ty: 4 held rows each) x 16 (tx)
constexpr int PP = BK + 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Pitch {  // floats per shared row: 16-byte aligned, consecutive rows 4 banks apart
  static constexpr int v = D + 4;
};

__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
// Rows [r0, r0 + R) of a [N, D] slice into shared memory as floats; rows past N are zero.
template <int D, int R>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int64_t r0, int64_t N) {
  constexpr int C = D / 4;
  for (int u = threadIdx.x; u < R * C; u += kT) {
    const int r = u / C, c = (u % C) * 4;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (r0 + r < N) load4(src + (r0 + r) * D + c, x);
    *reinterpret_cast<float4*>(dst + r * Pitch<D>::v + c) = make_float4(x[0], x[1], x[2], x[3]);
  }
}
// The same by asynchronous copies (zeros past N: nothing is read there).
template <int D, int R>
__device__ __forceinline__ void copy_tile(float* dst, const float* src, int64_t r0, int64_t N) {
  constexpr int C = D / 4;
  const uint32_t d = ptx::smem_u32(dst);
#pragma unroll
  for (int v = 0; v < R * C / kT; ++v) {
    const int u = v * kT + threadIdx.x, r = u / C, c = (u % C) * 4;
    const bool in = r0 + r < N;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + (r * Pitch<D>::v + c) * 4),
                 "l"(src + (in ? r0 + r : 0) * D + c), "r"(in ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}
// s[r][c] = sum_k A[4 ty + r][k] B[tx + 16 c][k]
template <int D>
__device__ __forceinline__ void scores(const float* A, const float* B, int ty, int tx, float (&s)[4][2]) {
  constexpr int P = Pitch<D>::v;
#pragma unroll
  for (int r = 0; r < 4; ++r) s[r][0] = s[r][1] = 0.f;
#pragma unroll 4
  for (int k = 0; k < D; k += 4) {
    float4 b[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) b[c] = *reinterpret_cast<const float4*>(B + (tx + 16 * c) * P + k);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float4 a = *reinterpret_cast<const float4*>(A + (4 * ty + r) * P + k);
#pragma unroll
      for (int c = 0; c < 2; ++c) s[r][c] = dot4(a, b[c], s[r][c]);
    }
  }
}
// acc[r][:] += sum_k T[4 ty + r][k] B[k][tx W ..], W = D / 16 columns per thread
template <int D>
__device__ __forceinline__ void accumulate(const float* T, const float* B, int ty, int tx, float (&acc)[4][D / 16]) {
  constexpr int W = D / 16, P = Pitch<D>::v;
#pragma unroll 2
  for (int k = 0; k < BK; k += 4) {
    float t[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) load4(T + (4 * ty + r) * PP + k, t[r]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* b = B + (k + u) * P + tx * W;
      float v[W];
      if constexpr (W == 2) {
        const float2 x = *reinterpret_cast<const float2*>(b);
        v[0] = x.x, v[1] = x.y;
      } else {
#pragma unroll
        for (int c = 0; c < W; c += 4) load4(b + c, reinterpret_cast<float(&)[4]>(v[c]));
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < W; ++c) acc[r][c] = fmaf(t[r][u], v[c], acc[r][c]);
    }
  }
}
template <int W>
__device__ __forceinline__ void store_row(float* dst, const float (&x)[W], float f) {
  if constexpr (W == 2) {
    *reinterpret_cast<float2*>(dst) = make_float2(x[0] * f, x[1] * f);
  } else {
#pragma unroll
    for (int c = 0; c < W; c += 4)
      *reinterpret_cast<float4*>(dst + c) = make_float4(x[c] * f, x[c + 1] * f, x[c + 2] * f, x[c + 3] * f);
  }
}

template <int D>
constexpr size_t fwd_smem() {
  return sizeof(float) * (2 * BQ * Pitch<D>::v + 2 * (2 * BK * Pitch<D>::v + BK * Pitch<2 * D>::v) + 2 * BQ * PP);
}

template <int D>
__global__ void __launch_bounds__(kT, 2)
    fwd_kernel(const float* __restrict__ Q, const float* __restrict__ K, const float* __restrict__ V,
               const float* __restrict__ lam, float* __restrict__ O, float* __restrict__ O2, float* __restrict__ lse,
               int64_t N, int64_t H, int nqb, int BH, int G, float scale, int causal, Band bd) {
  constexpr int DV = 2 * D, WV = DV / 16;
  extern __shared__ __align__(16) float sh[];
  float* sQ = sh;                                // [2][BQ]
  constexpr int kTile = 2 * BK * Pitch<D>::v + BK * Pitch<DV>::v;  // K_1, K_2, V
  float* sB = sQ + 2 * BQ * Pitch<D>::v;         // two tiles
  float* sP = sB + 2 * kTile;                    // [2][BQ]
  const tc::Order ord = tc::grid_order(BH, nqb);
  const int64_t bh = ord.bh, kvh = bh / G;
  const int64_t q0 = static_cast<int64_t>(nqb - 1 - ord.k) * BQ;  // heaviest blocks first
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float c = scale * kLog2e;
#pragma unroll
  for (int m = 0; m < 2; ++m)
    load_tile<D, BQ>(sQ + m * BQ * Pitch<D>::v, Q + (2 * bh + m) * N * D, q0, N);
  int64_t lo[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) lo[r] = causal ? bd.row_lo(bh, q0 + 4 * ty + r) : 0;
  const int64_t kend = causal ? (q0 + BQ < N ? q0 + BQ : N) : N;
  const int64_t kbeg = causal ? bd.row_lo(bh, q0) / BK * BK : 0;
  float mx[2][4], l[2][4], acc[2][4][WV];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      mx[m][r] = -INFINITY, l[m][r] = 0.f;
#pragma unroll
      for (int u = 0; u < WV; ++u) acc[m][r][u] = 0.f;
    }
  auto load = [&](int64_t k0, float* dst) {
#pragma unroll
    for (int m = 0; m < 2; ++m) copy_tile<D, BK>(dst + m * BK * Pitch<D>::v, K + (2 * kvh + m) * N * D, k0, N);
    copy_tile<DV, BK>(dst + 2 * BK * Pitch<D>::v, V + kvh * N * DV, k0, N);
    copies_commit();
  };
  load(kbeg, sB);
  int buf = 0;
  for (int64_t k0 = kbeg; k0 < kend; k0 += BK, buf ^= 1) {
    copies_wait();
    __syncthreads();  // this tile is there, the other buffer's has been read
    if (k0 + BK < kend) load(k0 + BK, sB + (buf ^ 1) * kTile);
    const float *sK = sB + buf * kTile, *sV = sK + 2 * BK * Pitch<D>::v;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float s[4][2];
      scores<D>(sQ + m * BQ * Pitch<D>::v, sK + m * BK * Pitch<D>::v, ty, tx, s);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t i = q0 + 4 * ty + r;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t j = k0 + tx + 16 * u;
          if (j >= N || (causal && (j > i || j < lo[r]))) s[r][u] = -INFINITY;
        }
        float t = fmaxf(s[r][0], s[r][1]);
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
        const float mn = fmaxf(mx[m][r], t);
        const float sub = mn == -INFINITY ? 0.f : mn;  // no visible key yet: every term is 2^-inf = 0
        const float alpha = ptx::ex2((mx[m][r] - sub) * c);
        const float p0 = ptx::ex2((s[r][0] - sub) * c), p1 = ptx::ex2((s[r][1] - sub) * c);
        mx[m][r] = mn;
        l[m][r] = l[m][r] * alpha + (p0 + p1);  // this thread's share; summed over tx at the end
#pragma unroll
        for (int u = 0; u < WV; ++u) acc[m][r][u] *= alpha;
        float* pr = sP + m * BQ * PP + (4 * ty + r) * PP + tx;
        pr[0] = p0, pr[16] = p1;
      }
    }
    __syncwarp();  // a row of P is written and read by the 16 threads of one ty, in one warp
#pragma unroll
    for (int m = 0; m < 2; ++m) accumulate<DV>(sP + m * BQ * PP, sV, ty, tx, acc[m]);
  }
  const float lm = lam[bh % H];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t i = q0 + 4 * ty + r;
    float inv[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float t = l[m][r];
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
      inv[m] = 1.f / t;
      if (i < N && tx == 0) lse[(2 * bh + m) * N + i] = mx[m][r] * scale + logf(t);
    }
    if (i < N) {
      float o[WV];
#pragma unroll
      for (int u = 0; u < WV; ++u) {
        acc[1][r][u] *= inv[1];
        o[u] = acc[0][r][u] * inv[0] - lm * acc[1][r][u];
      }
      store_row<WV>(O + (bh * N + i) * DV + tx * WV, o, 1.f);
      if (O2 != nullptr) store_row<WV>(O2 + (bh * N + i) * DV + tx * WV, acc[1][r], 1.f);
    }
  }
}

// Row statistics of the backward: (L_1, L_2, D_1, D_2), D_2 = dO.O_2, D_1 = dO.O + lam D_2;
// D = +inf marks a row with one visible key (its dS is 0).  16 threads per row.
template <int DV>
__global__ void __launch_bounds__(256)
    prep_kernel(const float* __restrict__ O, const float* __restrict__ O2, const float* __restrict__ dO,
                const float* __restrict__ lse, const float* __restrict__ lam, float4* __restrict__ stats, int64_t N,
                int64_t H, int64_t BH, int causal, Band bd) {
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = gid >> 4;
  const int part = static_cast<int>(gid & 15);
  const bool live = row < BH * N;
  float d = 0.f, d2 = 0.f;
  if (live) {
#pragma unroll
    for (int c = part * 4; c < DV; c += 64) {
      float g[4], o[4], o2[4];
      load4(dO + row * DV + c, g);
      load4(O + row * DV + c, o);
      load4(O2 + row * DV + c, o2);
#pragma unroll
      for (int u = 0; u < 4; ++u) d = fmaf(g[u], o[u], d), d2 = fmaf(g[u], o2[u], d2);
    }
  }
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) {
    d += __shfl_xor_sync(0xffffffffu, d, x);
    d2 += __shfl_xor_sync(0xffffffffu, d2, x);
  }
  if (live && part == 0) {
    const int64_t bh = row / N, i = row - bh * N;
    const bool one = diff_one_key(bd, causal, bh, i);
    stats[row] = make_float4(lse[2 * bh * N + i], lse[(2 * bh + 1) * N + i],
                             diff_mark_D(fmaf(lam[bh % H], d2, d), one), diff_mark_D(d2, one));
  }
}

template <int D>
constexpr size_t bwd_smem() {
  return sizeof(float) * ((2 * BQ + 4 * BK) * Pitch<D>::v + (BQ + 2 * BK) * Pitch<2 * D>::v + 2 * BQ * PP + 8 * BK + 8);
}

// COL = false: holds queries (Q_m, dO), streams keys (K_m, V), writes dQ_m and the block's
// share of dlam.  COL = true: holds keys, streams the queries of the G query heads that
// share them, writes dK_m, dV.
template <int D, bool COL>
__device__ __forceinline__ void bwd_pass(const float* __restrict__ Q, const float* __restrict__ K,
                                         const float* __restrict__ V, const float* __restrict__ dO,
                                         const float* __restrict__ lam, const float4* stats, float* __restrict__ out1,
                                         float* __restrict__ outV, float* __restrict__ partial, int64_t N, int64_t H,
                                         int nblk, int slices, int G, float scale, int causal, const Band& bd,
                                         int block) {
  constexpr int DV = 2 * D, W = D / 16, WV = DV / 16, PD = Pitch<D>::v;
  extern __shared__ __align__(16) float sh[];
  float* sA = sh;                      // [2][BQ] held Q_m or K_m
  float* sAV = sA + 2 * BQ * PD;       // [BQ]    held dO or V
  constexpr int kTile = 2 * BK * PD + BK * Pitch<DV>::v;  // K_m or Q_m, and V or dO
  float* sS = sAV + BQ * Pitch<DV>::v; // two streamed tiles
  float* sT = sS + 2 * kTile;          // [2][BQ] dS_m; then in the first P_1 - lam P_2 (COL)
  float4* sSt0 = reinterpret_cast<float4*>(sT + 2 * BQ * PP);  // [2][BK] streamed rows' statistics (COL)
  float* sRed = reinterpret_cast<float*>(sSt0 + 2 * BK);       // [4]
  const tc::Order ord = tc::grid_order_at(block, slices, nblk);
  const int64_t sl = ord.bh;                                      // query slice, or key/value slice
  const int64_t blk = COL || !causal ? ord.k : nblk - 1 - ord.k;  // heaviest first
  const int64_t a0 = blk * BQ;
  const int64_t kvh = COL ? sl : sl / G;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float c = scale * kLog2e;
  const float* heldM = COL ? K : Q;
  const float* heldV = COL ? V : dO;
#pragma unroll
  for (int m = 0; m < 2; ++m) load_tile<D, BQ>(sA + m * BQ * PD, heldM + (2 * sl + m) * N * D, a0, N);
  load_tile<DV, BQ>(sAV, heldV + sl * N * DV, a0, N);
  // the range of streamed rows, and per held row its bound among them
  int64_t b0 = 0, b1 = N, lim[4];
  float4 hst[4];
  if (causal) {
    if (COL) {
      b0 = a0 / BK * BK;
      b1 = static_cast<int64_t>(bd.key_hi(kvh, a0 + BQ - 1)) + 1;
    } else {
      b0 = bd.row_lo(kvh, a0) / BK * BK;
      b1 = a0 + BQ < N ? a0 + BQ : N;
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t a = a0 + 4 * ty + r;
    lim[r] = !causal ? 0 : (COL ? bd.key_hi(kvh, a) : bd.row_lo(kvh, a));
    hst[r] = (!COL && a < N) ? stats[sl * N + a] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float acc[2][4][W], accV[COL ? 4 : 1][WV];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int u = 0; u < W; ++u) acc[0][r][u] = acc[1][r][u] = 0.f;
    if constexpr (COL) {
#pragma unroll
      for (int u = 0; u < WV; ++u) accV[r][u] = 0.f;
    }
  }
  float dl = 0.f;
  auto load = [&](int g, int64_t k0, int buf) {
    const int64_t qs = COL ? kvh * G + g : sl;
    const float* strM = COL ? Q + 2 * qs * N * D : K + 2 * kvh * N * D;
    const float* strV = COL ? dO + qs * N * DV : V + kvh * N * DV;
    float* dst = sS + buf * kTile;
#pragma unroll
    for (int m = 0; m < 2; ++m) copy_tile<D, BK>(dst + m * BK * PD, strM + m * N * D, k0, N);
    copy_tile<DV, BK>(dst + 2 * BK * PD, strV, k0, N);
    if (COL && threadIdx.x < BK) {
      const bool in = k0 + threadIdx.x < N;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(sSt0 + buf * BK + threadIdx.x)),
                   "l"(stats + qs * N + (in ? k0 + threadIdx.x : 0)), "r"(in ? 16 : 0)
                   : "memory");
    }
    copies_commit();
  };
  load(0, b0, 0);
  int buf = 0;
  for (int g = 0; g < (COL ? G : 1); ++g) {
    const int64_t qs = COL ? kvh * G + g : sl;  // query slice
    const float lm = lam[qs % H];
    for (int64_t k0 = b0; k0 < b1; k0 += BK, buf ^= 1) {
      copies_wait();
      __syncthreads();  // this tile is there, the other buffer's has been read
      if (k0 + BK < b1)
        load(g, k0 + BK, buf ^ 1);
      else if (COL && g + 1 < G)
        load(g + 1, b0, buf ^ 1);
      const float *sB = sS + buf * kTile, *sBV = sB + 2 * BK * PD;
      const float4* sSt = sSt0 + buf * BK;
      float dp[4][2], w[4][2], sum = 0.f;  // sum: of P_2 dP in this tile (short chains of additions)
      scores<DV>(sAV, sBV, ty, tx, dp);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float s[4][2];
        scores<D>(sA + m * BQ * PD, sB + m * BK * PD, ty, tx, s);
        const float wm = m == 0 ? 1.f : -lm;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t b = k0 + tx + 16 * u;
          const float4 bst = COL ? sSt[tx + 16 * u] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t a = a0 + 4 * ty + r;
            const float4 st = COL ? bst : hst[r];
            const float L = m == 0 ? st.x : st.y, Dm = m == 0 ? st.z : st.w;
            bool see = a < N && b < N;
            if (causal) see = see && (COL ? (a <= b && b <= lim[r]) : (b <= a && b >= lim[r]));
            const float p = see ? ptx::ex2(fmaf(s[r][u], c, -L * kLog2e)) : 0.f;
            const float ds = (see && Dm != INFINITY) ? wm * p * (dp[r][u] - Dm) : 0.f;
            if (m == 1 && !COL) sum = fmaf(p, see ? dp[r][u] : 0.f, sum);
            sT[m * BQ * PP + (4 * ty + r) * PP + tx + 16 * u] = ds;
            if (COL) {
              w[r][u] = m == 0 ? p : fmaf(wm, p, w[r][u]);
            }
          }
        }
      }
      dl += sum;
      __syncwarp();
#pragma unroll
      for (int m = 0; m < 2; ++m) accumulate<D>(sT + m * BQ * PP, sB + m * BK * PD, ty, tx, acc[m]);
      if constexpr (COL) {
        __syncwarp();  // a row of sT is written and read by the 16 threads of one ty, in one warp
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int u = 0; u < 2; ++u) sT[(4 * ty + r) * PP + tx + 16 * u] = w[r][u];
        __syncwarp();
        accumulate<DV>(sT, sBV, ty, tx, accV);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t a = a0 + 4 * ty + r;
    if (a >= N) continue;
#pragma unroll
    for (int m = 0; m < 2; ++m) store_row<W>(out1 + ((2 * sl + m) * N + a) * D + tx * W, acc[m][r], scale);
    if constexpr (COL) store_row<WV>(outV + (sl * N + a) * DV + tx * WV, accV[r], 1.f);
  }
  if constexpr (!COL) {  // the block's sum of P_2 dP: lanes, then warps in order
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) dl += __shfl_xor_sync(0xffffffffu, dl, x);
    if ((threadIdx.x & 31) == 0) sRed[threadIdx.x >> 5] = dl;
    __syncthreads();
    if (threadIdx.x == 0) {
      float t = 0.f;
      for (int u = 0; u < kT / 32; ++u) t += sRed[u];
      partial[sl * nblk + blk] = t;
    }
  }
}

// Both passes in one launch: they read nothing of one another's, and a short sequence's blocks of
// one pass do not fill the SMs.  The column pass's blocks, the longer ones, come first.
template <int D>
__global__ void __launch_bounds__(kT, 2)
    bwd_kernel(const float* __restrict__ Q, const float* __restrict__ K, const float* __restrict__ V,
               const float* __restrict__ dO, const float* __restrict__ lam, const float4* stats,
               float* __restrict__ dQ, float* __restrict__ dK, float* __restrict__ dV, float* __restrict__ partial,
               int64_t N, int64_t H, int nblk, int BHkv, int G, float scale, int causal, Band bd) {
  const int ncol = nblk * BHkv, x = static_cast<int>(blockIdx.x);
  if (x < ncol)
    bwd_pass<D, true>(Q, K, V, dO, lam, stats, dK, dV, nullptr, N, H, nblk, BHkv, G, scale, causal, bd, x);
  else
    bwd_pass<D, false>(Q, K, V, dO, lam, stats, dQ, nullptr, partial, N, H, nblk, BHkv * G, G, scale, causal, bd,
                       x - ncol);
}

__global__ void __launch_bounds__(256)
    dlam_kernel(const float* partial, float* __restrict__ dlam, int64_t B, int64_t H, int64_t nblk) {
  ptx::grid_dependency_wait();  // the blocks' sums
  const int64_t h = blockIdx.x;
  float t = 0.f;
  for (int64_t b = 0; b < B; ++b)
    for (int64_t k = threadIdx.x; k < nblk; k += 256) t += partial[(b * H + h) * nblk + k];
  __shared__ float red[256];
  red[threadIdx.x] = t;
  __syncthreads();
  for (int s = 128; s > 0; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
    __syncthreads();
  }
  if (threadIdx.x == 0) dlam[h] = -red[0];
}

template <typename F>
cudaError_t set_smem(F kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <int D>
cudaError_t fwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, void* O, void* O2,
                float* lse, cudaStream_t st) {
  const int nqb = static_cast<int>((p.N + BQ - 1) / BQ);
  cudaError_t e = set_smem(fwd_kernel<D>, fwd_smem<D>());
  if (e != cudaSuccess) return e;
  fwd_kernel<D><<<static_cast<unsigned>(nqb * p.BH), kT, fwd_smem<D>(), st>>>(
      static_cast<const float*>(Q), static_cast<const float*>(K), static_cast<const float*>(V), lam, static_cast<float*>(O),
      static_cast<float*>(O2), lse, p.N, p.H, nqb, static_cast<int>(p.BH), p.group, p.scale, p.causal,
      make_band(p, eff_window(p), false));
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd(const Problem& p, const void* Q_, const void* K_, const void* V_, const float* lam, const void* O,
                const void* O2, const void* dO_, const float* lse, void* dQ, void* dK, void* dV, float* dlam,
                float4* stats, cudaStream_t st) {
  const float *Q = static_cast<const float*>(Q_), *K = static_cast<const float*>(K_), *V = static_cast<const float*>(V_);
  const float* dO = static_cast<const float*>(dO_);
  const int nblk = static_cast<int>((p.N + BQ - 1) / BQ);
  float* partial = reinterpret_cast<float*>(stats + p.BH * p.N);
  const int64_t threads = p.BH * p.N * 16;
  prep_kernel<2 * D><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, st>>>(
      static_cast<const float*>(O), static_cast<const float*>(O2), dO, lse, lam, stats, p.N, p.H, p.BH, p.causal,
      make_band(p, eff_window(p), false));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if ((e = set_smem(bwd_kernel<D>, bwd_smem<D>())) != cudaSuccess) return e;
  bwd_kernel<D><<<static_cast<unsigned>(nblk * (p.BH + p.BHkv)), kT, bwd_smem<D>(), st>>>(
      Q, K, V, dO, lam, stats, static_cast<float*>(dQ), static_cast<float*>(dK), static_cast<float*>(dV), partial, p.N,
      p.H, nblk, static_cast<int>(p.BHkv), p.group, p.scale, p.causal, make_band(p, eff_window(p), true));
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return diff_reduce_dlam(partial, dlam, p.B, p.H, nblk, st);
}

}  // namespace

cudaError_t diff_reduce_dlam(const float* partial, float* dlam, int64_t B, int64_t H, int64_t nblk, cudaStream_t st) {
  return launch_behind(dlam_kernel, H, 256, 0, st, partial, dlam, B, H, nblk);
}

size_t simt_diff_bwd_bytes(int64_t BH, int64_t N) {
  return static_cast<size_t>(BH) * N * sizeof(float4) + static_cast<size_t>(BH) * ((N + BQ - 1) / BQ) * sizeof(float);
}

cudaError_t simt_diff_fwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, void* O,
                          void* O2, float* lse, cudaStream_t st) {
  return p.d == 32 ? fwd<32>(p, Q, K, V, lam, O, O2, lse, st)
                   : fwd<64>(p, Q, K, V, lam, O, O2, lse, st);
}

cudaError_t simt_diff_bwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam,
                          const void* O, const void* O2, const void* dO, const float* lse, void* dQ, void* dK,
                          void* dV, float* dlam, void* ws, cudaStream_t st) {
  float4* s = static_cast<float4*>(ws);
  return p.d == 32 ? bwd<32>(p, Q, K, V, lam, O, O2, dO, lse, dQ, dK, dV, dlam, s, st)
                   : bwd<64>(p, Q, K, V, lam, O, O2, dO, lse, dQ, dK, dV, dlam, s, st);
}

}  // namespace fbd
