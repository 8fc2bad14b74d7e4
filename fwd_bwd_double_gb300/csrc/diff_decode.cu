// Differential attention of one new token over a key/value cache.
//
//   o_m = sum_j softmax_j(s q_m.k_mj) v_j over the keys lo <= j < len of the sequence,
//   O = o_1 - lam o_2;  a sequence with no key gives 0.
// Bound by reading the cache once: up to eight query heads that share a key/value head are
// handled together, both maps against the same V rows.  The keys of a sequence are split
// over `nsplit` CTAs, each leaving (max, sum, unnormalised o) per row and map, which a
// second launch joins; with one split the result is written at once.
//
// bf16 on warp-level matrix products (m16n8k16): rows 0-7 of a tile are the heads' first maps,
// rows 8-15 their second ones, so one product P V serves both maps, and S is Q_1 K_1^T with
// rows 8-15 zero and Q_2 K_2^T with rows 0-7 zero, of which the other rows are kept (zeros times an
// infinite key of the other map are NaN).  (tcgen05 has 128 rows to fill.)  Each of
// four warps takes 16 of a tile's 64 keys with a softmax of its own; the four are joined at
// the end.  Three 32 KB stages of 16-byte asynchronous copies, two CTAs an SM: 192 KB in
// flight on each SM.  P is rounded to bf16 for its product; sums, maxima and o are fp32.
// float32 on the CUDA cores, a key per lane, two stages.
#include <cuda_bf16.h>

#include "diff.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace fbd {
namespace {

constexpr int BK = 32;    // float32: keys per tile, one per lane
constexpr int MK = 64;    // bf16: keys per tile, 16 per warp
constexpr int NS = 3;     // bf16: stages
constexpr int RMAX = 8;   // query heads handled together
constexpr int kMaxSplits = 256;
constexpr int kT = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct Plan {
  int rows, chunks, nsplit;  // query heads per CTA; CTAs per key/value head for the group; splits of the keys
};
Plan make_plan(const Problem& p) {
  Plan q;
  q.rows = p.group < RMAX ? p.group : RMAX;
  q.chunks = (p.group + q.rows - 1) / q.rows;
  // Two waves of the CTAs that fit 152 SMs (bf16 two an SM, float32 three), a split no shorter than
  // 128 keys.  Measured at 3, 4, 6 and 8 CTAs an SM: 54.8, 52.6, 50.7, 52.6 us for 32 ragged contexts
  // of up to 8192 keys, 124, 120, 124, 128 us for one of 131072, 29.6, 30.1, 35.0, 39.1 us for one
  // key/value head and 8 query heads over 40000 (the join grows with the splits); float32, 64 heads
  // over 8192: 179, 152, 143, 127 us (that shape alone, so the rule stays at two waves for both types).
  const int64_t fit = p.dtype == ATTN_BF16 ? 2 : 3;
  const int64_t base = p.BHkv * q.chunks;
  const int64_t want = base > 0 ? (2 * fit * 152 + base - 1) / base : 1;
  const int64_t most = (p.N + 127) / 128;
  const int64_t n = want < most ? want : most;
  q.nsplit = static_cast<int>(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
  return q;
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

__device__ __forceinline__ void key_range(const int* lens, int b, int64_t cap, int64_t win, int64_t& lo, int64_t& n) {
  int64_t len = lens[b];
  len = len < 0 ? 0 : (len > cap ? cap : len);
  lo = win > 0 && len > win ? len - win : 0;
  n = len - lo;
}

// ------------------------------------------------------------------------- bf16
// 16 bytes global -> shared, or 16 bytes of zeros (nothing is read) where !in.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Byte offset of a 16-byte chunk in a tile of RB-byte rows, swizzled so that the same chunk of
// eight consecutive rows lies in eight different 16-byte columns.
template <int RB>
__device__ __forceinline__ uint32_t at(int row, int chunk) {
  return static_cast<uint32_t>(row * RB + ((chunk ^ (RB >= 128 ? row & 7 : (row >> 1) & 3)) << 4));
}

template <int D>
struct Stage {
  static constexpr int kK = MK * D * 2, kV = MK * D * 4, bytes = 2 * kK + kV;
};

// ws: o of every (b, h, map, split), 2d floats each, then their (max (scaled, in powers of two),
// sum) at `tail`.
template <int D>
__global__ void __launch_bounds__(kT, 2)
    mma_kernel(const __nv_bfloat16* __restrict__ Q, const __nv_bfloat16* __restrict__ K,
               const __nv_bfloat16* __restrict__ V, const float* __restrict__ lam, const int* __restrict__ lens,
               __nv_bfloat16* __restrict__ O, float* __restrict__ ws, float2* __restrict__ tail, int64_t cap, int H, int G, int rows, int nsplit,
               int64_t win, float c) {
  using St = Stage<D>;
  constexpr int DV = 2 * D, NT = DV / 8;  // 8-column tiles of o
  extern __shared__ __align__(128) uint8_t sh[];
  const uint32_t s0 = ptx::smem_u32(sh);
  ptx::grid_dependency_launch();
  const int split = blockIdx.x % nsplit, Hkv = H / G, chunks = (G + rows - 1) / rows;
  const int unit = blockIdx.x / nsplit;  // (b, key/value head, chunk of its query heads)
  const int r0 = unit % chunks * rows, n = unit / chunks % Hkv, b = unit / chunks / Hkv;
  const int R = min(rows, G - r0);
  const int64_t kvh = static_cast<int64_t>(b) * Hkv + n;
  const int64_t h0 = static_cast<int64_t>(b) * H + n * G + r0;  // first query head
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  int64_t lo, cnt;
  key_range(lens, b, cap, win, lo, cnt);
  const int64_t per = ((cnt + nsplit - 1) / nsplit + MK - 1) / MK * MK;
  const int64_t kb = lo + split * per, ke = min(lo + cnt, kb + per);
  const int nt = ke > kb ? static_cast<int>((ke - kb + MK - 1) / MK) : 0;
  const __nv_bfloat16* K0 = K + 2 * kvh * cap * D;  // map 1; map 2 is cap * D further on
  const __nv_bfloat16* V0 = V + kvh * cap * DV;
  auto load = [&](int t) {
    const uint32_t st = s0 + static_cast<uint32_t>((t % NS) * St::bytes);
    const int64_t k0 = kb + static_cast<int64_t>(t) * MK;
    // keys past the end are not read: zeros there (a cache row not yet written may hold anything)
#pragma unroll
    for (int u = 0; u < 2 * MK * D / 8 / kT; ++u) {
      const int x = u * kT + threadIdx.x, m = x / (MK * D / 8), y = x % (MK * D / 8), r = y / (D / 8), ch = y % (D / 8);
      const bool in = k0 + r < ke;
      copy16(st + m * St::kK + at<D * 2>(r, ch), K0 + (m * cap + (in ? k0 + r : kb)) * D + ch * 8, in);
    }
#pragma unroll
    for (int u = 0; u < MK * DV / 8 / kT; ++u) {
      const int x = u * kT + threadIdx.x, r = x / (DV / 8), ch = x % (DV / 8);
      const bool in = k0 + r < ke;
      copy16(st + 2 * St::kK + at<DV * 2>(r, ch), V0 + (in ? k0 + r : kb) * DV + ch * 8, in);
    }
  };
#pragma unroll
  for (int t = 0; t < NS - 1; ++t) {
    if (t < nt) load(t);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // The heads' queries as the A operand: row g their first maps, row g + 8 their second.
  uint32_t qa[2][D / 16][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        qa[m][k][x] =
            g < R ? *reinterpret_cast<const uint32_t*>(Q + (2 * (h0 + g) + m) * D + k * 16 + x * 8 + q4 * 2) : 0u;
  float mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of map 1, map 2 (l: this thread's keys)
  float o[NT][4];
#pragma unroll
  for (int u = 0; u < NT; ++u) o[u][0] = o[u][1] = o[u][2] = o[u][3] = 0.f;
  for (int t = 0; t < nt; ++t) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
    __syncthreads();
    if (t + NS - 1 < nt) load(t + NS - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const uint32_t st = s0 + static_cast<uint32_t>((t % NS) * St::bytes);
    float s[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float sm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t f[4];
          ldm4(st + m * St::kK + at<D * 2>(warp * 16 + u * 8 + (lane & 7), k * 4 + (lane >> 3)), f);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            mma(sm, m == 0 ? qa[0][2 * k + x][0] : 0u, m == 1 ? qa[1][2 * k + x][0] : 0u,
                m == 0 ? qa[0][2 * k + x][1] : 0u, m == 1 ? qa[1][2 * k + x][1] : 0u, f[2 * x], f[2 * x + 1]);
        }
        s[u][2 * m] = sm[2 * m], s[u][2 * m + 1] = sm[2 * m + 1];
      }
    if (t == nt - 1) {
      const int64_t k0 = kb + static_cast<int64_t>(t) * MK + warp * 16 + q4 * 2;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (k0 + u * 8 + (x & 1) >= ke) s[u][x] = -INFINITY;
    }
    float a[2], nm[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float v = fmaxf(fmaxf(s[0][2 * m], s[0][2 * m + 1]), fmaxf(s[1][2 * m], s[1][2 * m + 1])) * c;
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
      v = fmaxf(mx[m], v);
      const float sub = v == -INFINITY ? 0.f : v;  // no key of this warp's yet
      a[m] = ptx::ex2(mx[m] - sub);
      nm[m] = -sub;
      l[m] *= a[m];
      mx[m] = v;
    }
    if (__any_sync(0xffffffffu, a[0] != 1.f || a[1] != 1.f)) {
#pragma unroll
      for (int u = 0; u < NT; ++u) o[u][0] *= a[0], o[u][1] *= a[0], o[u][2] *= a[1], o[u][3] *= a[1];
    }
    uint32_t p[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float x = ptx::ex2(fmaf(s[u][2 * m], c, nm[m])), y = ptx::ex2(fmaf(s[u][2 * m + 1], c, nm[m]));
        l[m] += x + y;
        p[u][m] = ptx::pack_bf16(x, y);
      }
#pragma unroll
    for (int u = 0; u < NT; u += 2) {
      uint32_t f[4];
      ldm4t(st + 2 * St::kK + at<DV * 2>(warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), u + (lane >> 4)), f);
      mma(o[u], p[0][0], p[0][1], p[1][0], p[1][1], f[0], f[1]);
      mma(o[u + 1], p[0][0], p[0][1], p[1][0], p[1][1], f[2], f[3]);
    }
  }
  // The warps' parts joined through shared memory: row 8 m + head of each, o and (max, sum).
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float* so = reinterpret_cast<float*>(sh);            // [4][16][DV]
  float* sm = so + 4 * 16 * DV;                        // [4][16] max, [4][16] sum
  static_assert((4 * 16 * DV + 128) * 4 <= NS * St::bytes, "the join fits");
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float v = l[m];
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    if (q4 == 0) sm[warp * 16 + 8 * m + g] = mx[m], sm[64 + warp * 16 + 8 * m + g] = v;
#pragma unroll
    for (int u = 0; u < NT; ++u)
      *reinterpret_cast<float2*>(so + (warp * 16 + 8 * m + g) * DV + u * 8 + q4 * 2) =
          make_float2(o[u][2 * m], o[u][2 * m + 1]);
  }
  __syncthreads();
  constexpr int C = DV / 4;  // threads per row, four columns each
  for (int r = threadIdx.x / C; r < R; r += kT / C) {
    const int col = threadIdx.x % C * 4;
    float res[4], ll = 0.f, mm = -INFINITY;
    float4 first;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int row = 8 * m + r;
      mm = fmaxf(fmaxf(sm[row], sm[16 + row]), fmaxf(sm[32 + row], sm[48 + row]));
      const float sub = mm == -INFINITY ? 0.f : mm;
      ll = 0.f;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ptx::ex2(sm[w * 16 + row] - sub);
        const float4 v = *reinterpret_cast<const float4*>(so + (w * 16 + row) * DV + col);
        ll = fmaf(f, sm[64 + w * 16 + row], ll);
        x[0] = fmaf(f, v.x, x[0]), x[1] = fmaf(f, v.y, x[1]), x[2] = fmaf(f, v.z, x[2]), x[3] = fmaf(f, v.w, x[3]);
      }
      if (nsplit > 1) {
        const int64_t w = ((h0 + r) * 2 + m) * nsplit + split;
        *reinterpret_cast<float4*>(ws + w * DV + col) = make_float4(x[0], x[1], x[2], x[3]);
        if (col == 0) tail[w] = make_float2(mm, ll);
      } else {
        const float inv = ll > 0.f ? 1.f / ll : 0.f;
        if (m == 0) {
          first = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        } else {
          const float f = lam[n * G + r0 + r] * inv;
          res[0] = first.x - f * x[0], res[1] = first.y - f * x[1];
          res[2] = first.z - f * x[2], res[3] = first.w - f * x[3];
          *reinterpret_cast<uint2*>(O + (h0 + r) * DV + col) =
              make_uint2(ptx::pack_bf16(res[0], res[1]), ptx::pack_bf16(res[2], res[3]));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------- float32
template <int D>
__global__ void __launch_bounds__(kT)
    decode_kernel(const float* __restrict__ Q, const float* __restrict__ K, const float* __restrict__ V,
                  const float* __restrict__ lam, const int* __restrict__ lens, float* __restrict__ O,
                  float* __restrict__ ws, float2* __restrict__ tail, int64_t cap, int H, int G, int rows, int nsplit, int64_t win, float c) {
  constexpr int DV = 2 * D, PD = D + 4, PV = DV;
  constexpr int VC = DV / 64;  // a thread's columns: (t & 63) + 64 v of map t >> 6
  constexpr int kTile = 2 * BK * PD + BK * PV;  // K_1, K_2, V
  extern __shared__ __align__(128) uint8_t sh[];
  float* sB = reinterpret_cast<float*>(sh);  // two tiles
  float *sQ = sB + 2 * kTile, *sP = sQ + 2 * RMAX * D, *sA = sP + 2 * RMAX * BK, *sM = sA + 2 * RMAX, *sL = sM + 2 * RMAX;
  ptx::grid_dependency_launch();
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
  auto load = [&](int64_t k0, int buf) {
    // keys past the end are not read: zeros there (a cache row not yet written may hold anything)
    const uint32_t dst = ptx::smem_u32(sB + buf * kTile);
#pragma unroll
    for (int v = 0; v < 2 * BK * D / 4 / kT; ++v) {
      const int u = v * kT + threadIdx.x;
      const int m = u / (BK * D / 4), w = u % (BK * D / 4), r = w / (D / 4), cc = w % (D / 4) * 4;
      const bool in = k0 + r < ke;
      copy16(dst + ((m * BK + r) * PD + cc) * 4, K + ((2 * kvh + m) * cap + (in ? k0 + r : kb)) * D + cc, in);
    }
#pragma unroll
    for (int v = 0; v < BK * DV / 4 / kT; ++v) {
      const int u = v * kT + threadIdx.x, r = u / (DV / 4), cc = u % (DV / 4) * 4;
      const bool in = k0 + r < ke;
      copy16(dst + (2 * BK * PD + r * PV + cc) * 4, V + (kvh * cap + (in ? k0 + r : kb)) * DV + cc, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (kb < ke) load(kb, 0);
  int buf = 0;
  for (int64_t k0 = kb; k0 < ke; k0 += BK, buf ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // this tile is there, the other buffer's has been read
    if (k0 + BK < ke) load(k0 + BK, buf ^ 1);
    const float *sK = sB + buf * kTile, *sV = sK + 2 * BK * PD;
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
    // The tile's sums, then added to the running ones: a chain of additions as long as the
    // context would lose bits with its square root.
    float part[RMAX][VC];
#pragma unroll
    for (int r = 0; r < RMAX; ++r)
#pragma unroll
      for (int v = 0; v < VC; ++v) part[r][v] = 0.f;
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
        for (int v = 0; v < VC; ++v) part[r][v] = fmaf(p, x[v], part[r][v]);
      }
    }
#pragma unroll
    for (int r = 0; r < RMAX; ++r) {
      if (r >= R) break;
      const float a = sA[2 * r + pm];
#pragma unroll
      for (int v = 0; v < VC; ++v) acc[r][v] = fmaf(acc[r][v], a, part[r][v]);
    }
  }
  __syncthreads();
  if (nsplit > 1) {
#pragma unroll
    for (int r = 0; r < RMAX; ++r)
      if (r < R) {
        const int64_t w = ((h0 + r) * 2 + pm) * nsplit + split;
#pragma unroll
        for (int v = 0; v < VC; ++v) ws[w * DV + pc + 64 * v] = acc[r][v];
        if (pc == 0) tail[w] = make_float2(sM[2 * r + pm], sL[2 * r + pm]);
      }
    return;
  }
  // one split: map 2's rows through shared memory (the tiles are done), then the difference
  float* x2 = sB;  // [R][DV]
  static_assert(RMAX * DV <= kTile, "exchange fits");
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
          *(O + (h0 + r) * DV + pc + 64 * v) = acc[r][v] - lm * x2[r * DV + pc + 64 * v];
      }
  }
}

// One block per (b, h): the splits of both maps joined.  The splits' weights are formed once, in
// shared memory; then groups of threads, each four columns wide, sum every kGroups-th split with
// four loads in flight, and the groups are added in order.
template <int DV, typename T>
__global__ void __launch_bounds__(256)
    join_kernel(const float* ws, const float2* tail, const float* __restrict__ lam,
                T* __restrict__ O, int H, int nsplit) {
  constexpr int C = DV / 4, kGroups = 256 / C;
  __shared__ float w[2][kMaxSplits];
  __shared__ __align__(16) float part[kGroups][DV];
  const int64_t bh = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::grid_dependency_wait();  // the splits' parts
  if (warp < 2) {  // map `warp`: w = 2^(max_s - max) / sum, minus lam of that for the second
    const float2* t = tail + (bh * 2 + warp) * nsplit;
    float mx = -INFINITY, l = 0.f;
    for (int s = lane; s < nsplit; s += 32) mx = fmaxf(mx, t[s].x);
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float sub = mx == -INFINITY ? 0.f : mx;  // no key at all
    for (int s = lane; s < nsplit; s += 32) {
      const float f = ptx::ex2(t[s].x - sub);
      w[warp][s] = f;
      l = fmaf(f, t[s].y, l);
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    const float f = l > 0.f ? (warp == 0 ? 1.f : -lam[bh % H]) / l : 0.f;
    for (int s = lane; s < nsplit; s += 32) w[warp][s] *= f;
  }
  __syncthreads();
  const int g = threadIdx.x / C, col = threadIdx.x % C * 4;
  const float* x = ws + bh * 2 * nsplit * DV + col;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = g; s < 2 * nsplit; s += kGroups) {  // map 1's splits, then map 2's
    const float4 v = *reinterpret_cast<const float4*>(x + static_cast<int64_t>(s) * DV);
    const float f = s < nsplit ? w[0][s] : w[1][s - nsplit];
    a[0] = fmaf(f, v.x, a[0]), a[1] = fmaf(f, v.y, a[1]), a[2] = fmaf(f, v.z, a[2]), a[3] = fmaf(f, v.w, a[3]);
  }
  *reinterpret_cast<float4*>(&part[g][col]) = make_float4(a[0], a[1], a[2], a[3]);
  __syncthreads();
  for (int c = threadIdx.x; c < DV; c += 256) {
    float o = 0.f;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) o += part[u][c];
    st1(O + bh * DV + c, o);
  }
}

template <int D>
cudaError_t run(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, const int* lens,
                void* O, float* ws, cudaStream_t st) {
  const Plan q = make_plan(p);
  const unsigned grid = static_cast<unsigned>(p.BHkv * q.chunks * q.nsplit);
  const int H = static_cast<int>(p.H);
  const float c = p.scale * kLog2e;
  float2* tail = reinterpret_cast<float2*>(ws + p.BH * 2 * q.nsplit * 2 * D);
  cudaError_t e;
  if (p.dtype == ATTN_BF16) {
    using T = __nv_bfloat16;
    constexpr int smem = NS * Stage<D>::bytes;
    e = cudaFuncSetAttribute(mma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    mma_kernel<D><<<grid, kT, smem, st>>>(static_cast<const T*>(Q), static_cast<const T*>(K), static_cast<const T*>(V),
                                          lam, lens, static_cast<T*>(O), ws, tail, p.N, H, p.group, q.rows, q.nsplit,
                                          p.window, c);
    if ((e = cudaGetLastError()) != cudaSuccess || q.nsplit == 1) return e;
    return launch_behind(join_kernel<2 * D, T>, p.BH, 256, 0, st, ws, tail, lam, static_cast<T*>(O), H, q.nsplit);
  } else {
    using T = float;
    constexpr int smem = 4 * (2 * (2 * BK * (D + 4) + BK * 2 * D) + 2 * RMAX * (D + BK + 3));
    e = cudaFuncSetAttribute(decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    decode_kernel<D><<<grid, kT, smem, st>>>(static_cast<const T*>(Q), static_cast<const T*>(K), static_cast<const T*>(V),
                                          lam, lens, static_cast<T*>(O), ws, tail, p.N, H, p.group, q.rows, q.nsplit,
                                          p.window, c);
    if ((e = cudaGetLastError()) != cudaSuccess || q.nsplit == 1) return e;
    return launch_behind(join_kernel<2 * D, T>, p.BH, 256, 0, st, ws, tail, lam, static_cast<T*>(O), H, q.nsplit);
  }
}

}  // namespace

size_t diff_decode_bytes(const Problem& p) {
  const Plan q = make_plan(p);
  return q.nsplit == 1 ? 0 : static_cast<size_t>(p.BH) * 2 * q.nsplit * (2 * p.d + 2) * sizeof(float);
}

cudaError_t diff_decode(const Problem& p, const void* Q, const void* K, const void* V, const float* lam,
                        const int* lens, void* O, void* ws, cudaStream_t st) {
  return p.d == 32 ? run<32>(p, Q, K, V, lam, lens, O, static_cast<float*>(ws), st)
                   : run<64>(p, Q, K, V, lam, lens, O, static_cast<float*>(ws), st);
}

}  // namespace fbd
