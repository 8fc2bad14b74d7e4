// Differential attention backward, bf16, on the tensor cores, in one pass over key blocks.
//
// With P_m recomputed from the stored log-sum-exps, dP = dO V^T, w = (1, -lam) and
// D_2 = dO.O_2, D_1 = dO.O + lam D_2:
//   W_m = w_m P_m,  dS_m = W_m (dP - D_m);
//   dV = sum_m W_m^T dO,  dK_m = s dS_m^T Q_m,  dQ_m = s dS_m K_m,  dlam = -sum P_2 dP.
// One CTA holds 128 keys (K_1, K_2, V) and streams the blocks of 128 queries that see them,
// first those of map 1, then those of map 2; dV accumulates over both sweeps, dK_m over its
// own.  (Both maps at once would form dP and dV once instead of twice, ten products of
// 128 x 128 x 64 a block pair instead of fourteen, but S_1, S_2, dP, dV, dK_m and dQ_m take
// 768 TMEM columns of 512.)  Per query block and map:
//   S^T = K_m Q_m^T, dP^T = V dO^T    in TMEM, released as soon as they are in registers
//   dV += W^T dO, dK += dS^T Q_m      A from shared-memory tiles of W^T and dS^T
//   dQ = dS K_m                       the dS tile read M-major
// dQ's share (fp32) is reduce-added in L2 into an accumulator in the workspace, in the order
// the key blocks reach it, so dQ can differ between runs in its last bits; every other
// output is the same bits on every run (dlam: one partial sum per warp and block, added in a
// fixed order).  W and dS are rounded to bf16 for their products; dlam uses the fp32 P and dP.
//
// Warps 0-15 compute (warp w: TMEM lanes 32(w%4).., tile columns 32(w/4)..), warp 16 issues
// the TMA loads and reduces, warp 17 the tile products, warp 18 the output products.
#include <cuda_bf16.h>

#include <type_traits>

#include "diff.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace fbd {
namespace {

__device__ unsigned int g_err = 0;

constexpr int BW = 128;        // held keys and streamed queries
constexpr int NS = 2;          // stages of streamed blocks
constexpr int kCW = 16;        // compute warps
constexpr int kCompute = kCW * 32;
constexpr int kThreads = kCompute + 96;
constexpr int kC = 32;         // tile columns per compute warp
constexpr int kSlab = BW * 128;  // 64 bf16 columns of 128 rows: 16 KB
constexpr float kLog2e = 1.4426950408889634f;

// d = 32 runs with its maps' tiles zero-filled to 64 columns (TMA), DV = 64.
template <int DV>
struct Lay {
  static constexpr int kV = kSlab * (DV / 64);
  static constexpr int kStat = BW * 8;  // (-L log2 e, -D) of the block's rows, pair-interleaved
  static constexpr int kStage = kSlab + kV + kStat;  // Q_m, dO (then the fp32 dQ share), statistics
  static constexpr int oK = 0, oV = 2 * kSlab;
  static constexpr int odS = oV + kV, oW = odS + 2 * kSlab;
  static constexpr int oStage = oW + 2 * kSlab;
  static constexpr int oBar = oStage + NS * kStage;
  static constexpr int bytes = oBar + 256;
  // TMEM columns: S^T, dP^T, dQ, dK, dV
  static constexpr int cS = 0, cdP = 128, cdQ = 256, cdK = 320, cdV = 384;
};
static_assert(Lay<128>::bytes <= 232448 && Lay<128>::kStage % 1024 == 0 && Lay<64>::kStage % 1024 == 0, "layout");

struct Bars {
  uint64_t* held_full;
  uint64_t* full;      // [NS] stage loaded
  uint64_t* s_full;    // S^T, dP^T in TMEM
  uint64_t* consumed;  // ... in the compute registers
  uint64_t* ready;     // W^T and dS in shared memory
  uint64_t* dq_full;   // the block's output products done
  uint64_t* dq_empty;  // dQ copied out of TMEM
  uint64_t* stg_full;  // [NS] dQ staged in its stage
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  __device__ explicit Bars(uint8_t* b) {
    held_full = reinterpret_cast<uint64_t*>(b);
    full = held_full + 1;
    s_full = full + NS;
    consumed = s_full + 1;
    ready = consumed + 1;
    dq_full = ready + 1;
    dq_empty = dq_full + 1;
    stg_full = dq_empty + 1;
    tmem_slot = reinterpret_cast<uint32_t*>(stg_full + NS);
    abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  }
};

// Byte offset of (row, 16-byte chunk) in a 128-byte-swizzled tile of 128-byte lines.
__device__ __forceinline__ uint32_t sw128(int row, int chunk) {
  return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// WIN: a banded causal mask is in force (window and/or document bounds).
template <int DV, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
               const __grid_constant__ CUtensorMap tmSt, const __grid_constant__ CUtensorMap tmAcc,
               const float* __restrict__ lam, __nv_bfloat16* __restrict__ dK, __nv_bfloat16* __restrict__ dV,
               float* __restrict__ partial, int N, int H, int nb, int BHkv, float scale, float c, int causal, Band bd,
               int G) {
  using L = Lay<DV>;
  constexpr int D = DV / 2;  // a map's true width
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars br(sm + L::oBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const tc::Order ord = tc::grid_order(BHkv, nb);
  const int kvh = ord.bh;          // key/value slice; its query heads are kvh * G + h, h < G
  const int kb = ord.k;            // first key blocks have the most query blocks: first
  const int i0 = causal ? kb : 0;  // first query block that sees this key block
  const int ntile = ((WIN && causal) ? bd.key_hi(kvh, min(kb * BW + BW - 1, N - 1)) / BW + 1 : nb) - i0;
  const int hi_first = (WIN && causal) ? bd.key_hi(kvh, kb * BW) : 0;  // the first key's last query
  const int half = G * ntile;      // tiles of a map
  const int nt = 2 * half;         // tile t = (m, h, i - i0)

  if (threadIdx.x == 0) {
    ptx::mbar_init(br.held_full, 1);
    ptx::mbar_init(br.s_full, 1);
    ptx::mbar_init(br.consumed, kCompute);
    ptx::mbar_init(br.ready, kCompute);
    ptx::mbar_init(br.dq_full, 1);
    ptx::mbar_init(br.dq_empty, kCompute);
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(&br.full[s], 1);
      ptx::mbar_init(&br.stg_full[s], kCompute);
    }
    *br.abort_flag = (ptx::smem_u32(sm) & 1023u) ? 1 : 0;
    if (*br.abort_flag) atomicOr(&g_err, FBD_ERR_TIMEOUT);
    ptx::fence_mbar_init();
  }
  if (warp == kCW + 1) {
    ptx::tmem_alloc(br.tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *br.tmem_slot;
  const ptx::BoundedWait wait{br.abort_flag, &g_err};
  const bool ok = *br.abort_flag == 0;
  auto tile_at = [&](int t, int& m, int& bh, int& i) {
    m = t >= half ? 1 : 0;
    const int r = t - m * half, h = r / ntile;
    bh = kvh * G + h;
    i = i0 + r - h * ntile;
  };

  if (warp == kCW) {
    // ------------------------------------------------ TMA loads and dQ reduces
    if (lane == 0 && ok) {
      ptx::prefetch_tmap(&tmQ);
      ptx::prefetch_tmap(&tmdO);
      ptx::prefetch_tmap(&tmSt);
      ptx::prefetch_tmap(&tmAcc);
      ptx::mbar_expect_tx(br.held_full, 2 * kSlab + L::kV);
      for (int m = 0; m < 2; ++m)
        ptx::tma_load_3d(sm + L::oK + m * kSlab, &tmK, br.held_full, 0, kb * BW, 2 * kvh + m);
      for (int u = 0; u < DV / 64; ++u)
        ptx::tma_load_3d(sm + L::oV + u * kSlab, &tmV, br.held_full, u * 64, kb * BW, kvh);
      auto load = [&](int t) {
        int m, bh, i;
        tile_at(t, m, bh, i);
        const int s = t % NS;
        uint8_t* st = sm + L::oStage + s * L::kStage;
        ptx::mbar_expect_tx(&br.full[s], L::kStage);
        ptx::tma_load_3d(st, &tmQ, &br.full[s], 0, i * BW, 2 * bh + m);
        for (int u = 0; u < DV / 64; ++u)
          ptx::tma_load_3d(st + kSlab + u * kSlab, &tmdO, &br.full[s], u * 64, i * BW, bh);
        ptx::tma_load_3d(st + kSlab + L::kV, &tmSt, &br.full[s], 0, i * (BW / 2), 2 * bh + m);
      };
      for (int t = 0; t < nt && t < NS; ++t) load(t);
      for (int t = 0; t < nt; ++t) {
        // dQ of tile t staged in its stage: reduce-add its 32-column boxes, then refill the stage
        if (!wait(&br.stg_full[t % NS], (t / NS) & 1)) break;
        int m, bh, i;
        tile_at(t, m, bh, i);
        const uint8_t* st = sm + L::oStage + (t % NS) * L::kStage;
        ptx::tma_reduce_add_3d(&tmAcc, st, 0, i * BW, 2 * bh + m);
        if (D > 32) ptx::tma_reduce_add_3d(&tmAcc, st + kSlab, 32, i * BW, 2 * bh + m);
        ptx::bulk_commit_group();
        ptx::bulk_wait_group_read0();
        if (t + NS < nt) load(t + NS);
      }
      ptx::bulk_wait_group0();  // every reduce performed before the CTA ends
    }
  } else if (warp == kCW + 1) {
    // ---------------------------------------------------------- tile products
    if (ok) {
      constexpr uint32_t idS = ptx::idesc_bf16(BW, BW, 0, 0);
      const uint64_t dKk = tc::kmajor_desc(ptx::smem_u32(sm + L::oK), BW, 0);
      const uint64_t dVk = tc::kmajor_desc(ptx::smem_u32(sm + L::oV), BW, 0);
      const uint32_t sSt = ptx::smem_u32(sm + L::oStage);
      const uint64_t dQk = tc::kmajor_desc(sSt, BW, 0), ddOk = tc::kmajor_desc(sSt + kSlab, BW, 0);
      const uint32_t tS = tmem + L::cS, tdP = tmem + L::cdP;
      wait(br.held_full, 0);
      for (int t = 0; t < nt; ++t) {
        const int s = t % NS;
        const uint32_t so = static_cast<uint32_t>(s * L::kStage), ko = t >= half ? kSlab : 0;
        wait(&br.full[s], (t / NS) & 1);
        if (t > 0) wait(br.consumed, (t - 1) & 1);
        ptx::tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_ss_e(tS, tc::desc_add(dKk, ko + tc::kmajor_off(BW, k)), tc::desc_add(dQk, so + tc::kmajor_off(BW, k)),
                        idS, k > 0);
#pragma unroll
        for (int k = 0; k < DV / 16; ++k)
          ptx::mma_ss_e(tdP, tc::desc_add(dVk, tc::kmajor_off(BW, k)), tc::desc_add(ddOk, so + tc::kmajor_off(BW, k)),
                        idS, k > 0);
        ptx::mma_commit_e(br.s_full);
      }
    }
  } else if (warp == kCW + 2) {
    // -------------------------------------------------------- output products
    if (ok) {
      constexpr uint32_t idV = ptx::idesc_bf16(BW, DV, 0, 1);  // A K-major (W^T), B MN-major
      constexpr uint32_t idK = ptx::idesc_bf16(BW, 64, 0, 1);
      constexpr uint32_t idQ = ptx::idesc_bf16(BW, 64, 1, 1);  // A = dS read M-major
      const uint32_t sSt = ptx::smem_u32(sm + L::oStage), sdS = ptx::smem_u32(sm + L::odS);
      const uint64_t dQm = tc::mnmajor_desc(sSt, BW, 0), ddOm = tc::mnmajor_desc(sSt + kSlab, BW, 0);
      const uint64_t dSk = tc::kmajor_desc(sdS, BW, 0);   // dS^T: M = keys, K = queries (2 slabs)
      const uint64_t dSm = tc::mnmajor_desc(sdS, BW, 0);  // dS: M = queries (2 slabs), K = keys
      const uint64_t dWk = tc::kmajor_desc(ptx::smem_u32(sm + L::oW), BW, 0);
      const uint64_t dKm = tc::mnmajor_desc(ptx::smem_u32(sm + L::oK), BW, 0);
      const uint32_t tdV = tmem + L::cdV, tdK = tmem + L::cdK, tdQ = tmem + L::cdQ;
      wait(br.held_full, 0);
      for (int t = 0; t < nt; ++t) {
        const int s = t % NS;
        const uint32_t so = static_cast<uint32_t>(s * L::kStage), ko = t >= half ? kSlab : 0;
        wait(br.ready, t & 1);
        wait(&br.full[s], (t / NS) & 1);  // complete already: this warp's acquire of the loaded stage
        ptx::tc_fence_after();
#pragma unroll
        for (int k = 0; k < BW / 16; ++k) {
          ptx::mma_ss_e(tdV, tc::desc_add(dWk, tc::kmajor_off(BW, k)), tc::desc_add(ddOm, so + 2048 * k), idV,
                        (t > 0 || k > 0) ? 1u : 0u);
          ptx::mma_ss_e(tdK, tc::desc_add(dSk, tc::kmajor_off(BW, k)), tc::desc_add(dQm, so + 2048 * k), idK,
                        ((t > 0 && t != half) || k > 0) ? 1u : 0u);
        }
        if (t > 0) {
          wait(br.dq_empty, (t - 1) & 1);
          ptx::tc_fence_after();
        }
#pragma unroll
        for (int k = 0; k < BW / 16; ++k)
          ptx::mma_ss_e(tdQ, tc::desc_add(dSm, 2048 * k), tc::desc_add(dKm, ko + 2048 * k), idQ, k > 0 ? 1u : 0u);
        ptx::mma_commit_e(br.dq_full);
      }
    }
  } else {
    // ------------------------------------------------------------ compute
    const int qd = warp & 3, cg = warp >> 2;
    const int r = qd * 32 + lane;  // key row (TMEM lane) of the outputs
    const uint32_t lo = static_cast<uint32_t>(qd * 32) << 16;
    const int key = kb * BW + r;
    const int c0 = cg * kC;
    // Score tiles through the 16-lane shapes: a thread sees 8 queries of its 32 (pairs
    // 2(t%4) + 8k, k < 4) for 4 keys (rows t/4 + 8m of each 16-lane half).
    const int g4 = lane >> 2, q4 = lane & 3;
    const uint64_t c2 = tc::pk2f(c, c);
    int khi[2][2] = {{0, 0}, {0, 0}};  // last query each of the four keys is seen by
    if constexpr (WIN) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < 2; ++m) khi[h][m] = bd.key_hi(kvh, kb * BW + qd * 32 + g4 + 16 * h + 8 * m);
    }
    // dQ of tile t out of TMEM (query 32 qd + lane, columns 16 cg ..) into its stage as
    // 128-byte-swizzled fp32 boxes of 32 columns.
    auto drain = [&](int t) {
      uint32_t qv[16];
      ptx::tmem_ld16(tmem + L::cdQ + static_cast<uint32_t>(cg * 16) + lo, qv);
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      ptx::mbar_arrive(br.dq_empty);
      if (cg * 16 < D) {
        uint8_t* box = sm + L::oStage + (t % NS) * L::kStage + (cg >> 1) * kSlab;
        const int q = qd * 32 + lane;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4*>(box + sw128(q, (cg & 1) * 4 + u)) =
              make_uint4(qv[4 * u], qv[4 * u + 1], qv[4 * u + 2], qv[4 * u + 3]);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&br.stg_full[t % NS]);
    };
    auto store_dk = [&](int m) {
      uint32_t a[16];
      ptx::tmem_ld16(tmem + L::cdK + cg * 16 + lo, a);
      ptx::tmem_wait_ld();
      if (key < N && cg * 16 < D) {
        uint32_t o[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) o[u] = ptx::pack_bf16(scale * tc::f(a[2 * u]), scale * tc::f(a[2 * u + 1]));
        uint4* p = reinterpret_cast<uint4*>(dK + ((2 * static_cast<size_t>(kvh) + m) * N + key) * D + cg * 16);
        p[0] = make_uint4(o[0], o[1], o[2], o[3]);
        p[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    };
    uint64_t dl2 = 0;  // sums of P_2 dP
    for (int t = 0; t < nt; ++t) {
      const int s = t % NS;
      int m, bh, i;
      tile_at(t, m, bh, i);
      const float wm = m == 0 ? 1.f : -lam[bh % H];
      const uint64_t w2 = tc::pk2f(wm, wm);
      wait(br.s_full, t & 1);
      ptx::tc_fence_after();
      uint32_t sv[2][16], pv[2][16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t la = lo + (static_cast<uint32_t>(16 * h) << 16);
        ptx::tmem_ld16x256_x4(tmem + L::cS + c0 + la, sv[h]);
        ptx::tmem_ld16x256_x4(tmem + L::cdP + c0 + la, pv[h]);
      }
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      ptx::mbar_arrive(br.consumed);
      // float4 k: (-L, -L', -D, -D') of queries 2k, 2k + 1
      wait(&br.full[s], (t / NS) & 1);  // complete already: the acquire of the loaded statistics
      const float4* st = reinterpret_cast<const float4*>(sm + L::oStage + s * L::kStage + kSlab + L::kV) + c0 / 2;
      float4 A[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) A[k] = st[4 * k + q4];
      const int qbase = i * BW + c0 + 2 * q4;    // query of column (k = 0, col 0)
      const int kbase = kb * BW + qd * 32 + g4;  // key of (h = 0, row 0)
      uint32_t pk[2][8], dk[2][8];               // [h][2k + (row, row+8)]
      auto block = [&](auto masked) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int e = 4 * k + 2 * u;
              const float2 arg = tc::unpk2(tc::fma2(tc::pk2(sv[h][e], sv[h][e + 1]), c2, tc::pk2f(A[k].x, A[k].y)));
              float p0 = ptx::ex2(arg.x), p1 = ptx::ex2(arg.y);
              if constexpr (decltype(masked)::value) {
                const int q0 = qbase + 8 * k, kk = kbase + 16 * h + 8 * u;
                if ((causal ? (q0 < kk || (WIN && q0 > khi[h][u])) : kk >= N) || q0 >= N) p0 = 0.f;
                if ((causal ? (q0 + 1 < kk || (WIN && q0 + 1 > khi[h][u])) : kk >= N) || q0 + 1 >= N) p1 = 0.f;
              }
              const uint64_t P2 = tc::pk2f(p0, p1), dP2 = tc::pk2(pv[h][e], pv[h][e + 1]);
              if (m == 1) dl2 = tc::fma2(P2, dP2, dl2);
              const uint64_t W2 = tc::mul2(P2, w2);
              float2 ds = tc::unpk2(tc::mul2(W2, tc::add2(dP2, tc::pk2f(A[k].z, A[k].w))));
              if constexpr (decltype(masked)::value) {  // rows with one visible key
                if (A[k].z == -INFINITY) ds.x = 0.f;
                if (A[k].w == -INFINITY) ds.y = 0.f;
              }
              const float2 w = tc::unpk2(W2);
              pk[h][2 * k + u] = ptx::pack_bf16(w.x, w.y);
              dk[h][2 * k + u] = ptx::pack_bf16(ds.x, ds.y);
            }
      };
      // the diagonal block, a block past the first key's last query, past N, or with keys past N
      if ((causal && i == kb) || (WIN && causal && i * BW + BW - 1 > hi_first) || i * BW + c0 + kC > N ||
          (!causal && kb * BW + BW > N))
        block(std::true_type{});
      else
        block(std::false_type{});
      if (t > 0) {  // the previous block's products have read W^T, dS and its stage
        wait(br.dq_full, (t - 1) & 1);
        ptx::tc_fence_after();
      }
      if (t == half) store_dk(0);  // map 1's sweep is done (the next dK product waits for `ready`)
      {
        const uint32_t sdS = ptx::smem_u32(sm + L::odS), sW = ptx::smem_u32(sm + L::oW);
        const int qcol = c0 + 8 * (lane >> 3);  // first query of the chunk this lane addresses
        const uint32_t cb = static_cast<uint32_t>((qcol >> 6) * kSlab);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a = cb + sw128(qd * 32 + 16 * h + 8 * u + (lane & 7), (qcol & 63) >> 3);
            ptx::stmatrix_x4(sW + a, pk[h][u], pk[h][2 + u], pk[h][4 + u], pk[h][6 + u]);
            ptx::stmatrix_x4(sdS + a, dk[h][u], dk[h][2 + u], dk[h][4 + u], dk[h][6 + u]);
          }
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      ptx::mbar_arrive(br.ready);
      if (t > 0) drain(t - 1);
      if (m == 1 && i == i0 + ntile - 1) {  // head h's queries are done: this warp's share of its dlam
        const float2 x = tc::unpk2(dl2);
        float v = x.x + x.y;
#pragma unroll
        for (int u = 1; u < 32; u <<= 1) v += __shfl_xor_sync(0xffffffffu, v, u);
        if (lane == 0) partial[(static_cast<size_t>(bh) * nb + kb) * kCW + warp] = v;
        dl2 = 0;
      }
    }
    wait(br.dq_full, (nt - 1) & 1);
    ptx::tc_fence_after();
    drain(nt - 1);
    store_dk(1);
    constexpr int VG = DV / 4;  // dV columns per thread
#pragma unroll
    for (int u = 0; u < VG / 16; ++u) {
      uint32_t a[16], o[8];
      ptx::tmem_ld16(tmem + L::cdV + cg * VG + u * 16 + lo, a);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int x = 0; x < 8; ++x) o[x] = ptx::pack_bf16(tc::f(a[2 * x]), tc::f(a[2 * x + 1]));
      if (key < N) {
        uint4* p = reinterpret_cast<uint4*>(dV + (static_cast<size_t>(kvh) * N + key) * DV + cg * VG + u * 16);
        p[0] = make_uint4(o[0], o[1], o[2], o[3]);
        p[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kCW + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// D_m of every row and both maps' statistics, pair-interleaved and negated as the key-block
// pass reads them: float4 k of a map's slice = (-L log2 e, -L' log2 e, -D, -D') of rows 2k,
// 2k + 1 (zeros for the padding row of an odd N); the dQ accumulator's rows zeroed.  16
// threads per row.
template <int DV>
__global__ void __launch_bounds__(256)
    prep_kernel(const __nv_bfloat16* __restrict__ O, const __nv_bfloat16* __restrict__ O2,
                const __nv_bfloat16* __restrict__ dO, const float* __restrict__ lse, const float* __restrict__ lam,
                float* __restrict__ stats, float* __restrict__ acc, int64_t N, int64_t Np, int64_t H, int64_t BH,
                int causal, Band bd) {
  constexpr int W = DV / 16;  // columns per thread
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t rowg = gid >> 4;
  const int part = static_cast<int>(gid & 15);
  const bool valid = rowg < BH * Np;  // every lane stays for the shuffles below
  const int64_t bh = valid ? rowg / Np : 0, row = valid ? rowg - bh * Np : 0;
  const bool live = valid && row < N;
  float d = 0.f, d2 = 0.f;
  if (live) {
    const int64_t off = (bh * N + row) * DV + part * W;
#pragma unroll
    for (int u = 0; u < W; u += 4) {
      const uint2 g = *reinterpret_cast<const uint2*>(dO + off + u), o = *reinterpret_cast<const uint2*>(O + off + u),
                  p = *reinterpret_cast<const uint2*>(O2 + off + u);
      const uint32_t gw[2] = {g.x, g.y}, ow[2] = {o.x, o.y}, pw[2] = {p.x, p.y};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = tc::bf16_lo(gw[e]), y = tc::bf16_hi(gw[e]);
        d = fmaf(x, tc::bf16_lo(ow[e]), fmaf(y, tc::bf16_hi(ow[e]), d));
        d2 = fmaf(x, tc::bf16_lo(pw[e]), fmaf(y, tc::bf16_hi(pw[e]), d2));
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
      *reinterpret_cast<float4*>(acc + ((2 * bh + m) * N + row) * 64 + part * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) {
    d += __shfl_xor_sync(0xffffffffu, d, x);
    d2 += __shfl_xor_sync(0xffffffffu, d2, x);
  }
  if (valid && part < 2) {
    const int m = part;
    float L = 0.f, D = 0.f;
    if (live) {
      L = lse[(2 * bh + m) * N + row] * kLog2e;
      D = diff_mark_D(m == 0 ? fmaf(lam[bh % H], d2, d) : d2, diff_one_key(bd, causal, bh, row));
    }
    float* s = stats + ((2 * bh + m) * Np + (row & ~int64_t(1))) * 2 + (row & 1);
    s[0] = -L;
    s[2] = -D;
  }
}

// dQ = bf16(s acc), the d columns of each row, eight per thread.
__global__ void __launch_bounds__(256) dq_kernel(const float* __restrict__ acc, __nv_bfloat16* __restrict__ dQ,
                                                 int64_t rows, int d, float scale) {
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int per = d / 8;
  const int64_t row = gid / per;
  const int part = static_cast<int>(gid - row * per);
  if (row >= rows) return;
  const float4* a = reinterpret_cast<const float4*>(acc + row * 64 + part * 8);
  const float4 x = a[0], y = a[1];
  *reinterpret_cast<uint4*>(dQ + row * d + part * 8) =
      make_uint4(ptx::pack_bf16(scale * x.x, scale * x.y), ptx::pack_bf16(scale * x.z, scale * x.w),
                 ptx::pack_bf16(scale * y.x, scale * y.y), ptx::pack_bf16(scale * y.z, scale * y.w));
}

int64_t padded(int64_t N) { return (N + 1) & ~int64_t(1); }
int64_t blocks(int64_t N) { return (N + BW - 1) / BW; }

template <int DV>
cudaError_t run(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, const void* O,
                const void* O2, const void* dO, const float* lse, void* dQ, void* dK, void* dV, float* dlam, void* ws,
                cudaStream_t st) {
  constexpr int D = DV / 2;
  const int64_t N = p.N, BH = p.BH, Np = padded(N);
  float* stats = static_cast<float*>(ws);        // [2BH][Np / 2] float4
  float* acc = stats + 2 * BH * Np * 2;          // [2BH][N][64]
  float* partial = acc + 2 * BH * N * 64;        // [BH][blocks][kCW]
  alignas(64) CUtensorMap k, v, q, g, s, a;
  if (!make_tmap_bf16(&q, Q, N, D, 2 * BH, BW) || !make_tmap_bf16(&g, dO, N, DV, BH, BW) ||
      !make_tmap_bf16(&k, K, N, D, 2 * p.BHkv, BW) || !make_tmap_bf16(&v, V, N, DV, p.BHkv, BW) ||
      !make_tmap_stats(&s, stats, Np / 2, 2 * BH, BW / 2) || !make_tmap_f32_rows(&a, acc, N, 2 * BH, BW))
    return cudaErrorInvalidValue;
  const int64_t threads = BH * Np * 16;
  prep_kernel<DV><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, st>>>(
      static_cast<const __nv_bfloat16*>(O), static_cast<const __nv_bfloat16*>(O2),
      static_cast<const __nv_bfloat16*>(dO), lse, lam, stats, acc, N, Np, p.H, BH, p.causal,
      make_band(p, eff_window(p), false));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int nb = static_cast<int>(blocks(N));
  auto kern = banded(p) ? bwd_kernel<DV, true> : bwd_kernel<DV, false>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<DV>::bytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(nb * p.BHkv), kThreads, Lay<DV>::bytes, st>>>(
      k, v, q, g, s, a, lam, static_cast<__nv_bfloat16*>(dK), static_cast<__nv_bfloat16*>(dV), partial,
      static_cast<int>(N), static_cast<int>(p.H), nb, static_cast<int>(p.BHkv), p.scale, p.scale * kLog2e, p.causal,
      make_band(p, eff_window_tc(p), true), p.group);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t dqt = 2 * BH * N * (D / 8);
  dq_kernel<<<static_cast<unsigned>((dqt + 255) / 256), 256, 0, st>>>(acc, static_cast<__nv_bfloat16*>(dQ), 2 * BH * N,
                                                                      D, p.scale);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return diff_reduce_dlam(partial, dlam, p.B, p.H, static_cast<int64_t>(nb) * kCW, st);
}

}  // namespace

size_t tc_diff_bwd_bytes(int64_t BH, int64_t N) {
  return static_cast<size_t>(BH) * (padded(N) * 16 + N * 512 + blocks(N) * kCW * 4);
}

cudaError_t tc_diff_bwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, const void* O,
                        const void* O2, const void* dO, const float* lse, void* dQ, void* dK, void* dV, float* dlam,
                        void* ws, cudaStream_t st) {
  return p.d == 32 ? run<64>(p, Q, K, V, lam, O, O2, dO, lse, dQ, dK, dV, dlam, ws, st)
                   : run<128>(p, Q, K, V, lam, O, O2, dO, lse, dQ, dK, dV, dlam, ws, st);
}

uint32_t tc_diff_bwd_take_error() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err, &z, sizeof(z));
  return v;
}

}  // namespace fbd
