// Differential attention backward, bf16, on the tensor cores, in two passes.
//
// With P_m recomputed from the stored log-sum-exps, dP = dO V^T, w = (1, -lam) and
// D_2 = dO.O_2, D_1 = dO.O + lam D_2 (a first launch, into the workspace):
//   W_m = w_m P_m,  dS_m = W_m (dP - D_m);
//   dQ_m = s dS_m K_m,  dK_m = s dS_m^T Q_m,  dV = (W_1 + W_2)^T dO,  dlam = -sum P_2 dP.
// Both maps of a head are handled together, so that dP and dV are formed once.
//   row pass:     a CTA holds 128 queries (Q_1, Q_2, dO), streams key blocks; six products of
//                 128 x 128 x 64 a block: S_1, S_2, dP (two), dQ_1, dQ_2.  Also dlam's sums.
//   column pass:  a CTA holds 128 keys (K_1, K_2, V), streams the query blocks that see them;
//                 eight: S_1^T, S_2^T, dP^T (two), dV (two), dK_1, dK_2.
// (One pass with dQ summed over key blocks by reduce-adds in L2 needs ten, or fourteen with a
// map at a time, since both maps' tiles and accumulators take 768 TMEM columns of 512; at a map
// at a time its reduce-adds, 32 KB a block and map at about 3.6 TB/s, took longer than the
// products: 0.65 ms against 0.46 for the two passes at B4 H6 N4096 d64.)
// Every output is written once and is the same bits on every run.
//
// S and dP tiles go to registers as soon as they are done and their columns are released;
// S_1 and S_2 share one tile.  dS (and W) are rounded to bf16 for their products; P, dP, the
// exponents' arguments and dlam's sums are fp32.
//
// Warps 0-15 compute (warp w: TMEM lanes 32(w%4).., tile columns 32(w/4)..), warp 16 issues
// the TMA loads, warp 17 allocates TMEM and issues the products (elect.sync from the warp); in
// the column pass warp 18 brings the streamed rows' statistics.
#include <cuda_bf16.h>

#include <type_traits>

#include "diff.h"
#include "handover.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace fbd {
namespace {

__device__ unsigned int g_err = 0;

constexpr int BW = 128;          // held and streamed rows
constexpr int NS = 2;            // stages of streamed blocks
constexpr int kCW = 16;          // compute warps
constexpr int kC = 32;           // tile columns per compute warp
// Column pass: 640 threads launched with 96 registers; the compute warps take 104 (each
// thread's two maps of P alone are 64), the fifth warpgroup's warps keep 64:
// 512 * 104 + 128 * 64 = 640 * 96.
constexpr int kThreads = kCW * 32 + 128;
constexpr int kColRegs = 104, kColRegsOther = 64;
constexpr int kPlanes = 5;       // row statistics: -L_1 log2 e, -L_2 log2 e, -D_1, lam D_2, -D_2
constexpr int kSlab = BW * 128;  // 64 bf16 columns of 128 rows: 16 KB
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void st_shared4(uint32_t a, const uint32_t* v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Shared memory of both passes: the held block (two maps' 64-column tiles, d = 32 zero-filled
// by TMA, and the DV-column one), the column pass's dS_2 tile, the stages, the barriers.
template <int DV, bool COL>
struct Lay {
  static constexpr int kV = kSlab * (DV / 64);
  static constexpr int kBlock = 2 * kSlab + kV;
  static constexpr int oT = kBlock;
  static constexpr int oStage = oT + (COL ? 2 * kSlab : 0);
  static constexpr int oStat = oStage + NS * kBlock;  // column pass: the streamed queries' statistics
  static constexpr int oBar = oStat + (COL ? 4 * BW * 4 : 0);
  static constexpr int bytes = oBar + 256;
};
static_assert(Lay<128, true>::bytes <= 232448, "shared memory");

// 16 columns (from c0) of a thread's row r as bf16 into its 64-column tiles, scaled.
__device__ __forceinline__ void stage16(uint8_t* tiles, int r, int c0, const uint32_t (&a)[16], float f) {
  uint32_t o[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) o[u] = ptx::pack_bf16(f * tc::f(a[2 * u]), f * tc::f(a[2 * u + 1]));
  uint8_t* t = tiles + (c0 >> 6) * kSlab;
  *reinterpret_cast<uint4*>(t + tc::sw128(r, (c0 & 63) >> 3)) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(t + tc::sw128(r, ((c0 & 63) >> 3) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ void init_abort(uint8_t* sm, volatile int* abort_flag) {
  *abort_flag = (ptx::smem_u32(sm) & 1023u) ? 1 : 0;  // the swizzled tiles need 1024-byte alignment
  if (*abort_flag) atomicOr(&g_err, FBD_ERR_TIMEOUT);
}

// After the roles have met, in a CTA where a wait has given up: loads and products may still be on
// their way into its shared memory and TMEM, which others get when it ends.  started: the loads
// begun in each ring of stages; the first ones come with the held block's.
__device__ __forceinline__ void teardown(volatile int* abort_flag, uint64_t* settled, volatile int* started,
                                         uint64_t* held, uint64_t* ring0, uint64_t* ring1) {
  if (*abort_flag == 0) return;
  if (threadIdx.x == kCW * 32) {
    if (started[0] > 0) ptx::settle(held, 0);
    for (int s = 0; s < NS; ++s) {
      if (s < started[0]) ptx::settle(&ring0[s], handover::last_phase(started[0], NS, s));
      if (s < started[1]) ptx::settle(&ring1[s], handover::last_phase(started[1], NS, s));
    }
  }
  if (threadIdx.x / 32 == kCW + 1) {
    ptx::mma_commit_e(settled);
    ptx::settle(settled, 0);
  }
}

struct Args {
  const float* lam;
  const float* stats;
  float* partial;
  int N, H, nb, BHkv;
  float scale, c;
  int causal;
  Band bd;  // over key/value slices (the row pass asks by its key/value slice too)
  int G;
};

// ------------------------------------------------------------------ row pass
// TMEM columns: S (S_1, then S_2), dP, dS_1, dS_2 (bf16 pairs), dQ_1, dQ_2.
// WIN: a banded causal mask is in force (window and/or document bounds).
template <int DV, bool WIN>
__device__ __forceinline__ void row_pass(const Args& p, int block, const CUtensorMap& tmQ, const CUtensorMap& tmdO,
                                         const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmdQ) {
  using L = Lay<DV, false>;
  constexpr int D = DV / 2;
  constexpr uint32_t cS = 0, cdP = 128, cdS = 256, cdQ = 384;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* held_full = bars;
  uint64_t* k_full = bars + 1;        // [NS]
  uint64_t* v_full = k_full + NS;     // [NS]
  uint64_t* k_empty = v_full + NS;    // [NS] dQ_2 of the block done
  uint64_t* v_empty = k_empty + NS;   // [NS] dP of the block done
  uint64_t* s_full = v_empty + NS;    // [2] S_m in TMEM
  uint64_t* s_cons = s_full + 2;      // [2] ... in the compute registers
  uint64_t* dp_full = s_cons + 2;
  uint64_t* dp_cons = dp_full + 1;
  uint64_t* ds_ready = dp_cons + 1;   // [2] dS_m in TMEM
  uint64_t* dq_done = ds_ready + 2;   // [2] dS_m K_m done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dq_done + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sRed = reinterpret_cast<float*>(sm + L::oBar + 160);  // [kCW]
  uint64_t* settled = reinterpret_cast<uint64_t*>(sm + L::oBar + 224);  // see teardown()
  volatile int* started = reinterpret_cast<volatile int*>(settled + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float *lam = p.lam, *stats = p.stats;
  float* partial = p.partial;
  const int N = p.N, H = p.H, nrb = p.nb, causal = p.causal, G = p.G, BH = p.BHkv * p.G;
  const float scale = p.scale, c = p.c;
  const Band& bd = p.bd;
  const tc::Order ord = tc::grid_order_at(block, BH, nrb);
  const int bh = ord.bh, kvh = bh / G;
  const int rb = nrb - 1 - ord.k;  // heaviest row blocks first
  const int j0 = (WIN && causal) ? bd.row_lo(kvh, rb * BW) / BW : 0;
  const int lo_last = (WIN && causal) ? bd.row_lo(kvh, min(rb * BW + BW - 1, N - 1)) : 0;
  const int nt = (causal ? rb + 1 : nrb) - j0;

  auto load_v = [&](int t) {
    const int s = t % NS;
    ptx::mbar_expect_tx(&v_full[s], L::kV);
    for (int u = 0; u < DV / 64; ++u)
      ptx::tma_load_3d(sm + L::oStage + s * L::kBlock + (2 + u) * kSlab, &tmV, &v_full[s], u * 64, (j0 + t) * BW, kvh);
  };
  auto load_k = [&](int t) {
    const int s = t % NS;
    ptx::mbar_expect_tx(&k_full[s], 2 * kSlab);
    for (int m = 0; m < 2; ++m)
      ptx::tma_load_3d(sm + L::oStage + s * L::kBlock + m * kSlab, &tmK, &k_full[s], 0, (j0 + t) * BW, 2 * kvh + m);
  };
  // The TMA thread sets the barriers up and starts the first loads before the others are let in
  // (the TMEM allocation alone takes about a thousand cycles).
  if (threadIdx.x == kCW * 32) {
    ptx::mbar_init(held_full, 1);
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(&k_full[s], 1);
      ptx::mbar_init(&v_full[s], 1);
      ptx::mbar_init(&k_empty[s], 1);
      ptx::mbar_init(&v_empty[s], 1);
    }
    for (int m = 0; m < 2; ++m) {
      ptx::mbar_init(&s_full[m], 1);
      ptx::mbar_init(&s_cons[m], kCW * 32);
      ptx::mbar_init(&ds_ready[m], kCW * 32);
      ptx::mbar_init(&dq_done[m], 1);
    }
    ptx::mbar_init(dp_full, 1);
    ptx::mbar_init(dp_cons, kCW * 32);
    ptx::mbar_init(settled, 1);
    init_abort(sm, abort_flag);
    started[0] = started[1] = *abort_flag ? 0 : min(nt, NS);
    ptx::fence_mbar_init();
    if (!*abort_flag) {
      ptx::mbar_expect_tx(held_full, L::kBlock);
      for (int m = 0; m < 2; ++m) ptx::tma_load_3d(sm + m * kSlab, &tmQ, held_full, 0, rb * BW, 2 * bh + m);
      for (int u = 0; u < DV / 64; ++u)
        ptx::tma_load_3d(sm + (2 + u) * kSlab, &tmdO, held_full, u * 64, rb * BW, bh);
      for (int t = 0; t < nt && t < NS; ++t) {
        load_k(t);
        load_v(t);
      }
    }
  }
  if (warp == kCW + 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const ptx::BoundedWait wait{abort_flag, &g_err};
  const bool ok = *abort_flag == 0;

  if (warp == kCW) {
    // ------------------------------------------------------------ TMA loads
    if (lane == 0 && ok) {
      for (int t = NS; t < nt; ++t) {
        const int s = t % NS, ph = ((t / NS) - 1) & 1;
        if (!wait(&v_empty[s], ph)) break;
        load_v(t);
        started[1] = t + 1;
        if (!wait(&k_empty[s], ph)) break;
        load_k(t);
        started[0] = t + 1;
      }
    }
  } else if (warp == kCW + 1) {
    // ------------------------------------------------------------- products
    if (ok) {
      constexpr uint32_t idS = ptx::idesc_bf16(BW, BW, 0, 0);
      constexpr uint32_t idQ = ptx::idesc_bf16(BW, 64, 0, 1);
      const uint32_t sH = ptx::smem_u32(sm), sS = ptx::smem_u32(sm + L::oStage);
      const uint64_t dHk = tc::kmajor_desc(sH, BW, 0);    // held block, rows = M
      const uint64_t dSk = tc::kmajor_desc(sS, BW, 0);    // streamed block, rows = N
      const uint64_t dSm = tc::mnmajor_desc(sS, BW, 0);   // streamed block, rows = K
      auto S = [&](int m, int t) {
        const uint32_t so = static_cast<uint32_t>((t % NS) * L::kBlock + m * kSlab);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_ss_e(tmem + cS, tc::desc_add(dHk, m * kSlab + tc::kmajor_off(BW, k)),
                        tc::desc_add(dSk, so + tc::kmajor_off(BW, k)), idS, k > 0);
        ptx::mma_commit_e(&s_full[m]);
      };
      auto dP = [&](int t) {
        const uint32_t so = static_cast<uint32_t>((t % NS) * L::kBlock + 2 * kSlab);
#pragma unroll
        for (int k = 0; k < DV / 16; ++k)
          ptx::mma_ss_e(tmem + cdP, tc::desc_add(dHk, 2 * kSlab + tc::kmajor_off(BW, k)),
                        tc::desc_add(dSk, so + tc::kmajor_off(BW, k)), idS, k > 0);
        ptx::mma_commit_e(dp_full);
        ptx::mma_commit_e(&v_empty[t % NS]);
      };
      auto dQm = [&](int m, int t) {
        wait(&ds_ready[m], t & 1);
        ptx::tc_fence_after();
        const uint32_t so = static_cast<uint32_t>((t % NS) * L::kBlock + m * kSlab);
#pragma unroll
        for (int k = 0; k < BW / 16; ++k)
          ptx::mma_ts_e(tmem + cdQ + m * 64, tmem + cdS + m * 64 + k * 8, tc::desc_add(dSm, so + 2048 * k), idQ,
                        (t > 0 || k > 0) ? 1u : 0u);
        ptx::mma_commit_e(&dq_done[m]);
      };
      wait(held_full, 0);
      wait(&k_full[0], 0);
      ptx::tc_fence_after();
      S(0, 0);
      wait(&v_full[0], 0);
      ptx::tc_fence_after();
      dP(0);
      for (int t = 0; t < nt; ++t) {
        const int s1 = (t + 1) % NS, ph1 = ((t + 1) / NS) & 1;
        wait(&s_cons[0], t & 1);
        ptx::tc_fence_after();
        S(1, t);
        if (t + 1 < nt) {
          wait(dp_cons, t & 1);
          wait(&v_full[s1], ph1);
          ptx::tc_fence_after();
          dP(t + 1);
        }
        dQm(0, t);
        if (t + 1 < nt) {
          wait(&s_cons[1], t & 1);
          wait(&k_full[s1], ph1);
          ptx::tc_fence_after();
          S(0, t + 1);
        }
        dQm(1, t);
        ptx::mma_commit_e(&k_empty[t % NS]);
      }
    }
  } else if (warp < kCW) {
    // ------------------------------------- compute: a query row, 32 keys of a block
    const int qd = warp & 3, cg = warp >> 2, c0 = cg * kC;
    const uint32_t lo = static_cast<uint32_t>(qd * 32) << 16;
    const int row = rb * BW + qd * 32 + lane;
    const int lo_row = (WIN && causal) ? bd.row_lo(kvh, row) : 0;
    const float* st = stats + (static_cast<int64_t>(bh) * nrb + rb) * (kPlanes * BW) + qd * 32 + lane;
    const float lm = lam[bh % H];
    ptx::grid_dependency_wait();  // the statistics are the preparation's
    const bool one = st[2 * BW] == -INFINITY;  // the row sees one key: its dS is 0
    const uint64_t c2 = tc::pk2f(c, c);
    const uint64_t nL[2] = {tc::pk2f(st[0], st[0]), tc::pk2f(st[BW], st[BW])};
    const uint64_t nD[2] = {tc::pk2f(st[2 * BW], st[2 * BW]), tc::pk2f(st[4 * BW], st[4 * BW])};
    uint64_t dl2 = 0;
    for (int t = 0; t < nt; ++t) {
      const int kb = j0 + t;
      const bool diag = causal ? kb == rb : (t == nt - 1 && (N % BW) != 0);
      const bool low = WIN && causal && kb * BW < lo_last;
      const int klim = (causal ? row : N - 1) - kb * BW - c0;  // last visible key, from this warp's first
      const int klo = (WIN && causal) ? lo_row - kb * BW - c0 : 0;
      // bounds grow with the row: the warp's first row has the first last key, its last row the
      // last first one
      const bool masked = (diag || low) && (kC - 1 > __shfl_sync(0xffffffffu, klim, 0) ||
                                            0 < __shfl_sync(0xffffffffu, klo, 31));
      uint32_t dp[32];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t v[32], pk[16];
        uint64_t sum = 0;  // of P_2 dP in this block: short chains of additions (dlam is fp32)
        wait(&s_full[m], t & 1);
        ptx::tc_fence_after();
        ptx::tmem_ld32(tmem + cS + c0 + lo, v);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&s_cons[m]);
        if (m == 0) {
          wait(dp_full, t & 1);
          ptx::tc_fence_after();
          ptx::tmem_ld32(tmem + cdP + c0 + lo, dp);
        }
#pragma unroll
        for (int u = 0; u < 32; u += 2) {
          const float2 a = tc::unpk2(tc::fma2(tc::pk2(v[u], v[u + 1]), c2, nL[m]));
          v[u] = __float_as_uint(ptx::ex2(a.x));
          v[u + 1] = __float_as_uint(ptx::ex2(a.y));
        }
        if (m == 0) {
          ptx::tmem_wait_ld();
          ptx::tc_fence_before();
          ptx::mbar_arrive(dp_cons);
        }
        if (masked) {
          const uint32_t see = tc::bits_between(klo, klim);
#pragma unroll
          for (int u = 0; u < 32; ++u)
            if (!(see & (1u << u))) v[u] = 0u;
        }
#pragma unroll
        for (int u = 0; u < 32; u += 2) {
          const uint64_t P = tc::pk2(v[u], v[u + 1]), g = tc::pk2(dp[u], dp[u + 1]);
          if (m == 1) sum = tc::fma2(P, g, sum);
          const float2 d = tc::unpk2(tc::mul2(P, tc::add2(g, nD[m])));
          pk[u >> 1] = ptx::pack_bf16(d.x, d.y);
        }
        if (m == 1) dl2 = tc::add2(dl2, sum);
        if (masked && one) {
#pragma unroll
          for (int u = 0; u < 16; ++u) pk[u] = 0u;
        }
        if (t > 0) {  // the previous block's product has read dS_m
          wait(&dq_done[m], (t - 1) & 1);
          ptx::tc_fence_after();
        }
        ptx::tmem_st16(tmem + cdS + m * 64 + cg * 16 + lo, pk);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&ds_ready[m]);
      }
    }
    {  // this warp's share of dlam's sum
      const float2 x = tc::unpk2(dl2);
      float v = x.x + x.y;
#pragma unroll
      for (int u = 1; u < 32; u <<= 1) v += __shfl_xor_sync(0xffffffffu, v, u);
      if (lane == 0) sRed[warp] = v;
    }
    // dQ_m = s w_m (P_m (dP - D_m)) K_m: the weight -lam of map 2 enters here
    const float f[2] = {scale, -scale * lm};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      wait(&dq_done[m], (nt - 1) & 1);
      ptx::tc_fence_after();
      uint32_t a[16];
      ptx::tmem_ld16(tmem + cdQ + m * 64 + cg * 16 + lo, a);
      ptx::tmem_wait_ld();
      stage16(sm + L::oStage + m * kSlab, qd * 32 + lane, cg * 16, a, f[m]);
    }
    // (the stages are free: every block has been read)
    ptx::fence_proxy_async_smem();
    tc::named_sync(1, kCW * 32);
    if (threadIdx.x == 0) {
      for (int m = 0; m < 2; ++m) ptx::tma_store_3d(&tmdQ, sm + L::oStage + m * kSlab, 0, rb * BW, 2 * bh + m);
      ptx::bulk_commit_group();
      ptx::bulk_wait_group_read0();
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  teardown(abort_flag, settled, started, held_full, k_full, v_full);
  if (warp == kCW + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) {
    float v = 0.f;
    for (int u = 0; u < kCW; ++u) v += sRed[u];
    partial[static_cast<int64_t>(bh) * nrb + rb] = v;
  }
}

// --------------------------------------------------------------- column pass
// TMEM columns: S^T (S_1, then S_2), dP^T, dK_1, dK_2, dV.  W^T and dS_1^T (bf16 pairs) are
// written over dP^T by the warp that read it: of 16 queries' columns, W^T takes the first 8.  dS_2^T goes
// through shared memory, so that S_1 of the next block can be formed while this one's are read.
// Order of the products: S_1(t+1) while the compute warps finish block t; dV(t), dK_1(t),
// S_2(t+1), dP(t+1), dK_2(t) once they have, so the chain from one block's operands to the
// next's is dV, dK_1, S_2, dP and the last steps of the CUDA cores.  (dP(t+1) overwrites the
// operands of dV(t), dK_1(t): products of one thread run in order.)
template <int DV, bool WIN>
__device__ __forceinline__ void col_pass(const Args& p, int block, const CUtensorMap& tmQ, const CUtensorMap& tmdO,
                                         const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmdK,
                                         const CUtensorMap& tmdV) {
  using L = Lay<DV, true>;
  constexpr int D = DV / 2;
  constexpr uint32_t cS = 0, cX = 128, cdK = 256, cdV = 384;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* held_full = bars;
  uint64_t* a_full = bars + 1;       // [NS] Q_1, dO of the stage loaded
  uint64_t* b_full = a_full + NS;    // [NS] Q_2
  uint64_t* a_empty = b_full + NS;   // [NS] dV, dK_1 of the block done
  uint64_t* b_empty = a_empty + NS;  // [NS] dK_2 done
  uint64_t* s_full = b_empty + NS;   // [2] S_m^T in TMEM
  uint64_t* s_cons = s_full + 2;     // [2] ... in the compute registers
  uint64_t* dp_full = s_cons + 2;    // dP^T in TMEM (and the previous block's dV, dK_1 done)
  uint64_t* ready = dp_full + 1;     // W^T, dS_1^T in TMEM, dS_2^T in shared memory
  uint64_t* out_done = ready + 1;    // all products of the block done
  uint64_t* st_full = out_done + 1;  // the block's statistics in shared memory
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(st_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* settled = reinterpret_cast<uint64_t*>(sm + L::oBar + 224);  // see teardown()
  volatile int* started = reinterpret_cast<volatile int*>(settled + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float *lam = p.lam, *stats = p.stats;
  const int N = p.N, H = p.H, nb = p.nb, causal = p.causal, G = p.G, BHkv = p.BHkv;
  const float scale = p.scale, c = p.c;
  const Band& bd = p.bd;
  const tc::Order ord = tc::grid_order_at(block, BHkv, nb);
  const int kvh = ord.bh;          // key/value slice; its query heads are kvh * G + h, h < G
  const int kb = ord.k;            // first key blocks have the most query blocks: first
  const int i0 = causal ? kb : 0;  // first query block that sees this key block
  const int ntile = ((WIN && causal) ? bd.key_hi(kvh, min(kb * BW + BW - 1, N - 1)) / BW + 1 : nb) - i0;
  const int nt = G * ntile;        // tile t = (h, i - i0)

  auto load_a = [&](int t) {  // Q_1, dO
    const int s = t % NS, h = t / ntile, i = i0 + t - h * ntile;
    uint8_t* st = sm + L::oStage + s * L::kBlock;
    ptx::mbar_expect_tx(&a_full[s], kSlab + L::kV);
    ptx::tma_load_3d(st, &tmQ, &a_full[s], 0, i * BW, 2 * (kvh * G + h));
    for (int u = 0; u < DV / 64; ++u)
      ptx::tma_load_3d(st + (2 + u) * kSlab, &tmdO, &a_full[s], u * 64, i * BW, kvh * G + h);
  };
  auto load_b = [&](int t) {  // Q_2
    const int s = t % NS, h = t / ntile, i = i0 + t - h * ntile;
    ptx::mbar_expect_tx(&b_full[s], kSlab);
    ptx::tma_load_3d(sm + L::oStage + s * L::kBlock + kSlab, &tmQ, &b_full[s], 0, i * BW, 2 * (kvh * G + h) + 1);
  };
  // As in the row pass: the first loads before the others are let in.
  if (threadIdx.x == kCW * 32) {
    ptx::mbar_init(held_full, 1);
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(&a_full[s], 1);
      ptx::mbar_init(&b_full[s], 1);
      ptx::mbar_init(&a_empty[s], 1);
      ptx::mbar_init(&b_empty[s], 1);
    }
    for (int m = 0; m < 2; ++m) {
      ptx::mbar_init(&s_full[m], 1);
      ptx::mbar_init(&s_cons[m], kCW * 32);
    }
    ptx::mbar_init(dp_full, 1);
    ptx::mbar_init(ready, kCW * 32);
    ptx::mbar_init(out_done, 1);
    ptx::mbar_init(st_full, 32);
    ptx::mbar_init(settled, 1);
    init_abort(sm, abort_flag);
    started[0] = started[1] = *abort_flag ? 0 : min(nt, NS);
    ptx::fence_mbar_init();
    if (!*abort_flag) {
      ptx::mbar_expect_tx(held_full, L::kBlock);
      for (int m = 0; m < 2; ++m) ptx::tma_load_3d(sm + m * kSlab, &tmK, held_full, 0, kb * BW, 2 * kvh + m);
      for (int u = 0; u < DV / 64; ++u)
        ptx::tma_load_3d(sm + (2 + u) * kSlab, &tmV, held_full, u * 64, kb * BW, kvh);
      for (int t = 0; t < nt && t < NS; ++t) {
        load_a(t);
        load_b(t);
      }
    }
  }
  if (warp == kCW + 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const ptx::BoundedWait wait{abort_flag, &g_err};
  const bool ok = *abort_flag == 0;

  if (warp >= kCW) ptx::setmaxnreg_dec<kColRegsOther>();
  if (warp == kCW) {
    // ------------------------------------------------------------ TMA loads
    if (lane == 0 && ok) {
      for (int t = NS; t < nt; ++t) {
        const int s = t % NS, ph = ((t / NS) - 1) & 1;
        if (!wait(&a_empty[s], ph)) break;
        load_a(t);
        started[0] = t + 1;
        if (!wait(&b_empty[s], ph)) break;
        load_b(t);
        started[1] = t + 1;
      }
    }
  } else if (warp == kCW + 1) {
    // ------------------------------------------------------------- products
    if (ok) {
      constexpr uint32_t idS = ptx::idesc_bf16(BW, BW, 0, 0);
      constexpr uint32_t idV = ptx::idesc_bf16(BW, DV, 0, 1);
      constexpr uint32_t idK = ptx::idesc_bf16(BW, 64, 0, 1);
      const uint32_t sH = ptx::smem_u32(sm), sS = ptx::smem_u32(sm + L::oStage);
      uint64_t dHk = tc::kmajor_desc(sH, BW, 0);   // held block, rows = M
      uint64_t dSk = tc::kmajor_desc(sS, BW, 0);   // streamed block, rows = N
      uint64_t dSm = tc::mnmajor_desc(sS, BW, 0);  // streamed block, rows = K
      uint64_t dTk = tc::kmajor_desc(ptx::smem_u32(sm + L::oT), BW, 0);  // dS_2^T
      auto S = [&](int m, int t) {
        const uint32_t so = static_cast<uint32_t>((t % NS) * L::kBlock + m * kSlab);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_ss_e(tmem + cS, tc::desc_add(dHk, m * kSlab + tc::kmajor_off(BW, k)),
                        tc::desc_add(dSk, so + tc::kmajor_off(BW, k)), idS, k > 0);
        ptx::mma_commit_e(&s_full[m]);
      };
      auto dP = [&](int t) {
        const uint32_t so = static_cast<uint32_t>((t % NS) * L::kBlock + 2 * kSlab);
#pragma unroll
        for (int k = 0; k < DV / 16; ++k)
          ptx::mma_ss_e(tmem + cX, tc::desc_add(dHk, 2 * kSlab + tc::kmajor_off(BW, k)),
                        tc::desc_add(dSk, so + tc::kmajor_off(BW, k)), idS, k > 0);
        ptx::mma_commit_e(dp_full);
      };
      wait(held_full, 0);
      wait(&a_full[0], 0);
      ptx::tc_fence_after();
      S(0, 0);
      dP(0);
      wait(&s_cons[0], 0);
      wait(&b_full[0], 0);
      ptx::tc_fence_after();
      S(1, 0);
      for (int t = 0; t < nt; ++t) {
        const int s1 = (t + 1) % NS, ph1 = ((t + 1) / NS) & 1;
        const uint32_t so = static_cast<uint32_t>((t % NS) * L::kBlock);
        // The steps' descriptors are formed in the loop, one add each: hoisted out of it they
        // would take more registers than this warp keeps.
        asm volatile("" : "+l"(dHk), "+l"(dSk), "+l"(dSm), "+l"(dTk));
        if (t + 1 < nt) {
          wait(&s_cons[1], t & 1);
          wait(&a_full[s1], ph1);
          ptx::tc_fence_after();
          S(0, t + 1);
        }
        wait(ready, t & 1);
        ptx::tc_fence_after();
#pragma unroll
        for (int k = 0; k < BW / 16; ++k)
          ptx::mma_ts_e(tmem + cdV, tmem + cX + k * 16,
                        tc::desc_add(dSm, so + 2 * kSlab + 2048 * k), idV, (t > 0 || k > 0) ? 1u : 0u);
#pragma unroll
        for (int k = 0; k < BW / 16; ++k)
          ptx::mma_ts_e(tmem + cdK, tmem + cX + k * 16 + 8, tc::desc_add(dSm, so + 2048 * k), idK,
                        (t > 0 || k > 0) ? 1u : 0u);
        ptx::mma_commit_e(&a_empty[t % NS]);
        if (t + 1 < nt) {
          wait(&s_cons[0], (t + 1) & 1);
          wait(&b_full[s1], ph1);
          ptx::tc_fence_after();
          S(1, t + 1);
          dP(t + 1);
        }
#pragma unroll
        for (int k = 0; k < BW / 16; ++k)
          ptx::mma_ss_e(tmem + cdK + 64, tc::desc_add(dTk, tc::kmajor_off(BW, k)),
                        tc::desc_add(dSm, so + kSlab + 2048 * k), idK, (t > 0 || k > 0) ? 1u : 0u);
        ptx::mma_commit_e(&b_empty[t % NS]);
        ptx::mma_commit_e(out_done);
      }
    }
  } else if (warp == kCW + 2) {
    // -------------------- the streamed queries' statistics (four planes) into shared memory:
    // loaded a block ahead, written once the compute warps are done with the previous block
    float4* dst = reinterpret_cast<float4*>(sm + L::oStat);
    auto src = [&](int t) {
      const int h = t / ntile, i = i0 + t - h * ntile;
      return reinterpret_cast<const float4*>(stats + ((static_cast<int64_t>(kvh) * G + h) * nb + i) * (kPlanes * BW));
    };
    float4 v[4];
    ptx::grid_dependency_wait();  // the statistics are the preparation's
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = src(0)[32 * u + lane];
    for (int t = 0; t < nt; ++t) {
      if (t > 0) wait(ready, (t - 1) & 1);
#pragma unroll
      for (int u = 0; u < 4; ++u) dst[32 * u + lane] = v[u];
      ptx::mbar_arrive(st_full);
      const float4* next = src(min(t + 1, nt - 1));
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = next[32 * u + lane];
    }
  } else if (warp < kCW) {
    ptx::setmaxnreg_inc<kColRegs>();
    // ----------------------------------- compute: a key row, 32 queries of a block
    const int qd = warp & 3, cg = warp >> 2;
    const uint32_t lo = static_cast<uint32_t>(qd * 32) << 16;
    const int r = qd * 32 + lane, key = kb * BW + r;
    const int c0 = cg * kC;
    const uint64_t c2 = tc::pk2f(c, c);
    const int khi = (WIN && causal) ? bd.key_hi(kvh, key) : 0;  // the key's last query
    const int khi_first = __shfl_sync(0xffffffffu, khi, 0);     // (they grow with the key)
    const uint32_t sT = ptx::smem_u32(sm + L::oT) + static_cast<uint32_t>((c0 >> 6) * kSlab);
    const float* sSt = reinterpret_cast<const float*>(sm + L::oStat) + c0;
    int t = 0;
    for (int h = 0; h < G; ++h) {
      const int64_t bh = static_cast<int64_t>(kvh) * G + h;
      const float wl = -lam[bh % H];
      const uint64_t w2 = tc::pk2f(wl, wl);
      for (int i = i0; i < i0 + ntile; ++i, ++t) {
        wait(st_full, t & 1);
        // Some of the warp's 32 keys x 32 queries are not visible: queries before the last key,
        // past the first key's last query, past N, or keys past N.
        const int q0 = i * BW + c0, k0 = kb * BW + qd * 32;
        const bool masked = (causal ? q0 < k0 + 31 || (WIN && q0 + kC - 1 > khi_first) : k0 + 32 > N) || q0 + kC > N;
        auto probs = [&](auto mk, int m, uint32_t (&v)[32]) {
          wait(&s_full[m], t & 1);
          ptx::tc_fence_after();
          ptx::tmem_ld32(tmem + cS + c0 + lo, v);
          ptx::tmem_wait_ld();
          ptx::tc_fence_before();
          ptx::mbar_arrive(&s_cons[m]);
          // queries u of the block's 32 the key is seen by: from .. to
          const int from = causal ? key - i * BW - c0 : (key < N ? 0 : kC);
          const int to = min((WIN && causal ? khi : N - 1), N - 1) - i * BW - c0;
          const uint32_t see = tc::bits_between(from, to);
#pragma unroll
          for (int u = 0; u < kC; u += 4) {
            const float4 L = *reinterpret_cast<const float4*>(sSt + m * BW + u);
            const float2 a = tc::unpk2(tc::fma2(tc::pk2(v[u], v[u + 1]), c2, tc::pk2f(L.x, L.y)));
            const float2 b = tc::unpk2(tc::fma2(tc::pk2(v[u + 2], v[u + 3]), c2, tc::pk2f(L.z, L.w)));
            float p[4] = {ptx::ex2(a.x), ptx::ex2(a.y), ptx::ex2(b.x), ptx::ex2(b.y)};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if constexpr (decltype(mk)::value)
                if (!(see & (1u << (u + x)))) p[x] = 0.f;
              v[u + x] = __float_as_uint(p[x]);
            }
          }
        };
        auto block = [&](auto mk) {
          uint32_t p1[32], p2[32];
          probs(mk, 0, p1);
          probs(mk, 1, p2);
          wait(dp_full, t & 1);
          ptx::tc_fence_after();
          if (t > 0) wait(out_done, (t - 1) & 1);  // dS_2's tile has been read
#pragma unroll
          for (int x = 0; x < 2; ++x) {  // 16 queries at a time: the maps' P hold 64 registers
            uint32_t pw[8], d1[8], d2[8];
#pragma unroll
            for (int z = 0; z < 16; z += 8) {
              uint32_t g[8];
              ptx::tmem_ld8(tmem + cX + c0 + 16 * x + z + lo, g);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 8; u += 4) {
                const int q = 16 * x + z + u;
                const float4 D1 = *reinterpret_cast<const float4*>(sSt + 2 * BW + q);
                const float4 D2 = *reinterpret_cast<const float4*>(sSt + 3 * BW + q);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int e = q + 2 * y, o = (z + u + 2 * y) >> 1;
                  const uint64_t dp = tc::pk2(g[u + 2 * y], g[u + 2 * y + 1]);
                  const uint64_t n1 = y == 0 ? tc::pk2f(D1.x, D1.y) : tc::pk2f(D1.z, D1.w);
                  const uint64_t n2 = y == 0 ? tc::pk2f(D2.x, D2.y) : tc::pk2f(D2.z, D2.w);
                  const uint64_t P1 = tc::pk2(p1[e], p1[e + 1]), P2 = tc::pk2(p2[e], p2[e + 1]);
                  float2 a = tc::unpk2(tc::mul2(P1, tc::add2(dp, n1)));      // P_1 (dP - D_1)
                  float2 b = tc::unpk2(tc::mul2(P2, tc::fma2(dp, w2, n2)));  // -lam P_2 (dP - D_2)
                  const float2 w = tc::unpk2(tc::fma2(P2, w2, P1));
                  if constexpr (decltype(mk)::value) {  // rows with one visible key
                    const float2 d = tc::unpk2(n1);
                    if (d.x == -INFINITY) a.x = b.x = 0.f;
                    if (d.y == -INFINITY) a.y = b.y = 0.f;
                  }
                  pw[o] = ptx::pack_bf16(w.x, w.y);
                  d1[o] = ptx::pack_bf16(a.x, a.y);
                  d2[o] = ptx::pack_bf16(b.x, b.y);
                }
              }
            }
            // W over the 8 columns' worth of dP just read, dS_1 over the next 8
            ptx::tmem_st8(tmem + cX + c0 + 16 * x + lo, pw);
            ptx::tmem_st8(tmem + cX + c0 + 16 * x + 8 + lo, d1);
#pragma unroll
            for (int y = 0; y < 2; ++y)
              st_shared4(sT + tc::sw128(r, ((c0 & 63) >> 3) + 2 * x + y), &d2[4 * y]);
          }
        };
        if (masked)
          block(std::true_type{});
        else
          block(std::false_type{});
        ptx::fence_proxy_async_smem();
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ready);
      }
    }
    wait(out_done, (nt - 1) & 1);
    ptx::tc_fence_after();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t a[16];
      ptx::tmem_ld16(tmem + cdK + m * 64 + cg * 16 + lo, a);
      ptx::tmem_wait_ld();
      stage16(sm + L::oStage + m * kSlab, r, cg * 16, a, scale);
    }
    constexpr int VG = DV / 4;  // dV columns per thread
#pragma unroll
    for (int u = 0; u < VG / 16; ++u) {
      uint32_t a[16];
      ptx::tmem_ld16(tmem + cdV + cg * VG + u * 16 + lo, a);
      ptx::tmem_wait_ld();
      stage16(sm + L::oStage + 2 * kSlab, r, cg * VG + u * 16, a, 1.f);
    }
    // (the stages are free: every block has been read)
    ptx::fence_proxy_async_smem();
    tc::named_sync(1, kCW * 32);
    if (threadIdx.x == 0) {
      for (int m = 0; m < 2; ++m) ptx::tma_store_3d(&tmdK, sm + L::oStage + m * kSlab, 0, kb * BW, 2 * kvh + m);
      for (int u = 0; u < DV / 64; ++u)
        ptx::tma_store_3d(&tmdV, sm + L::oStage + (2 + u) * kSlab, u * 64, kb * BW, kvh);
      ptx::bulk_commit_group();
      ptx::bulk_wait_group_read0();
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  teardown(abort_flag, settled, started, held_full, a_full, b_full);
  if (warp == kCW + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Both passes in one launch: they read the same statistics and nothing of one another's, so the
// row pass's blocks fill the SMs that the column pass's last ones leave, and the other way round
// for short sequences.  The column pass's blocks, the longer ones, come first.
template <int DV, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
               const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ CUtensorMap tmdQ, const __grid_constant__ CUtensorMap tmdK,
               const __grid_constant__ CUtensorMap tmdV, const __grid_constant__ Args p) {
  ptx::grid_dependency_launch();
  const int ncol = p.nb * p.BHkv, x = static_cast<int>(blockIdx.x);
  if (x < ncol)
    col_pass<DV, WIN>(p, x, tmQ, tmdO, tmK, tmV, tmdK, tmdV);
  else
    row_pass<DV, WIN>(p, x - ncol, tmQ, tmdO, tmK, tmV, tmdQ);
}

template <int N>
__device__ __forceinline__ void load_words(const __nv_bfloat16* p, uint32_t (&x)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
}

// The row statistics both passes read, kPlanes rows of 128 per block of queries (zeros past N):
// -L_1 log2 e, -L_2 log2 e, -D_1, lam D_2, -D_2.  16 threads per row, 16 rows of a head per block.
template <int DV>
__global__ void __launch_bounds__(256)
    prep_kernel(const __nv_bfloat16* __restrict__ O, const __nv_bfloat16* __restrict__ O2,
                const __nv_bfloat16* __restrict__ dO, const float* __restrict__ lse, const float* __restrict__ lam,
                float* __restrict__ stats, int64_t N, unsigned per_head, unsigned H, int causal, Band bd) {
  constexpr int W = DV / 16;  // columns per thread
  ptx::grid_dependency_launch();
  const unsigned bh = blockIdx.x / per_head, blk = blockIdx.x - bh * per_head;
  const int row = static_cast<int>(blk * 16 + (threadIdx.x >> 4)), part = static_cast<int>(threadIdx.x & 15);
  const bool live = row < N;
  float d = 0.f, d2 = 0.f;
  if (live) {
    const int64_t off = (bh * N + row) * DV + part * W;
    uint32_t g[W / 2], o[W / 2], o2[W / 2];
    load_words<W / 2>(dO + off, g);
    load_words<W / 2>(O + off, o);
    load_words<W / 2>(O2 + off, o2);
#pragma unroll
    for (int e = 0; e < W / 2; ++e) {
      const float x = tc::bf16_lo(g[e]), y = tc::bf16_hi(g[e]);
      d = fmaf(x, tc::bf16_lo(o[e]), fmaf(y, tc::bf16_hi(o[e]), d));
      d2 = fmaf(x, tc::bf16_lo(o2[e]), fmaf(y, tc::bf16_hi(o2[e]), d2));
    }
  }
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) {
    d += __shfl_xor_sync(0xffffffffu, d, x);
    d2 += __shfl_xor_sync(0xffffffffu, d2, x);
  }
  if (part < kPlanes) {
    float v = 0.f;
    if (live) {
      const float lm = lam[bh % H];
      const bool one = diff_one_key(bd, causal, bh, row);
      v = part < 2 ? -lse[(2 * static_cast<int64_t>(bh) + part) * N + row] * kLog2e
          : part == 2 ? -diff_mark_D(fmaf(lm, d2, d), one)
          : part == 3 ? lm * d2
                      : -diff_mark_D(d2, one);
    }
    stats[(static_cast<int64_t>(bh) * (per_head / 8) + row / BW) * (kPlanes * BW) + part * BW + row % BW] = v;
  }
}

int64_t blocks(int64_t N) { return (N + BW - 1) / BW; }

template <int DV>
cudaError_t run(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, const void* O,
                const void* O2, const void* dO, const float* lse, void* dQ, void* dK, void* dV, float* dlam, void* ws,
                cudaStream_t st) {
  constexpr int D = DV / 2;
  const int64_t N = p.N, BH = p.BH;
  const int64_t Np = blocks(N) * BW;
  float* stats = static_cast<float*>(ws);          // [BH][blocks][kPlanes][BW]
  float* partial = stats + BH * kPlanes * Np;      // [BH][blocks]
  alignas(64) CUtensorMap k, v, q, g, mdq, mdk, mdv;
  if (!make_tmap_bf16(&q, Q, N, D, 2 * BH, BW) || !make_tmap_bf16(&g, dO, N, DV, BH, BW) ||
      !make_tmap_bf16(&k, K, N, D, 2 * p.BHkv, BW) || !make_tmap_bf16(&v, V, N, DV, p.BHkv, BW) ||
      !make_tmap_bf16(&mdq, dQ, N, D, 2 * BH, BW) || !make_tmap_bf16(&mdk, dK, N, D, 2 * p.BHkv, BW) ||
      !make_tmap_bf16(&mdv, dV, N, DV, p.BHkv, BW))
    return cudaErrorInvalidValue;
  const int64_t per_head = Np / 16;
  prep_kernel<DV><<<static_cast<unsigned>(BH * per_head), 256, 0, st>>>(
      static_cast<const __nv_bfloat16*>(O), static_cast<const __nv_bfloat16*>(O2),
      static_cast<const __nv_bfloat16*>(dO), lse, lam, stats, N, static_cast<unsigned>(per_head),
      static_cast<unsigned>(p.H), p.causal, make_band(p, eff_window(p), false));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int nb = static_cast<int>(blocks(N));
  const Args args{lam,      stats,  partial, static_cast<int>(N), static_cast<int>(p.H), nb, static_cast<int>(p.BHkv),
                  p.scale,  p.scale * kLog2e, p.causal, make_band(p, eff_window_tc(p), true), p.group};
  auto kern = banded(p) ? bwd_kernel<DV, true> : bwd_kernel<DV, false>;
  constexpr int smem = Lay<DV, true>::bytes;
  static_assert(smem >= Lay<DV, false>::bytes, "one launch, one size");
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
  e = launch_behind(kern, nb * (BH + p.BHkv), kThreads, smem, st, q, g, k, v, mdq, mdk, mdv, args);
  if (e != cudaSuccess) return e;
  return diff_reduce_dlam(partial, dlam, p.B, p.H, nb, st);
}

}  // namespace

size_t tc_diff_bwd_bytes(int64_t BH, int64_t N) {
  return static_cast<size_t>(BH) * blocks(N) * (kPlanes * BW + 1) * sizeof(float);
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
