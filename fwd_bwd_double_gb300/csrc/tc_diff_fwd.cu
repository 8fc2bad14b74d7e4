// Differential attention forward, bf16, on the tensor cores.
//
//   A_m = softmax(s Q_m K_m^T + mask), m = 1, 2;   O = (A_1 - lam A_2) V,  O_2 = A_2 V.
// One CTA owns 128 query rows of a head and streams blocks of 128 keys (K_1, K_2 and V, so
// that V is read once for both maps).  Per block and map
//   S_m = Q_m K_m^T          A and B from shared memory, accumulator in TMEM
//   P_m = 2^(S_m c - M_m c)  online softmax, one query row per thread, bf16 over S_m's columns
//   O_m += P_m V             A = P_m from TMEM, B = V (MN-major)
// The two maps take turns: while four warps exponentiate S_1, the tensor cores run P_2 V and
// the next S_2, and the other way round (six products of 128 x 128 x 64 a block).  TMEM is
// full: S_1, S_2 (128 columns each, P_m over the first half of S_m) and O_1, O_2 (2d each).
// A CTA takes row blocks one after another, heaviest first, each next one by cluster launch
// control: its loads and first products run under this one's epilogue, and the uneven blocks
// spread over the SMs as separate CTAs would (a CTA per row block: 143 against 130 us at B4 H6
// N4096, 98 against 88 us for a window of 1024 in 8000; row blocks dealt out in a fixed order:
// 241 against 166 us at B1 H2 N16384).
// The MMA warp issues S_m of block j + 1 behind P_m V of block j; products of one thread
// run in order, so S_m overwrites P_m only once it has been read.  P_m V starts on the first
// 64 keys' P while the rest is exponentiated.
//
// The reference maximum M_m moves only when a row's maximum passes it so far that the new largest P
// would be above a quarter of the row's sum so far (or above 2^8; P_m <= 2^8, l and O_m in fp32):
// most blocks then rescale nothing, and a weight that makes up more than a fifth of its row is 1
// exactly, so its product is not rounded.  That matters where attention is nearly one-hot (keys with
// a shared mean of norm 40, queries near copies of keys): dQ within 1.89e-2 and 1.97e-2 of 64-bit
// values, as with a maximum that always moves (1.88e-2, 1.96e-2); 2.07e-2 and 2.10e-2 at 2^8 alone.
// B4 H6 N8192: 447 us, 563 if it always moves, 445 at 2^8 alone; H48 N8000, window 1024: 290, 333, 282.
// P is rounded to bf16 for its product; the sums l are of the unrounded fp32 values.
#include <cuda_bf16.h>

#include <type_traits>

#include "diff.h"
#include "handover.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace fbd {
namespace {

__device__ unsigned int g_err = 0;

constexpr int BM = 128, BN = 128;
constexpr int NS = 2;
// Warps 0-3: map 1, 4-7: map 2, 8: TMA, 9: MMA.  384 threads launched with 168 registers; the
// softmax warps (a row of 128 scores each thread) take 208, the third warpgroup's keep 80:
// 256 * 208 + 128 * 80 <= 384 * 168.
constexpr int kThreads = 384;
constexpr int kRegs = 208, kRegsOther = 80;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 256.f;  // the largest P
constexpr float kShare = .25f;   // ... and its share of the row's sum so far, where it is above 1

template <int D>
struct Lay {
  static constexpr int DV = 2 * D;
  static constexpr int kQ = BM * 128;         // a map's tile: 64 columns (d = 32: the rest zero-filled)
  static constexpr int kV = BN * DV * 2;
  static constexpr int kStage = 2 * kQ + kV;  // K_1, K_2, V
  static constexpr int oStage = 2 * kQ;
  static constexpr int oOut = oStage + NS * kStage;  // O, O_2 on their way out
  static constexpr int oInv = oOut + 2 * BM * DV * 2;  // 1 / l_2 of every row
  static constexpr int oBar = oInv + BM * 4;
  static constexpr int oClc = oBar + 192;
  static constexpr int bytes = oClc + 16;
  static constexpr uint32_t cS = 0, cO = 2 * BN;  // S_m at cS + m BN, O_m at cO + m DV
};
static_assert(Lay<64>::bytes <= 232448, "shared memory");

// The primitives of a role in the hand-over to the next row block (handover.h): a whole warp's, or
// one thread's.
template <bool WARP>
struct Role {
  ptx::BoundedWait wait;
  uint64_t *known, *free;
  const void* answer_at;
  int lane;
  __device__ __forceinline__ bool wait_free(int n) const { return wait(free, n & 1); }
  __device__ __forceinline__ bool wait_known(int n) const {
    const bool ok = wait(known, n & 1);
    return WARP ? __all_sync(0xffffffffu, ok) : ok;
  }
  __device__ __forceinline__ void request() const {
    ptx::mbar_expect_tx(known, 16);
    ptx::clc_request(const_cast<void*>(answer_at), known);
  }
  __device__ __forceinline__ int answer() const {
    const int x = ptx::clc_block(answer_at);
    ptx::fence_proxy_async_smem();
    return x;
  }
  __device__ __forceinline__ void taken() const {
    if (WARP) __syncwarp();
    if (!WARP || lane == 0) ptx::mbar_arrive(free);
  }
};

// WIN: a banded causal mask is in force (window and/or document bounds).
template <int D, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
               const __grid_constant__ CUtensorMap tmO2, const float* __restrict__ lam, float* __restrict__ lse,
               int with_O2, int N, int H, int nrb, int BH, float scale,
               float c, int causal, Band bd, int G) {
  using L = Lay<D>;
  constexpr int DV = L::DV;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;            // [NS]
  uint64_t* v_full = k_full + NS;         // [NS]
  uint64_t* empty = v_full + NS;          // [NS] both maps' P V of the stage done
  uint64_t* s_full = empty + NS;          // [2] S_m in TMEM (and the previous P_m V done)
  uint64_t* p_half = s_full + 2;          // [2] P_m of the first 64 keys in TMEM, O_m rescaled
  uint64_t* p_ready = p_half + 2;         // [2] of all keys
  uint64_t* o_full = p_ready + 2;
  uint64_t* o_empty = o_full + 1;         // O_1, O_2 read by the epilogue
  uint64_t* q_empty = o_empty + 1;        // the row block's last S_1, S_2 done
  uint64_t* x_full = q_empty + 1;         // the next row block is known
  uint64_t* x_empty = x_full + 1;         // ... and every role has taken it
  uint64_t* settled = x_empty + 1;        // after a wait that gave up: the products in flight done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(settled + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* started = abort_flag + 1;  // Q loads, key blocks' loads, requests (the TMA thread's)
  float* sInv = reinterpret_cast<float*>(sm + L::oInv);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // A row block: its slices, and the key blocks j0 + j, j < nkv, it sees.
  struct Item {
    int bh, kvh, rb, j0, nkv;
  };
  auto item_at = [&](int x) {
    const tc::Order ord = tc::grid_order_at(x, BH, nrb);
    Item it;
    it.bh = ord.bh, it.kvh = ord.bh / G;
    it.rb = nrb - 1 - ord.k;  // heaviest row blocks first
    it.j0 = (WIN && causal) ? bd.row_lo(it.bh, it.rb * BM) / BN : 0;
    it.nkv = (causal ? it.rb + 1 : nrb) - it.j0;
    return it;
  };
  // A role's side of the hand-over to the next row block, for a whole warp or for one thread of it.
  auto role = [&](const ptx::BoundedWait& w, auto whole) {
    return Role<decltype(whole)::value>{w, x_full, x_empty, sm + L::oClc, lane};
  };

  auto load_q = [&](const Item& it) {
    ptx::mbar_expect_tx(q_full, 2 * L::kQ);
    for (int m = 0; m < 2; ++m) ptx::tma_load_3d(sm + m * L::kQ, &tmQ, q_full, 0, it.rb * BM, 2 * it.bh + m);
  };
  auto load = [&](const Item& it, int j, int T) {  // key block j; T: blocks so far, the ring's position
    const int s = T % NS;
    uint8_t* st = sm + L::oStage + s * L::kStage;
    ptx::mbar_expect_tx(&k_full[s], 2 * L::kQ);
    for (int m = 0; m < 2; ++m) ptx::tma_load_3d(st + m * L::kQ, &tmK, &k_full[s], 0, (it.j0 + j) * BN, 2 * it.kvh + m);
    ptx::mbar_expect_tx(&v_full[s], L::kV);
    for (int u = 0; u < DV / 64; ++u)
      ptx::tma_load_3d(st + 2 * L::kQ + u * BN * 128, &tmV, &v_full[s], u * 64, (it.j0 + j) * BN, it.kvh);
  };
  // The TMA thread sets the barriers up and starts the first loads before the others are let in
  // (the TMEM allocation alone takes about a thousand cycles).
  if (threadIdx.x == 8 * 32) {
    ptx::mbar_init(q_full, 1);
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(&k_full[s], 1);
      ptx::mbar_init(&v_full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int m = 0; m < 2; ++m) {
      ptx::mbar_init(&s_full[m], 1);
      ptx::mbar_init(&p_half[m], 128);
      ptx::mbar_init(&p_ready[m], 128);
    }
    ptx::mbar_init(o_full, 1);
    ptx::mbar_init(o_empty, 256);
    ptx::mbar_init(q_empty, 1);
    ptx::mbar_init(x_full, 1);
    ptx::mbar_init(x_empty, 10);  // the TMA thread, the MMA warp, eight softmax warps
    ptx::mbar_init(settled, 1);
    started[0] = started[1] = started[2] = 0;
    *abort_flag = (ptx::smem_u32(sm) & 1023u) ? 1 : 0;  // the swizzled tiles need 1024-byte alignment
    if (*abort_flag) atomicOr(&g_err, FBD_ERR_TIMEOUT);
    ptx::fence_mbar_init();
    if (!*abort_flag) {
      const Item it = item_at(static_cast<int>(blockIdx.x));
      load_q(it);
      for (int j = 0; j < it.nkv && j < NS; ++j) load(it, j, j);
    }
  }
  if (warp == 9) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const ptx::BoundedWait wait{abort_flag, &g_err};
  const bool ok = *abort_flag == 0;

  if (warp >= 8) ptx::setmaxnreg_dec<kRegsOther>();
  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && ok) {
      const auto me = role(wait, std::false_type{});
      int T = 0, nq = 1, asked = 0;
      for (int x = static_cast<int>(blockIdx.x), n = 0; x >= 0; ++n) {
        const Item it = item_at(x);
        if (n > 0) {
          if (!wait(q_empty, (n - 1) & 1)) break;
          load_q(it);
          ++nq;
        }
        int j = 0;
        for (; j < it.nkv; ++j, ++T) {
          if (n == 0 && j < NS) continue;  // (issued above)
          if (T >= NS && !wait(&empty[T % NS], ((T / NS) - 1) & 1)) break;
          load(it, j, T);
        }
        // Ask for the next row block now, a few key blocks before this one ends: asked for sooner,
        // it would wait here while other SMs run out.
        if (j < it.nkv || !handover::ask(me, n)) break;
        ++asked;
        x = handover::take(me, n);
      }
      started[0] = nq, started[1] = T, started[2] = asked;
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------- MMA issuer
    if (ok) {
      constexpr uint32_t idS = ptx::idesc_bf16(BM, BN, 0, 0);
      constexpr uint32_t idO = ptx::idesc_bf16(BM, DV, 0, 1);
      const uint64_t dQ = tc::kmajor_desc(ptx::smem_u32(sm), BM, 0);
      const uint64_t dK = tc::kmajor_desc(ptx::smem_u32(sm + L::oStage), BN, 0);
      const uint64_t dV = tc::mnmajor_desc(ptx::smem_u32(sm + L::oStage + 2 * L::kQ), BN, 0);
      auto issue_s = [&](int m, int T) {
        const uint32_t so = static_cast<uint32_t>((T % NS) * L::kStage + m * L::kQ);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_ss_e(tmem + L::cS + m * BN, tc::desc_add(dQ, m * L::kQ + tc::kmajor_off(BM, k)),
                        tc::desc_add(dK, so + tc::kmajor_off(BN, k)), idS, k > 0 ? 1u : 0u);
        ptx::mma_commit_e(&s_full[m]);
      };
      const auto me = role(wait, std::true_type{});
      int T = 0;
      for (int x = static_cast<int>(blockIdx.x), n = 0; x >= 0; x = handover::take(me, n), ++n) {
        const int nkv = item_at(x).nkv;
        wait(q_full, n & 1);
        wait(&k_full[T % NS], (T / NS) & 1);
        ptx::tc_fence_after();
        issue_s(0, T);
        issue_s(1, T);
        if (nkv == 1) ptx::mma_commit_e(q_empty);
        for (int j = 0; j < nkv; ++j, ++T) {
          const int s = T % NS;
          const uint32_t so = static_cast<uint32_t>(s * L::kStage);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            wait(&p_half[m], T & 1);
            if (m == 0) wait(&v_full[s], (T / NS) & 1);
            if (m == 0 && j == 0 && n > 0) wait(o_empty, (n - 1) & 1);
            ptx::tc_fence_after();
#pragma unroll
            for (int k = 0; k < BN / 16; ++k) {
              if (k == BN / 32) {
                wait(&p_ready[m], T & 1);
                ptx::tc_fence_after();
              }
              ptx::mma_ts_e(tmem + L::cO + m * DV, tmem + L::cS + m * BN + k * 8, tc::desc_add(dV, so + k * 2048), idO,
                            (j > 0 || k > 0) ? 1u : 0u);
            }
            if (m == 1) ptx::mma_commit_e(&empty[s]);
            if (j + 1 < nkv) {
              if (m == 0) {
                wait(&k_full[(T + 1) % NS], ((T + 1) / NS) & 1);
                ptx::tc_fence_after();
              }
              issue_s(m, T + 1);
              if (m == 1 && j + 2 == nkv) ptx::mma_commit_e(q_empty);
            }
          }
        }
        ptx::mma_commit_e(o_full);
      }
    }
  } else if (warp < 8) {
    ptx::setmaxnreg_inc<kRegs>();
    // --------------------------- softmax of map m: thread r owns query row r
    const int m = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + L::cS + m * BN + lane_off, tO = tmem + L::cO + lane_off;
    const uint64_t c2 = tc::pk2f(c, c);
    // A row block with this thread's row's bound, the last row's, and its head's lam: looked up
    // before the last row block's epilogue (after it: 292 against 283 us at H48 N8000 for a window of 1024).
    struct Row {
      Item it;
      int lo_row, lo_last;
      float lm;
    };
    auto row_at = [&](int x) {
      Row w;
      w.it = item_at(x);
      w.lm = lam[w.it.bh % H];
      w.lo_row = (WIN && causal) ? bd.row_lo(w.it.bh, static_cast<int64_t>(w.it.rb) * BM + r) : 0;
      w.lo_last = (WIN && causal) ? bd.row_lo(w.it.bh, min(w.it.rb * BM + BM - 1, N - 1)) : 0;
      return w;
    };
    const auto me = role(wait, std::true_type{});
    int T = 0;
    Row next = row_at(static_cast<int>(blockIdx.x));
    for (int x = static_cast<int>(blockIdx.x), n = 0; x >= 0; ++n) {
      const Item it = next.it;
      const int bh = it.bh, rb = it.rb, j0 = it.j0, nkv = it.nkv, lo_row = next.lo_row, lo_last = next.lo_last;
      const float lm = next.lm;
      const int64_t row = static_cast<int64_t>(rb) * BM + r;
      float mref = -INFINITY, l = 0.f;
      for (int j = 0; j < nkv; ++j, ++T) {
        const int kb = j0 + j;
        const bool diag = causal ? kb == rb : (j == nkv - 1 && (N % BN) != 0);
        const bool low = WIN && causal && kb * BN < lo_last;
        const int klim = causal ? (WIN ? rb * BM + r - kb * BN : r) : N - 1 - kb * BN;  // last visible key
        const int klo = (WIN && causal) ? lo_row - kb * BN : 0;                         // first one
        wait(&s_full[m], T & 1);
        ptx::tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) ptx::tmem_ld32(tS + ch * 32, v[ch]);
        ptx::tmem_wait_ld();
        if (diag || low) {
          // bounds grow with the row: the warp's first row has the first last key, its last row
          // the last first one, and 32 keys between the two need no masking
          const int klim0 = __shfl_sync(0xffffffffu, klim, 0), klo31 = __shfl_sync(0xffffffffu, klo, 31);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
            if (ch * 32 + 31 > klim0 || ch * 32 < klo31) {
              // (two comparisons a score: 314 against 292 us at H48 N8000 for a window of 1024)
              const uint32_t see = tc::bits_between(klo - ch * 32, klim - ch * 32);
#pragma unroll
              for (int t = 0; t < 32; ++t)
                if (!(see & (1u << t))) v[ch][t] = __float_as_uint(-INFINITY);
            }
        }
        float mx[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
#pragma unroll
          for (int t = 0; t < 32; t += 16)
#pragma unroll
            for (int u = 0; u < 8; ++u) mx[u] = fmaxf(mx[u], fmaxf(tc::f(v[ch][t + u]), tc::f(v[ch][t + 8 + u])));
#pragma unroll
        for (int u = 1; u < 8; ++u) mx[0] = fmaxf(mx[0], mx[u]);
        // (always at the first visible key: mref = -inf)
        const bool moved = ptx::ex2((mx[0] - mref) * c) > fminf(fmaxf(kShare * l, 1.f), kSlack);
        const float mnew = moved ? mx[0] : mref;
        const float alpha = moved ? ptx::ex2((mref - mnew) * c) : 1.f;
        if (j > 0 && __any_sync(0xffffffffu, moved)) {
          const uint64_t a2 = tc::pk2f(alpha, alpha);
#pragma unroll 1
          for (int c0 = 0; c0 < DV; c0 += 16) {  // 16 columns at a time: the scores hold 128 registers
            uint32_t o[16];
            ptx::tmem_ld16(tO + m * DV + c0, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
              const float2 x = tc::unpk2(tc::mul2(tc::pk2(o[t], o[t + 1]), a2));
              o[t] = __float_as_uint(x.x);
              o[t + 1] = __float_as_uint(x.y);
            }
            ptx::tmem_st16(tO + m * DV + c0, o);
          }
        }
        l *= alpha;
        mref = mnew;
        // a row that has seen no key yet subtracts 0, not -inf: every term is 2^-inf = 0
        const float nm = mref == -INFINITY ? 0.f : -mref * c;
        const uint64_t nm2 = tc::pk2f(nm, nm);
        uint64_t rs[4] = {0, 0, 0, 0};
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int t = 0; t < 32; t += 2) {
            const float2 arg = tc::unpk2(tc::fma2(tc::pk2(v[ch][t], v[ch][t + 1]), c2, nm2));
            const float p0 = ptx::ex2(arg.x), p1 = ptx::ex2(arg.y);
            rs[(t >> 1) & 3] = tc::add2(rs[(t >> 1) & 3], tc::pk2f(p0, p1));
            pk[t >> 1] = ptx::pack_bf16(p0, p1);
          }
          ptx::tmem_st16(tS + ch * 16, pk);
          if (ch & 1) {
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(ch == 1 ? &p_half[m] : &p_ready[m]);
          }
        }
        const float2 x = tc::unpk2(tc::add2(tc::add2(rs[0], rs[1]), tc::add2(rs[2], rs[3])));
        l += x.x + x.y;
      }
      // ------------------------------------------------------------------ epilogue
      x = handover::take(me, n);
      if (x >= 0) next = row_at(x);
      const float inv = 1.f / l;
      if (row < N) lse[(2 * static_cast<int64_t>(bh) + m) * N + row] = mref * scale + logf(l);
      wait(o_full, n & 1);
      if (m == 1) sInv[r] = inv;  // (map 1 is done with the last row block's: it has taken part in this one)
      // (both maps' warps go on to the same row block, or none does: they meet at barriers in each)
      x = handover::agree(x, [](bool some) { return tc::named_all(1, 256, some); });
      ptx::tc_fence_after();
      if (m == 0 || with_O2) {
        const float w = m == 0 ? -lm * sInv[r] : inv;  // of O_2's columns
        // Through shared memory as 64-column tiles, and out by TMA: a row per thread straight to
        // memory, 16 bytes at a time, took 5.6 thousand cycles of each row block.
        uint8_t* out = sm + L::oOut + m * BM * DV * 2;
        if (r == 0) ptx::bulk_wait_group_read0();  // the last row block's has left
        tc::named_sync(2 + m, 128);
#pragma unroll
        for (int ch = 0; ch < DV / 32; ++ch) {
          uint32_t a[32], b[32];
          ptx::tmem_ld32(tO + DV + ch * 32, b);
          if (m == 0) ptx::tmem_ld32(tO + ch * 32, a);
          ptx::tmem_wait_ld();
          if (ch == DV / 32 - 1) {
            ptx::tc_fence_before();
            ptx::mbar_arrive(o_empty);
          }
          uint32_t pk[16];
#pragma unroll
          for (int t = 0; t < 32; t += 2) {
            float x0 = tc::f(b[t]) * w, x1 = tc::f(b[t + 1]) * w;
            if (m == 0) x0 = fmaf(tc::f(a[t]), inv, x0), x1 = fmaf(tc::f(a[t + 1]), inv, x1);
            pk[t >> 1] = ptx::pack_bf16(x0, x1);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(out + (ch >> 1) * BM * 128 + tc::sw128(r, (ch & 1) * 4 + u)) =
                make_uint4(pk[u * 4], pk[u * 4 + 1], pk[u * 4 + 2], pk[u * 4 + 3]);
        }
        ptx::fence_proxy_async_smem();
        tc::named_sync(2 + m, 128);
        if (r == 0) {
          for (int u = 0; u < DV / 64; ++u)
            ptx::tma_store_3d(m == 0 ? &tmO : &tmO2, out + u * BM * 128, u * 64, rb * BM, bh);
          ptx::bulk_commit_group();
        }
      } else {
        ptx::mbar_arrive(o_empty);
      }
    }
    if (r == 0) ptx::bulk_wait_group_read0();
  }

  ptx::tc_fence_before();
  __syncthreads();
  // A wait has given up: loads, an answer and products may still be on their way into this CTA's
  // shared memory and TMEM, which others get when it ends.
  if (*abort_flag != 0) {
    if (threadIdx.x == 8 * 32) {
      const int nq = started[0], T = started[1], asked = started[2];
      if (nq > 0) ptx::settle(q_full, (nq - 1) & 1);
      for (int s = 0; s < NS && s < T; ++s) {
        ptx::settle(&k_full[s], handover::last_phase(T, NS, s));
        ptx::settle(&v_full[s], handover::last_phase(T, NS, s));
      }
      if (asked > 0) ptx::settle(x_full, (asked - 1) & 1);
    }
    if (warp == 9) {
      ptx::mma_commit_e(settled);
      ptx::settle(settled, 0);
    }
  }
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, void* O, void* O2,
                   float* lse, cudaStream_t st) {
  alignas(64) CUtensorMap mq, mk, mv, mo, mo2;
  if (!make_tmap_bf16(&mq, Q, p.N, D, 2 * p.BH, BM) || !make_tmap_bf16(&mk, K, p.N, D, 2 * p.BHkv, BN) ||
      !make_tmap_bf16(&mv, V, p.N, 2 * D, p.BHkv, BN) || !make_tmap_bf16(&mo, O, p.N, 2 * D, p.BH, BM) ||
      !make_tmap_bf16(&mo2, O2 != nullptr ? O2 : O, p.N, 2 * D, p.BH, BM))
    return cudaErrorInvalidValue;
  const int nrb = static_cast<int>((p.N + BM - 1) / BM);
  auto kern = banded(p) ? fwd_kernel<D, true> : fwd_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::bytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(nrb * p.BH), kThreads, Lay<D>::bytes, st>>>(
      mq, mk, mv, mo, mo2, lam, lse, O2 != nullptr ? 1 : 0, static_cast<int>(p.N),
      static_cast<int>(p.H), nrb, static_cast<int>(p.BH), p.scale, p.scale * kLog2e, p.causal,
      make_band(p, eff_window_tc(p), false), p.group);
  return cudaGetLastError();
}

}  // namespace

cudaError_t tc_diff_fwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, void* O,
                        void* O2, float* lse, cudaStream_t st) {
  return p.d == 32 ? launch<32>(p, Q, K, V, lam, O, O2, lse, st) : launch<64>(p, Q, K, V, lam, O, O2, lse, st);
}

uint32_t tc_diff_fwd_take_error() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err, &z, sizeof(z));
  return v;
}

}  // namespace fbd
