// Attention of new tokens over a paged cache, bf16, on the tensor cores.
//
//   O = softmax(s Q K^T + mask) V over each sequence's pages
// A tile's 128 rows are tokens times the query heads that share a key/value head, so that K and V are
// loaded once for all of them.  Two tiles at once, per block of 128 keys and tile
//   S_m = Q_m K^T            A and B from shared memory, accumulator in TMEM
//   P_m = 2^(S_m c - M_m c)  online softmax, one row per thread, bf16 over S_m's columns
//   O_m += P_m V             A = P_m from TMEM, B = V (MN-major)
// The tiles take turns: while four warps exponentiate S_0, the tensor cores run P_1 V and the next S_1,
// and the other way round.  Items of more tokens than a tile holds fill two tiles that see the same
// blocks; of smaller ones both "tiles" hold the same rows and take the blocks in turn, and the two
// softmaxes are joined at the end.
//
// Pages: a block is fetched in boxes of as many keys as divide the page's (16 .. 128), one lane of the
// loading warp per box, which looks its page up; keys that the sequence does not hold, and entries
// that are no page, are coordinates outside the tensor, which read as zeros without traffic.  The lanes'
// copies are issued one after another (about 75 cycles each), so where the strides allow it a box takes all
// d columns, in groups of eight keys (group, slab of 64 columns, key: MMA operands of either major), else
// a slab of them.  Keys hidden from a row are masked in its scores.  Their values are multiplied by weights of 0, which would make
// an infinity or NaN there a NaN: in blocks that some row does not see whole, a warp makes such
// elements 0 before the product (and rows behind the last key, which may hold anything), and the
// rows that do see them add them at the end.
//
// 8192 tokens over 32192 keys, 16 heads of 128 in groups of 4: 1.27 ms, 1.49 PFLOP/s (77 % of what a plain product
// reaches), bound by the chain S -> softmax -> P V of each tile.  12 sequences of up to 1500 tokens behind up to 9000 keys,
// window 2000, 12 heads of 96 (run as 128): 142 us, 0.52 PFLOP/s, bound by the items' starts and epilogues and by
// blocks that are partly masked.
// CTAs take the stretches of paged.cuh.  The reference maximum M_m moves as in the differential forward
// (tc_diff_fwd.cu): when the new largest P would be above a quarter of the row's sum so far, or above 2^8.
#include <cuda_bf16.h>

#include "handover.h"
#include "tc_paged.cuh"

namespace fbd {
namespace paged {
namespace {

__device__ unsigned int g_err = 0;

// Warps 0-3: tile 0, 4-7: tile 1, 8: TMA, 9, 10: MMA of a tile each, 11: values that a row must not see.  384 threads
// launched with 168 registers; the softmax warps (a row of 128 scores each thread) take 208, the third
// warpgroup's keep 80: 256 * 208 + 128 * 80 <= 384 * 168.
constexpr int kThreads = 384;
constexpr int kRegs = 208, kRegsOther = 80;

template <int D>
struct Lay {
  static constexpr int kTile = BM * D * 2;       // Q tile, and a K or V entry of the ring
  static constexpr int NS = D == 64 ? 8 : 4;
  static constexpr int oRing = 2 * kTile;
  static constexpr int oOut = oRing + NS * kTile;
  static constexpr int oStat = oOut + 8 * kOut;  // [2][128] (max, sum) of the second half of an item's blocks, of two items
  static constexpr int oBar = oStat + 2 * BM * 8;
  static constexpr int oItem = oBar + 512;
  static constexpr int bytes = oItem + 8 * 64;
  static constexpr uint32_t cS = 0, cO = 2 * BN;  // S_m at cS + m BN, O_m at cO + m D
};
static_assert(Lay<128>::bytes <= 232448 && Lay<64>::bytes <= 232448, "shared memory");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const Work w, const Space sp, const Out out,
                 const __nv_bfloat16* __restrict__ Vg, int64_t vs0, int64_t vs1, int64_t vs2, int d, Pages pg,
                 float scale, float c) {
  using L = Lay<D>;
  constexpr int NS = L::NS, SL = D / 64;  // slabs of 64 columns
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;      // the item's last products with Q done
  uint64_t* s_full = bars + 2;       // [2] S_m in TMEM (and the previous P_m V done)
  uint64_t* p_half = s_full + 2;     // [2] P_m of the first 64 keys in TMEM, O_m rescaled
  uint64_t* p_ready = p_half + 2;    // [2] of all keys
  uint64_t* o_full = p_ready + 2;
  uint64_t* o_empty = o_full + 1;    // O_0, O_1 read by the epilogue
  uint64_t* x_full = o_empty + 1;    // [2] tile 1's maxima and sums are there for tile 0, in each buffer of stat
  uint64_t* settled = x_full + 2;    // after a wait that gave up: the products in flight done
  uint64_t* full = settled + 1;      // [NS]
  uint64_t* empty = full + NS;       // [NS]
  uint64_t* v_ok = empty + NS;       // [NS] values that some row does not see are finite
  uint64_t* known = v_ok + NS;       // [8] items
  uint64_t* turn = known + 8;        // [2] tile m may issue its next products
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(turn + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* started = abort_flag + 1;                                 // Q loads, ring entries (the TMA warp's)
  volatile uint8_t* hidden = reinterpret_cast<volatile uint8_t*>(started + 2);  // [2][8] of tile m's blocks: 16-key runs without a page
  volatile int* spoilt = reinterpret_cast<volatile int*>(hidden + 16);    // [8] of items: n + 1 where values were made 0
  float2* stat = reinterpret_cast<float2*>(sm + L::oStat);
  Item* items = reinterpret_cast<Item*>(sm + L::oItem);
  static_assert(sizeof(Item) == 64 && (13 + 3 * NS + 10) * 8 + 4 * 4 + 16 + 32 <= 512, "the barriers' region");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, p = blockIdx.x;
  const int gt = w.cut.gt, tq = w.cut.tile;
  ptx::grid_dependency_launch();
  if (threadIdx.x == 8 * 32) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 2);  // each tile's
    for (int m = 0; m < 2; ++m) {
      ptx::mbar_init(&s_full[m], 2);  // the products' end and the warp that issued them
      ptx::mbar_init(&p_half[m], 128);
      ptx::mbar_init(&p_ready[m], 128);
      ptx::mbar_init(&turn[m], 1);
    }
    ptx::mbar_init(o_full, 4);
    ptx::mbar_init(o_empty, 256);
    for (int s = 0; s < 2; ++s) ptx::mbar_init(&x_full[s], 128);
    ptx::mbar_init(settled, 2);
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 3);  // each tile's, and the warp's that looks at values
      ptx::mbar_init(&v_ok[s], 1);
    }
    for (int s = 0; s < 8; ++s) ptx::mbar_init(&known[s], 1), spoilt[s] = 0;
    started[0] = started[1] = 0;
    *abort_flag = (ptx::smem_u32(sm) & 1023u) ? 1 : 0;  // the swizzled tiles need 1024-byte alignment
    if (*abort_flag) atomicOr(&g_err, FBD_ERR_TIMEOUT);
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  Plan planned{};
  if (warp == 8) planned = plan(w, p);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const ptx::BoundedWait wait{abort_flag, &g_err};
  const bool ok = *abort_flag == 0;
  // Item n, once it is known (ring of 8: the loading warp is three items ahead at most, since it waits for the
  // products with Q of the one before, and those for the softmax of the one before that).
  auto item = [&](int n) -> const Item* {
    wait(&known[n & 7], (n >> 3) & 1);
    const Item* it = items + (n & 7);
    // (a whole warp goes on or leaves; warps may leave at different times, since they meet only at barriers
    // whose waits are bounded)
    return __all_sync(0xffffffffu, *abort_flag == 0 && *reinterpret_cast<const volatile int*>(&it->n) > 0) ? it : nullptr;
  };

  if (warp >= 8) ptx::setmaxnreg_dec<kRegsOther>();
  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    Walk it;
    Tail tail{0, 0, 0, 0};
    bool more = it.begin(w, planned) && ok, go = true;
    int E = 0, n = 0, nq = 0, T0 = 0, T1 = 0;
    const int per = BN / pg.box;                                                // boxes of an entry along its keys
    const int c0 = pg.whole ? 0 : lane % SL, g0 = pg.whole ? lane : lane / SL;  // this lane's box
    auto box = [&](int kb) { return box_at(w, pg, it.s, it.b, kb * BN, g0, per); };
    // The next entry: K (for tiles m0 .. m1) or V.
    auto load = [&](const CUtensorMap* map, int m0, int m1, const Box& x, int kvh) {
      const int s = E % NS;
      if (E >= NS) go = wait(&empty[s], ((E / NS) - 1) & 1) && go;
      go = __all_sync(0xffffffffu, go);
      if (!go) return;
      if (lane == 0) {
        if (m0 <= m1) {
          if (m0 == 0) hidden[T0 & 7] = static_cast<uint8_t>(x.hidden);
          if (m1 == 1) hidden[8 + (T1 & 7)] = static_cast<uint8_t>(x.hidden);
        }
        ptx::mbar_expect_tx(&full[s], L::kTile);
      }
      if (m0 <= m1) T0 += m0 == 0, T1 += m1 == 1;
      __syncwarp();
      load_box(sm + L::oRing + s * L::kTile, map, &full[s], pg, x, g0, per, c0, kvh);
      ++E;
    };
    for (; more && go; more = it.next(w), ++n) {
      const int tiles = it.pair ? 2 : 1, kvh = it.vh / w.cut.per_kv, nb = it.k1 - it.k0, b0 = it.j0 + it.k0;
      if (n > 0) go = wait(q_empty, (n - 1) & 1) && go;
      go = __all_sync(0xffffffffu, go);
      if (!go) break;
      ++nq;
      if (lane == 0) {
        Item& x = items[n & 7];
        x.n = nb, x.b0 = b0, x.pair = it.pair, x.t0 = it.t0, x.t1 = it.t1, x.start = it.s.start, x.len = it.s.len;
        const int64_t p0 = static_cast<int64_t>(it.s.start) + it.t0, p1 = static_cast<int64_t>(it.s.start) + it.t1 - 1;
        x.last = w.causal ? static_cast<int>(min(p0, static_cast<int64_t>(it.s.len) - 1)) : it.s.len - 1;
        x.first = w.window > 0 ? static_cast<int>(max(p1 - w.window + 1, static_cast<int64_t>(0))) : 0;
        x.slot = it.whole() ? -1 : it.slot(p);
        x.b = it.b, x.batch = it.s.batch, x.row0 = it.s.row0, x.vh = it.vh, x.kvh = kvh;
        ptx::mbar_arrive(&known[n & 7]);
        if (!it.whole() && it.k0 == 0) tail = Tail{it.b, it.tile, it.vh, it.parts(p)};
        ptx::mbar_expect_tx(q_full, tiles * SL * gt * tq * 128);
        for (int m = 0; m < tiles; ++m)
          for (int u = 0; u < SL; ++u)
            ptx::tma_load_5d(sm + m * L::kTile + u * BM * 128, &tmQ, q_full, u * 64, 0, it.s.row0 + it.t0 + m * tq, it.vh,
                             it.s.batch);
      }
      // (a block's pages are looked up before the wait for room in the ring)
      Box x = box(b0);
      if (tiles == 2) {
        for (int j = 0; j < nb && go; ++j) {
          load(&tmK, 0, 1, x, kvh);
          if (go) load(&tmV, 1, 0, x, kvh);
          if (j + 1 < nb) x = box(b0 + j + 1);
        }
      } else {
        Box y = x;
        load(&tmK, 0, 0, x, kvh);
        if (nb > 1) y = box(b0 + 1);
        if (go && nb > 1) load(&tmK, 1, 1, y, kvh);
        for (int j = 0; j < nb && go; ++j) {
          Box z = y;
          if (j + 2 < nb) z = box(b0 + j + 2);
          load(&tmV, 1, 0, x, kvh);
          if (go && j + 2 < nb) load(&tmK, j & 1, j & 1, z, kvh);
          x = y, y = z;
        }
      }
    }
    if (lane == 0) {
      if (go) {
        items[n & 7].n = 0;
        ptx::mbar_arrive(&known[n & 7]);
      }
      sp.tail[p] = tail;
      started[0] = nq, started[1] = E;
    }
  } else if (warp == 9 || warp == 10) {
    // ------------------------------------------------- MMA issuer of tile m
    // (one warp for both tiles spends 1700 cycles of each product pair issuing, the products take 1024)
    const int m = warp - 9;
    constexpr uint32_t idS = ptx::idesc_bf16(BM, BN, 0, 0);
    constexpr uint32_t idO = ptx::idesc_bf16(BM, D, 0, 1);
    const uint64_t dQ = tc::kmajor_desc(ptx::smem_u32(sm), BM, 0);
    const uint64_t dK = ptx::sdesc_sw128(ptx::smem_u32(sm + L::oRing), 16, pg.sbo);
    const uint64_t dV = ptx::sdesc_sw128(ptx::smem_u32(sm + L::oRing), pg.slab, pg.sbo);
    const uint32_t tS = tmem + L::cS + m * BN, tO = tmem + L::cO + m * D;
    int base = 0, n = 0, T = 0, masked = 0, seen = 0, turns = 0;
    // Entry e, after those before it that are the other tile's.  A parity tells two neighbouring phases apart, so each
    // consumer looks at every entry in turn, and an entry is filled again once all three have done with it.
    auto pass = [&](int e) {
      for (; seen < e; ++seen) {
        wait(&full[seen % NS], (seen / NS) & 1);
        if (lane == 0) ptx::mbar_arrive(&empty[seen % NS]);
      }
    };
    auto loaded = [&](int e) {
      pass(e);
      wait(&full[e % NS], (e / NS) & 1);
      seen = e + 1;
    };
    for (const Item* it; (it = item(n)) != nullptr; ++n) {
      const Order o{base, it->n, it->pair != 0};
      const int b0 = it->b0, nb = it->count(m);
      const uint32_t qo = o.pair && m == 1 ? L::kTile : 0;
      auto issue_s = [&](int j) {
        const int e = o.K(o.block(m, j)), s = e % NS;
        loaded(e);
        ptx::tc_fence_after();
        const uint32_t so = static_cast<uint32_t>(s * L::kTile);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_ss_e(tS, tc::desc_add(dQ, qo + tc::kmajor_off(BM, k)), tc::desc_add(dK, so + (k >> 2) * pg.slab + (k & 3) * 32),
                        idS, k > 0 ? 1u : 0u);
        ptx::mma_commit_e(&s_full[m]);
        if (lane == 0) ptx::mbar_arrive(&s_full[m]);
        ptx::mma_commit_e(&empty[s]);
      };
      int block = 0;  // blocks of the item whose values have been waited for
      wait(q_full, n & 1);
      if (nb > 0) issue_s(0);
      if (nb <= 1) ptx::mma_commit_e(q_empty);
      for (int j = 0; j < nb; ++j, ++T) {
        const int i = o.block(m, j), e = o.V(i), s = e % NS;
        loaded(e);
        for (; block <= i; ++block)  // (in turn, too)
          if (it->hides(b0 + block)) {
            wait(&v_ok[masked % NS], (masked / NS) & 1);
            ++masked;
          }
        wait(&p_half[m], T & 1);
        if (j == 0 && n > 0) wait(o_empty, (n - 1) & 1);
        // Two tiles take turns, P V and the next S at a time: left to themselves their softmaxes fall into step,
        // and the products wait for both at once.
        if (o.pair && (m == 1 || turns > 0)) wait(&turn[m], (turns - 1 + m) & 1);
        ptx::tc_fence_after();
        const uint32_t so = static_cast<uint32_t>(s * L::kTile);
#pragma unroll
        for (int k = 0; k < BN / 16; ++k) {
          if (k == BN / 32) {
            wait(&p_ready[m], T & 1);
            ptx::tc_fence_after();
          }
          ptx::mma_ts_e(tO, tS + k * 8, tc::desc_add(dV, so + k * 2 * pg.sbo), idO, (j > 0 || k > 0) ? 1u : 0u);
        }
        ptx::mma_commit_e(&empty[s]);
        if (j + 1 < nb) {
          issue_s(j + 1);
          if (j + 2 == nb) ptx::mma_commit_e(q_empty);
        }
        if (o.pair) {
          if (lane == 0) ptx::mbar_arrive(&turn[1 - m]);
          ++turns;
        }
      }
      for (; block < o.n; ++block)  // (the other tile's last one)
        if (it->hides(b0 + block)) {
          wait(&v_ok[masked % NS], (masked / NS) & 1);
          ++masked;
        }
      base += 2 * o.n;
      pass(base);
      if (nb == 0 && n > 0) wait(o_empty, (n - 1) & 1);  // (every item's, for the same reason)
      ptx::mma_commit_e(o_full);
      if (lane == 0) ptx::mbar_arrive(o_full);
    }
  } else if (warp == 11) {
    // ------------------------- values that some row does not see: made 0 where they are not finite
    int base = 0, n = 0, masked = 0, seen = 0;
    for (const Item* it; (it = item(n)) != nullptr; ++n) {
      const Order o{base, it->n, it->pair != 0};
      const int b0 = it->b0;
      for (int i = 0; i < o.n; ++i) {
        const int e = o.V(i), s = e % NS;
        for (; seen < e; ++seen) {  // (every entry in turn, as above)
          wait(&full[seen % NS], (seen / NS) & 1);
          if (lane == 0) ptx::mbar_arrive(&empty[seen % NS]);
        }
        if (!it->hides(b0 + i)) continue;
        wait(&full[s], (e / NS) & 1);
        const bool some = hide_values(sm + L::oRing + s * L::kTile, BN, min(max(it->len - (b0 + i) * BN, 0), BN), SL, pg);
        if (some) spoilt[n & 7] = n + 1;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&v_ok[masked % NS]);
        ++masked;
      }
      base += 2 * o.n;
      for (; seen < base; ++seen) {
        wait(&full[seen % NS], (seen / NS) & 1);
        if (lane == 0) ptx::mbar_arrive(&empty[seen % NS]);
      }
    }
  } else {
    ptx::setmaxnreg_inc<kRegs>();
    // --------------------------- softmax of tile m: thread r owns row r
    const int m = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + L::cS + m * BN + lane_off, tO = tmem + L::cO + lane_off;
    const uint64_t c2 = tc::pk2f(c, c);
    const int rt = r / gt, rh = r - rt * gt;  // this row's token of the tile, and its head
    uint8_t* stage = sm + L::oOut + warp * kOut;
    int T = 0, shared = 0;
    const Item* it;
    for (int n = 0; (it = item(n)) != nullptr; ++n) {
      const int nb = it->count(m);
      const bool pair = it->pair != 0;
      // the keys that this row sees: its token's position less the window, up to that position or the last key
      int last, first;
      {
        const int tok = it->t0 + (pair ? m * tq : 0) + rt;
        const int64_t at = static_cast<int64_t>(it->start) + tok, end = it->len - 1;
        last = static_cast<int>(w.causal ? max(min(at, end), static_cast<int64_t>(-1)) : end);
        const int64_t f = w.window > 0 ? at - w.window + 1 : 0;
        first = static_cast<int>(min(max(f, static_cast<int64_t>(0)), static_cast<int64_t>(0x7fffffff)));
      }
      // bounds grow with the row: the warp's first row has the first last key, its last row the last first one
      const int last0 = __shfl_sync(0xffffffffu, last, 0), first31 = __shfl_sync(0xffffffffu, first, 31);
      int key0 = (it->b0 + (pair ? 0 : m)) * BN;
      float mref = -INFINITY, l = 0.f;
      for (int j = 0; j < nb; ++j, ++T, key0 += pair ? BN : 2 * BN) {
        wait(&s_full[m], T & 1);
        ptx::tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) ptx::tmem_ld32(tS + ch * 32, v[ch]);
        const uint32_t hid = hidden[m * 8 + (T & 7)];
        ptx::tmem_wait_ld();
        if (key0 + BN - 1 > last0 || key0 < first31 || hid != 0) {
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
            if (key0 + ch * 32 + 31 > last0 || key0 + ch * 32 < first31 || hid != 0) {
              uint32_t see = tc::bits_between(first - key0 - ch * 32, last - key0 - ch * 32);
              if (hid & (1u << (2 * ch))) see &= 0xffff0000u;
              if (hid & (2u << (2 * ch))) see &= 0x0000ffffu;
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
          for (int x0 = 0; x0 < D; x0 += 16) {  // 16 columns at a time: the scores hold 128 registers
            uint32_t q[16];
            ptx::tmem_ld16(tO + m * D + x0, q);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
              const float2 x = tc::unpk2(tc::mul2(tc::pk2(q[t], q[t + 1]), a2));
              q[t] = __float_as_uint(x.x);
              q[t + 1] = __float_as_uint(x.y);
            }
            ptx::tmem_st16(tO + m * D + x0, q);
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
      float a0 = 1.f, a1 = 0.f;  // weights of this tile's sums and of the other's
      // Tile 1 hands over for the next such item before tile 0 has looked at this one where it has one block there, whose
      // S needs nothing of tile 0's; for the one after that it needs this item's epilogue, tile 0's o_empty: two buffers, each
      // with its barrier.
      if (!pair && it->n > 1) {
        const int buf = handover::buffer_of(shared, 2);
        float2* mine = stat + buf * BM + r;
        if (m == 1) {
          *mine = make_float2(mref, l);
          ptx::mbar_arrive(&x_full[buf]);
        } else {
          wait(&x_full[buf], handover::parity_of(shared, 2));
          const float2 z = *mine;
          const float top = fmaxf(mref, z.x), sub = top == -INFINITY ? 0.f : top * c;
          a0 = mref == -INFINITY ? 0.f : ptx::ex2(fmaf(mref, c, -sub)), a1 = z.x == -INFINITY ? 0.f : ptx::ex2(fmaf(z.x, c, -sub));
          l = l * a0 + z.y * a1, mref = top;
        }
        ++shared;
      }
      wait(o_full, n & 1);
      ptx::tc_fence_after();
      if (pair || m == 0) {
        const int slot = it->slot, tok = it->t0 + (pair ? m * tq : 0) + rt;
        const bool both = !pair && it->n > 1, live = rt < tq && tok < it->t1;
        const int64_t h = static_cast<int64_t>(it->vh) * gt + rh, pos = it->row0 + tok;
        const float inv = slot >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;  // (a row that sees no key: 0)
        a0 *= inv, a1 *= inv;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.O) + it->batch * out.os[0] + h * out.os[1] + pos * out.os[2];
        float* part = slot >= 0 ? sp.o(slot, (pair ? m * BM : 0) + r) : nullptr;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t a[32], b[32];
          ptx::tmem_ld32(tO + (pair ? m * D : 0) + ch * 32, a);
          if (both) ptx::tmem_ld32(tO + D + ch * 32, b);
          ptx::tmem_wait_ld();
          if (ch == D / 32 - 1) {
            ptx::tc_fence_before();
            ptx::mbar_arrive(o_empty);
          }
          if (ch * 32 >= d) continue;  // columns past d are padding
#pragma unroll
          for (int t = 0; t < 32; ++t) {
            float x = tc::f(a[t]) * a0;
            if (both) x = fmaf(tc::f(b[t]), a1, x);
            a[t] = l == 0.f ? 0u : __float_as_uint(x);
          }
          // Through shared memory, so that four threads write 64 bytes of a row: a row per thread straight to memory
          // took 12 thousand cycles of an item.
          if (part == nullptr) {
            uint32_t pk[16];
#pragma unroll
            for (int t = 0; t < 16; ++t) pk[t] = ptx::pack_bf16(tc::f(a[2 * t]), tc::f(a[2 * t + 1]));
            put_rows(stage, pk, reinterpret_cast<uint8_t*>(dst) + ch * 64, live);
          } else {
            put_rows(stage, reinterpret_cast<const uint32_t(&)[16]>(a[0]), reinterpret_cast<uint8_t*>(part) + ch * 128, live);
            put_rows(stage, reinterpret_cast<const uint32_t(&)[16]>(a[16]), reinterpret_cast<uint8_t*>(part) + ch * 128 + 64, live);
          }
        }
        __syncwarp();
        if (live) {
          if (spoilt[n & 7] == n + 1) add_spoilt(w, *it, first, last, Vg + it->kvh * vs1, vs0, vs2, d, dst, part);
          if (part != nullptr)
            *sp.ml(slot, (pair ? m * BM : 0) + r) = make_float2(mref == -INFINITY ? mref : mref * c, l);
          else if (out.lse != nullptr)
            out.lse[it->batch * out.ls[0] + h * out.ls[1] + pos] = l == 0.f ? -INFINITY : fmaf(mref, scale, logf(l));
        }
      } else {
        ptx::mbar_arrive(o_empty);
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  // A wait has given up: loads and products may still be on their way into this CTA's shared memory and
  // TMEM, which others get when it ends.
  if (*abort_flag != 0) {
    if (threadIdx.x == 8 * 32) {
      const int nq = started[0], E = started[1];
      if (nq > 0) ptx::settle(q_full, (nq - 1) & 1);
      for (int s = 0; s < NS && s < E; ++s) ptx::settle(&full[s], handover::last_phase(E, NS, s));
    }
    if (warp == 9 || warp == 10) {
      ptx::mma_commit_e(settled);
      ptx::settle(settled, 0);
    }
    __syncthreads();
  }
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const PagedArgs& a, const Work& w, const Space& sp, const Out& out, cudaStream_t st) {
  alignas(64) CUtensorMap mq, mk, mv;
  Pages pg;
  if (!make_maps(a, w.cut, BN, D / 64, &mq, &mk, &mv, pg)) return cudaErrorInvalidValue;
  auto kern = paged_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::bytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(w.cut.ctas), kThreads, Lay<D>::bytes, st>>>(mq, mk, mv, w, sp, out,
                    static_cast<const __nv_bfloat16*>(a.V), a.vs[0], a.vs[1], a.vs[2], a.d, pg, a.scale, a.scale * kLog2e);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return join(w, sp, out, a.dtype, a.d, BM, a.max_new, st);
}

Work work_of(const PagedArgs& a) {
  Work w;
  const int g = a.H / a.Hkv;
  w.seqs = a.seqs, w.causal = a.causal, w.window = a.window;
  w.cut.gt = heads_together(g, BM, a.max_new);
  w.cut.nv = a.H / w.cut.gt, w.cut.per_kv = g / w.cut.gt;
  w.cut.tile = BM / w.cut.gt, w.cut.step = 2 * w.cut.tile;
  // An item's start, epilogue and idle half cost about four blocks: 146 us for the ragged window with 1, 142 with 4, 144 with 8
  // and 16; long chunks do not care.
  w.cut.shift = 7, w.cut.over = 4, w.cut.least = 8, w.cut.ctas = 152;
  return w;
}

}  // namespace

size_t tc_bytes(const PagedArgs& a) { return Space::bytes(152, 2 * BM, a.d <= 64 ? 64 : 128); }

cudaError_t tc_paged(const PagedArgs& a, void* ws, cudaStream_t st) {
  const Work w = work_of(a);
  const Space sp = Space::at(ws, w.cut.ctas, 2 * BM, a.d <= 64 ? 64 : 128);
  const Out out{a.O, a.lse, {a.os[0], a.os[1], a.os[2]}, {a.ls[0], a.ls[1]}};
  // d = 32 runs the kernel of 64 columns and d = 96 that of 128: TMA fills the columns past d with zeros.
  return a.d <= 64 ? launch<64>(a, w, sp, out, st) : launch<128>(a, w, sp, out, st);
}

}  // namespace paged

uint32_t tc_paged_take_error() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, paged::g_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(paged::g_err, &z, sizeof(z));
  return v;
}

}  // namespace fbd
