// Attention of new tokens over a paged cache at d = 256, bf16, on the tensor cores (tc_paged.cu has the
// method; d = 256 leaves TMEM room for one tile's O, 256 columns).
//
// One tile of 128 rows over blocks of 64 keys; S of the next block is formed while this one is
// exponentiated, in the other of two S (P over the S it came from), by a warp of its own, P V by another: 1024 cycles
// of products a block.  What bounds it is the way of K and V into shared memory, 64 KB a block, so Q lies in
// TMEM (128 columns, written by the softmax threads, a row each), and shared memory is a ring of six entries
// of 64 keys.  With Q in shared memory and four such entries a block took 3600 cycles: 126 us for 2 x 1000 tokens over
// 4500 keys, 8 heads in pairs, 84 us so (0.87 PFLOP/s).  O is rescaled, where
// the maximum moved, once the product before has ended.
#include <cuda_bf16.h>

#include "handover.h"
#include "tc_paged.cuh"

namespace fbd {
namespace paged {
namespace {

__device__ unsigned int g_err = 0;

constexpr int D = 256, KN = 64;  // columns; keys of a block and of an entry
// Warps 0-3: softmax, 4: TMA, 5: S, 6: P V, 7: values that a row must not see.
constexpr int kThreads = 256;
constexpr int NS = 6, SL = D / 64;
constexpr int kEntry = KN * D * 2;
constexpr int oOut = NS * kEntry, oBar = oOut + 4 * kOut, oItem = oBar + 512, kBytes = oItem + 8 * 64;
static_assert(kBytes <= 232448, "shared memory");
constexpr uint32_t cS = 0, cQ = 2 * KN, cO = cQ + D / 2;  // S of an even (odd) block at cS (+ KN)

__global__ void __launch_bounds__(kThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Work w, const Space sp,
                const Out out, const __nv_bfloat16* __restrict__ Q, int64_t qs0, int64_t qs1, int64_t qs2,
                const __nv_bfloat16* __restrict__ Vg, int64_t vs0, int64_t vs1, int64_t vs2, Pages pg, float scale, float c) {
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + oBar);
  uint64_t* q_full = bars;          // Q in TMEM
  uint64_t* s_full = bars + 1;      // [2] S in TMEM
  uint64_t* p_ready = s_full + 2;   // [2] P in TMEM, O rescaled
  uint64_t* pv_done = p_ready + 2;  // [2] the block's P V done
  uint64_t* o_full = pv_done + 2;
  uint64_t* o_empty = o_full + 1;   // O read by the epilogue
  uint64_t* settled = o_empty + 1;  // after a wait that gave up: the products in flight done
  uint64_t* full = settled + 1;     // [NS]
  uint64_t* empty = full + NS;      // [NS]
  uint64_t* v_ok = empty + NS;      // [NS] values that some row does not see are finite
  uint64_t* known = v_ok + NS;      // [8] items
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(known + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* started = abort_flag + 1;                                       // ring entries (the TMA warp's)
  volatile uint8_t* hidden = reinterpret_cast<volatile uint8_t*>(started + 1);  // [8] of blocks: 16-key runs without a page
  volatile int* spoilt = reinterpret_cast<volatile int*>(hidden + 8);           // [8] of items: n + 1 where values were made 0
  Item* items = reinterpret_cast<Item*>(sm + oItem);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, p = blockIdx.x;
  const int gt = w.cut.gt, tq = w.cut.tile;
  ptx::grid_dependency_launch();
  if (threadIdx.x == 4 * 32) {
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    ptx::mbar_init(q_full, 128);
    for (int m = 0; m < 2; ++m) {
      ptx::mbar_init(&s_full[m], 2);  // the products' end and the warp that issued them
      ptx::mbar_init(&p_ready[m], 128);
      ptx::mbar_init(&pv_done[m], 1);
    }
    ptx::mbar_init(o_full, 2);
    ptx::mbar_init(o_empty, 128);
    ptx::mbar_init(settled, 2);
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 3);  // of the three consumers: S, P V and the warp that looks at values
      ptx::mbar_init(&v_ok[s], 1);
    }
    for (int s = 0; s < 8; ++s) ptx::mbar_init(&known[s], 1), spoilt[s] = 0;
    *started = 0;
    *abort_flag = (ptx::smem_u32(sm) & 1023u) ? 1 : 0;  // the swizzled tiles need 1024-byte alignment
    if (*abort_flag) atomicOr(&g_err, FBD_ERR_TIMEOUT);
    ptx::fence_mbar_init();
  }
  if (warp == 5) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  Plan planned{};
  if (warp == 4) planned = plan(w, p);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const ptx::BoundedWait wait{abort_flag, &g_err};
  const bool ok = *abort_flag == 0;
  // Item n, once it is known (tc_paged.cu).
  auto item = [&](int n) -> const Item* {
    wait(&known[n & 7], (n >> 3) & 1);
    const Item* it = items + (n & 7);
    return __all_sync(0xffffffffu, *abort_flag == 0 && *reinterpret_cast<const volatile int*>(&it->n) > 0) ? it : nullptr;
  };

  // A consumer's entries up to the e-th that are another's.  A parity tells two neighbouring phases apart, so each
  // consumer looks at every entry in turn, and an entry is filled again once all three have done with it.
  int seen = 0;
  auto pass = [&](int e) {
    for (; seen < e; ++seen) {
      wait(&full[seen % NS], (seen / NS) & 1);
      if (lane == 0) ptx::mbar_arrive(&empty[seen % NS]);
    }
  };
  auto loaded = [&](int e) {
    wait(&full[e % NS], (e / NS) & 1);
    seen = e + 1;
  };

  if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    Walk it;
    Tail tail{0, 0, 0, 0};
    bool more = it.begin(w, planned) && ok, go = true;
    int E = 0, n = 0, T = 0;
    const int per = KN / pg.box;                                                // boxes of an entry along its keys
    const int c0 = pg.whole ? 0 : lane % SL, g0 = pg.whole ? lane : lane / SL;  // this lane's box
    // The next entry: block kb of K or V.
    auto load = [&](const CUtensorMap* map, bool key, int kb, int kvh) {
      const Box x = box_at(w, pg, it.s, it.b, kb * KN, g0, per);  // (looked up before the wait for room in the ring)
      const int s = E % NS;
      if (E >= NS) go = wait(&empty[s], ((E / NS) - 1) & 1) && go;
      go = __all_sync(0xffffffffu, go);
      if (!go) return;
      if (lane == 0) {
        if (key) hidden[T & 7] = static_cast<uint8_t>(x.hidden);
        ptx::mbar_expect_tx(&full[s], kEntry);
      }
      __syncwarp();
      load_box(sm + s * kEntry, map, &full[s], pg, x, g0, per, c0, kvh);
      ++E, T += key;
    };
    for (; more && go; more = it.next(w), ++n) {
      const int kvh = it.vh / w.cut.per_kv, nb = it.k1 - it.k0, b0 = it.j0 + it.k0;
      // (the ring of items is longer than the loads' lead, half the entries)
      if (lane == 0) {
        Item& x = items[n & 7];
        x.n = nb, x.b0 = b0, x.pair = 0, x.t0 = it.t0, x.t1 = it.t1, x.start = it.s.start, x.len = it.s.len;
        const int64_t p0 = static_cast<int64_t>(it.s.start) + it.t0, p1 = static_cast<int64_t>(it.s.start) + it.t1 - 1;
        x.last = w.causal ? static_cast<int>(min(p0, static_cast<int64_t>(it.s.len) - 1)) : it.s.len - 1;
        x.first = w.window > 0 ? static_cast<int>(max(p1 - w.window + 1, static_cast<int64_t>(0))) : 0;
        x.slot = it.whole() ? -1 : it.slot(p);
        x.b = it.b, x.batch = it.s.batch, x.row0 = it.s.row0, x.vh = it.vh, x.kvh = kvh;
        ptx::mbar_arrive(&known[n & 7]);
        if (!it.whole() && it.k0 == 0) tail = Tail{it.b, it.tile, it.vh, it.parts(p)};
      }
      // K_0 K_1 V_0 K_2 V_1 ...
      for (int i = 0; i < nb + 2 && go; ++i) {
        if (i >= 2) load(&tmV, false, b0 + i - 2, kvh);
        if (go && i < nb) load(&tmK, true, b0 + i, kvh);
      }
    }
    if (lane == 0) {
      if (go) {
        items[n & 7].n = 0;
        ptx::mbar_arrive(&known[n & 7]);
      }
      sp.tail[p] = tail;
      *started = E;
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ S = Q K^T
    constexpr uint32_t idS = ptx::idesc_bf16(BM, KN, 0, 0);
    const uint64_t dK = ptx::sdesc_sw128(ptx::smem_u32(sm), 16, pg.sbo);
    int base = 0, n = 0, T = 0;
    for (const Item* it; (it = item(n)) != nullptr; ++n) {
      const Order o{base, it->n, false};
      wait(q_full, n & 1);
      for (int j = 0; j < o.n; ++j, ++T) {
        const int e = o.K(j), s = e % NS;
        pass(e);
        loaded(e);
        // the block before the last has been multiplied with V: its P's columns are free
        if (T >= 2) wait(&pv_done[T & 1], ((T >> 1) - 1) & 1);
        ptx::tc_fence_after();
        const uint32_t so = static_cast<uint32_t>(s * kEntry);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_ts_e(tmem + cS + (T & 1) * KN, tmem + cQ + k * 8, tc::desc_add(dK, so + (k >> 2) * pg.slab + (k & 3) * 32), idS,
                        k > 0 ? 1u : 0u);
        ptx::mma_commit_e(&s_full[T & 1]);
        if (lane == 0) ptx::mbar_arrive(&s_full[T & 1]);
        ptx::mma_commit_e(&empty[s]);
      }
      base += 2 * o.n;
      pass(base);
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------ O += P V
    constexpr uint32_t idO = ptx::idesc_bf16(BM, D, 0, 1);
    const uint64_t dV = ptx::sdesc_sw128(ptx::smem_u32(sm), pg.slab, pg.sbo);
    int base = 0, n = 0, T = 0, masked = 0;
    for (const Item* it; (it = item(n)) != nullptr; ++n) {
      const Order o{base, it->n, false};
      for (int j = 0; j < o.n; ++j, ++T) {
        const int b = T & 1, e = o.V(j), s = e % NS;
        pass(e);
        loaded(e);
        if (it->hides(it->b0 + j, KN)) {
          wait(&v_ok[masked % NS], (masked / NS) & 1);
          ++masked;
        }
        wait(&p_ready[b], (T >> 1) & 1);
        if (j == 0 && n > 0) wait(o_empty, (n - 1) & 1);
        ptx::tc_fence_after();
        const uint32_t so = static_cast<uint32_t>(s * kEntry);
#pragma unroll
        for (int k = 0; k < KN / 16; ++k)
          ptx::mma_ts_e(tmem + cO, tmem + cS + b * KN + k * 8, tc::desc_add(dV, so + k * 2 * pg.sbo), idO, (j > 0 || k > 0) ? 1u : 0u);
        ptx::mma_commit_e(&empty[s]);
        ptx::mma_commit_e(&pv_done[b]);
      }
      ptx::mma_commit_e(o_full);
      if (lane == 0) ptx::mbar_arrive(o_full);
      base += 2 * o.n;
      pass(base);
    }
  } else if (warp == 7) {
    // ------------------------- values that some row does not see: made 0 where they are not finite
    int base = 0, n = 0, masked = 0;
    for (const Item* it; (it = item(n)) != nullptr; ++n) {
      const Order o{base, it->n, false};
      for (int j = 0; j < o.n; ++j) {
        const int e = o.V(j), key0 = (it->b0 + j) * KN;
        pass(e);
        if (!it->hides(it->b0 + j, KN)) continue;
        wait(&full[e % NS], (e / NS) & 1);
        const bool some = hide_values(sm + e % NS * kEntry, KN, min(max(it->len - key0, 0), KN), SL, pg);
        if (some) spoilt[n & 7] = n + 1;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&v_ok[masked % NS]);
        ++masked;
      }
      base += 2 * o.n;
      pass(base);
    }
  } else {
    // --------------------------- softmax: thread r owns row r
    const int r = threadIdx.x;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tO = tmem + cO + lane_off;
    const uint64_t c2 = tc::pk2f(c, c);
    const int rt = r / gt, rh = r - rt * gt;  // this row's token of the tile, and its head
    uint8_t* stage = sm + oOut + warp * kOut;
    // This row's queries of an item to TMEM (the products with the last item's have ended: their last S has been seen).
    auto bring_q = [&](const Item* it) {
      const bool live = rt < tq && it->t0 + rt < it->t1;
      const __nv_bfloat16* q =
          Q + it->batch * qs0 + (static_cast<int64_t>(it->vh) * gt + rh) * qs1 + static_cast<int64_t>(it->row0 + it->t0 + rt) * qs2;
#pragma unroll 1
      for (int x0 = 0; x0 < D / 2; x0 += 32) {
        uint32_t v[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 y = live ? *reinterpret_cast<const uint4*>(q + 2 * x0 + u * 8) : make_uint4(0, 0, 0, 0);
          v[4 * u] = y.x, v[4 * u + 1] = y.y, v[4 * u + 2] = y.z, v[4 * u + 3] = y.w;
        }
        ptx::tmem_st32(tmem + cQ + lane_off + x0, v);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(q_full);
    };
    int T = 0;
    const Item* it = item(0);
    if (it != nullptr) bring_q(it);
    for (int n = 0; it != nullptr; ++n) {
      const int nb = it->n;
      // the keys that this row sees: its token's position less the window, up to that position or the last key
      int last, first;
      {
        const int64_t at = static_cast<int64_t>(it->start) + it->t0 + rt, end = it->len - 1;
        last = static_cast<int>(w.causal ? max(min(at, end), static_cast<int64_t>(-1)) : end);
        const int64_t f = w.window > 0 ? at - w.window + 1 : 0;
        first = static_cast<int>(min(max(f, static_cast<int64_t>(0)), static_cast<int64_t>(0x7fffffff)));
      }
      const int last0 = __shfl_sync(0xffffffffu, last, 0), first31 = __shfl_sync(0xffffffffu, first, 31);
      int key0 = it->b0 * KN;
      float mref = -INFINITY, l = 0.f;
      for (int j = 0; j < nb; ++j, ++T, key0 += KN) {
        const int b = T & 1;
        const uint32_t tS = tmem + cS + b * KN + lane_off;
        wait(&s_full[b], (T >> 1) & 1);
        ptx::tc_fence_after();
        uint32_t v[2][32];
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) ptx::tmem_ld32(tS + ch * 32, v[ch]);
        const uint32_t hid = hidden[T & 7];
        ptx::tmem_wait_ld();
        if (key0 + KN - 1 > last0 || key0 < first31 || hid != 0) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
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
        for (int u = 0; u < 8; ++u) mx[u] = fmaxf(tc::f(v[0][u]), tc::f(v[1][u]));
#pragma unroll
        for (int t = 8; t < 32; t += 8)
#pragma unroll
          for (int u = 0; u < 8; ++u) mx[u] = fmaxf(mx[u], fmaxf(tc::f(v[0][t + u]), tc::f(v[1][t + u])));
#pragma unroll
        for (int u = 1; u < 8; ++u) mx[0] = fmaxf(mx[0], mx[u]);
        // (always at the first visible key: mref = -inf)
        const bool moved = ptx::ex2((mx[0] - mref) * c) > fminf(fmaxf(kShare * l, 1.f), kSlack);
        const float mnew = moved ? mx[0] : mref;
        const float alpha = moved ? ptx::ex2((mref - mnew) * c) : 1.f;
        l *= alpha;
        mref = mnew;
        // a row that has seen no key yet subtracts 0, not -inf: every term is 2^-inf = 0
        const float nm = mref == -INFINITY ? 0.f : -mref * c;
        const uint64_t nm2 = tc::pk2f(nm, nm);
        uint64_t rs[4] = {0, 0, 0, 0};
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int t = 0; t < 32; t += 2) {
            const float2 arg = tc::unpk2(tc::fma2(tc::pk2(v[ch][t], v[ch][t + 1]), c2, nm2));
            const float p0 = ptx::ex2(arg.x), p1 = ptx::ex2(arg.y);
            rs[(t >> 1) & 3] = tc::add2(rs[(t >> 1) & 3], tc::pk2f(p0, p1));
            pk[t >> 1] = ptx::pack_bf16(p0, p1);
          }
          ptx::tmem_st16(tS + ch * 16, pk);
        }
        // (waited for only here: S of the block before came behind the product two before that, so the phase is not
        // mistaken for an older one)
        if (j > 0 && __any_sync(0xffffffffu, moved)) {
          wait(&pv_done[b ^ 1], ((T - 1) >> 1) & 1);
          ptx::tc_fence_after();
          const uint64_t a2 = tc::pk2f(alpha, alpha);
#pragma unroll 1
          for (int x0 = 0; x0 < D; x0 += 32) {
            uint32_t q[32];
            ptx::tmem_ld32(tO + x0, q);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 32; t += 2) {
              const float2 x = tc::unpk2(tc::mul2(tc::pk2(q[t], q[t + 1]), a2));
              q[t] = __float_as_uint(x.x);
              q[t + 1] = __float_as_uint(x.y);
            }
            ptx::tmem_st32(tO + x0, q);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&p_ready[b]);
        const float2 x = tc::unpk2(tc::add2(tc::add2(rs[0], rs[1]), tc::add2(rs[2], rs[3])));
        l += x.x + x.y;
      }
      // The next item's queries, so that its first S are formed under this one's epilogue.
      const Item* then = item(n + 1);
      if (then != nullptr) bring_q(then);
      // ------------------------------------------------------------------ epilogue
      wait(o_full, n & 1);
      ptx::tc_fence_after();
      const int slot = it->slot, tok = it->t0 + rt;
      const bool live = rt < tq && tok < it->t1;
      const int64_t h = static_cast<int64_t>(it->vh) * gt + rh, pos = it->row0 + tok;
      const float inv = slot >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;  // (a row that sees no key: 0)
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.O) + it->batch * out.os[0] + h * out.os[1] + pos * out.os[2];
      float* part = slot >= 0 ? sp.o(slot, r) : nullptr;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t a[32];
        ptx::tmem_ld32(tO + ch * 32, a);
        ptx::tmem_wait_ld();
        if (ch == D / 32 - 1) {
          ptx::tc_fence_before();
          ptx::mbar_arrive(o_empty);
        }
#pragma unroll
        for (int t = 0; t < 32; ++t) a[t] = l == 0.f ? 0u : __float_as_uint(tc::f(a[t]) * inv);
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
        if (spoilt[n & 7] == n + 1) add_spoilt(w, *it, first, last, Vg + it->kvh * vs1, vs0, vs2, D, dst, part, KN);
        if (part != nullptr)
          *sp.ml(slot, r) = make_float2(mref == -INFINITY ? mref : mref * c, l);
        else if (out.lse != nullptr)
          out.lse[it->batch * out.ls[0] + h * out.ls[1] + pos] = l == 0.f ? -INFINITY : fmaf(mref, scale, logf(l));
      }
      it = then;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  // A wait has given up: loads and products may still be on their way into this CTA's shared memory and
  // TMEM, which others get when it ends.
  if (*abort_flag != 0) {
    if (threadIdx.x == 4 * 32)
      for (int s = 0; s < NS && s < *started; ++s) ptx::settle(&full[s], handover::last_phase(*started, NS, s));
    if (warp == 5 || warp == 6) {
      ptx::mma_commit_e(settled);
      ptx::settle(settled, 0);
    }
    __syncthreads();
  }
  if (warp == 5) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

Work work_of(const PagedArgs& a) {
  Work w;
  const int g = a.H / a.Hkv;
  w.seqs = a.seqs, w.causal = a.causal, w.window = a.window;
  w.cut.gt = heads_together(g, BM, a.max_new);
  w.cut.nv = a.H / w.cut.gt, w.cut.per_kv = g / w.cut.gt;
  w.cut.tile = w.cut.step = BM / w.cut.gt;
  // An item's start and epilogue cost about eight blocks of 64 keys: 89.7 us for 2 x 1000 tokens over 4500 keys with 2,
  // 88.2 with 8, 89.5 with 16.
  w.cut.shift = 6, w.cut.over = 8, w.cut.least = 8, w.cut.ctas = 152;
  return w;
}

}  // namespace

size_t tc_wide_bytes(const PagedArgs& a) { return Space::bytes(152, BM, D); }

cudaError_t tc_paged_wide(const PagedArgs& a, void* ws, cudaStream_t st) {
  const Work w = work_of(a);
  const Space sp = Space::at(ws, w.cut.ctas, BM, D);
  const Out out{a.O, a.lse, {a.os[0], a.os[1], a.os[2]}, {a.ls[0], a.ls[1]}};
  alignas(64) CUtensorMap mk, mv;
  Pages pg;
  if (!make_maps(a, w.cut, KN, SL, nullptr, &mk, &mv, pg)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  wide_kernel<<<static_cast<unsigned>(w.cut.ctas), kThreads, kBytes, st>>>(
      mk, mv, w, sp, out, static_cast<const __nv_bfloat16*>(a.Q), a.qs[0], a.qs[1], a.qs[2], static_cast<const __nv_bfloat16*>(a.V),
      a.vs[0], a.vs[1], a.vs[2], pg, a.scale, a.scale * kLog2e);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return join(w, sp, out, a.dtype, D, BM, a.max_new, st);
}

}  // namespace paged

uint32_t tc_paged_wide_take_error() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, paged::g_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(paged::g_err, &z, sizeof(z));
  return v;
}

}  // namespace fbd
