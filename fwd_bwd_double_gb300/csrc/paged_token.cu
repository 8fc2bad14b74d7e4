// Attention of one or a few new tokens per sequence over a paged cache, bf16: up to 16 rows (tokens times the query
// heads that share a key/value head), on warp-level matrix products (m16n8k16; tcgen05 has 128 rows to fill).
//
// Bound by reading the cache once.  A loading warp fetches tiles of 64 keys by TMA into a ring; of each, a warp
// of four forms the scores of 16 keys, the four agree on the rows' maxima, each writes its
// weights (bf16) to shared memory, and each multiplies all 64 with its quarter of V's columns: no sums are joined
// at the end, where a batch of short contexts would spend its time.
// 64 contexts of up to 8191 keys, 4 key/value heads of 128 (544 MB): 90 us, 6.05 TB/s; one of 131001 keys (268 MB): 52 us,
// 5.1 TB/s, of which the start, the join and the last waves of copies are the rest.
// CTAs take the stretches of paged.cuh.
#include <cuda_bf16.h>

#include "handover.h"
#include "tc_paged.cuh"

namespace fbd {
namespace paged {
namespace {

__device__ unsigned int g_err = 0;

constexpr int MK = 64;        // keys of a tile
constexpr int kThreads = 160;  // warps 0-3: products, 4: TMA
constexpr int kRows = 16;

template <int D>
struct Lay {
  static constexpr int kTile = MK * D * 2;  // K or V
  static constexpr int NS = D == 64 ? 6 : 3;
  static constexpr int oP = NS * 2 * kTile;     // [16][64] bf16
  static constexpr int oMax = oP + kRows * MK * 2;  // [4][16] maxima of the warps' keys (at the end, their sums)
  static constexpr int oBar = oMax + 4 * kRows * 4;
  static constexpr int oItem = oBar + 256;
  static constexpr int bytes = oItem + 8 * 64;
  static constexpr int per_sm = D == 256 ? 1 : 2;
};
static_assert(Lay<128>::bytes + 1024 <= 233472 / 2 && Lay<64>::bytes + 1024 <= 233472 / 2 && Lay<256>::bytes <= 232448, "shared memory");

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
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kThreads, Lay<D>::per_sm)
    token_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Work w, const Space sp,
                 const Out out, const __nv_bfloat16* __restrict__ Q, int64_t qs0, int64_t qs1, int64_t qs2,
                 const __nv_bfloat16* __restrict__ Vg, int64_t vs0, int64_t vs1, int64_t vs2, int d, Pages pg, float scale,
                 float c) {
  using L = Lay<D>;
  constexpr int NS = L::NS, SL = D / 64, NT = D / 32;  // slabs; 8-column tiles of a warp's quarter of the columns
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::oBar);  // [NS]
  uint64_t* empty = full + NS;                                 // [NS]
  uint64_t* known = empty + NS;                                // [8] items
  volatile int* abort_flag = reinterpret_cast<volatile int*>(known + 8);
  volatile int* started = abort_flag + 1;
  volatile int* spoilt = abort_flag + 2;                       // n + 1 of the last item in which values were made 0
  volatile uint8_t* hidden = reinterpret_cast<volatile uint8_t*>(abort_flag + 3);  // [NS] 16-key runs without a page
  float* sMax = reinterpret_cast<float*>(sm + L::oMax);
  Item* items = reinterpret_cast<Item*>(sm + L::oItem);
  static_assert((2 * NS + 8) * 8 + 12 + NS <= 256, "the barriers' region");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, p = blockIdx.x, gt = w.cut.gt;
  ptx::grid_dependency_launch();
  if (threadIdx.x == 4 * 32) {
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 4);
    }
    for (int s = 0; s < 8; ++s) ptx::mbar_init(&known[s], 1);
    *spoilt = 0, *started = 0;
    *abort_flag = (ptx::smem_u32(sm) & 1023u) ? 1 : 0;  // the swizzled tiles need 1024-byte alignment
    if (*abort_flag) atomicOr(&g_err, FBD_ERR_TIMEOUT);
    ptx::fence_mbar_init();
  }
  Plan planned{};
  if (warp == 4) planned = plan(w, p);
  __syncthreads();
  const ptx::BoundedWait wait{abort_flag, &g_err};

  if (warp == 4) {
    // ------------------------------------------------------------ plan and loads
    Walk it;
    bool more = it.begin(w, planned) && *abort_flag == 0, go = true;
    int E = 0, n = 0;
    const int per = MK / pg.box;
    const int c0 = pg.whole ? 0 : lane % SL, g0 = pg.whole ? lane : lane / SL;  // this lane's box
    Tail tail{0, 0, 0, 0};
    for (; more && go; more = it.next(w), ++n) {
      const int kvh = it.vh / w.cut.per_kv, nb = it.k1 - it.k0, b0 = it.j0 + it.k0;
      // (an item of n - 8 has been left: at least one tile of n - 4 is in the ring or has left it)
      if (lane == 0) {
        Item& x = items[n & 7];
        x.n = nb, x.b0 = b0, x.pair = 0, x.t0 = it.t0, x.t1 = it.t1, x.start = it.s.start, x.len = it.s.len;
        const int64_t p0 = static_cast<int64_t>(it.s.start) + it.t0, p1 = static_cast<int64_t>(it.s.start) + it.t1 - 1;
        x.last = w.causal ? static_cast<int>(min(p0, static_cast<int64_t>(it.s.len) - 1)) : it.s.len - 1;
        x.first = w.window > 0 ? static_cast<int>(max(p1 - w.window + 1, static_cast<int64_t>(0))) : 0;
        x.slot = it.whole() ? -1 : it.slot(p);
        x.b = it.b, x.batch = it.s.batch, x.row0 = it.s.row0, x.vh = it.vh, x.kvh = kvh;
        ptx::mbar_arrive(&known[n & 7]);
      }
      if (!it.whole() && it.k0 == 0) tail = Tail{it.b, it.tile, it.vh, it.parts(p)};
      Box x = box_at(w, pg, it.s, it.b, b0 * MK, g0, per);
      for (int j = 0; j < nb; ++j, ++E) {
        const int s = E % NS;
        if (E >= NS) go = wait(&empty[s], ((E / NS) - 1) & 1) && go;
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        if (lane == 0) {
          hidden[s] = static_cast<uint8_t>(x.hidden);
          ptx::mbar_expect_tx(&full[s], 2 * L::kTile);
        }
        __syncwarp();
        load_box(sm + s * 2 * L::kTile, &tmK, &full[s], pg, x, g0, per, c0, kvh);
        load_box(sm + (s * 2 + 1) * L::kTile, &tmV, &full[s], pg, x, g0, per, c0, kvh);
        if (j + 1 < nb) x = box_at(w, pg, it.s, it.b, (b0 + j + 1) * MK, g0, per);  // (looked up before the wait)
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
  } else {
    // ------------------------------------------------------------ products
    const int g = lane >> 2, q4 = lane & 3;
    const uint32_t s0 = ptx::smem_u32(sm), sP = s0 + L::oP;
    int E = 0;
    for (int n = 0;; ++n) {
      wait(&known[n & 7], (n >> 3) & 1);
      const Item* it = items + (n & 7);
      // (all four warps go on to an item or none: they meet at barriers)
      if (!tc::named_all(1, 128, *abort_flag == 0 && *reinterpret_cast<const volatile int*>(&it->n) > 0)) break;
      const int nb = it->n, rows = (it->t1 - it->t0) * gt;
      const int64_t h0 = static_cast<int64_t>(it->vh) * gt;
      uint32_t qa[D / 16][4];
      int last[2], first[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // rows g and g + 8
        const int r = g + 8 * x, t = r / gt;
        const __nv_bfloat16* q = Q + it->batch * qs0 + (h0 + r - t * gt) * qs1 + static_cast<int64_t>(it->row0 + it->t0 + t) * qs2;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int col = k * 16 + y * 8 + q4 * 2;
            qa[k][x + 2 * y] = r < rows && col < d ? *reinterpret_cast<const uint32_t*>(q + col) : 0u;
          }
        const int64_t at = static_cast<int64_t>(it->start) + it->t0 + t, end = it->len - 1;
        last[x] = static_cast<int>(w.causal ? max(min(at, end), static_cast<int64_t>(-1)) : end);
        const int64_t f = w.window > 0 ? at - w.window + 1 : 0;
        first[x] = static_cast<int>(min(max(f, static_cast<int64_t>(0)), static_cast<int64_t>(0x7fffffff)));
      }
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // (l: of this thread's keys)
      float o[NT][4];
#pragma unroll
      for (int u = 0; u < NT; ++u) o[u][0] = o[u][1] = o[u][2] = o[u][3] = 0.f;
      for (int j = 0; j < nb; ++j, ++E) {
        const int s = E % NS, key0 = (it->b0 + j) * MK;
        wait(&full[s], (E / NS) & 1);
        const uint32_t K = s0 + s * 2 * L::kTile, V = K + L::kTile;
        const bool hides = it->hides(it->b0 + j, MK);
        const bool gone = hidden[s] >> warp & 1;  // this warp's 16 keys have no page
        float sc[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          sc[u][0] = sc[u][1] = sc[u][2] = sc[u][3] = 0.f;
          const uint32_t row = K + (warp * 2 + u) * pg.sbo + (lane & 7) * 128;
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t f[4];
            ldm4(row + (k >> 1) * pg.slab + ((((k & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4), f);
            mma(sc[u], qa[2 * k], f[0], f[1]);
            mma(sc[u], qa[2 * k + 1], f[2], f[3]);
          }
        }
        if (hides || gone) {
          const int k0 = key0 + warp * 16 + q4 * 2;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = k0 + u * 8 + (x & 1);
              if (gone || key > last[x >> 1] || key < first[x >> 1]) sc[u][x] = -INFINITY;
            }
          if (hides) {  // this warp's 16 values
            const int r = warp * 16 + (lane & 15), held = it->len - key0;
            uint8_t* row = sm + s * 2 * L::kTile + L::kTile + (r >> 3) * pg.sbo + (r & 7) * 128;
            bool some = false;
            for (int u = lane >> 4; u < 2 * SL; u += 2) {  // half a slab at a time
              uint4* at = reinterpret_cast<uint4*>(row + (u >> 1) * pg.slab + (u & 1) * 64);
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                uint4 x = at[ch ^ (r & 3)];
                const uint32_t top = ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                                     ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
                if (r >= held) {
                  at[ch ^ (r & 3)] = make_uint4(0, 0, 0, 0);
                } else if (top & 0x80008000u) {
                  some = true;
                  uint16_t* e = reinterpret_cast<uint16_t*>(at + (ch ^ (r & 3)));
                  for (int k = 0; k < 8; ++k)
                    if ((e[k] & 0x7f80u) == 0x7f80u) e[k] = 0;
                }
              }
            }
            if (some) *spoilt = n + 1;
            ptx::fence_proxy_async_smem();  // (before the next copy into this stage)
          }
        }
        float mx[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = fmaxf(fmaxf(sc[0][2 * x], sc[0][2 * x + 1]), fmaxf(sc[1][2 * x], sc[1][2 * x + 1]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          if (q4 == 0) sMax[warp * kRows + g + 8 * x] = v;
          mx[x] = v;
        }
        tc::named_sync(1, 128);
        float nm[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float* v = sMax + g + 8 * x;
          const float top = fmaxf(fmaxf(fmaxf(v[0], v[kRows]), fmaxf(v[2 * kRows], v[3 * kRows])) * c, m[x]);
          const float sub = top == -INFINITY ? 0.f : top;  // no key of this row's yet
          const float a = ptx::ex2(m[x] - sub);
          nm[x] = -sub, m[x] = top, l[x] *= a;
#pragma unroll
          for (int u = 0; u < NT; ++u) o[u][2 * x] *= a, o[u][2 * x + 1] *= a;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float e0 = ptx::ex2(fmaf(sc[u][2 * x], c, nm[x])), e1 = ptx::ex2(fmaf(sc[u][2 * x + 1], c, nm[x]));
            l[x] += e0 + e1;
            const int r = g + 8 * x;
            *reinterpret_cast<uint32_t*>(sm + L::oP + r * 128 + (((warp * 2 + u) ^ (r & 7)) << 4) + q4 * 4) = ptx::pack_bf16(e0, e1);
          }
        tc::named_sync(1, 128);
#pragma unroll
        for (int k = 0; k < MK / 16; ++k) {
          uint32_t a[4];
          const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
          ldm4(sP + r * 128 + (((k * 2 + (lane >> 4)) ^ (r & 7)) << 4), a);
          const uint32_t row = V + (k * 2 + ((lane >> 3) & 1)) * pg.sbo + (lane & 7) * 128;
#pragma unroll
          for (int u = 0; u < NT; u += 2) {
            const int ch = warp * NT + u + (lane >> 4);  // 8-column chunk
            uint32_t f[4];
            ldm4t(row + (ch >> 3) * pg.slab + (((ch & 7) ^ (lane & 7)) << 4), f);
            mma(o[u], a, f[0], f[1]);
            mma(o[u + 1], a, f[2], f[3]);
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&empty[s]);
      }
      // The rows' sums, over the warps' keys.
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (q4 == 0) sMax[warp * kRows + g + 8 * x] = l[x];
      }
      tc::named_sync(1, 128);
      const int slot = it->slot;
      const bool bad = *spoilt == n + 1;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = g + 8 * x, t = r / gt;
        if (r >= rows) continue;
        const float* v = sMax + r;
        const float sum = (v[0] + v[kRows]) + (v[2 * kRows] + v[3 * kRows]);
        const float inv = sum == 0.f ? 0.f : slot >= 0 ? 1.f : 1.f / sum;  // (a row that sees no key: 0)
        const int64_t h = h0 + r - t * gt, pos = it->row0 + it->t0 + t;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.O) + it->batch * out.os[0] + h * out.os[1] + pos * out.os[2];
        float* part = slot >= 0 ? sp.o(slot, r) : nullptr;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          const int col = (warp * NT + u) * 8 + q4 * 2;
          if (col >= d) continue;
          const float y0 = sum == 0.f ? 0.f : o[u][2 * x] * inv, y1 = sum == 0.f ? 0.f : o[u][2 * x + 1] * inv;
          if (part != nullptr) *reinterpret_cast<float2*>(part + col) = make_float2(y0, y1);
          else *reinterpret_cast<uint32_t*>(dst + col) = ptx::pack_bf16(y0, y1);
        }
        if (warp == 0 && q4 == 0) {
          if (part != nullptr) *sp.ml(slot, r) = make_float2(m[x], sum);
          else if (out.lse != nullptr)
            out.lse[it->batch * out.ls[0] + h * out.ls[1] + pos] = sum == 0.f ? -INFINITY : (m[x] + log2f(sum)) * 0.69314718055994531f;
        }
      }
      if (bad) {  // values made 0 for the rows that do not see them
        tc::named_sync(1, 128);
        __threadfence_block();
        const int r = threadIdx.x, t = r / gt;
        if (r < rows) {
          const int64_t at = static_cast<int64_t>(it->start) + it->t0 + t, end = it->len - 1;
          const int hi = static_cast<int>(w.causal ? max(min(at, end), static_cast<int64_t>(-1)) : end);
          const int64_t f = w.window > 0 ? at - w.window + 1 : 0;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.O) + it->batch * out.os[0] + (h0 + r - t * gt) * out.os[1] +
                               static_cast<int64_t>(it->row0 + it->t0 + t) * out.os[2];
          add_spoilt(w, *it, static_cast<int>(f > 0 ? f : 0), hi, Vg + it->kvh * vs1, vs0, vs2, d, dst,
                     slot >= 0 ? sp.o(slot, r) : nullptr, MK);
        }
      }
    }
  }
  __syncthreads();
  // A wait has given up: copies may still be on their way into this CTA's shared memory.
  if (*abort_flag != 0 && threadIdx.x == 0)
    for (int s = 0; s < NS && s < *started; ++s) ptx::settle(&full[s], handover::last_phase(*started, NS, s));
}

template <int D>
cudaError_t launch(const PagedArgs& a, const Work& w, const Space& sp, const Out& out, cudaStream_t st) {
  alignas(64) CUtensorMap mk, mv;
  Pages pg;
  if (!make_maps(a, w.cut, MK, D / 64, nullptr, &mk, &mv, pg)) return cudaErrorInvalidValue;
  auto kern = token_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::bytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(w.cut.ctas), kThreads, Lay<D>::bytes, st>>>(
      mk, mv, w, sp, out, static_cast<const __nv_bfloat16*>(a.Q), a.qs[0], a.qs[1], a.qs[2], static_cast<const __nv_bfloat16*>(a.V),
      a.vs[0], a.vs[1], a.vs[2], a.d, pg, a.scale, a.scale * kLog2e);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return join(w, sp, out, a.dtype, a.d, kRows, a.max_new, st);
}

int columns(const PagedArgs& a) { return a.d <= 64 ? 64 : a.d <= 128 ? 128 : 256; }

Work work_of(const PagedArgs& a) {
  Work w;
  const int g = a.H / a.Hkv;
  w.seqs = a.seqs, w.causal = a.causal, w.window = a.window;
  w.cut.gt = heads_together(g, kRows, a.max_new);
  w.cut.nv = a.H / w.cut.gt, w.cut.per_kv = g / w.cut.gt;
  w.cut.tile = w.cut.step = kRows / w.cut.gt;
  w.cut.shift = 6, w.cut.over = 1, w.cut.least = 4, w.cut.ctas = 152 * (columns(a) == 256 ? 1 : 2);
  return w;
}

}  // namespace

size_t token_bytes(const PagedArgs& a) { return Space::bytes(work_of(a).cut.ctas, kRows, columns(a)); }

cudaError_t token_paged(const PagedArgs& a, void* ws, cudaStream_t st) {
  const Work w = work_of(a);
  const Space sp = Space::at(ws, w.cut.ctas, kRows, columns(a));
  const Out out{a.O, a.lse, {a.os[0], a.os[1], a.os[2]}, {a.ls[0], a.ls[1]}};
  // d = 32 and 96: the columns past d are zeros (TMA fills them).
  return a.d <= 64 ? launch<64>(a, w, sp, out, st) : a.d <= 128 ? launch<128>(a, w, sp, out, st) : launch<256>(a, w, sp, out, st);
}

}  // namespace paged

uint32_t token_paged_take_error() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, paged::g_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(paged::g_err, &z, sizeof(z));
  return v;
}

}  // namespace fbd
