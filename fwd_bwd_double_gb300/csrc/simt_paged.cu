// Attention of new tokens over a paged cache in float32, on the CUDA cores: online softmax over blocks of 64
// keys, fp32 throughout.
//
// A CTA of 256 threads holds R rows (tokens times the query heads that share a key/value head) and streams
// K and V through shared memory; a row belongs to 16 threads of a half-warp, R / 16 rows to a thread,
// so that scores, maxima and probabilities pass between them by shuffles and a row of shared memory.
// Keys that the sequence does not hold are not read; a key hidden from a row has weight 0 there and its
// value is left out of the sum, whatever it is.
#include "paged_launch.h"

namespace fbd {
namespace paged {
namespace {

constexpr int kT = 256, BN = 64;

template <int D, int R>
struct Lay {
  static constexpr int PK = D + 4, PP = BN + 4;
  static constexpr int kStage = BN * (PK + D);      // K and V of a block
  static constexpr int NB = D <= 128 ? 2 : 1;       // blocks: the next one's copies run behind this one's sums
  static constexpr int oQ = 0, oStage = oQ + R * D, oP = oStage + NB * kStage;
  static constexpr int bytes = 4 * (oP + R * PP);
};

// 16 bytes global -> shared, or 16 bytes of zeros (nothing is read) where !in.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void put2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }

template <int D, int R>
__global__ void __launch_bounds__(kT, (D <= 64 ? 2 : 1))
    paged_kernel(const Work w, const Space sp, const Out out, const float* __restrict__ Q, const float* __restrict__ K,
                 const float* __restrict__ V, int64_t qs0, int64_t qs1, int64_t qs2, int64_t ks0, int64_t ks1, int64_t ks2,
                 int64_t vs0, int64_t vs1, int64_t vs2, float c) {
  using L = Lay<D, R>;
  constexpr int RT = R / 16, C2 = D / 32;  // rows, pairs of columns of a thread
  extern __shared__ __align__(16) float sh[];
  float *sQ = sh + L::oQ, *sP = sh + L::oP;
  __shared__ Plan planned;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, p = blockIdx.x, gt = w.cut.gt;
  ptx::grid_dependency_launch();
  if (threadIdx.x < 32) {
    const Plan r = plan(w, p);
    if (threadIdx.x == 0) planned = r;
  }
  __syncthreads();
  Tail tail{0, 0, 0, 0};
  Walk it;
  for (bool more = it.begin(w, planned); more; more = it.next(w)) {
    const Seq& s = it.s;
    const int rows = (it.t1 - it.t0) * gt, kvh = it.vh / w.cut.per_kv;
    const int64_t h0 = static_cast<int64_t>(it.vh) * gt;
    __syncthreads();
    for (int u = threadIdx.x; u < R * D / 4; u += kT) {
      const int r = u / (D / 4), cc = u % (D / 4) * 4, t = r / gt;
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) q = load4(Q + s.batch * qs0 + (h0 + r - t * gt) * qs1 + static_cast<int64_t>(s.row0 + it.t0 + t) * qs2 + cc);
      *reinterpret_cast<float4*>(sQ + r * D + cc) = make_float4(q.x * c, q.y * c, q.z * c, q.w * c);
    }
    int first[RT], last[RT];  // keys that the thread's rows see
    float m[RT], l[RT], acc[RT][C2][2];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int t = it.t0 + (ty * RT + i) / gt;
      const int64_t at = static_cast<int64_t>(s.start) + t;
      last[i] = w.causal ? static_cast<int>(at < s.len ? at : s.len - 1) : s.len - 1;
      const int64_t f = w.window > 0 ? at - w.window + 1 : 0;
      first[i] = static_cast<int>(f > 0 ? f : 0);
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int x = 0; x < C2; ++x) acc[i][x][0] = acc[i][x][1] = 0.f;
    }
    const int64_t at0 = static_cast<int64_t>(s.start) + it.t0, at1 = static_cast<int64_t>(s.start) + it.t1 - 1;
    // Block k's copies into its buffer; the 16-key runs of it without a page or behind the last key.
    auto load = [&](int k) {
      const int64_t key0 = static_cast<int64_t>(it.j0 + k) * BN;
      const uint32_t dst = ptx::smem_u32(sh + L::oStage + (L::NB == 2 ? k & 1 : 0) * L::kStage);
      unsigned gone = 0;
      int page[BN / 16], slot[BN / 16];
#pragma unroll
      for (int g = 0; g < BN / 16; ++g) {
        const int64_t j = key0 + g * 16;
        const int e = static_cast<int>(j) / w.seqs.page;
        page[g] = j < s.len ? page_at(w.seqs, it.b, e) : -1, slot[g] = static_cast<int>(j) - e * w.seqs.page;
        if (page[g] < 0) gone |= 1u << g;
      }
      constexpr int C = D / 4, kStep = kT / C;  // 16-byte pieces of a key; keys a step
#pragma unroll
      for (int r0 = 0; r0 < BN; r0 += kStep) {
        const int r = r0 + threadIdx.x / C, cc = threadIdx.x % C * 4;
        if (kT % C != 0 && (threadIdx.x / C >= kStep || r >= BN)) continue;
        int pg = page[0], sl = slot[0];
#pragma unroll
        for (int g = 1; g < BN / 16; ++g)
          if (r >> 4 == g) pg = page[g], sl = slot[g];
        // keys that the sequence does not hold are not read: zeros there (a cache row not yet written may hold anything)
        const bool in = pg >= 0 && key0 + r < s.len;
        const int64_t at = in ? sl + (r & 15) : 0;
        copy16(dst + (r * L::PK + cc) * 4, in ? K + pg * ks0 + kvh * ks1 + at * ks2 + cc : K, in);
        copy16(dst + (BN * L::PK + r * D + cc) * 4, in ? V + pg * vs0 + kvh * vs1 + at * vs2 + cc : V, in);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return gone;
    };
    unsigned gone = load(it.k0), then = 0;
    for (int k = it.k0; k < it.k1; ++k, gone = then) {
      const int64_t key0 = static_cast<int64_t>(it.j0 + k) * BN;
      const float *sK = sh + L::oStage + (L::NB == 2 ? k & 1 : 0) * L::kStage, *sV = sK + BN * L::PK;
      if (L::NB == 1 && k > it.k0) {
        __syncthreads();  // the block before has been read
        gone = load(k);
      }
      if (L::NB == 2 && k + 1 < it.k1) {
        then = load(k + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      // some row does not see some key of the block
      const bool part = gone != 0 || key0 + BN > s.len || (w.causal && key0 + BN - 1 > at0) || (w.window > 0 && key0 <= at1 - w.window);
      float sc[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[i][x] = 0.f;
#pragma unroll 8
      for (int d = 0; d < D; d += 4) {
        float4 kk[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) kk[x] = *reinterpret_cast<const float4*>(sK + (tx + 16 * x) * L::PK + d);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(sQ + (ty * RT + i) * D + d);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            sc[i][x] = fmaf(q.x, kk[x].x, fmaf(q.y, kk[x].y, fmaf(q.z, kk[x].z, fmaf(q.w, kk[x].w, sc[i][x]))));
        }
      }
      float alpha[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (part) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int64_t j = key0 + tx + 16 * x;
            if (j < first[i] || j > last[i] || (gone >> x & 1)) sc[i][x] = -INFINITY;  // (key tx + 16 x: run x)
          }
        }
        float t = fmaxf(fmaxf(sc[i][0], sc[i][1]), fmaxf(sc[i][2], sc[i][3]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
        const float mn = fmaxf(m[i], t), sub = mn == -INFINITY ? 0.f : mn;
        alpha[i] = ptx::ex2(m[i] - sub);
        m[i] = mn;
        float z = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float e = ptx::ex2(sc[i][x] - sub);
          z += e;
          sP[(ty * RT + i) * L::PP + tx + 16 * x] = e;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        l[i] = fmaf(l[i], alpha[i], z);
      }
      __syncwarp();
      // The block's sums, then added to the running ones: a chain of additions as long as the context would
      // lose bits with its square root.
      float o[RT][C2][2];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int x = 0; x < C2; ++x) o[i][x][0] = o[i][x][1] = 0.f;
      for (int j = 0; j < BN; j += 4) {
        float4 e[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) e[i] = *reinterpret_cast<const float4*>(sP + (ty * RT + i) * L::PP + j);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float2 v[C2];
#pragma unroll
          for (int x = 0; x < C2; ++x) v[x] = *reinterpret_cast<const float2*>(sV + (j + u) * D + tx * 2 + 32 * x);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float f = u == 0 ? e[i].x : u == 1 ? e[i].y : u == 2 ? e[i].z : e[i].w;
            if (part && f == 0.f) continue;  // (hidden: 0 times an infinity would be NaN)
#pragma unroll
            for (int x = 0; x < C2; ++x) o[i][x][0] = fmaf(f, v[x].x, o[i][x][0]), o[i][x][1] = fmaf(f, v[x].y, o[i][x][1]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int x = 0; x < C2; ++x)
          acc[i][x][0] = fmaf(acc[i][x][0], alpha[i], o[i][x][0]), acc[i][x][1] = fmaf(acc[i][x][1], alpha[i], o[i][x][1]);
      if (L::NB == 2) __syncthreads();  // (this block's buffer is the next but one's)
    }
    const bool whole = it.whole();
    const int slot = it.slot(p);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty * RT + i;
      if (r >= rows) break;
      if (!whole) {
#pragma unroll
        for (int x = 0; x < C2; ++x) put2(sp.o(slot, r) + tx * 2 + 32 * x, acc[i][x][0], acc[i][x][1]);
        if (tx == 0) *sp.ml(slot, r) = make_float2(m[i], l[i]);
        continue;
      }
      const int t = r / gt;
      const int64_t h = h0 + r - t * gt, pos = s.row0 + it.t0 + t;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // (a row that sees no key: 0)
      float* dst = static_cast<float*>(out.O) + s.batch * out.os[0] + h * out.os[1] + pos * out.os[2];
#pragma unroll
      for (int x = 0; x < C2; ++x) put2(dst + tx * 2 + 32 * x, acc[i][x][0] * inv, acc[i][x][1] * inv);
      if (tx == 0 && out.lse != nullptr)
        out.lse[s.batch * out.ls[0] + h * out.ls[1] + pos] =
            l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
    }
    if (!whole && it.k0 == 0) tail = Tail{it.b, it.tile, it.vh, it.parts(p)};
  }
  if (threadIdx.x == 0) sp.tail[p] = tail;
}

template <int D, int R>
cudaError_t launch(const PagedArgs& a, const Work& w, const Space& sp, const Out& out, cudaStream_t st) {
  auto kern = paged_kernel<D, R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, R>::bytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(w.cut.ctas), kT, Lay<D, R>::bytes, st>>>(w, sp, out, static_cast<const float*>(a.Q), static_cast<const float*>(a.K),
                    static_cast<const float*>(a.V), a.qs[0], a.qs[1], a.qs[2], a.ks[0], a.ks[1], a.ks[2], a.vs[0], a.vs[1],
                    a.vs[2], a.scale * kLog2e);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return join(w, sp, out, a.dtype, D, R, a.max_new, st);
}

template <int D>
cudaError_t rows(const PagedArgs& a, const Work& w, const Space& sp, const Out& out, cudaStream_t st) {
  return sp.rows == 16 ? launch<D, 16>(a, w, sp, out, st) : launch<D, 64>(a, w, sp, out, st);
}

// 16 rows a tile where the new tokens of a sequence fit them, else 64.
int tile_rows(const PagedArgs& a) { return a.max_new * (a.H / a.Hkv) <= 16 ? 16 : 64; }

Work work_of(const PagedArgs& a) {
  Work w;
  const int R = tile_rows(a), g = a.H / a.Hkv;
  w.seqs = a.seqs, w.causal = a.causal, w.window = a.window;
  w.cut.gt = heads_together(g, R, R == 16 ? a.max_new : 0);
  w.cut.nv = a.H / w.cut.gt, w.cut.per_kv = g / w.cut.gt;
  w.cut.tile = w.cut.step = R / w.cut.gt;
  w.cut.shift = 6, w.cut.over = 1, w.cut.least = 4;
  w.cut.ctas = 152 * (a.d <= 64 ? 2 : 1);  // CTAs that fit an SM
  return w;
}

}  // namespace

size_t simt_bytes(const PagedArgs& a) {
  const Work w = work_of(a);
  return Space::bytes(w.cut.ctas, tile_rows(a), a.d);
}

cudaError_t simt_paged(const PagedArgs& a, void* ws, cudaStream_t st) {
  const Work w = work_of(a);
  const Space sp = Space::at(ws, w.cut.ctas, tile_rows(a), a.d);
  const Out out{a.O, a.lse, {a.os[0], a.os[1], a.os[2]}, {a.ls[0], a.ls[1]}};
  return a.d == 32 ? rows<32>(a, w, sp, out, st) : a.d == 64 ? rows<64>(a, w, sp, out, st) : a.d == 96 ? rows<96>(a, w, sp, out, st)
         : a.d == 128 ? rows<128>(a, w, sp, out, st) : rows<256>(a, w, sp, out, st);
}

}  // namespace paged
}  // namespace fbd
