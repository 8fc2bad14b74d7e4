// Attention of new tokens over a paged cache in float32, on the CUDA cores: online softmax over blocks of
// keys, fp32 throughout.  A CTA of 256 threads holds R rows (tokens times the query heads that share a
// key/value head) and streams K and V through shared memory, the next block's copies behind this one's sums.
// Keys that the sequence does not hold are not read; a key hidden from a row has weight 0 there and its
// value is left out of the sum, whatever it is.
//
// R = 64 (paged_kernel): a row belongs to 16 threads of a half-warp, four rows to a thread, so that scores, maxima and
// probabilities pass between them by shuffles and a row of shared memory.  Bound by the reads of shared memory beside the
// multiply-adds (32 cycles of reads for 16 of products; two floats an instruction made it slower, 652 -> 830 us): 4 x 1000
// tokens over 3000 keys, 8 heads of 64 in pairs (20 GFLOP) 604 us, 34 TFLOP/s; at d = 256 2.3 ms (2.6 with the test for
// hidden keys in every block's products).
// R = 4, 8, 16 (few_kernel): one or a few tokens, bound by reading the cache.  A warp takes an eighth of a block's keys
// for all rows, so that K and V are read from shared memory once, not by every warp, and keeps maxima, sums and
// outputs of its own, which meet at the end of the item.  32 tokens over 100 to 4000 keys, 16 heads in groups of 4: at
// d = 128 (269 MB) 83 us, 3.2 TB/s, at d = 64 51 us (with rows dealt to half-warps as above 248 and 116), bound by
// the instructions a key (half of the issue slots) and the waits of their chains.
#include <type_traits>

#include "paged_launch.h"

namespace fbd {
namespace paged {
namespace {

constexpr int kT = 256, BN = 64;

template <int D, int R>
struct Lay {
  static constexpr int PK = D + 4, PP = BN + 4;  // pitches of K and P
  static constexpr int kStage = BN * (PK + D);      // K and V of a block
  static constexpr int NB = D <= 128 ? 2 : 1;       // blocks: the next one's copies run behind this one's sums
  static constexpr int oQ = 0, oStage = oQ + R * D, oP = oStage + NB * kStage;
  static constexpr int bytes = 4 * (oP + R * PP);
};

// 16 bytes global -> shared, or 16 bytes of zeros (nothing is read) where !in.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// A block's K and V to shared memory (pitches PK, D).  A warp looks up the pages of 32 runs of 16 keys at a time, a lane
// each, and those of the next 32 before it needs them, so that the copies wait for no page.
struct Runs {
  int page, slot;  // page < 0: none, or behind the last key
};
__device__ __forceinline__ Runs run_at(const Work& w, const Walk& it, int64_t key) {
  Runs r{-1, 0};
  if (key < it.s.len) {
    const int e = static_cast<int>(key) / w.seqs.page;
    r.page = page_at(w.seqs, it.b, e), r.slot = static_cast<int>(key) - e * w.seqs.page;
  }
  return r;
}
template <int KN>
struct Lookup {  // of blocks k0, k0 + 1, ... of an item, in order
  Runs now, then;
  int64_t key;  // of this lane's run of `then`
  int at;       // the lane of the next block's first run
  __device__ __forceinline__ Lookup(const Work& w, const Walk& it) {
    key = static_cast<int64_t>(it.j0 + it.k0) * KN + threadIdx.x % 32 * 16;
    now = run_at(w, it, key);
    key += 512;
    then = run_at(w, it, key);
    at = 0;
  }
  __device__ __forceinline__ void next(const Work& w, const Walk& it) {
    at += KN / 16;
    if (at < 32) return;
    at = 0, now = then, key += 512;
    then = run_at(w, it, key);
  }
};
// This thread's part of the copies, from the addresses of its piece of a key of the head (first: its key of a step); their
// group.  The runs without a page.  Keys that the sequence does not hold are not read: zeros there (a cache row
// not yet written may hold anything).
template <int D, int KN, int PK>
__device__ __forceinline__ unsigned copy_block(const Walk& it, int k, const Runs& x, int lane0, const float* K, const float* V, int64_t ks0,
                                               int64_t ks2, int64_t vs0, int64_t vs2, float* to) {
  constexpr int C = D / 4, kStep = kT / C, NR = KN / 16;  // 16-byte pieces of a key; keys a step
  const int first = threadIdx.x / C, held = static_cast<int>(min(static_cast<int64_t>(KN), it.s.len - static_cast<int64_t>(it.j0 + k) * KN));
  const uint32_t dst = ptx::smem_u32(to) + (first * PK + threadIdx.x % C * 4) * 4;
  const uint32_t dst_v = ptx::smem_u32(to) + (KN * PK + first * D + threadIdx.x % C * 4) * 4;
  const unsigned gone = (__ballot_sync(0xffffffffu, x.page < 0) >> lane0) & ((1u << NR) - 1);
  int64_t ko = 0, vo = 0;
#pragma unroll
  for (int r0 = 0; r0 < KN; r0 += kStep) {
    const int r = r0 + first;
    constexpr bool kOne = 16 % kStep == 0;  // a step lies in one run
    if (!kOne || r0 % 16 == 0) {
      const int g = kOne ? r0 / 16 : min(r / 16, NR - 1);
      const int page = max(__shfl_sync(0xffffffffu, x.page, lane0 + g), 0), slot = __shfl_sync(0xffffffffu, x.slot, lane0 + g);
      const int64_t at = slot + (kOne ? first : r % 16);
      ko = page * ks0 + at * ks2, vo = page * vs0 + at * vs2;
    }
    if (kT % C != 0 && (first >= kStep || r >= KN)) continue;
    const bool in = r < held && !(gone >> (kOne ? r0 / 16 : r / 16) & 1);
    const int more = kOne ? r0 % 16 : 0;
    copy16(dst + r0 * PK * 4, K + ko + more * ks2, in);
    copy16(dst_v + r0 * D * 4, V + vo + more * vs2, in);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  return gone;
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
    const float *Kh = K + kvh * ks1 + threadIdx.x % (D / 4) * 4, *Vh = V + kvh * vs1 + threadIdx.x % (D / 4) * 4;
    Lookup<BN> runs(w, it);
    auto load = [&](int k) {
      const unsigned gone = copy_block<D, BN, L::PK>(it, k, runs.now, runs.at, Kh, Vh, ks0, ks2, vs0, vs2,
                                                     sh + L::oStage + (L::NB == 2 ? k & 1 : 0) * L::kStage);
      runs.next(w, it);
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
      auto products = [&](auto some) {  // some: keys may be hidden
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
              if (some.value && f == 0.f) continue;  // (hidden: 0 times an infinity would be NaN)
#pragma unroll
              for (int x = 0; x < C2; ++x) o[i][x][0] = fmaf(f, v[x].x, o[i][x][0]), o[i][x][1] = fmaf(f, v[x].y, o[i][x][1]);
            }
          }
        }
      };
      if (part) products(std::true_type{}); else products(std::false_type{});
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

// The few rows' shared memory: a ring of blocks of 64 or 32 keys; at an item's end the warps' outputs over it.
constexpr int few_keys(int D) { return D <= 64 ? 64 : 32; }
constexpr int few_per_sm(int D, int R) { return D <= 64 || (D <= 128 && R <= 8) ? 2 : 1; }  // CTAs whose registers fit an SM
template <int D, int R>
struct Few {
  static constexpr int KN = few_keys(D), KW = KN / 8, LK = 32 / KW;  // keys of a warp, lanes of a key (its 16-byte pieces go round them)
  static constexpr int kStage = KN * 2 * D;
  static constexpr int kFit = (few_per_sm(D, R) == 2 ? 98304 : 196608) / (4 * kStage), NS = kFit < 8 ? kFit : 8;
  static constexpr int oQ = 0, oStage = oQ + R * D, oP = oStage + NS * kStage, oML = oP + 8 * R * KW;  // P, (m, l) of a warp
  static constexpr int bytes = 4 * (oML + 8 * R * 2);
  static constexpr int VW = D % 128 == 0 ? 4 : D == 64 ? 2 : 1, NX = D / 32 / VW;  // a lane's columns: NX runs of VW
  static_assert(NS >= 3 && 8 * R * D <= NS * kStage, "the ring");
  static_assert((bytes + 2048) * few_per_sm(D, R) <= 233472, "shared memory");
};
template <int VW>
__device__ __forceinline__ void take(const float* p, float* v) {
  if constexpr (VW == 4) {
    const float4 x = load4(p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else if constexpr (VW == 2) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x, v[1] = x.y;
  } else {
    v[0] = *p;
  }
}

template <int D, int R>
__global__ void __launch_bounds__(kT, few_per_sm(D, R))
    few_kernel(const Work w, const Space sp, const Out out, const float* __restrict__ Q, const float* __restrict__ K,
               const float* __restrict__ V, int64_t qs0, int64_t qs1, int64_t qs2, int64_t ks0, int64_t ks1, int64_t ks2,
               int64_t vs0, int64_t vs1, int64_t vs2, float c) {
  using L = Few<D, R>;
  constexpr int KN = L::KN, KW = L::KW, LK = L::LK, VW = L::VW, NX = L::NX, NC = VW * NX, NS = L::NS;
  constexpr int NR = KN / 16, K4 = D / 4 / LK;  // runs of a block; 16-byte pieces of a key that a lane holds
  extern __shared__ __align__(16) float sh[];
  __shared__ Plan planned;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, p = blockIdx.x, gt = w.cut.gt;
  const int key = warp * KW + lane / LK, part = lane % LK;  // this lane's key of a block, its share of the columns
  const int odd = LK == 4 ? (lane & 4) : 0;  // odd keys take their pieces the other way round: two keys' would share banks
  float *sQ = sh + L::oQ, *sP = sh + L::oP + warp * R * KW;
  float2* sML = reinterpret_cast<float2*>(sh + L::oML);
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
    __syncthreads();  // the item before has been joined
    const float *Kh = K + kvh * ks1 + threadIdx.x % (D / 4) * 4, *Vh = V + kvh * vs1 + threadIdx.x % (D / 4) * 4;
    Lookup<KN> runs(w, it);
    unsigned gone = 0;  // runs without a page of the blocks on their way, NR bits each
    int ahead = it.k0, into = 0, from = 0;
    auto load = [&] {
      if (ahead < it.k1) {
        gone |= copy_block<D, KN, D>(it, ahead, runs.now, runs.at, Kh, Vh, ks0, ks2, vs0, vs2, sh + L::oStage + into * L::kStage)
                << (NR * (NS - 2));
        runs.next(w, it);
        ++ahead, into = into + 1 == NS ? 0 : into + 1;
      } else {
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
    };
#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) {
      gone >>= NR;
      load();
    }
    for (int u = threadIdx.x; u < R * D / 4; u += kT) {
      const int r = u / (D / 4), cc = u % (D / 4) * 4, t = r / gt;
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) q = load4(Q + s.batch * qs0 + (h0 + r - t * gt) * qs1 + static_cast<int64_t>(s.row0 + it.t0 + t) * qs2 + cc);
      *reinterpret_cast<float4*>(sQ + r * D + cc) = make_float4(q.x * c, q.y * c, q.z * c, q.w * c);
    }
    const int64_t at0 = static_cast<int64_t>(s.start) + it.t0, at1 = static_cast<int64_t>(s.start) + it.t1 - 1;
    float m[R], l[R], acc[R][NC];  // of the warp's keys; l: of this lane's key's place alone
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int x = 0; x < NC; ++x) acc[i][x] = 0.f;
    }
    for (int k = it.k0; k < it.k1; ++k) {
      const int64_t key0 = static_cast<int64_t>(it.j0 + k) * KN;
      const float *sK = sh + L::oStage + from * L::kStage, *sV = sK + KN * D;
      from = from + 1 == NS ? 0 : from + 1;
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
      __syncthreads();  // ... and the block before has been read
      const unsigned none = gone & ((1u << NR) - 1);
      gone >>= NR;
      load();
      // some row does not see some key of the block
      const bool cut = none != 0 || key0 + KN > s.len || (w.causal && key0 + KN - 1 > at0) || (w.window > 0 && key0 <= at1 - w.window);
      float sc[R], alpha[R];
      {
        float4 kk[K4];
#pragma unroll
        for (int x = 0; x < K4; ++x) kk[x] = load4(sK + key * D + ((x * LK + part) ^ odd) * 4);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          float a = 0.f;
#pragma unroll
          for (int x = 0; x < K4; ++x) {
            const float4 q = load4(sQ + i * D + ((x * LK + part) ^ odd) * 4);
            a = fmaf(q.x, kk[x].x, fmaf(q.y, kk[x].y, fmaf(q.z, kk[x].z, fmaf(q.w, kk[x].w, a))));
          }
#pragma unroll
          for (int o = 1; o < LK; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
          sc[i] = a;
        }
      }
      if (cut) {
        const int64_t j = key0 + key;
        const bool held = !(none >> (key >> 4) & 1) && j < s.len;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int64_t at = at0 + i / gt;
          if (!held || (w.causal && j > at) || (w.window > 0 && j <= at - w.window)) sc[i] = -INFINITY;
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float t = sc[i];
#pragma unroll
        for (int o = LK; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
        const float mn = fmaxf(m[i], t), sub = mn == -INFINITY ? 0.f : mn;
        alpha[i] = ptx::ex2(m[i] - sub);
        m[i] = mn;
        const float e = ptx::ex2(sc[i] - sub);
        l[i] = fmaf(l[i], alpha[i], e);
        if (part == 0) sP[i * KW + lane / LK] = e;
      }
      __syncwarp();
      // The block's sums, then added to the running ones (as above).
      float v[KW][NC];
#pragma unroll
      for (int j = 0; j < KW; ++j)
#pragma unroll
        for (int x = 0; x < NX; ++x) take<VW>(sV + (warp * KW + j) * D + (x * 32 + lane) * VW, v[j] + x * VW);
      auto products = [&](auto some) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          float e[KW], o[NC];
#pragma unroll
          for (int j = 0; j < KW; j += 4) take<4>(sP + i * KW + j, e + j);
#pragma unroll
          for (int x = 0; x < NC; ++x) o[x] = 0.f;
#pragma unroll
          for (int j = 0; j < KW; ++j) {
            if (some.value && e[j] == 0.f) continue;  // (hidden: 0 times an infinity would be NaN)
#pragma unroll
            for (int x = 0; x < NC; ++x) o[x] = fmaf(e[j], v[j][x], o[x]);
          }
#pragma unroll
          for (int x = 0; x < NC; ++x) acc[i][x] = fmaf(acc[i][x], alpha[i], o[x]);
        }
      };
      if (cut) products(std::true_type{}); else products(std::false_type{});
    }
    // The warps' outputs meet.
    __syncthreads();
    float* sO = sh + L::oStage;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i >= rows) break;
#pragma unroll
      for (int o = LK; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      if (lane == 0) sML[warp * R + i] = make_float2(m[i], l[i]);
#pragma unroll
      for (int x = 0; x < NC; ++x) sO[(warp * R + i) * D + (x / VW * 32 + lane) * VW + x % VW] = acc[i][x];
    }
    __syncthreads();
    const bool whole = it.whole();
    const int slot = it.slot(p);
    for (int u = threadIdx.x; u < rows * (D / 4); u += kT) {
      const int r = u / (D / 4), cc = u % (D / 4) * 4;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, sML[k * R + r].x);
      const float sub = top == -INFINITY ? 0.f : top;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 z = sML[k * R + r];
        const float f = ptx::ex2(z.x - sub);
        const float4 x = load4(sO + (k * R + r) * D + cc);
        sum = fmaf(f, z.y, sum);
        o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y), o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
      }
      if (!whole) {
        *reinterpret_cast<float4*>(sp.o(slot, r) + cc) = o;
        if (cc == 0) *sp.ml(slot, r) = make_float2(top, sum);
        continue;
      }
      const int t = r / gt;
      const int64_t h = h0 + r - t * gt, pos = s.row0 + it.t0 + t;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (a row that sees no key: 0)
      *reinterpret_cast<float4*>(static_cast<float*>(out.O) + s.batch * out.os[0] + h * out.os[1] + pos * out.os[2] + cc) =
          make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      if (cc == 0 && out.lse != nullptr)
        out.lse[s.batch * out.ls[0] + h * out.ls[1] + pos] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    }
    if (!whole && it.k0 == 0) tail = Tail{it.b, it.tile, it.vh, it.parts(p)};
  }
  if (threadIdx.x == 0) sp.tail[p] = tail;
}

template <int D, int R>
cudaError_t launch(const PagedArgs& a, const Work& w, const Space& sp, const Out& out, cudaStream_t st) {
  auto kern = paged_kernel<D, 64>;
  int bytes = Lay<D, 64>::bytes;
  if constexpr (R < 64) kern = few_kernel<D, R>, bytes = Few<D, R>::bytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(w.cut.ctas), kT, bytes, st>>>(w, sp, out, static_cast<const float*>(a.Q), static_cast<const float*>(a.K),
                    static_cast<const float*>(a.V), a.qs[0], a.qs[1], a.qs[2], a.ks[0], a.ks[1], a.ks[2], a.vs[0], a.vs[1],
                    a.vs[2], a.scale * kLog2e);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return join(w, sp, out, a.dtype, D, R, a.max_new, st);
}

template <int D>
cudaError_t rows(const PagedArgs& a, const Work& w, const Space& sp, const Out& out, cudaStream_t st) {
  return sp.rows == 4 ? launch<D, 4>(a, w, sp, out, st) : sp.rows == 8 ? launch<D, 8>(a, w, sp, out, st)
         : sp.rows == 16 ? launch<D, 16>(a, w, sp, out, st) : launch<D, 64>(a, w, sp, out, st);
}

// As few rows a tile as the new tokens of a sequence fit, else 64.
int tile_rows(const PagedArgs& a) {
  const int64_t n = a.max_new * (a.H / a.Hkv);
  return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 64;
}

Work work_of(const PagedArgs& a) {
  Work w;
  const int R = tile_rows(a), g = a.H / a.Hkv;
  w.seqs = a.seqs, w.causal = a.causal, w.window = a.window;
  w.cut.gt = heads_together(g, R, R < 64 ? a.max_new : 0);
  w.cut.nv = a.H / w.cut.gt, w.cut.per_kv = g / w.cut.gt;
  w.cut.tile = w.cut.step = R / w.cut.gt;
  w.cut.shift = R < 64 && few_keys(a.d) == 32 ? 5 : 6, w.cut.over = 1, w.cut.least = 4;
  w.cut.ctas = 152 * (R < 64 ? few_per_sm(a.d, R) : a.d <= 64 ? 2 : 1);  // CTAs that fit an SM
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
