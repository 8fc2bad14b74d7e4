// RMS norm of each head's vector and its rotary positions in one pass, to [B, heads, N, d] views or
// into the pages of a cache:  z = w x r,  r = (mean x^2 + eps)^(-1/2),  y = R(angle) z,
// and its gradient:  dz = R(-angle) dy,  dw = sum of dz x r,  dx = r (w dz - x r^2 mean(w dz x)).
//
// Bound by reading and writing each element once.  A group of threads (a power of two of them, so
// that a warp holds whole groups; at d = 96 a quarter of them idle) takes a token: a thread holds
// 16 bytes of each half of the head (neighbouring pairs: 32 bytes in a row), so that both
// coordinates of its pairs are its own and the sum of squares is a few shuffles.  The sines of its
// pairs, times the weights, serve all its heads; arithmetic goes two floats an instruction.  Each thread brings its
// own 16-byte pieces by asynchronous copies to a ring in shared memory that only it reads (no barrier), the first
// ones before the tables and the token's place are looked up, and the next token's behind this one's: held in
// registers, half as many bytes were on their way.  Squares, sums and r are fp32; each output is rounded once.
//
// 24 heads of 64 over 32768 tokens in bf16 (201 MB): 39 us, 5.2 TB/s; the gradient (302 MB) 55 us, 5.5 TB/s (with the
// next pieces in registers 41 and 78 us); 19.8 thousand prompt tokens of 16 + 4 + 4 heads of 128 into pages (243 MB)
// 57 us, 4.3 TB/s (with registers 55).  float32: 71 us, 5.7 TB/s; 101 us, 6.0 TB/s; 90 us, 5.4 TB/s.  Half of the issue slots are
// the sums, turns and conversions; that does not bound it, the cut does (split): the 24 heads' blocks take three or four
// groups of tokens where 3.4 would be even, and the SMs are active for 78 % of the time.
#include <cuda_bf16.h>

#include "angle.cuh"
#include "diff.h"
#include "paged.h"

namespace fbd {
namespace {

constexpr int kT = 256;
constexpr int kMaxPairs = 128;

// Threads per token: its pairs in pieces of W, rounded up to a power of two.
__host__ __device__ inline int group_threads(int d, int W) {
  int n = 1;
  while (n * W < d / 2) n *= 2;
  return n;
}

template <int LG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 16 bytes as pairs of floats, and back.
__device__ __forceinline__ void widen2(const uint4& v, uint64_t* x, float) { x[0] = tc::pk2(v.x, v.y), x[1] = tc::pk2(v.z, v.w); }
__device__ __forceinline__ void widen2(const uint4& v, uint64_t* x, __nv_bfloat16) {
  x[0] = tc::bf2_to_f2(v.x), x[1] = tc::bf2_to_f2(v.y), x[2] = tc::bf2_to_f2(v.z), x[3] = tc::bf2_to_f2(v.w);
}
__device__ __forceinline__ uint32_t pack2(uint64_t x) {
  const float2 f = tc::unpk2(x);
  return ptx::pack_bf16(f.x, f.y);
}
__device__ __forceinline__ void put2(float* p, const uint64_t* x) {
  const float2 a = tc::unpk2(x[0]), b = tc::unpk2(x[1]);
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void put2(__nv_bfloat16* p, const uint64_t* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
}
__device__ __forceinline__ uint64_t both(float v) { return tc::pk2f(v, v); }

// The frequencies' turns per step and their axes (outside 0 .. axes - 1: -1).
__device__ __forceinline__ void angle_tables(const float* freq, const int* axis, int pairs, int axes,
                                             unsigned long long* sT, int* sAx) {
  for (int i = threadIdx.x; i < pairs; i += kT) {
    sT[i] = angle::turns_per_step(freq[i]);
    const int ax = axis[i];
    sAx[i] = ax < axes ? ax : -1;
  }
}

// A thread's part of a head: W packed pairs, of its first piece and then of its second.  Its coordinate pair u is
// HALF: elements u of both pieces; else the neighbours 2u, 2u + 1 of the two in a row.
template <typename T, bool HALF>
struct Part {
  static constexpr int W = 16 / sizeof(T);  // pairs of coordinates, and packed words
  // (x0, x1) -> (x0 a + x1 nb, x0 c + x1 d) of every pair
  uint64_t p[W], q[W];  // HALF: a, nb then c, d of two pairs each; else (a, c), (nb, d) of a pair each
  __device__ __forceinline__ void set(int u, float a, float nb, float c, float d) {
    if (HALF) {
      const int k = u / 2;
      const float2 A = tc::unpk2(p[k]), B = tc::unpk2(q[k]), C = tc::unpk2(p[W / 2 + k]), E = tc::unpk2(q[W / 2 + k]);
      p[k] = u % 2 ? tc::pk2f(A.x, a) : tc::pk2f(a, 0.f), q[k] = u % 2 ? tc::pk2f(B.x, nb) : tc::pk2f(nb, 0.f);
      p[W / 2 + k] = u % 2 ? tc::pk2f(C.x, c) : tc::pk2f(c, 0.f), q[W / 2 + k] = u % 2 ? tc::pk2f(E.x, d) : tc::pk2f(d, 0.f);
    } else {
      p[u] = tc::pk2f(a, c), q[u] = tc::pk2f(nb, d);
    }
  }
  __device__ __forceinline__ void apply(const uint64_t (&x)[W], uint64_t (&y)[W]) const {
    if (HALF) {
#pragma unroll
      for (int k = 0; k < W / 2; ++k) {
        y[k] = tc::fma2(x[W / 2 + k], q[k], tc::mul2(x[k], p[k]));
        y[W / 2 + k] = tc::fma2(x[W / 2 + k], q[W / 2 + k], tc::mul2(x[k], p[W / 2 + k]));
      }
    } else {
#pragma unroll
      for (int u = 0; u < W; ++u) {
        const float2 v = tc::unpk2(x[u]);
        y[u] = tc::fma2(both(v.y), q[u], tc::mul2(both(v.x), p[u]));
      }
    }
  }
};

template <int W>
__device__ __forceinline__ float sum_squares(const uint64_t (&x)[W]) {
  uint64_t s = tc::mul2(x[0], x[0]);
#pragma unroll
  for (int k = 1; k < W; ++k) s = tc::fma2(x[k], x[k], s);
  const float2 f = tc::unpk2(s);
  return f.x + f.y;
}

// W floats of a table from c0 on and W from c1 on (ones where it is null).
template <int W>
__device__ __forceinline__ void weights(const float* w, int c0, int c1, float (&w0)[W], float (&w1)[W]) {
#pragma unroll
  for (int u = 0; u < W; ++u) w0[u] = w1[u] = 1.f;
  if (w == nullptr) return;
#pragma unroll
  for (int u = 0; u < W; ++u) w0[u] = __ldg(w + c0 + u), w1[u] = __ldg(w + c1 + u);  // (aligned to 4 bytes only)
}

constexpr int kNear = 512;    // sequences of an append that are looked up in shared memory
constexpr int kAhead = 6;     // heads on their way (the gradient: four of x and of dy)
constexpr int kAheadGrad = 4;

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, bool HALF, bool APPEND, int LG>
__global__ void __launch_bounds__(kT, 2) head_kernel(const HeadArgs a) {
  using P = Part<T, HALF>;
  constexpr int W = P::W;
  __shared__ unsigned long long sT[kMaxPairs];
  __shared__ int sAx[kMaxPairs];
  __shared__ int sCu[APPEND ? kNear + 1 : 1], sLens[APPEND ? kNear : 1];
  const int pairs = a.d / 2, per = pairs / W;
  int t = 0;
  while (static_cast<int>(blockIdx.y) >= a.first[t + 1]) ++t;
  const HeadTensor& z = a.t[t];
  const int hb = (blockIdx.y - a.first[t]) * a.per[t], heads = min(a.per[t], z.heads - hb);
  const int part = threadIdx.x & (LG - 1);
  const bool mine = part < per;  // (the others take part in the shuffles, on the first one's elements)
  const int own = mine ? part : 0;
  const int c0 = HALF ? own * W : 2 * own * W, c1 = HALF ? c0 + pairs : c0 + W;
  const bool packed = APPEND && a.seqs.cu != nullptr;
  const int64_t tokens = a.B * a.N;
  constexpr int step = kT / LG;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * step;
  struct Token {
    int64_t i, b, n;
    const T* x;
  };
  auto token_at = [&](int64_t base) {  // (behind the last one: the last one)
    Token k;
    k.i = min(base + threadIdx.x / LG, tokens - 1);
    k.b = packed ? 0 : k.i / a.N, k.n = k.i - k.b * a.N;
    k.x = static_cast<const T*>(z.x) + k.b * z.xs[0] + hb * z.xs[1] + k.n * z.xs[2];
    return k;
  };
  // This thread's ring: head i of its sequence of (token, head) in place i % kAhead.
  extern __shared__ __align__(16) uint4 ring[];
  uint4* own_ring = ring + threadIdx.x;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * step;
  struct {
    int64_t base;
    const T* x;
    int h, place;
  } ahead;
  ahead.base = first, ahead.h = 0, ahead.place = 0;
  Token tok = token_at(first);
  ahead.x = tok.x;
  auto fetch = [&] {
    if (ahead.base < tokens) {
      copy16(own_ring + ahead.place * 2 * kT, ahead.x + c0);
      copy16(own_ring + (ahead.place * 2 + 1) * kT, ahead.x + c1);
      ahead.place = ahead.place + 1 == kAhead ? 0 : ahead.place + 1;
      ahead.x += z.xs[1];
      if (++ahead.h == heads) {
        ahead.h = 0, ahead.base += stride;
        ahead.x = token_at(ahead.base).x;
      }
    }
    copy_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kAhead - 1; ++i) fetch();
  // Behind those loads: the tables.
  const bool turn = z.turn;
  if (turn) angle_tables(a.freq, a.axis, pairs, a.axes, sT, sAx);
  float w0[W], w1[W];
  weights<W>(z.norm ? z.w : nullptr, c0, c1, w0, w1);
  const float inv = 1.f / static_cast<float>(a.d);
  Seqs q = a.seqs;
  if (APPEND && q.B <= kNear) {
    for (int i = threadIdx.x; i <= q.B; i += kT) {
      if (packed) sCu[i] = q.cu[i];
      if (i < q.B) sLens[i] = q.lens[i];
    }
    if (packed) q.cu = sCu;
    q.lens = sLens;
  }
  if (turn || APPEND) __syncthreads();
  // A token's position in its sequence and its place in the cache (page as the table holds it, unused where
  // it is none).
  struct Place {
    int at, page, slot;
    bool live;
  };
  auto place_at = [&](const Token& k, int64_t base) {
    Place x{0, -1, 0, mine && base + threadIdx.x / LG < tokens};
    if (!APPEND) return x;
    int s = static_cast<int>(packed ? 0 : k.b);
    if (packed) {  // the last sequence that begins at or before this row
      int lo = 0, hi = q.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.cu[mid] <= k.i) lo = mid; else hi = mid;
      }
      s = lo;
    }
    const Seq e = seq_at(q, s);
    const int64_t i = k.n - e.row0, p = e.start + i;
    x.live = x.live && i >= 0 && i < e.n;  // (a row of no sequence)
    x.at = static_cast<int>(p);
    if (z.paged && x.live && p >= 0 && p < q.cap) {
      const int entry = x.at / q.page;
      x.page = __ldg(q.table + s * q.width + entry), x.slot = x.at - entry * q.page;
    }
    return x;
  };
  Place place = place_at(tok, first);
  int at_ring = 0;
  for (int64_t base = first; base < tokens; base += stride) {
    const bool live = place.live;
    const int at = place.at, slot = place.slot, page = place.page < q.pages ? place.page : -1;
    P m;
    {
      int pos[W];
#pragma unroll
      for (int u = 0; u < W; ++u) {
        const int ax = turn ? sAx[own * W + u] : -1;
        pos[u] = ax < 0 ? 0 : APPEND && a.pos == nullptr ? at : a.pos[ax * a.pos_axis + tok.b * a.pos_batch + tok.n];
      }
#pragma unroll
      for (int u = 0; u < W; ++u) {
        float cs = 1.f, sn = 0.f;
        if (turn && sAx[own * W + u] >= 0) angle::sincos_at(pos[u], sT[own * W + u], &sn, &cs);
        // the pair's weights: of its elements in the two pieces, or in a row through both
        const float wa = HALF ? w0[u] : u < W / 2 ? w0[2 * u % W] : w1[2 * u % W];
        const float wb = HALF ? w1[u] : u < W / 2 ? w0[(2 * u + 1) % W] : w1[(2 * u + 1) % W];
        m.set(u, wa * cs, -wb * sn, wa * sn, wb * cs);
      }
    }
    const bool put = live && !(APPEND && z.paged && page < 0);
    T* y = static_cast<T*>(z.y) + hb * z.ys[1] +
           (APPEND && z.paged ? page * z.ys[0] + slot * z.ys[2] : tok.b * z.ys[0] + tok.n * z.ys[2]);
    tok = token_at(base + stride);
    if (APPEND) place = place_at(tok, base + stride);  // (its page is not waited for here)
    else place.live = mine && base + stride + threadIdx.x / LG < tokens;
    for (int h = 0; h < heads; ++h, y += z.ys[1]) {
      copy_wait<kAhead - 2>();
      const uint4 lo = own_ring[at_ring * 2 * kT], hi = own_ring[(at_ring * 2 + 1) * kT];
      at_ring = at_ring + 1 == kAhead ? 0 : at_ring + 1;
      fetch();
      if (z.norm || turn) {
        uint64_t v[W], o[W];
        widen2(lo, v, T{}), widen2(hi, v + W / 2, T{});
        m.apply(v, o);
        if (z.norm) {
          const float ss = sum_squares(v);
          const float r = rsqrtf(fmaf(group_sum<LG>(mine ? ss : 0.f), inv, a.eps));
#pragma unroll
          for (int u = 0; u < W; ++u) o[u] = tc::mul2(o[u], both(r));
        }
        if (put) {
          put2(y + c0, o);
          put2(y + c1, o + W / 2);
        }
      } else if (put) {
        *reinterpret_cast<uint4*>(y + c0) = lo;
        *reinterpret_cast<uint4*>(y + c1) = hi;
      }
    }
  }
  copy_wait<0>();
}

template <typename T, bool HALF, int LG>
__global__ void __launch_bounds__(kT, 2) grad_kernel(const HeadGradArgs a) {
  constexpr int W = 16 / sizeof(T);
  __shared__ unsigned long long sT[kMaxPairs];
  __shared__ int sAx[kMaxPairs];
  __shared__ float sum[kT / 32][2 * kMaxPairs];
  __shared__ __align__(16) float sW[2 * kMaxPairs];
  ptx::grid_dependency_launch();
  const int pairs = a.d / 2, per = pairs / W;
  int t = 0;
  while (static_cast<int>(blockIdx.y) >= a.first[t + 1]) ++t;
  const HeadGrad& z = a.t[t];
  const int hb = (blockIdx.y - a.first[t]) * a.per[t], heads = min(a.per[t], z.heads - hb);
  const int part = threadIdx.x & (LG - 1);
  const bool mine = part < per, turn = a.freq != nullptr;
  const int own = mine ? part : 0;
  const int c0 = HALF ? own * W : 2 * own * W, c1 = HALF ? c0 + pairs : c0 + W;
  const int64_t tokens = a.B * a.N;
  constexpr int step = kT / LG;
  struct Token {
    int64_t b, n;
    const T *x, *dy;
  };
  auto token_at = [&](int64_t base) {  // (behind the last one: the last one)
    Token k;
    const int64_t i = min(base + threadIdx.x / LG, tokens - 1);
    k.b = i / a.N, k.n = i - k.b * a.N;
    k.x = static_cast<const T*>(z.x) + k.b * z.xs[0] + hb * z.xs[1] + k.n * z.xs[2];
    k.dy = static_cast<const T*>(z.dy) + k.b * z.dys[0] + hb * z.dys[1] + k.n * z.dys[2];
    return k;
  };
  extern __shared__ __align__(16) uint4 ring[];  // (as in head_kernel: x's two pieces and dy's)
  uint4* own_ring = ring + threadIdx.x;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * step, stride = static_cast<int64_t>(gridDim.x) * step;
  Token tok = token_at(first);
  struct {
    int64_t base;
    const T *x, *dy;
    int h, place;
  } ahead;
  ahead.base = first, ahead.h = 0, ahead.place = 0, ahead.x = tok.x, ahead.dy = tok.dy;
  auto fetch = [&] {
    if (ahead.base < tokens) {
      uint4* to = own_ring + ahead.place * 4 * kT;
      copy16(to, ahead.x + c0), copy16(to + kT, ahead.x + c1);
      copy16(to + 2 * kT, ahead.dy + c0), copy16(to + 3 * kT, ahead.dy + c1);
      ahead.place = (ahead.place + 1) % kAheadGrad;
      ahead.x += z.xs[1], ahead.dy += z.dys[1];
      if (++ahead.h == heads) {
        ahead.h = 0, ahead.base += stride;
        const Token k = token_at(ahead.base);
        ahead.x = k.x, ahead.dy = k.dy;
      }
    }
    copy_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kAheadGrad - 1; ++i) fetch();
  int at_ring = 0;
  if (turn) angle_tables(a.freq, a.axis, pairs, a.axes, sT, sAx);
  for (int i = threadIdx.x; i < a.d; i += kT) sW[i] = z.w != nullptr ? z.w[i] : 1.f;
  uint64_t g[W];
#pragma unroll
  for (int k = 0; k < W; ++k) g[k] = 0;
  __syncthreads();
  const float inv = 1.f / static_cast<float>(a.d);
  for (int64_t base = first; base < tokens; base += stride) {
    const bool live = mine && base + threadIdx.x / LG < tokens;
    float cs[W], sn[W];
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const int i = own * W + u, ax = turn ? sAx[i] : -1;
      cs[u] = 1.f, sn[u] = 0.f;
      if (ax >= 0) angle::sincos_at(a.pos[ax * a.pos_axis + tok.b * a.pos_batch + tok.n], sT[i], &sn[u], &cs[u]);
    }
    T* dx = static_cast<T*>(z.dx) + tok.b * z.dxs[0] + hb * z.dxs[1] + tok.n * z.dxs[2];
    for (int h = 0; h < heads; ++h, dx += z.dxs[1]) {
      uint64_t x[W], y[W], f[W];
      copy_wait<kAheadGrad - 2>();
      {
        const uint4* from = own_ring + at_ring * 4 * kT;
        widen2(from[0], x, T{}), widen2(from[kT], x + W / 2, T{});
        widen2(from[2 * kT], y, T{}), widen2(from[3 * kT], y + W / 2, T{});
      }
      at_ring = (at_ring + 1) % kAheadGrad;
      fetch();
      if (HALF) {  // the turn back
#pragma unroll
        for (int k = 0; k < W / 2; ++k) {
          const uint64_t c2 = tc::pk2f(cs[2 * k], cs[2 * k + 1]), s2 = tc::pk2f(sn[2 * k], sn[2 * k + 1]);
          const uint64_t n2 = tc::pk2f(-sn[2 * k], -sn[2 * k + 1]);
          f[k] = tc::fma2(y[W / 2 + k], s2, tc::mul2(y[k], c2));
          f[W / 2 + k] = tc::fma2(y[k], n2, tc::mul2(y[W / 2 + k], c2));
        }
      } else {
#pragma unroll
        for (int u = 0; u < W; ++u) {
          const float2 v = tc::unpk2(y[u]);
          f[u] = tc::pk2f(fmaf(v.y, sn[u], v.x * cs[u]), fmaf(-v.x, sn[u], v.y * cs[u]));
        }
      }
      uint64_t dots = 0;
#pragma unroll
      for (int k = 0; k < W; k += 2) {
        const uint4 w = *reinterpret_cast<const uint4*>(sW + (k < W / 2 ? c0 + 2 * k : c1 + 2 * (k - W / 2)));
        y[k] = tc::mul2(tc::pk2(w.x, w.y), f[k]), y[k + 1] = tc::mul2(tc::pk2(w.z, w.w), f[k + 1]);
        dots = tc::fma2(y[k], x[k], dots), dots = tc::fma2(y[k + 1], x[k + 1], dots);
      }
      const float2 dd = tc::unpk2(dots);
      const float sq = sum_squares(x);
      const float ss = group_sum<LG>(mine ? sq : 0.f), dot = group_sum<LG>(mine ? dd.x + dd.y : 0.f);
      const float r = rsqrtf(fmaf(ss, inv, a.eps));
      if (live) {
        const uint64_t r2 = both(r), nm = both(-dot * inv * r * r);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          g[k] = tc::fma2(f[k], tc::mul2(x[k], r2), g[k]);
          y[k] = tc::mul2(tc::fma2(x[k], nm, y[k]), r2);
        }
        put2(dx + c0, y);
        put2(dx + c1, y + W / 2);
      }
    }
    tok = token_at(base + stride);
  }
  copy_wait<0>();
  if (z.dw == nullptr) return;
  // This block's share of dw: over the groups of a warp, then over the warps.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int o = LG; o < 32; o <<= 1) g[k] = tc::add2(g[k], __shfl_xor_sync(0xffffffffu, g[k], o));
  if (lane < per) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float2 v = tc::unpk2(g[k]);
      const int c = k < W / 2 ? c0 + 2 * k : c1 + 2 * (k - W / 2);
      sum[warp][c] = v.x, sum[warp][c + 1] = v.y;
    }
  }
  __syncthreads();
  float* out = a.ws + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.d;
  for (int i = threadIdx.x; i < a.d; i += kT) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kT / 32; ++k) v += sum[k][i];
    out[i] = v;
  }
}

// dw of a tensor: its blocks' shares, in a fixed order.
__global__ void __launch_bounds__(1024) weight_kernel(const HeadGradArgs a) {
  __shared__ float part[1024];
  ptx::grid_dependency_wait();
  const int t = blockIdx.x, d = a.d, groups = 1024 / d;
  const HeadGrad& z = a.t[t];
  if (z.dw == nullptr) return;
  const int64_t from = static_cast<int64_t>(a.first[t]) * a.cols, to = static_cast<int64_t>(a.first[t + 1]) * a.cols;
  const int g = threadIdx.x / d, c = threadIdx.x - g * d;
  float v = 0.f;
  if (g < groups) {
#pragma unroll 4
    for (int64_t s = from + g; s < to; s += groups) v += a.ws[s * d + c];
  }
  part[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < d) {
    for (int k = 1; k < groups; ++k) v += part[k * d + threadIdx.x];
    z.dw[threadIdx.x] = v;
  }
}

// How a call's heads and tokens are dealt to blocks: block rows of up to `per` heads of a tensor, and block columns, each
// of which takes groups of tokens one after another behind one set of tables, two blocks an SM.  The most heads
// a row that end soonest: a group costs its heads and its sines (about two and a half heads' time).  For 24 heads
// of 32768 tokens one wave took 41 us when columns for 2, 4 and 8 waves took 43, 44, 47 (39 since the ring).
struct Split {
  int per[4], first[5], cols;
};
Split split(int64_t groups, const int64_t* heads, int count) {
  Split best{};
  double least = 0;
  for (int most = 1; most <= 12; ++most) {
    Split s{};
    int widest = 0;
    for (int t = 0; t < 4; ++t) {
      const int h = t < count ? static_cast<int>(heads[t]) : 0, rows = (h + most - 1) / most;
      s.per[t] = rows > 0 ? (h + rows - 1) / rows : 1;
      s.first[t + 1] = s.first[t] + (h + s.per[t] - 1) / s.per[t];
      if (h > 0 && s.per[t] > widest) widest = s.per[t];
    }
    const int64_t rows = s.first[4], fit = 152 * 2, wave = rows > 0 && rows < fit ? fit / rows : 1;
    s.cols = static_cast<int>(groups < wave ? groups : wave);
    const int64_t blocks = rows * s.cols, each = s.cols > 0 ? (groups + s.cols - 1) / s.cols : 0;
    const double cost = static_cast<double>((blocks + fit - 1) / fit) * each * (widest + 2.5);
    if (most == 1 || cost <= least) best = s, least = cost;
  }
  return best;
}

template <typename T, bool HALF, bool APPEND, int LG>
cudaError_t run(const HeadArgs& a, dim3 grid, cudaStream_t st) {
  constexpr int smem = kAhead * 2 * kT * 16;
  const cudaError_t e = cudaFuncSetAttribute(head_kernel<T, HALF, APPEND, LG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  head_kernel<T, HALF, APPEND, LG><<<grid, kT, smem, st>>>(a);
  return cudaGetLastError();
}
template <typename T, bool HALF, bool APPEND>
cudaError_t run(const HeadArgs& a, int LG, dim3 grid, cudaStream_t st) {
  constexpr int S = sizeof(T) / 2;  // threads per token: d = 32, 64, 96 and 128, 256
  return LG == 2 * S   ? run<T, HALF, APPEND, 2 * S>(a, grid, st)
         : LG == 4 * S ? run<T, HALF, APPEND, 4 * S>(a, grid, st)
         : LG == 8 * S ? run<T, HALF, APPEND, 8 * S>(a, grid, st)
                       : run<T, HALF, APPEND, 16 * S>(a, grid, st);
}
template <typename T>
cudaError_t run(HeadArgs a, bool half, bool append, cudaStream_t st) {
  const int LG = group_threads(a.d, 16 / static_cast<int>(sizeof(T)));
  const int step = kT / LG;
  int64_t heads[4];
  for (int t = 0; t < 4; ++t) heads[t] = a.t[t].heads;
  const Split p = split((a.B * a.N + step - 1) / step, heads, 4);
  for (int t = 0; t < 4; ++t) a.per[t] = p.per[t];
  for (int t = 0; t < 5; ++t) a.first[t] = p.first[t];
  const dim3 grid(static_cast<unsigned>(p.cols), static_cast<unsigned>(p.first[4]));
  if (append) return half ? run<T, true, true>(a, LG, grid, st) : run<T, false, true>(a, LG, grid, st);
  return half ? run<T, true, false>(a, LG, grid, st) : run<T, false, false>(a, LG, grid, st);
}

Split grad_split(int64_t B, int64_t N, int64_t d, int dtype, const int64_t* heads, int count) {
  const int step = kT / group_threads(static_cast<int>(d), dtype == ATTN_BF16 ? 8 : 4);
  return split((B * N + step - 1) / step, heads, count);
}

template <typename T, bool HALF, int LG>
cudaError_t run_grad(const HeadGradArgs& a, dim3 grid, cudaStream_t st) {
  constexpr int smem = kAheadGrad * 4 * kT * 16;
  const cudaError_t e = cudaFuncSetAttribute(grad_kernel<T, HALF, LG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  grad_kernel<T, HALF, LG><<<grid, kT, smem, st>>>(a);
  return cudaGetLastError();
}
template <typename T, bool HALF>
cudaError_t run_grad(const HeadGradArgs& a, int LG, dim3 grid, cudaStream_t st) {
  constexpr int S = sizeof(T) / 2;
  return LG == 2 * S   ? run_grad<T, HALF, 2 * S>(a, grid, st)
         : LG == 4 * S ? run_grad<T, HALF, 4 * S>(a, grid, st)
         : LG == 8 * S ? run_grad<T, HALF, 8 * S>(a, grid, st)
                       : run_grad<T, HALF, 16 * S>(a, grid, st);
}

}  // namespace

cudaError_t head_norm(const HeadArgs& a, int dtype, bool half, bool append, cudaStream_t st) {
  return dtype == ATTN_BF16 ? run<__nv_bfloat16>(a, half, append, st) : run<float>(a, half, append, st);
}

size_t head_norm_bwd_bytes(int64_t B, int64_t N, int64_t d, int dtype, const int64_t* heads, int count) {
  const Split p = grad_split(B, N, d, dtype, heads, count);
  return static_cast<size_t>(p.first[4]) * p.cols * d * sizeof(float);
}

cudaError_t head_norm_bwd(const HeadGradArgs& args, int dtype, bool half, cudaStream_t st) {
  HeadGradArgs a = args;
  int64_t heads[4] = {0, 0, 0, 0};
  bool dw = false;
  for (int t = 0; t < a.count; ++t) heads[t] = a.t[t].heads, dw = dw || a.t[t].dw != nullptr;
  const Split p = grad_split(a.B, a.N, a.d, dtype, heads, a.count);
  for (int t = 0; t < 4; ++t) a.per[t] = p.per[t];
  for (int t = 0; t < 5; ++t) a.first[t] = p.first[t];
  a.cols = p.cols;
  const dim3 grid(static_cast<unsigned>(p.cols), static_cast<unsigned>(p.first[4]));
  const int LG = group_threads(a.d, dtype == ATTN_BF16 ? 8 : 4);
  cudaError_t e;
  if (dtype == ATTN_BF16) e = half ? run_grad<__nv_bfloat16, true>(a, LG, grid, st) : run_grad<__nv_bfloat16, false>(a, LG, grid, st);
  else e = half ? run_grad<float, true>(a, LG, grid, st) : run_grad<float, false>(a, LG, grid, st);
  if (e != cudaSuccess || !dw) return e;
  return launch_behind(weight_kernel, a.count, 1024, 0, st, a);
}

}  // namespace fbd
