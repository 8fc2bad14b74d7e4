// The planning launch of the attention over a paged cache (one block), and the launch that joins the
// parts of items that several CTAs shared.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "paged_launch.h"

namespace fbd {
namespace paged {
namespace {

constexpr int kT = 1024;

constexpr int kNear = 2048;  // sequences whose ends are kept in shared memory

__global__ void __launch_bounds__(kT) plan_kernel(const Work w, const Space sp) {
  __shared__ int64_t carry, part[kT / 32], near[kNear];
  ptx::grid_dependency_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, B = w.seqs.B, step = w.cut.step;
  int64_t* ends = B <= kNear ? near : sp.ends;
  if (threadIdx.x == 0) carry = 0;
  for (int b0 = 0; b0 < B; b0 += kT) {
    const int b = b0 + threadIdx.x;
    // A sequence's tiles: its thread's, the warp's together where they are many.
    int64_t v = 0;
    Seq s{};
    if (b < B) s = seq_at(w.seqs, b);
    for (int t = 0; t < 4 && static_cast<int64_t>(t) * step < s.n; ++t) v += tile_units(w, s, t);
    for (unsigned many = __ballot_sync(0xffffffffu, s.n > 4ll * step); many != 0; many &= many - 1) {
      const int from = __ffs(many) - 1;
      const Seq q = seq_at(w.seqs, b0 + warp * 32 + from);
      int64_t u = 0;
      for (int64_t t = 4 + lane; t * step < q.n; t += 32) u += tile_units(w, q, static_cast<int>(t));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
      if (lane == from) v += u;
    }
    v = warp_scan(v * w.cut.nv, lane);
    __syncthreads();  // `part` and `carry` of the round before
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) part[lane] = warp_scan(part[lane], lane);
    __syncthreads();
    v += carry + (warp > 0 ? part[warp - 1] : 0);
    if (b < B) ends[b] = v;
    __syncthreads();
    if (threadIdx.x == kT - 1) carry = v;
  }
  __syncthreads();
  const int64_t total = carry;
  const int64_t even = (total + w.cut.ctas - 1) / w.cut.ctas, stretch = even > w.cut.least ? even : w.cut.least;
  if (threadIdx.x == 0) *sp.head = Head{total, stretch};
  for (int p = warp; p < w.cut.ctas; p += kT / 32) {
    const int64_t x = stretch * p;
    if (lane == 0) sp.tail[p] = Tail{0, 0, 0, 0};
    if (x >= total) {
      if (lane == 0) sp.start[p] = Start{0, -1, 0, 0, 0};
      continue;
    }
    int hi = B - 1;  // the first sequence that ends behind x
    for (int lo = -1; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > x) hi = mid; else lo = mid;
    }
    const Seq s = seq_at(w.seqs, hi);
    int64_t at = hi > 0 ? ends[hi - 1] : 0;
    for (int64_t t0 = 0; t0 * step < s.n; t0 += 32) {  // ... and its tile that does
      const int64_t t = t0 + lane;
      const int64_t u = t * step < s.n ? tile_units(w, s, static_cast<int>(t)) : 0, cum = at + warp_scan(u * w.cut.nv, lane);
      const unsigned behind = __ballot_sync(0xffffffffu, cum > x);
      if (behind != 0) {
        if (lane == __ffs(behind) - 1) {
          const int64_t b = cum - u * w.cut.nv, vh = (x - b) / u;
          sp.start[p] = Start{b + vh * u, hi, static_cast<int>(t), static_cast<int>(vh), 0};
        }
        break;
      }
      at = __shfl_sync(0xffffffffu, cum, 31);
    }
  }
}

__device__ __forceinline__ void put(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16(v.x, v.y), ptx::pack_bf16(v.z, v.w));
}

constexpr int kJ = 256;

// Block (p, y): every gridDim.y-th run of `per` rows of the item that begins in CTA p's stretch and goes on behind it.  A row's columns
// are d / 4 threads' (rounded up to a power of two); such groups take a row each, or, where the
// parts are many, parts of one row after another.
template <typename T>
__global__ void __launch_bounds__(kJ) join_kernel(const Work w, const Space sp, const Out out, int d, int tile_rows, int per) {
  __shared__ float4 sum[kJ];
  __shared__ float sl[kJ], sm[kJ];
  ptx::grid_dependency_wait();
  const Tail q = sp.tail[blockIdx.x];
  if (q.parts == 0) return;
  const Seq s = seq_at(w.seqs, q.b);
  const int t0 = q.tile * w.cut.step, t1 = min(s.n, t0 + w.cut.step), gt = w.cut.gt;
  const int rows = (t1 - t0) * gt, p = blockIdx.x;
  int C = 8;
  while (C * 4 < d) C *= 2;
  const int groups = kJ / C, g = threadIdx.x / C, col = (threadIdx.x & (C - 1)) * 4;
  const bool wide = q.parts > 2 * groups;  // groups share a row
  for (int r0 = blockIdx.y * per; r0 < rows; r0 += gridDim.y * per)
  for (int rr = r0, r1 = min(rows, r0 + per); rr < r1; rr += wide ? 1 : groups) {
    const int row = rr + (wide ? 0 : g);
    const bool live = row < r1;
    const int t = live ? row / gt : 0, hh = live ? row - t * gt : 0;
    const int tl = t / w.cut.tile, at = tl * tile_rows + (t - tl * w.cut.tile) * gt + hh;  // in a slot
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
#pragma unroll 4
      for (int k = wide ? g : 0; k < q.parts; k += wide ? groups : 1) {
        const int slot = k == 0 ? 2 * p + 1 : 2 * (p + k);
        const float2 x = *sp.ml(slot, at);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < d) v = *reinterpret_cast<const float4*>(sp.o(slot, at) + col);
        const float mn = fmaxf(m, x.x), sub = mn == -INFINITY ? 0.f : mn;
        const float a = ptx::ex2(m - sub), b = ptx::ex2(x.x - sub);
        m = mn, l = fmaf(l, a, x.y * b);
        o.x = fmaf(o.x, a, v.x * b), o.y = fmaf(o.y, a, v.y * b);
        o.z = fmaf(o.z, a, v.z * b), o.w = fmaf(o.w, a, v.w * b);
      }
    }
    if (wide) {
      __syncthreads();  // the row before has been read
      sum[threadIdx.x] = o, sm[threadIdx.x] = m, sl[threadIdx.x] = l;
      __syncthreads();
      if (g == 0) {
        for (int k = 1; k < groups; ++k) {
          const int u = k * C + threadIdx.x;
          const float4 v = sum[u];
          const float mn = fmaxf(m, sm[u]), sub = mn == -INFINITY ? 0.f : mn;
          const float a = ptx::ex2(m - sub), b = ptx::ex2(sm[u] - sub);
          m = mn, l = fmaf(l, a, sl[u] * b);
          o.x = fmaf(o.x, a, v.x * b), o.y = fmaf(o.y, a, v.y * b);
          o.z = fmaf(o.z, a, v.z * b), o.w = fmaf(o.w, a, v.w * b);
        }
      }
    }
    if (live && (!wide || g == 0)) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (a row that sees no key: 0)
      const int64_t h = static_cast<int64_t>(q.vh) * gt + hh, pos = s.row0 + t0 + t;
      if (col < d)
        put(static_cast<T*>(out.O) + s.batch * out.os[0] + h * out.os[1] + pos * out.os[2] + col,
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
      if (col == 0 && out.lse != nullptr)
        out.lse[s.batch * out.ls[0] + h * out.ls[1] + pos] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

}  // namespace

cudaError_t plan(const Work& w, const Space& sp, cudaStream_t st) {
  plan_kernel<<<1, kT, 0, st>>>(w, sp);
  return cudaGetLastError();
}

cudaError_t join(const Work& w, const Space& sp, const Out& out, int dtype, int d, int tile_rows, int64_t few, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  // A row a block where items have few (each then has many parts), else eight.
  const int64_t rows = (few < w.cut.step ? few : w.cut.step) * w.cut.gt;
  const int per = rows <= 32 ? 1 : 8;
  cfg.gridDim = dim3(static_cast<unsigned>(w.cut.ctas), static_cast<unsigned>((rows + per - 1) / per));
  cfg.blockDim = dim3(kJ);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return dtype == ATTN_BF16 ? cudaLaunchKernelEx(&cfg, join_kernel<__nv_bfloat16>, w, sp, out, d, tile_rows, per)
                            : cudaLaunchKernelEx(&cfg, join_kernel<float>, w, sp, out, d, tile_rows, per);
}

}  // namespace paged

size_t paged_bytes(const PagedArgs& a) {
  return a.dtype != ATTN_BF16 ? paged::simt_bytes(a) : paged::few_rows(a) ? paged::token_bytes(a) : a.d <= 128 ? paged::tc_bytes(a) : paged::tc_wide_bytes(a);
}
cudaError_t paged_attention(const PagedArgs& a, void* ws, cudaStream_t st) {
  return a.dtype != ATTN_BF16 ? paged::simt_paged(a, ws, st)
         : paged::few_rows(a) ? paged::token_paged(a, ws, st)
         : a.d <= 128         ? paged::tc_paged(a, ws, st)
                              : paged::tc_paged_wide(a, ws, st);
}

}  // namespace fbd
