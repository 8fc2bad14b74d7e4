// The launch that joins the parts of items that several CTAs shared, and the choice of a kernel for the
// attention over a paged cache.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "paged_launch.h"

namespace fbd {
namespace paged {
namespace {

__device__ __forceinline__ void put(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16(v.x, v.y), ptx::pack_bf16(v.z, v.w));
}

constexpr int kJ = 256;

// A row of an item: its token and head, and its place in a slot.
struct Row {
  int t, head, at;
  __device__ __forceinline__ Row(const Cut& c, int row, int tile_rows) {
    t = c.gt == 1 ? row : row / c.gt, head = row - t * c.gt;
    const int tl = t < c.tile ? 0 : t / c.tile;
    at = tl * tile_rows + (t - tl * c.tile) * c.gt + head;
  }
};
template <typename T>
__device__ __forceinline__ void put_row(const Work& w, const Out& out, const Seq& s, const Tail& q, const Row& row, int t0, int col,
                                        int d, float4 o, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;  // (a row that sees no key: 0)
  const int64_t h = static_cast<int64_t>(q.vh) * w.cut.gt + row.head, pos = s.row0 + t0 + row.t;
  if (col < d)
    put(static_cast<T*>(out.O) + s.batch * out.os[0] + h * out.os[1] + pos * out.os[2] + col,
        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (col == 0 && out.lse != nullptr)
    out.lse[s.batch * out.ls[0] + h * out.ls[1] + pos] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

constexpr int kFewRows = 16;  // items of at most as many rows may have many parts

// Block (p, y): every gridDim.y-th run of rows of the item that begins in CTA p's stretch and goes on behind it.  A
// row's columns are d / 4 threads' (rounded up to a power of two); such groups take a row each, or, of an
// item of few rows and many parts, the parts of one row after another, whose weights are formed once.
template <typename T>
__global__ void __launch_bounds__(kJ) join_kernel(const Work w, const Space sp, const Out out, int d, int tile_rows) {
  __shared__ float weight[kMaxCtas];
  __shared__ float4 sum[kJ];
  __shared__ float total[2];
  ptx::grid_dependency_wait();
  const Tail q = sp.tail[blockIdx.x];
  if (q.parts == 0) return;
  const Seq s = seq_at(w.seqs, q.b);
  const int t0 = q.tile * w.cut.step, t1 = min(s.n, t0 + w.cut.step);
  const int rows = (t1 - t0) * w.cut.gt, p = blockIdx.x, parts = q.parts;
  int C = 8;
  while (C * 4 < d) C *= 2;
  const int groups = kJ / C, g = threadIdx.x / C, col = (threadIdx.x & (C - 1)) * 4;
  auto slot_of = [&](int k) { return k == 0 ? 2 * p + 1 : 2 * (p + k); };
  if (parts <= 4 || rows > kFewRows) {
    for (int r = blockIdx.y * groups + g; r < rows; r += gridDim.y * groups) {
      const Row row(w.cut, r, tile_rows);
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = 0; k0 < parts; k0 += 4) {  // four parts' loads at once
        float2 x[4];
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[k] = make_float2(-INFINITY, 0.f), v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + k >= parts) continue;
          x[k] = *sp.ml(slot_of(k0 + k), row.at);
          if (col < d) v[k] = *reinterpret_cast<const float4*>(sp.o(slot_of(k0 + k), row.at) + col);
        }
        const float top = fmaxf(fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)), m), sub = top == -INFINITY ? 0.f : top;
        const float a = ptx::ex2(m - sub);
        m = top, l *= a;
        o.x *= a, o.y *= a, o.z *= a, o.w *= a;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float f = ptx::ex2(x[k].x - sub);
          l = fmaf(f, x[k].y, l);
          o.x = fmaf(f, v[k].x, o.x), o.y = fmaf(f, v[k].y, o.y), o.z = fmaf(f, v[k].z, o.z), o.w = fmaf(f, v[k].w, o.w);
        }
      }
      put_row<T>(w, out, s, q, row, t0, col, d, o, m, l);
    }
    return;
  }
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    const Row row(w.cut, r, tile_rows);
    __syncthreads();  // the row before has been read
    if (threadIdx.x < 32) {
      float m = -INFINITY, l = 0.f;
      for (int k = threadIdx.x; k < parts; k += 32) m = fmaxf(m, sp.ml(slot_of(k), row.at)->x);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      const float sub = m == -INFINITY ? 0.f : m;
      for (int k = threadIdx.x; k < parts; k += 32) {
        const float2 x = *sp.ml(slot_of(k), row.at);
        const float f = ptx::ex2(x.x - sub);
        weight[k] = f, l = fmaf(f, x.y, l);
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
      if (threadIdx.x == 0) total[0] = m, total[1] = l;
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < d) {
#pragma unroll 8
      for (int k = g; k < parts; k += groups) {
        const float4 v = *reinterpret_cast<const float4*>(sp.o(slot_of(k), row.at) + col);
        const float f = weight[k];
        o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
      }
    }
    sum[threadIdx.x] = o;
    __syncthreads();
    if (g == 0) {
      for (int k = 1; k < groups; ++k) {
        const float4 v = sum[k * C + threadIdx.x];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      }
      put_row<T>(w, out, s, q, row, t0, col, d, o, total[0], total[1]);
    }
  }
}

}  // namespace

cudaError_t join(const Work& w, const Space& sp, const Out& out, int dtype, int d, int tile_rows, int64_t few, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  // Up to four blocks an item of few rows (their parts may be many), else two rows for each of a block's groups
  // (one, two, four, eight: 92, 90, 90, 90 us at d = 256, 50, 51, 54, 54 us for the float32 chunk).
  const int64_t rows = (few < w.cut.step ? few : w.cut.step) * w.cut.gt;
  const int groups = d <= 32 ? kJ / 8 : d <= 64 ? kJ / 16 : d <= 128 ? kJ / 32 : kJ / 64;
  cfg.gridDim = dim3(static_cast<unsigned>(w.cut.ctas), static_cast<unsigned>(rows <= kFewRows ? (rows < 4 ? rows : 4) : (rows + 2 * groups - 1) / (2 * groups)));
  cfg.blockDim = dim3(kJ);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return dtype == ATTN_BF16 ? cudaLaunchKernelEx(&cfg, join_kernel<__nv_bfloat16>, w, sp, out, d, tile_rows)
                            : cudaLaunchKernelEx(&cfg, join_kernel<float>, w, sp, out, d, tile_rows);
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
