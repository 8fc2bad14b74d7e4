// C ABI of differential attention and the rotary positions (declared in include/fbd.h):
// argument validation and dispatch.
#include <cuda_runtime.h>

#include <initializer_list>

#include "checks.h"
#include "diff.h"
#include "fbd.h"
#include "rope.h"

namespace {

using namespace fbd;

// check_desc, then what differential attention adds.  `p` counts differential heads.
attn_status_t check_diff(const attn_desc_t* desc, Problem& p) {
  attn_status_t s = check_desc(desc, p);
  if (s != ATTN_OK) return s;
  if (!diff_supports(p.d)) return fail(ATTN_ERR_UNSUPPORTED, "differential attention: d must be 32 or 64%s");
  // 2H maps in a tensor-map extent; the backward's preparation takes eight blocks per 128 rows of a head
  if (p.BH >= (int64_t(1) << 30) || p.BH * ((p.N + 127) / 128) >= (int64_t(1) << 28))
    return fail(ATTN_ERR_INVALID_ARG, "B*H must be < 2^30 and B*H*ceil(N/128) < 2^28%s");
  return ATTN_OK;
}

// A pointer that needs only its 4-byte element's alignment.
attn_status_t check_small(const char* name, const void* p) {
  if (p == nullptr) return fail(ATTN_ERR_INVALID_ARG, "pointer %s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return fail(ATTN_ERR_ALIGNMENT, "pointer %s is not 4-byte aligned", name);
  return ATTN_OK;
}
// No overlap between an array of 4-byte elements and any of `others`, one of the two written.
attn_status_t check_apart(const Span& a, const Span* others, int n) {
  for (int k = 0; k < n; ++k)
    if (a.lo < others[k].hi && others[k].lo < a.hi)
      return fail(ATTN_ERR_INVALID_ARG, "%s overlaps an output, or is one and overlaps an input", a.name);
  return ATTN_OK;
}

// The 16-byte aligned inputs of a call, the document bounds among them when they are given.
struct Inputs {
  Span s[9];
  int n = 0;
  Inputs(std::initializer_list<Span> l, const Problem& p) {
    for (const Span& x : l) s[n++] = x;
    if (p.seg_lo != nullptr) {
      const size_t b = static_cast<size_t>(p.B * p.N) * sizeof(int);
      s[n++] = span("seg_lo", p.seg_lo, b);
      s[n++] = span("seg_hi", p.seg_hi, b);
    }
  }
};

struct Sizes {
  size_t q, k, v, o, s;  // bytes of Q, K, V, O and lse
  Sizes(const Problem& p, int64_t queries) {
    const size_t e = elem_size(p);
    q = static_cast<size_t>(2 * p.BH * queries * p.d) * e;
    k = v = static_cast<size_t>(2 * p.BHkv * p.N * p.d) * e;
    o = q;
    s = static_cast<size_t>(2 * p.BH * queries) * sizeof(float);
  }
};

}  // namespace

extern "C" {

attn_status_t attn_diff_fwd(const attn_desc_t* desc, const void* Q, const void* K, const void* V, const float* lam,
                            void* O, void* O2, float* lse, void* stream) {
  Problem p;
  attn_status_t s = check_diff(desc, p);
  if (s != ATTN_OK) return s;
  if (p.BH * p.N == 0) return ATTN_OK;
  if ((s = check_small("lam", lam)) != ATTN_OK) return s;
  const Sizes z(p, p.N);
  const Inputs in({span("Q", Q, z.q), span("K", K, z.k), span("V", V, z.v)}, p);
  Span out[3] = {span("O", O, z.o), span("lse", lse, z.s)};
  int nout = 2;
  if (O2 != nullptr) out[nout++] = span("O2", O2, z.o);
  if ((s = check_ptrs(in.s, in.n, out, nout)) != ATTN_OK) return s;
  if ((s = check_apart(span("lam", lam, p.H * sizeof(float)), out, nout)) != ATTN_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(p.dtype == ATTN_BF16 ? tc_diff_fwd(p, Q, K, V, lam, O, O2, lse, st)
                                            : simt_diff_fwd(p, Q, K, V, lam, O, O2, lse, st));
}

size_t attn_diff_bwd_workspace_bytes(const attn_desc_t* desc) {
  if (desc == nullptr || desc->B < 0 || desc->H < 0 || desc->N < 0) return 0;
  return desc->dtype == ATTN_BF16 ? tc_diff_bwd_bytes(desc->B * desc->H, desc->N)
                                  : simt_diff_bwd_bytes(desc->B * desc->H, desc->N);
}

attn_status_t attn_diff_bwd(const attn_desc_t* desc, const void* Q, const void* K, const void* V, const float* lam,
                            const void* O, const void* O2, const void* dO, const float* lse, void* dQ, void* dK,
                            void* dV, float* dlam, void* workspace, size_t workspace_bytes, void* stream) {
  Problem p;
  attn_status_t s = check_diff(desc, p);
  if (s != ATTN_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.H == 0) return ATTN_OK;
  if ((s = check_small("dlam", dlam)) != ATTN_OK) return s;
  if (p.B * p.N == 0) return launch_status(cudaMemsetAsync(dlam, 0, p.H * sizeof(float), st));
  if ((s = check_small("lam", lam)) != ATTN_OK) return s;
  const size_t need = attn_diff_bwd_workspace_bytes(desc);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace NULL or smaller than attn_diff_bwd_workspace_bytes()%s");
  const Sizes z(p, p.N);
  const Inputs in({span("Q", Q, z.q), span("K", K, z.k), span("V", V, z.v), span("O", O, z.o), span("O2", O2, z.o),
                   span("dO", dO, z.o), span("lse", lse, z.s)}, p);
  const Span out[] = {span("dQ", dQ, z.q), span("dK", dK, z.k), span("dV", dV, z.v),
                      span("workspace", workspace, need)};
  if ((s = check_ptrs(in.s, in.n, out, 4)) != ATTN_OK) return s;
  const Span la = span("lam", lam, p.H * sizeof(float)), dl = span("dlam", dlam, p.H * sizeof(float));
  if ((s = check_apart(la, out, 4)) != ATTN_OK || (s = check_apart(dl, out, 4)) != ATTN_OK ||
      (s = check_apart(dl, in.s, in.n)) != ATTN_OK || (s = check_apart(dl, &la, 1)) != ATTN_OK)
    return s;
  return launch_status(p.dtype == ATTN_BF16
                           ? tc_diff_bwd(p, Q, K, V, lam, O, O2, dO, lse, dQ, dK, dV, dlam, workspace, st)
                           : simt_diff_bwd(p, Q, K, V, lam, O, O2, dO, lse, dQ, dK, dV, dlam, workspace, st));
}

size_t attn_diff_decode_workspace_bytes(const attn_desc_t* desc) {
  Problem p;
  if (check_diff(desc, p) != ATTN_OK || p.BH == 0) return 0;
  return diff_decode_bytes(p);
}

attn_status_t attn_diff_decode(const attn_desc_t* desc, const void* Q, const void* K, const void* V, const float* lam,
                               const int32_t* lens, void* O, void* workspace, size_t workspace_bytes, void* stream) {
  Problem p;
  attn_status_t s = check_diff(desc, p);
  if (s != ATTN_OK) return s;
  if (p.causal != 1) return fail(ATTN_ERR_UNSUPPORTED, "a token over a cache is causal (causal = 1)%s");
  if (p.seg_lo != nullptr) return fail(ATTN_ERR_UNSUPPORTED, "no document mask over a cache%s");
  if (p.BH == 0) return ATTN_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Sizes z(p, 1);
  if (p.N == 0) {  // no cache: every sequence is empty
    const Span out[] = {span("O", O, z.o)};
    if ((s = check_ptrs(nullptr, 0, out, 1)) != ATTN_OK) return s;
    return launch_status(cudaMemsetAsync(O, 0, z.o, st));
  }
  if ((s = check_small("lam", lam)) != ATTN_OK || (s = check_small("lens", lens)) != ATTN_OK) return s;
  const size_t need = diff_decode_bytes(p);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(ATTN_ERR_WORKSPACE, "workspace NULL or smaller than attn_diff_decode_workspace_bytes()%s");
  const Span in[] = {span("Q", Q, z.q), span("K", K, z.k), span("V", V, z.v)};
  const Span out[] = {span("O", O, z.o), span("workspace", workspace, need)};
  const int nout = need > 0 ? 2 : 1;
  if ((s = check_ptrs(in, 3, out, nout)) != ATTN_OK) return s;
  if ((s = check_apart(span("lam", lam, p.H * sizeof(float)), out, nout)) != ATTN_OK ||
      (s = check_apart(span("lens", lens, p.B * sizeof(int32_t)), out, nout)) != ATTN_OK)
    return s;
  return launch_status(diff_decode(p, Q, K, V, lam, lens, O, workspace, st));
}

attn_status_t attn_rope(const attn_rope_desc_t* desc, const attn_rope_tensor_t* tensors, int count,
                        const int32_t* pos, const float* freq, const int32_t* axis, void* stream) {
  if (desc == nullptr) return fail(ATTN_ERR_INVALID_ARG, "desc is NULL%s");
  const int64_t B = desc->B, N = desc->N, d = desc->d, lim = int64_t(1) << 31;
  if (B < 0 || N < 0 || B >= lim || N >= lim || (N > 0 && B > (int64_t(1) << 33) / N))
    return fail(ATTN_ERR_INVALID_ARG, "B and N must be >= 0 and < 2^31, B*N <= 2^33%s");
  if (d != 32 && d != 64 && d != 96 && d != 128 && d != 256)
    return fail(ATTN_ERR_UNSUPPORTED, "head dim must be 32, 64, 96, 128 or 256%s");
  if (desc->dtype != ATTN_F32 && desc->dtype != ATTN_BF16) return fail(ATTN_ERR_UNSUPPORTED, "unknown dtype%s");
  if (desc->paired != ATTN_ROPE_HALF && desc->paired != ATTN_ROPE_NEIGHBOUR)
    return fail(ATTN_ERR_UNSUPPORTED, "paired must be ATTN_ROPE_HALF or ATTN_ROPE_NEIGHBOUR%s");
  if (desc->inverse != 0 && desc->inverse != 1) return fail(ATTN_ERR_UNSUPPORTED, "inverse must be 0 or 1%s");
  if (desc->axes < 1 || desc->axes > 64) return fail(ATTN_ERR_INVALID_ARG, "axes must be 1 .. 64%s");
  if (desc->pos_batch_stride != 0 && desc->pos_batch_stride != N)
    return fail(ATTN_ERR_INVALID_ARG, "pos_batch_stride must be 0 or N%s");
  if (tensors == nullptr || count < 1 || count > ATTN_ROPE_MAX_TENSORS)
    return fail(ATTN_ERR_INVALID_ARG, "1 to ATTN_ROPE_MAX_TENSORS tensors%s");
  RopeArgs a{};
  a.B = B, a.N = N, a.d = static_cast<int>(d), a.axes = desc->axes, a.inverse = desc->inverse != 0;
  a.pos_batch = desc->pos_batch_stride;
  a.pos_axis = desc->pos_batch_stride == 0 ? N : B * N;
  const int64_t e = desc->dtype == ATTN_F32 ? 4 : 2;
  int64_t heads = 0;
  for (int t = 0; t < count; ++t) {
    const int64_t h = tensors[t].heads;
    if (h < 0 || h > 65535 || (heads += h) > 65535) return fail(ATTN_ERR_INVALID_ARG, "0 to 65535 heads in all%s");
  }
  if (heads * B * N == 0) return ATTN_OK;
  // Byte ranges without gaps: what each y writes and each x reads where its strides leave none, and the
  // tables.  (Views with gaps may lie between one another, as a projection's heads do: not checked.)
  struct Range {
    uintptr_t lo, hi;
    bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
  };
  const auto table = [](const void* p, int64_t words) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return Range{at, at + static_cast<uintptr_t>(4 * words)};
  };
  const Range tables[3] = {table(pos, a.axes * a.pos_axis), table(freq, d / 2), table(axis, d / 2)};
  Range xr[ATTN_ROPE_MAX_TENSORS], yr[ATTN_ROPE_MAX_TENSORS];
  int nx = 0, ny = 0;
  bool meet = false;
  int n = 0;
  for (int t = 0; t < count; ++t) {
    const attn_rope_tensor_t& z = tensors[t];
    if (z.heads == 0) continue;
    if (z.x == nullptr || z.y == nullptr) return fail(ATTN_ERR_INVALID_ARG, "pointer %s is NULL", z.x ? "y" : "x");
    const uintptr_t ax = reinterpret_cast<uintptr_t>(z.x), ay = reinterpret_cast<uintptr_t>(z.y);
    if (ax % 16 || ay % 16) return fail(ATTN_ERR_ALIGNMENT, "pointer %s is not 16-byte aligned", ax % 16 ? "x" : "y");
    const int64_t size[3] = {B, z.heads, N};
    RopeTensor& r = a.t[n++];
    r.x = z.x, r.y = z.y, r.heads = static_cast<int>(z.heads);
    bool same = ax == ay;
    int64_t xe = d, ye = d;  // elements from the first to behind the last
    int64_t xn = d;          // elements of x, one that it repeats counted once
    for (int k = 0; k < 3; ++k) {
      if (size[k] == 1) continue;  // a stride that is never taken (left 0)
      const int64_t sx = z.x_stride[k], sy = z.y_stride[k], most = (int64_t(1) << 58) / size[k];
      if (sx < 0 || sy < 0 || sx > most || sy > most)
        return fail(ATTN_ERR_INVALID_ARG, "strides must be >= 0, within 2^58 elements%s");
      if (sx * e % 16 || sy * e % 16) return fail(ATTN_ERR_ALIGNMENT, "strides must be multiples of 16 bytes%s");
      r.xs[k] = sx, r.ys[k] = sy;
      xe += sx * (size[k] - 1), ye += sy * (size[k] - 1);
      if (sx > 0) xn *= size[k];
      same = same && sx == sy;
    }
    // y's rows apart: in order of stride, each stride past all that lies below it
    int order[3] = {0, 1, 2};
    for (int u = 0; u < 2; ++u)
      for (int k = 0; k < 2 - u; ++k)
        if (r.ys[order[k]] > r.ys[order[k + 1]]) {
          const int o = order[k];
          order[k] = order[k + 1], order[k + 1] = o;
        }
    int64_t below = d;
    for (int k : order) {
      if (size[k] == 1) continue;
      if (r.ys[k] < below) return fail(ATTN_ERR_INVALID_ARG, "y's strides make its rows overlap%s");
      below += r.ys[k] * (size[k] - 1);
    }
    const int64_t elems = B * z.heads * N * d;
    const Range x{ax, ax + static_cast<uintptr_t>(xe * e)}, y{ay, ay + static_cast<uintptr_t>(ye * e)};
    if (xe == xn && !same) {  // (x and y the same: y's checks below are x's)
      for (int k = 0; k < ny; ++k) meet = meet || x.meets(yr[k]);
      xr[nx++] = x;
    }
    if (ye == elems) {
      for (int k = 0; k < nx; ++k) meet = meet || y.meets(xr[k]);
      for (int k = 0; k < ny; ++k) meet = meet || y.meets(yr[k]);
      for (int k = 0; k < 3; ++k) meet = meet || y.meets(tables[k]);
      yr[ny++] = y;
    }
  }
  if (meet) return fail(ATTN_ERR_INVALID_ARG, "an output overlaps an input, a table or another output%s");
  a.heads = static_cast<int>(heads);
  attn_status_t s;
  if ((s = check_small("pos", pos)) != ATTN_OK || (s = check_small("freq", freq)) != ATTN_OK ||
      (s = check_small("axis", axis)) != ATTN_OK)
    return s;
  return launch_status(rope(a, desc->dtype, desc->paired == ATTN_ROPE_HALF, pos, freq, axis,
                            static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
