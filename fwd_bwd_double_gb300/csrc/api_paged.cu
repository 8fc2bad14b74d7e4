// C ABI of the paged cache and of the normed heads (declared in include/fbd.h): argument checks and
// kernel launches.
#include <cmath>

#include "checks.h"
#include "paged.h"

using namespace fbd;

namespace {

// Byte ranges of a call's arrays and of its views without gaps (views with gaps may lie between one
// another, as a projection's heads do: not checked).
struct Ranges {
  struct Range {
    const char* name;
    uintptr_t lo, hi;
    bool out;
  } r[24];
  int n = 0;
  void add(const char* name, const void* p, uint64_t bytes, bool out) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (p != nullptr && bytes > 0 && n < 24) r[n++] = Range{name, at, at + bytes, out};
  }
  attn_status_t apart() const {
    for (int i = 0; i < n; ++i)
      for (int k = 0; k < n; ++k)
        if (i != k && r[i].out && r[i].lo < r[k].hi && r[k].lo < r[i].hi)
          return fail(ATTN_ERR_INVALID_ARG, "output %s overlaps another array", r[i].name);
    return ATTN_OK;
  }
};

// A view of rows of d elements with `size` and `stride` in three dimensions: its checks, its strides as
// the kernels take them (0 where a stride is never taken), its range where it has no gaps.  `same`: the
// view that it may equal exactly (address and strides), which then has the range.
struct View {
  const char* name;
  const void* p;
  int64_t size[3];
  const int64_t* stride;
  bool out;
};
bool same_view(const View& a, const View& b) {
  bool same = a.p == b.p;
  for (int k = 0; k < 3; ++k) same = same && (a.size[k] == 1 || a.stride[k] == b.stride[k]);
  return same;
}
attn_status_t check_view(const View& v, int64_t d, int64_t e, bool broadcast, int64_t* eff, Ranges& ranges,
                         bool skip_range = false) {
  if (v.p == nullptr) return fail(ATTN_ERR_INVALID_ARG, "pointer %s is NULL", v.name);
  if (reinterpret_cast<uintptr_t>(v.p) % 16 != 0) return fail(ATTN_ERR_ALIGNMENT, "pointer %s is not 16-byte aligned", v.name);
  int64_t span = d, distinct = d, order[3][2];
  int n = 0;
  for (int k = 0; k < 3; ++k) {
    eff[k] = 0;
    if (v.size[k] == 1) continue;
    const int64_t s = v.stride[k], most = (int64_t(1) << 58) / v.size[k];
    if (s < 0 || s > most || (s == 0 && !(broadcast && !v.out)))
      return fail(ATTN_ERR_INVALID_ARG, "strides of %s must be positive, within 2^58 elements", v.name);
    if (s * e % 16 != 0) return fail(ATTN_ERR_ALIGNMENT, "strides of %s must be multiples of 16 bytes", v.name);
    eff[k] = s;
    span += s * (v.size[k] - 1);
    if (s > 0) distinct *= v.size[k];
    int i = n++;
    for (; i > 0 && order[i - 1][0] > s; --i) order[i][0] = order[i - 1][0], order[i][1] = order[i - 1][1];
    order[i][0] = s, order[i][1] = v.size[k];
  }
  if (v.out) {  // rows apart: in order of stride, each past all that lies below it
    int64_t below = d;
    for (int i = 0; i < n; ++i) {
      if (order[i][0] < below) return fail(ATTN_ERR_INVALID_ARG, "the strides of %s make its rows overlap", v.name);
      below += order[i][0] * (order[i][1] - 1);
    }
  }
  if (span == distinct && !skip_range) ranges.add(v.name, v.p, static_cast<uint64_t>(span) * e, v.out);
  return ATTN_OK;
}

attn_status_t check_words(const char* name, const void* p) {
  if (p == nullptr) return fail(ATTN_ERR_INVALID_ARG, "pointer %s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return fail(ATTN_ERR_ALIGNMENT, "pointer %s is not 4-byte aligned", name);
  return ATTN_OK;
}

attn_status_t check_eps(float eps) {
  return std::isfinite(eps) && eps >= 0.f ? ATTN_OK : fail(ATTN_ERR_INVALID_ARG, "eps must be finite and >= 0%s");
}

bool supported_d(int64_t d) { return d == 32 || d == 64 || d == 96 || d == 128 || d == 256; }

// The parts of a rotary descriptor that the normed heads share.
attn_status_t check_rope_desc(const attn_rope_desc_t* desc) {
  if (desc == nullptr) return fail(ATTN_ERR_INVALID_ARG, "desc is NULL%s");
  const int64_t B = desc->B, N = desc->N, lim = int64_t(1) << 31;
  if (B < 0 || N < 0 || B >= lim || N >= lim || (N > 0 && B > (int64_t(1) << 33) / N))
    return fail(ATTN_ERR_INVALID_ARG, "B and N must be >= 0 and < 2^31, B*N <= 2^33%s");
  if (!supported_d(desc->d)) return fail(ATTN_ERR_UNSUPPORTED, "head dim must be 32, 64, 96, 128 or 256%s");
  if (desc->dtype != ATTN_F32 && desc->dtype != ATTN_BF16) return fail(ATTN_ERR_UNSUPPORTED, "unknown dtype%s");
  if (desc->paired != ATTN_ROPE_HALF && desc->paired != ATTN_ROPE_NEIGHBOUR)
    return fail(ATTN_ERR_UNSUPPORTED, "paired must be ATTN_ROPE_HALF or ATTN_ROPE_NEIGHBOUR%s");
  if (desc->inverse != 0) return fail(ATTN_ERR_UNSUPPORTED, "inverse must be 0%s");
  return ATTN_OK;
}
// ... and the tables that turn the heads.
attn_status_t check_tables(int axes, int64_t pos_batch_stride, int64_t N, const int32_t* pos, bool own_pos, const float* freq,
                           const int32_t* axis, int64_t pos_words, int64_t d, Ranges& ranges) {
  if (axes < 1 || axes > 64) return fail(ATTN_ERR_INVALID_ARG, "axes must be 1 .. 64%s");
  if (pos_batch_stride != 0 && pos_batch_stride != N) return fail(ATTN_ERR_INVALID_ARG, "pos_batch_stride must be 0 or N%s");
  attn_status_t s;
  if ((!own_pos && (s = check_words("pos", pos)) != ATTN_OK) || (s = check_words("freq", freq)) != ATTN_OK ||
      (s = check_words("axis", axis)) != ATTN_OK)
    return s;
  if (!own_pos) ranges.add("pos", pos, 4ull * axes * pos_words, false);
  ranges.add("freq", freq, 2ull * d, false);
  ranges.add("axis", axis, 2ull * d, false);
  return ATTN_OK;
}

attn_status_t check_heads(const int64_t* heads, int count, int64_t& all) {
  all = 0;
  for (int t = 0; t < count; ++t)
    if (heads[t] < 0 || heads[t] > 65535 || (all += heads[t]) > 65535)
      return fail(ATTN_ERR_INVALID_ARG, "0 to 65535 heads in all%s");
  return ATTN_OK;
}

// A paged call's problem: descriptor and cache.
struct Paged {
  Seqs seqs;
  int64_t B, H, Hkv, N, d, e;
  int dtype, causal, window;
  float scale;
};
attn_status_t check_paged_desc(const attn_desc_t* desc, Paged& p) {
  if (desc == nullptr) return fail(ATTN_ERR_INVALID_ARG, "desc is NULL%s");
  attn_desc_t one = *desc;  // (its limits on B H N are those of a grid that these calls do not launch)
  one.B = one.N = 1;
  Problem q;
  const attn_status_t s = check_desc(&one, q);
  if (s != ATTN_OK) return s;
  if (desc->seg_lo != nullptr) return fail(ATTN_ERR_UNSUPPORTED, "no document mask over a cache%s");
  const int64_t lim = int64_t(1) << 31;
  if (desc->B < 0 || desc->N < 0 || desc->B >= lim / 64 || desc->N > lim - 4096 || desc->H > 65535)  // (a tile's end behind the last token is an int too)
    return fail(ATTN_ERR_INVALID_ARG, "0 <= B < 2^25, 0 <= N <= 2^31 - 4096, H <= 65535%s");
  p.B = desc->B, p.H = desc->H, p.Hkv = desc->H / q.group, p.N = desc->N, p.d = desc->d;
  p.dtype = desc->dtype, p.e = desc->dtype == ATTN_F32 ? 4 : 2;
  p.causal = desc->causal, p.window = desc->window, p.scale = q.scale;
  return ATTN_OK;
}
attn_status_t check_cache(const attn_cache_t* c, Paged& p, const int32_t* cu, const int32_t* lens, bool written,
                          int64_t (&ks)[3], int64_t (&vs)[3], Ranges& ranges) {
  if (c == nullptr) return fail(ATTN_ERR_INVALID_ARG, "cache is NULL%s");
  const int64_t lim = int64_t(1) << 31;
  if (c->page_size < 16 || c->page_size % 16 != 0 || c->page_size > (1 << 20))
    return fail(ATTN_ERR_UNSUPPORTED, "keys of a page must be a multiple of 16, up to 2^20%s");
  if (c->pages < 0 || c->pages >= lim || c->width < 0 || c->width >= lim || c->width * c->page_size > lim - 4096)
    return fail(ATTN_ERR_INVALID_ARG, "0 <= pages < 2^31, 0 <= width * page_size <= 2^31 - 4096%s");
  attn_status_t s;
  if ((s = check_words("lens", lens)) != ATTN_OK) return s;
  if (c->width > 0 && (s = check_words("table", c->table)) != ATTN_OK) return s;
  if (cu != nullptr && (s = check_words("cu", cu)) != ATTN_OK) return s;
  for (int k = 0; k < 3; ++k) ks[k] = vs[k] = 0;
  if (c->pages > 0) {
    const View k{"K of the cache", c->K, {c->pages, p.Hkv, c->page_size}, c->k_stride, written};
    const View v{"V of the cache", c->V, {c->pages, p.Hkv, c->page_size}, c->v_stride, written};
    if ((s = check_view(k, p.d, p.e, false, ks, ranges)) != ATTN_OK) return s;
    if ((s = check_view(v, p.d, p.e, false, vs, ranges)) != ATTN_OK) return s;
  }
  ranges.add("table", c->table, 4ull * p.B * c->width, false);
  ranges.add("lens", lens, 4ull * p.B, false);
  ranges.add("cu", cu, 4ull * (p.B + 1), false);
  p.seqs = Seqs{cu,
                lens,
                c->table,
                c->width,
                static_cast<int>(p.B),
                static_cast<int>(p.N),
                static_cast<int>(c->page_size),
                static_cast<int>(c->pages),
                static_cast<int>(c->width * c->page_size)};
  return ATTN_OK;
}

PagedArgs paged_args(const Paged& p, int64_t max_new) {
  PagedArgs a{};
  a.seqs = p.seqs;
  a.H = static_cast<int>(p.H), a.Hkv = static_cast<int>(p.Hkv), a.d = static_cast<int>(p.d);
  a.dtype = p.dtype, a.causal = p.causal, a.window = p.window, a.scale = p.scale;
  a.max_new = max_new > 0 && max_new < p.N ? max_new : p.N;
  return a;
}

}  // namespace

extern "C" {

attn_status_t attn_qk_norm(const attn_rope_desc_t* desc, const attn_norm_tensor_t* tensors, int count, float eps,
                           const int32_t* pos, const float* freq, const int32_t* axis, void* stream) {
  attn_status_t s = check_rope_desc(desc);
  if (s != ATTN_OK || (s = check_eps(eps)) != ATTN_OK) return s;
  if (tensors == nullptr || count < 1 || count > ATTN_ROPE_MAX_TENSORS)
    return fail(ATTN_ERR_INVALID_ARG, "1 to ATTN_ROPE_MAX_TENSORS tensors%s");
  int64_t heads[4] = {0, 0, 0, 0}, all;
  for (int t = 0; t < count; ++t) heads[t] = tensors[t].heads;
  if ((s = check_heads(heads, count, all)) != ATTN_OK) return s;
  const int64_t B = desc->B, N = desc->N, d = desc->d, e = desc->dtype == ATTN_F32 ? 4 : 2;
  if (all * B * N == 0) return ATTN_OK;
  Ranges ranges;
  HeadArgs a{};
  a.B = B, a.N = N, a.d = static_cast<int>(d), a.axes = desc->axes, a.eps = eps;
  a.pos_batch = desc->pos_batch_stride, a.pos_axis = desc->pos_batch_stride == 0 ? N : B * N;
  a.pos = pos, a.freq = freq, a.axis = axis;
  if (freq != nullptr || pos != nullptr || axis != nullptr)
    if ((s = check_tables(desc->axes, desc->pos_batch_stride, N, pos, false, freq, axis, a.pos_axis, d, ranges)) != ATTN_OK)
      return s;
  int n = 0;
  for (int t = 0; t < count; ++t) {
    const attn_norm_tensor_t& z = tensors[t];
    if (z.heads == 0) continue;
    HeadTensor& r = a.t[n++];
    r.x = z.x, r.y = z.y, r.w = z.w, r.heads = static_cast<int>(z.heads), r.norm = true, r.turn = freq != nullptr;
    const View x{"x", z.x, {B, z.heads, N}, z.x_stride, false}, y{"y", z.y, {B, z.heads, N}, z.y_stride, true};
    if ((s = check_view(x, d, e, true, r.xs, ranges, same_view(x, y))) != ATTN_OK) return s;
    if ((s = check_view(y, d, e, false, r.ys, ranges)) != ATTN_OK) return s;
    if (z.w != nullptr && (s = check_words("w", z.w)) != ATTN_OK) return s;
    ranges.add("w", z.w, 4ull * d, false);
  }
  if ((s = ranges.apart()) != ATTN_OK) return s;
  return launch_status(head_norm(a, desc->dtype, desc->paired == ATTN_ROPE_HALF, false, static_cast<cudaStream_t>(stream)));
}

size_t attn_qk_norm_bwd_workspace_bytes(const attn_rope_desc_t* desc, const attn_norm_grad_t* tensors, int count) {
  if (check_rope_desc(desc) != ATTN_OK || tensors == nullptr || count < 1 || count > ATTN_ROPE_MAX_TENSORS) return 0;
  int64_t heads[4] = {0, 0, 0, 0}, all;
  for (int t = 0; t < count; ++t) heads[t] = tensors[t].heads;
  if (check_heads(heads, count, all) != ATTN_OK || all * desc->B * desc->N == 0) return 0;
  return head_norm_bwd_bytes(desc->B, desc->N, desc->d, desc->dtype, heads, count);
}

attn_status_t attn_qk_norm_bwd(const attn_rope_desc_t* desc, const attn_norm_grad_t* tensors, int count, float eps,
                               const int32_t* pos, const float* freq, const int32_t* axis, void* workspace,
                               size_t workspace_bytes, void* stream) {
  attn_status_t s = check_rope_desc(desc);
  if (s != ATTN_OK || (s = check_eps(eps)) != ATTN_OK) return s;
  if (tensors == nullptr || count < 1 || count > ATTN_ROPE_MAX_TENSORS)
    return fail(ATTN_ERR_INVALID_ARG, "1 to ATTN_ROPE_MAX_TENSORS tensors%s");
  int64_t heads[4] = {0, 0, 0, 0}, all;
  for (int t = 0; t < count; ++t) heads[t] = tensors[t].heads;
  if ((s = check_heads(heads, count, all)) != ATTN_OK) return s;
  const int64_t B = desc->B, N = desc->N, d = desc->d, e = desc->dtype == ATTN_F32 ? 4 : 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Ranges ranges;
  for (int t = 0; t < count; ++t) {
    const attn_norm_grad_t& z = tensors[t];
    if (z.w != nullptr && (s = check_words("w", z.w)) != ATTN_OK) return s;
    if (z.dw != nullptr && (s = check_words("dw", z.dw)) != ATTN_OK) return s;
    ranges.add("w", z.w, 4ull * d, false);
    ranges.add("dw", z.dw, 4ull * d, true);
  }
  if (all * B * N == 0) {  // nothing to sum over
    if ((s = ranges.apart()) != ATTN_OK) return s;
    for (int t = 0; t < count; ++t)
      if (tensors[t].dw != nullptr && (s = launch_status(cudaMemsetAsync(tensors[t].dw, 0, d * 4, st))) != ATTN_OK) return s;
    return ATTN_OK;
  }
  HeadGradArgs a{};
  a.B = B, a.N = N, a.d = static_cast<int>(d), a.axes = desc->axes, a.eps = eps, a.count = count;
  a.pos_batch = desc->pos_batch_stride, a.pos_axis = desc->pos_batch_stride == 0 ? N : B * N;
  a.pos = pos, a.freq = freq, a.axis = axis;
  if (freq != nullptr || pos != nullptr || axis != nullptr)
    if ((s = check_tables(desc->axes, desc->pos_batch_stride, N, pos, false, freq, axis, a.pos_axis, d, ranges)) != ATTN_OK)
      return s;
  for (int t = 0; t < count; ++t) {
    const attn_norm_grad_t& z = tensors[t];
    HeadGrad& r = a.t[t];
    r.x = z.x, r.dy = z.dy, r.dx = z.dx, r.w = z.w, r.dw = z.dw, r.heads = static_cast<int>(z.heads);
    if (z.heads == 0) continue;
    const View x{"x", z.x, {B, z.heads, N}, z.x_stride, false}, dy{"dy", z.dy, {B, z.heads, N}, z.dy_stride, false},
        dx{"dx", z.dx, {B, z.heads, N}, z.dx_stride, true};
    if ((s = check_view(x, d, e, true, r.xs, ranges, same_view(x, dx))) != ATTN_OK) return s;
    if ((s = check_view(dy, d, e, true, r.dys, ranges, same_view(dy, dx))) != ATTN_OK) return s;
    if ((s = check_view(dx, d, e, false, r.dxs, ranges)) != ATTN_OK) return s;
  }
  const size_t need = head_norm_bwd_bytes(B, N, d, desc->dtype, heads, count);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace NULL or smaller than attn_qk_norm_bwd_workspace_bytes()%s");
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return fail(ATTN_ERR_ALIGNMENT, "pointer %s is not 16-byte aligned", "workspace");
  ranges.add("workspace", workspace, need, true);
  if ((s = ranges.apart()) != ATTN_OK) return s;
  a.ws = static_cast<float*>(workspace);
  return launch_status(head_norm_bwd(a, desc->dtype, desc->paired == ATTN_ROPE_HALF, st));
}

attn_status_t attn_cache_append(const attn_desc_t* desc, const attn_new_tokens_t* t, const attn_cache_t* cache,
                                const int32_t* cu, const int32_t* lens, void* stream) {
  Paged p;
  attn_status_t s = check_paged_desc(desc, p);
  if (s != ATTN_OK) return s;
  if (t == nullptr) return fail(ATTN_ERR_INVALID_ARG, "the new tokens are NULL%s");
  if ((s = check_eps(t->eps)) != ATTN_OK) return s;
  if (t->normed != 0 && t->normed != 1) return fail(ATTN_ERR_UNSUPPORTED, "normed must be 0 or 1%s");
  if (t->paired != ATTN_ROPE_HALF && t->paired != ATTN_ROPE_NEIGHBOUR)
    return fail(ATTN_ERR_UNSUPPORTED, "paired must be ATTN_ROPE_HALF or ATTN_ROPE_NEIGHBOUR%s");
  const int64_t batch = cu != nullptr ? 1 : p.B;
  if (p.N > 0 && batch > (int64_t(1) << 33) / p.N) return fail(ATTN_ERR_INVALID_ARG, "B*N must be <= 2^33%s");
  if (batch * p.N * p.H * p.B == 0) return ATTN_OK;
  Ranges ranges;
  HeadArgs a{};
  const bool turned = t->freq != nullptr || t->axis != nullptr || t->pos != nullptr;
  a.B = batch, a.N = p.N, a.d = static_cast<int>(p.d), a.axes = t->axes, a.eps = t->eps;
  a.pos_batch = t->pos_batch_stride, a.pos_axis = t->pos_batch_stride == 0 ? p.N : batch * p.N;
  a.pos = t->pos, a.freq = t->freq, a.axis = t->axis;
  if (turned) {
    if (t->pos == nullptr && t->axes != 1) return fail(ATTN_ERR_INVALID_ARG, "positions in the sequences have one axis%s");
    if ((s = check_tables(t->axes, t->pos_batch_stride, p.N, t->pos, t->pos == nullptr, t->freq, t->axis, a.pos_axis, p.d,
                          ranges)) != ATTN_OK)
      return s;
  }
  HeadTensor &k = a.t[0], &v = a.t[1], &q = a.t[2];
  if ((s = check_cache(cache, p, cu, lens, true, k.ys, v.ys, ranges)) != ATTN_OK) return s;
  k.x = t->K, k.y = cache->K, k.w = t->k_weight, k.heads = static_cast<int>(p.Hkv), k.norm = t->normed != 0, k.turn = turned;
  v.x = t->V, v.y = cache->V, v.heads = static_cast<int>(p.Hkv);
  k.paged = v.paged = true;
  const int64_t kv = p.Hkv;
  if ((s = check_view(View{"K", t->K, {batch, kv, p.N}, t->k_stride, false}, p.d, p.e, true, k.xs, ranges)) != ATTN_OK) return s;
  if ((s = check_view(View{"V", t->V, {batch, kv, p.N}, t->v_stride, false}, p.d, p.e, true, v.xs, ranges)) != ATTN_OK) return s;
  if (t->Q != nullptr || t->Q_out != nullptr) {
    q.x = t->Q, q.y = t->Q_out, q.w = t->q_weight, q.heads = static_cast<int>(p.H), q.norm = t->normed != 0, q.turn = turned;
    const View x{"Q", t->Q, {batch, p.H, p.N}, t->q_stride, false}, y{"Q_out", t->Q_out, {batch, p.H, p.N}, t->q_out_stride, true};
    if ((s = check_view(x, p.d, p.e, true, q.xs, ranges, same_view(x, y))) != ATTN_OK) return s;
    if ((s = check_view(y, p.d, p.e, false, q.ys, ranges)) != ATTN_OK) return s;
  }
  if (k.heads + v.heads + q.heads > 65535) return fail(ATTN_ERR_INVALID_ARG, "0 to 65535 heads in all%s");
  if (t->normed) {
    if (t->k_weight != nullptr && (s = check_words("k_weight", t->k_weight)) != ATTN_OK) return s;
    if (t->q_weight != nullptr && (s = check_words("q_weight", t->q_weight)) != ATTN_OK) return s;
    ranges.add("k_weight", t->k_weight, 4ull * p.d, false);
    ranges.add("q_weight", t->q_weight, 4ull * p.d, false);
  }
  if ((s = ranges.apart()) != ATTN_OK) return s;
  a.seqs = p.seqs;
  return launch_status(head_norm(a, p.dtype, t->paired == ATTN_ROPE_HALF, true, static_cast<cudaStream_t>(stream)));
}

size_t attn_paged_workspace_bytes(const attn_desc_t* desc, int64_t max_new) {
  Paged p;
  if (check_paged_desc(desc, p) != ATTN_OK || p.B * p.N * p.H == 0) return 0;
  p.seqs = Seqs{};
  p.seqs.B = static_cast<int>(p.B), p.seqs.N = static_cast<int>(p.N);
  return paged_bytes(paged_args(p, max_new));
}

attn_status_t attn_paged(const attn_desc_t* desc, const void* Q, const int64_t* q_stride, const attn_cache_t* cache,
                         const int32_t* cu, const int32_t* lens, int64_t max_new, void* O, const int64_t* o_stride,
                         float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  Paged p;
  attn_status_t s = check_paged_desc(desc, p);
  if (s != ATTN_OK) return s;
  if (max_new < 0) return fail(ATTN_ERR_INVALID_ARG, "max_new must be >= 0 (0: not known)%s");
  if (q_stride == nullptr || o_stride == nullptr) return fail(ATTN_ERR_INVALID_ARG, "strides are NULL%s");
  const int64_t batch = cu != nullptr ? 1 : p.B;
  if (batch * p.N * p.H * p.B == 0) return ATTN_OK;
  Ranges ranges;
  PagedArgs a{};
  int64_t qs[3], os[3], ks[3], vs[3];
  if ((s = check_cache(cache, p, cu, lens, false, ks, vs, ranges)) != ATTN_OK) return s;
  if ((s = check_view(View{"Q", Q, {batch, p.H, p.N}, q_stride, false}, p.d, p.e, false, qs, ranges)) != ATTN_OK) return s;
  if ((s = check_view(View{"O", O, {batch, p.H, p.N}, o_stride, true}, p.d, p.e, false, os, ranges)) != ATTN_OK) return s;
  if (lse != nullptr) {
    if ((s = check_words("lse", lse)) != ATTN_OK) return s;
    ranges.add("lse", lse, 4ull * batch * p.H * p.N, true);
  }
  a = paged_args(p, cu != nullptr ? max_new : p.N);
  const size_t need = paged_bytes(a);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace NULL or smaller than attn_paged_workspace_bytes()%s");
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return fail(ATTN_ERR_ALIGNMENT, "pointer %s is not 16-byte aligned", "workspace");
  ranges.add("workspace", workspace, need, true);
  if ((s = ranges.apart()) != ATTN_OK) return s;
  a.Q = Q, a.K = cache->K, a.V = cache->V, a.O = O, a.lse = lse;
  for (int k = 0; k < 3; ++k) a.qs[k] = qs[k], a.os[k] = os[k], a.ks[k] = ks[k], a.vs[k] = vs[k];
  a.ls[0] = p.H * p.N, a.ls[1] = p.N;
  return launch_status(paged_attention(a, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
