// Paged caches: the sequences of a call, their pages, and the launch interface between the C ABI
// (api_paged.cu) and the kernels.
//
// A cache holds K and V as [pages, Hkv, page, d] views; row b of the table lists the pages of sequence
// b, so that its key j lies in slot j % page of page table[b][j / page].  The new tokens of a sequence
// are its last n keys: token t stands at position lens[b] - n + t.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "fbd.h"

namespace fbd {

// The sequences of a call.  Packed: sequence b has the rows cu[b] .. cu[b + 1] - 1 of one batch row of N;
// else (cu == nullptr) the N rows of batch row b.
struct Seqs {
  const int* cu;
  const int* lens;
  const int* table;
  int64_t width;  // entries of a sequence's row of the table
  int B, N;
  int page, pages;
  int cap;        // width * page
};

// Rows row0 .. row0 + n - 1 of batch row `batch`; token t at position start + t (below 0: it sees nothing
// and is not stored); keys 0 .. len - 1.
struct Seq {
  int batch, row0, n, start, len;
};

#ifdef __CUDACC__
__device__ __forceinline__ Seq seq_at(const Seqs& a, int b) {
  Seq s;
  s.batch = a.cu != nullptr ? 0 : b;
  s.row0 = 0, s.n = a.N;
  if (a.cu != nullptr) {  // (whatever it holds, no row outside the tensor is touched)
    s.row0 = min(max(a.cu[b], 0), a.N);
    s.n = min(max(a.cu[b + 1], s.row0), a.N) - s.row0;
  }
  const int l = a.lens[b];
  s.len = min(max(l, 0), a.cap);
  s.start = l < 0 ? -s.n : l - s.n;
  return s;
}
// The page of entry e of sequence b's row, -1 where there is none.
__device__ __forceinline__ int page_at(const Seqs& a, int b, int e) {
  if (e < 0 || e >= a.width) return -1;
  const int p = __ldg(a.table + b * a.width + e);
  return p >= 0 && p < a.pages ? p : -1;
}
#endif

// The heads of new tokens, normed and turned, to where they belong (headnorm.cu).
struct HeadTensor {
  const void* x;
  void* y;
  const float* w;  // weight of the norm (may be null: ones)
  int heads;
  bool norm, turn;
  bool paged;      // y is a cache: strides of (page, head, slot); else of (batch, head, position)
  int64_t xs[3], ys[3];
};
struct HeadArgs {
  HeadTensor t[4];
  int64_t B, N;
  int64_t pos_axis, pos_batch;  // strides of pos, in elements
  const int* pos;               // null: the tokens' positions in their sequences
  const float* freq;            // null: nothing turns
  const int* axis;
  int d, axes;
  float eps;
  int per[4], first[5];         // heads per thread and first block row of each tensor (set by the launcher)
  Seqs seqs;                    // of an append (else unused)
};
cudaError_t head_norm(const HeadArgs& a, int dtype, bool half, bool append, cudaStream_t st);

struct HeadGrad {
  const void* x;
  const void* dy;
  void* dx;
  const float* w;
  float* dw;  // may be null
  int heads;
  int64_t xs[3], dys[3], dxs[3];
};
struct HeadGradArgs {
  HeadGrad t[4];
  int64_t B, N;
  int64_t pos_axis, pos_batch;
  const int* pos;
  const float* freq;
  const int* axis;
  int d, axes, count;
  float eps;
  float* ws;
  // set by the launcher: heads per block row and the first block row of each tensor, block columns
  int per[4], first[5], cols;
};
size_t head_norm_bwd_bytes(int64_t B, int64_t N, int64_t d, int dtype, const int64_t* heads, int count);
cudaError_t head_norm_bwd(const HeadGradArgs& a, int dtype, bool half, cudaStream_t st);

// Attention of new tokens over their pages.
struct PagedArgs {
  Seqs seqs;
  const void *Q, *K, *V;
  void* O;
  float* lse;                          // may be null
  int64_t qs[3], os[3], ks[3], vs[3];  // strides: (batch, head, position) and (page, head, slot)
  int64_t ls[2];                       // of lse: (batch, head); positions are neighbours
  int H, Hkv, d, dtype, causal, window;
  float scale;
  int64_t max_new;                     // the most new tokens of a sequence, as far as the host knows
};
size_t paged_bytes(const PagedArgs& a);
cudaError_t paged_attention(const PagedArgs& a, void* ws, cudaStream_t st);
uint32_t tc_paged_take_error();
uint32_t tc_paged_wide_take_error();
uint32_t token_paged_take_error();

}  // namespace fbd
