// Launches of the attention over a paged cache: its kernels, and the join behind each.
#pragma once
#include "paged.cuh"

namespace fbd {
namespace paged {

// tile_rows: rows of a slot that a tile takes; few: the most new tokens of a sequence, as far as is known.
cudaError_t join(const Work& w, const Space& sp, const Out& out, int dtype, int d, int tile_rows, int64_t few, cudaStream_t st);

// The query heads handled together by a kernel whose tiles have `rows` rows: all that share a key/value head where
// `few` new tokens of them fit a tile (K and V are then read once), else the most that leave no more than a
// sixteenth of a tile's rows empty: the more heads, the fewer tokens a tile spans, and so the fewer keys that
// some of its rows do not see, and the less of a sequence's last tile is empty (three heads of 42 tokens against one of
// 128: 184 us against 217 for the ragged window).
inline int heads_together(int group, int rows, int64_t few) {
  if (few > 0 && few * group <= rows) return group;
  int best = 1;
  for (int k = 1; k <= group && k <= rows; ++k)
    if (group % k == 0 && rows / k * k * 16 >= rows * 15) best = k;
  return best;
}

// The kernels: CUDA cores (simt_paged.cu, float32), tensor cores (tc_paged.cu, bf16 up to d = 128; tc_paged_wide.cu, d = 256).
size_t simt_bytes(const PagedArgs& a);
cudaError_t simt_paged(const PagedArgs& a, void* ws, cudaStream_t st);
size_t tc_bytes(const PagedArgs& a);
cudaError_t tc_paged(const PagedArgs& a, void* ws, cudaStream_t st);
// ... and warp-level products for up to 16 rows of a sequence (paged_token.cu, bf16).
inline bool few_rows(const PagedArgs& a) { return a.max_new * (a.H / a.Hkv) <= 16; }
size_t token_bytes(const PagedArgs& a);
cudaError_t token_paged(const PagedArgs& a, void* ws, cudaStream_t st);
size_t tc_wide_bytes(const PagedArgs& a);
cudaError_t tc_paged_wide(const PagedArgs& a, void* ws, cudaStream_t st);

}  // namespace paged
}  // namespace fbd
