// Tensor maps of bf16 views with strides of their own (defined in api.cu).
#pragma once
#include <cstdint>

namespace fbd {

// `rank` dimensions, the first one contiguous; strides of the others in elements (0: a dimension of one
// element, or one that is not stepped along); 128-byte swizzle, boxes of 64 elements along the first.
// Returns false if the driver entry point is missing or the encode fails.
bool make_tmap_view(void* map_out /* CUtensorMap* */, const void* base, int rank, const int64_t* dims, const int64_t* strides,
                    const int* box);

}  // namespace fbd
