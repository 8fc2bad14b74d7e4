// Argument checks and status reporting shared by the C entry points (defined in api.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "fbd.h"
#include "internal.h"

namespace fbd {

// Records `fmt` (with `what`) as the calling thread's attn_last_error() detail; returns s.
attn_status_t fail(attn_status_t s, const char* fmt, const char* what = "");

struct Span {
  const char* name;
  uintptr_t lo, hi;  // [lo, hi)
};
Span span(const char* name, const void* ptr, size_t bytes);

// Shape/type checks shared by every entry point.  Fills `p` on success.
attn_status_t check_desc(const attn_desc_t* desc, Problem& p);

size_t elem_size(const Problem& p);

// Non-NULL, 16-byte aligned, pairwise non-overlapping outputs vs everything.
attn_status_t check_ptrs(const Span* in, int nin, const Span* out, int nout);

attn_status_t launch_status(cudaError_t e);

}  // namespace fbd
