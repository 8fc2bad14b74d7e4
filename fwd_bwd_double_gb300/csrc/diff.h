// Differential attention: launch interface between the C ABI (api_diff.cu) and the kernels.
//
// A differential head h holds two softmax maps over one value head of twice their width:
//   A_m = softmax(s Q_m K_m^T + mask), m = 1, 2;   O = (A_1 - lam_h A_2) V.
// The maps of head h are the neighbouring slices 2h and 2h + 1 of Q [B,2H,N,d]; those of a
// key/value head n are 2n and 2n + 1 of K [B,2H/g,N,d]; V is [B,H/g,N,2d], O [B,H,N,2d].
// In `Problem` H, BH, group and BHkv count differential heads (BH = B H, BHkv = B H / g) and
// d is the width of a map.
#pragma once
#include <cmath>

#include "internal.h"

namespace fbd {

// The widths with kernels.
inline bool diff_supports(int64_t d) { return d == 32 || d == 64; }

// bf16 tensor-core kernels (tc_diff_fwd.cu, tc_diff_bwd.cu).
cudaError_t tc_diff_fwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, void* O,
                        void* O2, float* lse, cudaStream_t st);
uint32_t tc_diff_fwd_take_error();
cudaError_t tc_diff_bwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, const void* O,
                        const void* O2, const void* dO, const float* lse, void* dQ, void* dK, void* dV, float* dlam,
                        void* ws, cudaStream_t st);
size_t tc_diff_bwd_bytes(int64_t BH, int64_t N);
uint32_t tc_diff_bwd_take_error();

// CUDA-core kernels for float32 (simt_diff.cu).
cudaError_t simt_diff_fwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam, void* O,
                          void* O2, float* lse, cudaStream_t st);
cudaError_t simt_diff_bwd(const Problem& p, const void* Q, const void* K, const void* V, const float* lam,
                          const void* O, const void* O2, const void* dO, const float* lse, void* dQ, void* dK,
                          void* dV, float* dlam, void* ws, cudaStream_t st);
size_t simt_diff_bwd_bytes(int64_t BH, int64_t N);

// The rows whose dS is zero whatever their values: a softmax over one visible key is
// constant.  Formed as P (dP - D) from rounded O their dS would be noise, so the
// backward's preparation marks them with D = +inf and the kernels set dS = 0 there (a D
// that overflowed to +inf by its values is made NaN, as its gradients are).
__device__ __forceinline__ float diff_mark_D(float D, bool one_key) {
  return one_key ? INFINITY : (D == INFINITY ? __int_as_float(0x7fc00000) : D);
}
__device__ __forceinline__ bool diff_one_key(const Band& bd, int causal, int64_t slice, int64_t i) {
  return causal ? bd.row_lo(slice, i) == i : bd.N == 1;
}

// dlam_h = -sum over batch rows and blocks of partial[(b H + h) nblk + k], summed in a
// fixed order by one block per head.
cudaError_t diff_reduce_dlam(const float* partial, float* dlam, int64_t B, int64_t H, int64_t nblk, cudaStream_t st);

// A launch that may be set up while the kernel before it in the stream ends: it may read what
// that kernel wrote only behind ptx::grid_dependency_wait().  The kernel before it may let it in with
// ptx::grid_dependency_launch() as soon as its own blocks have all started: 13.6 against 14.7 us
// for the backward of B1 H2 N257 d32, 6.0 to 6.3 against 6.6 us for one token over 1024 keys, 6 heads.
template <typename... P, typename... A>
inline cudaError_t launch_behind(void (*kern)(P...), int64_t grid, int block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// One token over a cache (diff_decode.cu).  p.N is the cache's capacity.
size_t diff_decode_bytes(const Problem& p);
cudaError_t diff_decode(const Problem& p, const void* Q, const void* K, const void* V, const float* lam,
                        const int* lens, void* O, void* ws, cudaStream_t st);

}  // namespace fbd
