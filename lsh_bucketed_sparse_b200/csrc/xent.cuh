// Shared by the cross-entropy kernels.
#pragma once

#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace lsh {

// The row's target, -1 for one outside [0, vocab) (the row is ignored).
template <typename I>
__device__ __forceinline__ int target_of(const I* targets, long long row, int vocab) {
  const I t = targets[row];
  return t >= 0 && t < (I)vocab ? (int)t : -1;
}

// (m, s) stands for s exp(m); adds (m2, s2).  A NaN goes into the sum.
__device__ __forceinline__ void lse_add(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.f : top;  // nothing but exp(-inf) so far
  s = s * expf(m - ref) + s2 * expf(m2 - ref);
  m = top;
}

// clean[rows][d] = x with zeros in the rows that have no target, so that what
// stands there (padding may hold anything) takes no part in a product.
cudaError_t launch_xent_clean(const TableProblem& p, const void* x, const void* targets,
                              void* clean, cudaStream_t st);

// ---- CUDA cores (xent_portable.cu) ---------------------------------------------
// Forward: part[slice][row] = (maximum, sum) over the slice's logits, zt[row]
// the target's logit where the row has a target.
int xent_portable_slices(const TableProblem& p);
cudaError_t launch_xent_portable(const TableProblem& p, const void* x, const void* table,
                                 const void* targets, float2* part, float* zt, cudaStream_t st);
size_t xent_portable_backward_bytes(const TableProblem& p);
cudaError_t launch_xent_portable_backward(const TableProblem& p, const void* x, const void* table,
                                          const void* targets, const float* lse,
                                          const float* dloss, void* dx, void* dtable,
                                          void* workspace, cudaStream_t st);

}  // namespace lsh
