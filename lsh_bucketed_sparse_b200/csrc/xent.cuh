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

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The forward's logits are in units of log2: (m, s) stands for s 2^m.  Adds
// (m2, s2).  A NaN goes into the sum.
__device__ __forceinline__ void lse_add(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.f : top;  // nothing but 2^-inf so far
  s = s * exp2f(m - ref) + s2 * exp2f(m2 - ref);
  m = top;
}

// clean[rows][d] = x with zeros in the rows that have no target, so that what
// stands there (padding may hold anything) takes no part in a product.
cudaError_t launch_xent_clean(const TableProblem& p, const void* x, const void* targets,
                              void* clean, cudaStream_t st);

// Forward, of any kind: part[slice][row] = (maximum, sum) over the slice's logits
// except the target's, which stands in zt[row] where the row has a target, as the
// product left it, without scale (where scale is 0 the sum has it too).

// Most bytes of g in a piece of the backward: `most`, or less by the test hook.
size_t xent_piece_bytes(size_t most);
unsigned long long set_xent_piece_bytes(unsigned long long bytes);  // returns the previous limit

// ---- tensor cores (xent_tc.cu) ---------------------------------------------------
bool xent_tc_supported(const TableProblem& p);
// Sets the limit of the MMA thread's first wait (test hook); returns the
// previous limit.
unsigned long long set_xent_first_wait_ns(unsigned long long ns);
int xent_tc_slices(const TableProblem& p);
size_t xent_tc_bytes(const TableProblem& p);  // of scratch
cudaError_t launch_xent_tc(const TableProblem& p, const void* x, const void* table,
                           const void* targets, float2* part, float* zt, void* scratch,
                           cudaStream_t st);
size_t xent_tc_backward_bytes(const TableProblem& p);
cudaError_t launch_xent_tc_backward(const TableProblem& p, const void* x, const void* table,
                                    const void* targets, const float* lse, const float* dloss,
                                    void* dx, void* dtable, void* workspace, cudaStream_t st);

// ---- few float32 rows (xent_few.cu) ----------------------------------------------
bool xent_few_supported(const TableProblem& p);
int xent_few_slices(const TableProblem& p);
cudaError_t launch_xent_few(const TableProblem& p, const void* x, const void* table,
                            const void* targets, float2* part, float* zt, cudaStream_t st);
size_t xent_few_backward_bytes(const TableProblem& p);
cudaError_t launch_xent_few_backward(const TableProblem& p, const void* x, const void* table,
                                     const void* targets, const float* lse, const float* dloss,
                                     void* dx, void* dtable, void* workspace, cudaStream_t st);

// ---- CUDA cores (xent_portable.cu) ---------------------------------------------
int xent_portable_slices(const TableProblem& p);
cudaError_t launch_xent_portable(const TableProblem& p, const void* x, const void* table,
                                 const void* targets, float2* part, float* zt, cudaStream_t st);
size_t xent_portable_backward_bytes(const TableProblem& p);
cudaError_t launch_xent_portable_backward(const TableProblem& p, const void* x, const void* table,
                                          const void* targets, const float* lse,
                                          const float* dloss, void* dx, void* dtable,
                                          void* workspace, cudaStream_t st);

}  // namespace lsh
